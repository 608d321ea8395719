// What the kernels of differential attention share: the layout of their partial rows
// and the combines that join them.
#pragma once

#include "k8v4_ops.cuh"

namespace k8v4 {

// A partial row: o[256] (rotated space, unnormalised, relative to 2^m), m (a base-2
// exponent, -inf: no cell seen), l (the sum of 2^(score - m)), two unused floats.
constexpr int kDiffRow = 260;

// the CTA pairs that a ragged batch is planned for, at most, and the ranges that a row has
// then (2 * pairs / H, rounded up)
constexpr int kDiffMostPairs = 128, kDiffMostRanges = 2 * kDiffMostPairs + 2;

// Single queries over the line of their tiles (k8v4_diff.cu): of each pair (query, KV head) its
// first block and their number, and the blocks of 16 partial rows (map, query head).
struct DiffPieces {
  int2* pairs;
  float* rows;
  int blocks;                 // that there is room for
};
size_t place_pieces(DiffPieces* p, uint8_t* ws, int64_t n_pairs, int num_sms);
// a ragged batch's: the sequence and the packed token of each query, and how many there are (device)
struct DiffQueries {
  const int32_t* seq = nullptr;
  const int32_t* tok = nullptr;
  const int32_t* count = nullptr;
};
int launch_diff_split(const Launch& L, const CacheView& C, const void* q, int q_dtype, const int32_t* pt, int64_t max_pages,
                      const int32_t* lens, const DiffQueries& rows, int n_seqs, int max_seq_len, float sm_scale,
                      const DiffPieces& ws);

// four or eight fp16 block scales: nonzero where one is at least 2^13 in size, so that 8 d does not fit fp16
__device__ __forceinline__ uint32_t larger_of(uint32_t a, uint32_t b) {                    // in size, of each half
  const __half2 r = __hmax2(__habs2(*reinterpret_cast<const __half2*>(&a)), __habs2(*reinterpret_cast<const __half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t big_blocks(uint32_t a, uint32_t b) { return (larger_of(a, b) + 0x10001000u) & 0x80008000u; }
__device__ __forceinline__ uint32_t big_blocks(const uint4& d) { return big_blocks(larger_of(d.x, d.y), larger_of(d.z, d.w)); }
__device__ __forceinline__ uint32_t eighth_of(uint32_t d) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&d), __halves2half2(__ushort_as_half(0x3000), __ushort_as_half(0x3000)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// a warp: exp(q1 . k1) (term 0) or exp(q2 . k2) of a query head, 0 without vectors
__device__ __forceinline__ float diff_lambda_term(const k8v4_diff& d, int hq, int term, int lane) {
  if (!d.lambda_q1) return 0.0f;
  const int64_t at = (d.n_lambda > 1 ? hq * 128 : 0) + 4 * lane;
  const float4 a = *reinterpret_cast<const float4*>((term ? d.lambda_q2 : d.lambda_q1) + at);
  const float4 b = *reinterpret_cast<const float4*>((term ? d.lambda_k2 : d.lambda_k1) + at);
  float dot = a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  return expf(dot);
}

// A ragged batch's rows: each packed token's tile, or -1 (no sequence's), or -2 - query (one of the
// single queries above); and the tiles of 8 words: [1] the first token, [3] ranges, [4] the first
// block.  Range s of map m of query head h, KV head g, is in block first + (2 g + m) * ranges + s,
// row (token - first token) * 8 + h, blocks of 256 rows.
struct DiffRagged {
  const float* lambdas;       // of each query head
  const int32_t* tok_tile;
  const int32_t* tiles;
};
int launch_diff_combine_ragged(const Launch& L, const float* ws, const DiffRagged& r, const DiffPieces& pieces,
                               const int32_t* lens, int n_tok, int H, bool few, const k8v4_diff& diff, void* out);

}  // namespace k8v4
