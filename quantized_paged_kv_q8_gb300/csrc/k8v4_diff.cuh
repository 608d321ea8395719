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

// A ragged batch's rows: each packed token's tile (-1: no sequence's), and the tiles of 8
// words: [1] the first token, [3] ranges, [4] the first block.  Range s of map m of query head
// h, KV head g, is in block first + (2 g + m) * ranges + s, row (token - first token) * 8 + h,
// blocks of 256 rows.
struct DiffRagged {
  const int32_t* tok_tile;
  const int32_t* tiles;
};
int launch_diff_combine_ragged(const Launch& L, const float* ws, const DiffRagged& r, int n_tok, int H, bool wide,
                               const k8v4_diff& diff, void* out);

}  // namespace k8v4
