// Internal definitions shared by the k8v4 CUDA translation units: the device
// view of a cache, the page-layout offsets, the device status word, small PTX
// wrappers, and the host-side launch functions the C ABI calls.
#pragma once

#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/k8v4.h"

namespace k8v4 {

constexpr int kD = 256;   // head_dim
constexpr int kGqa = 8;   // query heads per KV head

// Bytes per (cell, head) of each format.  K8V4: 256 K codes + 8 (two fp32
// scales) + 128 V nibbles + 16 (eight fp16 scales) = 408; INT8: 256 + 8 + 256 +
// 8 = 528; Q4: 128 + 16 + 128 + 16 = 288.
__host__ __device__ constexpr int cell_head_bytes(int fmt) {
  return fmt == K8V4_FORMAT_K8V4 ? 408 : fmt == K8V4_FORMAT_Q4 ? 288 : 528;
}

// Device view of a cache.  Page p starts at pages + p * page_bytes; inside it
// the runs are K ([P][H][256] int8 codes, or [P][H][8][16] nibbles for Q4),
// K scales ([P][H][2] f32, or [P][H][8] f16 for Q4), V ([P][H][8][16] nibbles,
// or [P][H][256] int8 codes for INT8) and V scales ([P][H][8] f16, or [P][H][2]
// f32 for INT8).  r = slot * H + head indexes a (cell, head) inside a run.
struct CacheView {
  uint8_t* pages;
  int64_t n_pages;
  int64_t page_bytes;
  int P;
  int H;
  int fmt;

  __host__ __device__ int k_row_bytes() const { return fmt == K8V4_FORMAT_Q4 ? 128 : 256; }
  __host__ __device__ int ks_row_bytes() const { return fmt == K8V4_FORMAT_Q4 ? 16 : 8; }
  __host__ __device__ int v_row_bytes() const { return fmt == K8V4_FORMAT_INT8 ? 256 : 128; }
  __host__ __device__ int vs_row_bytes() const { return fmt == K8V4_FORMAT_INT8 ? 8 : 16; }
  __host__ __device__ int64_t ks_off() const { return static_cast<int64_t>(k_row_bytes()) * H * P; }
  __host__ __device__ int64_t v_off() const { return static_cast<int64_t>(k_row_bytes() + ks_row_bytes()) * H * P; }
  __host__ __device__ int64_t vs_off() const {
    return static_cast<int64_t>(k_row_bytes() + ks_row_bytes() + v_row_bytes()) * H * P;
  }
};

// ---------------------------------------------------------------- division
// Division by a kernel-invariant divisor d >= 1 for dividends below 2^31, by the
// round-up multiply-high method: s = ceil(log2 d), m = floor(2^32 (2^s - d) / d)
// + 1, q = (umulhi(n, m) + n) >> s (exact for every n < 2^31; the sum stays
// below 2^32).  Three instructions instead of a 64-bit division routine.
struct FastDiv {
  uint32_t d = 1, m = 1;
  int s = 0;
  FastDiv() = default;
  __host__ explicit FastDiv(uint32_t div) : d(div) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

// ---------------------------------------------------------------- status word
// Kernels record the first device-side error here (compare-and-swap from 0) and
// skip the offending access; the host reads and clears it.
__device__ __forceinline__ void record_status(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// ---------------------------------------------------------------- PTX helpers
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---------------------------------------------------------------- host side
struct Launch {
  cudaStream_t stream;
  int* status;      // device status word of the current device
  int num_sms;
};

// Launch a kernel whose first act on memory is griddepcontrol.wait: its CTAs may
// take their places while the kernel before it in the stream drains.  (Its own
// launch, about 1 us, is then hidden behind that kernel: a decode step is a chain
// of kernels of a few microseconds.)  Such a kernel is on the device while that one
// still writes, so nothing it reads may go through the read-only path (__ldg, const
// __restrict__ pointers).
template <typename... P, typename... A>
int launch_behind(const Launch& L, void (*kernel)(P...), dim3 grid, dim3 block, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return K8V4_ECUDA;
  return cudaGetLastError() == cudaSuccess ? K8V4_OK : K8V4_ECUDA;
}

// mirror != null: a streamed cache -- pt holds host-mirror page ids, every row is
// written to the mirror and, where slot_of_page[page] >= 0, to that slot of C
int launch_append(const Launch& L, const CacheView& C, const int32_t* pt, int64_t max_pages, int n_seqs,
                  const int64_t* pos, int n_tok, const void* k, const void* v, int dtype,
                  const CacheView* mirror = nullptr, const int32_t* slot_of_page = nullptr);
// streamed caches: look up the pages the sequences read (resident slot, or a copy
// from the host mirror M into a staging slot of C) and copy the misses
int launch_stream_resolve(const Launch& L, const CacheView& M, const CacheView& C, const int32_t* slot_of_page,
                          int n_resident, const int32_t* pt, int64_t max_pages, const int32_t* lens, int n_seqs,
                          int max_seq_len, int32_t* dev_pt, void* ws);
int launch_stream_copy(const Launch& L, const CacheView& M, const CacheView& C, const int32_t* pages, int n);
size_t stream_ws_bytes(int n_seqs, int64_t max_pages);
int launch_dequant(const Launch& L, const CacheView& C, const int32_t* pt, int64_t max_pages, int64_t start,
                   int64_t n_cells, float* k_out, float* v_rot_out, float* v_out);

struct AttendPlan {
  int n_q, n_groups, warps, splits, cells_per_split;
  size_t ws_bytes;
};
// most cell ranges that a sequence's decode, and a shared prefix, are split into
constexpr int kDecodeMaxSplits = 1024, kPrefixMaxSplits = 256;
AttendPlan plan_attend(const CacheView& C, int n_seqs, int n_q, int max_seq_len, int num_sms);
// k_new / v_new (n_q = 1 only): append each sequence's newest token (cell
// steps[b] - 1) from them before attending -- the fused decode step
int launch_attend(const Launch& L, const CacheView& C, const AttendPlan& plan, const void* q, int q_dtype,
                  const int32_t* pt, int64_t max_pages, const int32_t* steps, int n_seqs, int max_seq_len,
                  float sm_scale, float* out, void* ws, const void* k_new = nullptr, const void* v_new = nullptr,
                  int kv_dtype = K8V4_BF16);
AttendPlan plan_verify(const CacheView& C, int n_seqs, int n_q, int max_seq_len, int num_sms);
int launch_verify(const Launch& L, const CacheView& C, const AttendPlan& plan, const void* q, int q_dtype,
                  const int32_t* pt, int64_t max_pages, const int32_t* steps, int n_seqs, int max_seq_len,
                  float sm_scale, float* out, void* ws);
AttendPlan plan_verify_tc(const CacheView& C, int n_seqs, int n_q, int max_seq_len, int num_sms);
int launch_verify_tc(const Launch& L, const CacheView& C, const AttendPlan& plan, const void* q,
                     const int32_t* pt, int64_t max_pages, const int32_t* steps, int n_seqs, int max_seq_len,
                     float sm_scale, float* out, void* ws);
// the warp-specialised TMA decode kernel (k8v4_decode.cu): one query per
// sequence over the K8V4 or INT8 format; spin = mbarrier poll limit (0: default)
bool decode_ws_supported(const CacheView& C);
AttendPlan plan_decode(const CacheView& C, int n_seqs, int max_seq_len, int num_sms);
int launch_decode(const Launch& L, const CacheView& C, const AttendPlan& plan, const void* q, int q_dtype,
                  const int32_t* pt, int64_t max_pages, const int32_t* steps, int n_seqs, int max_seq_len,
                  float sm_scale, float* out, void* ws, const void* k_new, const void* v_new, int kv_dtype,
                  uint32_t spin);
// cells [cell_begin, cell_end) of every sequence only, merged into unnormalised
// partial rows [n_seqs][8 H][260] (o[256], m as a base-2 exponent, l); the plan
// is plan_decode over cell_end - cell_begin cells
int launch_decode_partial(const Launch& L, const CacheView& C, const AttendPlan& plan, const void* q, int q_dtype,
                          const int32_t* pt, int64_t max_pages, const int32_t* steps, int n_seqs,
                          int max_seq_len, int cell_begin, int cell_end, float sm_scale, float* partial, void* ws,
                          uint32_t wait_ns);
// the team-of-warps TMA verify kernel (k8v4_decode.cu): 2..8 queries per
// sequence over the K8V4 format with bf16 queries
bool verify_ws_supported(const CacheView& C, int n_q, int q_dtype);
AttendPlan plan_verify_ws(const CacheView& C, int n_seqs, int n_q, int max_seq_len, int num_sms);
int launch_verify_ws(const Launch& L, const CacheView& C, const void* q, const int32_t* pt, int64_t max_pages,
                     const int32_t* steps, int n_seqs, int n_q, int max_seq_len, float sm_scale, float* out, void* ws);
// the bound of the mbarrier waits in the tensor-memory and TMA kernels (ns; 0: default)
uint32_t wait_limit_ns();
// diagnostics: nonzero makes the TMA decode kernel withhold its first CTA's first copy
int withheld_copy();
// weighted sum of split partials (o[256], m, l rows of 260 floats) -> out, launched programmatically dependent
int launch_combine(const Launch& L, const float* ws, int splits, int n_seqs, int n_q, int H, float* out);
// the same for one query per sequence, a CTA per row: many rows of tens of splits
int launch_combine_rows(const Launch& L, const float* ws, int splits, int n_seqs, int H, float* out);
// the splits of a one-query decode merged into one unnormalised partial row per (sequence, query head)
int launch_combine_partial(const Launch& L, const float* ws, int splits, int n_seqs, int H, float* partial);
// gathered partials [n_parts][n_seqs][rows][260] -> out [n_seqs][rows][256]
int launch_combine_parts(const Launch& L, const float* parts, int n_parts, int n_seqs, int n_rows_per_seq,
                         float* out);
// decode with a shared prefix (k8v4_shared.cu): the first `cells` cells through the
// pair kernel, which writes partial rows [n_seqs][ws_splits][8 H][260], the first
// plan.splits of each sequence
struct SharedPlan {
  int cells = 0, splits = 0, tiles_per_split = 0;
  size_t acc_bytes = 0;      // running sums of the kernel's CTAs, behind the partial rows
};
bool shared_prefix_supported(const CacheView& C);
int shared_prefix_slots();   // CTA pairs at a time on the current device; 0 while the kernel's set-up fails
SharedPlan plan_shared(const CacheView& C, int n_seqs, int shared_len, int max_seq_len, int slots);
int launch_shared_prefix(const Launch& L, const CacheView& C, const SharedPlan& plan, const void* q, const int32_t* pt,
                         int64_t max_pages, const int32_t* lens, int n_seqs, int max_seq_len, float sm_scale, float* ws,
                         int ws_splits, float* acc, bool behind_splits);
// the cells from cell_begin on of every sequence as split partials (no merge):
// splits first_split .. of [n_seqs][ws_splits][8 H][260]; the plan is plan_decode
// over those cells
int launch_decode_splits(const Launch& L, const CacheView& C, const AttendPlan& plan, const void* q, int q_dtype,
                         const int32_t* pt, int64_t max_pages, const int32_t* steps, int n_seqs, int max_seq_len,
                         int cell_begin, float sm_scale, float* ws, int ws_splits, int first_split, uint32_t wait_ns);
// queries and keys: per-head RMS norm (weights may be null) and position rotation
int launch_norm_rope(const Launch& L, const void* q, int64_t q_stride, int n_q, const void* k, int64_t k_stride,
                     int n_k, int dtype, const float* q_weight, const float* k_weight, float eps, const int64_t* pos,
                     int n_seqs, int n_tok, const k8v4_rope& rope, void* q_out, void* k_out);
// the append with K normed (k_weight not null) and rotated on the way
int launch_append_rope(const Launch& L, const CacheView& C, const int32_t* pt, int64_t max_pages, int n_seqs,
                       const int64_t* pos, int n_tok, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                       int dtype, const float* k_weight, float eps, const k8v4_rope& rope);
// acceptance of drafted tokens
int launch_accept(const Launch& L, const void* p, const void* q, int dtype, const int32_t* drafts,
                  const int32_t* n_drafts, const float* u_accept, const float* u_sample, int n_seqs, int max_drafts,
                  int vocab, int32_t* tokens, int32_t* n_accepted);
int launch_prefill(const Launch& L, const CacheView& C, const void* q, const int32_t* pt, int64_t max_pages,
                   int seq_len, int n_q_tok, const int32_t* steps, float sm_scale, float* out);

}  // namespace k8v4
