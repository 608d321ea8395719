// Host-side launch functions of the calls of a ragged batch's step: page planning,
// appends through slots, differential attention and the norm between blocks.
#pragma once

#include <climits>

#include "k8v4_common.cuh"

namespace k8v4 {

struct PlanArgs {
  int P;
  int64_t n_pages;
  int32_t* free_pages;
  const int32_t* n_free;
  int32_t* pt;
  int64_t max_pages;
  const int32_t* lens;
  const int32_t* n_new;
  const int32_t* n_borrowed;   // or null
  int n_seqs, max_tokens;
  int32_t* offsets;
  int64_t* positions;
  int64_t* slots;
  int32_t* granted;
  int32_t* new_lens;
  int32_t* n_free_out;
};
constexpr int kPlanMaxSeqs = 8192;
int launch_plan(const Launch& L, const PlanArgs& a);

int launch_append_slots(const Launch& L, const CacheView& C, const int64_t* slots, int n_tok, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, int dtype);

// differential attention: one query per sequence, and a ragged batch
bool diff_supported(const CacheView& C);
// The longest length that the kernels take (a larger bound counts as this one): cell numbers, rounded up to a tile,
// stay within 31 bits
constexpr int kDiffMostCells = INT_MAX - 255;
size_t diff_decode_ws_bytes(const CacheView& C, int n_seqs, int num_sms);
int launch_diff_decode(const Launch& L, const CacheView& C, const void* q, int q_dtype, const int32_t* pt, int64_t max_pages,
                       const int32_t* lens, int n_seqs, int max_seq_len, float sm_scale, const k8v4_diff& diff, void* out,
                       void* ws);
size_t diff_ws_bytes(const CacheView& C, int n_seqs, int n_tok, int max_seq_len, int num_sms);
int launch_diff(const Launch& L, const CacheView& C, const void* q, int q_dtype, const int32_t* offsets, int n_tok,
                const int32_t* pt, int64_t max_pages, const int32_t* lens, const int32_t* steps, int n_seqs,
                int max_seq_len, float sm_scale, const k8v4_diff& diff, void* out, void* ws);

struct BlockNormArgs {
  const void* y;
  int64_t y_stride;
  int n_tok, dim;
  const float* post_weight;
  const void* gate;
  int64_t gate_stride;
  int gate_act;
  const void* residual;
  float residual_scale;
  const float* pre_weight;
  float eps;
  void* h_out;
  void* n_out;
};
constexpr int kBlockNormMaxDim = 32768;
int launch_block_norm(const Launch& L, const BlockNormArgs& a, int y_dtype, int dtype);

}  // namespace k8v4
