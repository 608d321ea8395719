// kv_append_k8v4_rope: the append with the position rotation (and the per-head
// key norm, when a weight is given) applied to K on the way into the cache.
//
// The bytes written are those of qk_norm_rope_k8v4 on K followed by
// kv_append_k8v4: the rotated row is rounded to K's type in registers and goes
// straight into the append's row quantisers, so the rotated keys are neither
// written to memory nor read back (1,024 B a cell each way in bf16).  K and V
// rows may be slices of a packed projection (a stride between tokens).
//
// What bounds it: the instructions of a row (the exact rotation and quantisation of
// V, as in the plain append, and the rotation of K with its errors carried), issued on
// 69% of the clocks while CTAs are resident; on the others the 24 warps of an SM wait
// for one another's fixed latencies or for loads.  No single unit is full.  The table
// row of a token is shared by its heads through L1.  Measured: 32,768 tokens of 2 heads
// in bf16, all 256 elements rotated: 64 us (127 MB, 2.0 TB/s), 46 for the plain append;
// 32 sequences of one token: 4.3 us.
#include <algorithm>

#include "k8v4_quant.cuh"
#include "k8v4_rope.cuh"

namespace k8v4 {
namespace {

constexpr int kWarps = 8;
constexpr int kBulkCtas = 3;      // resident CTAs per SM of the bulk kernel

struct AppendRopeParams {
  CacheView C;
  const int32_t* pt;
  int64_t max_pages;
  const int64_t* pos;
  int n_seqs, n_tok;
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;    // elements between tokens
  const float* k_weight;         // fp32 [256], or null
  float eps;
  const float* table;
  int64_t n_pos;
  int half;
  FastDiv div_h, div_tok, div_p;
  int* status;
};

// Short appends (a decode step's tokens) and fp32 rows: a warp per (token,
// head), or, for short ones, a warp pair (K half, V half), as append_kernel.
template <bool BF16, int FMT, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) append_rope_kernel(const AppendRopeParams p, int split_kv) {
  __shared__ __align__(16) long long stage[kWarps][kRotScratch];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const CacheView& C = p.C;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t wi = static_cast<int64_t>(blockIdx.x) * kWarps + w;
  const int64_t total = static_cast<int64_t>(p.n_seqs) * p.n_tok * C.H;
  if (wi >= (split_kv ? 2 * total : total)) return;
  const int role = split_kv ? static_cast<int>(wi & 1) : 2;             // 0: K only, 1: V only, 2: both
  const uint32_t item = static_cast<uint32_t>(split_kv ? wi >> 1 : wi);  // (seq, token, head)
  const uint32_t tok = p.div_h.div(item);
  const int g = static_cast<int>(item - tok * static_cast<uint32_t>(C.H));
  const uint32_t b = p.div_tok.div(tok);
  const int t = static_cast<int>(tok - b * static_cast<uint32_t>(p.n_tok));
  const int64_t cell = p.pos[b] + t;
  if (cell < 0 || cell >= p.max_pages * C.P || cell >= p.n_pos) {
    if (lane == 0) record_status(p.status, K8V4_ERANGE);
    return;
  }
  const uint32_t pidx = p.div_p.div(static_cast<uint32_t>(cell));
  const int cslot = static_cast<int>(static_cast<uint32_t>(cell) - pidx * static_cast<uint32_t>(C.P));
  const int64_t page = p.pt[static_cast<int64_t>(b) * p.max_pages + pidx];
  if (page < 0 || page >= C.n_pages) {
    if (lane == 0) record_status(p.status, K8V4_ERANGE);
    return;
  }
  uint8_t* base = C.pages + page * C.page_bytes;
  const int64_t r = static_cast<int64_t>(cslot) * C.H + g;
  long long* ts = stage[w];
  if (role != 1) {
    const RopeLane rl = rope_lane<INTER>(lane, p.half);
    RopeFactors<INTER> f;
    float x[8];
    load8<BF16>(p.k, static_cast<int64_t>(tok) * p.k_stride + g * kD + 8 * lane, x);
    rope_load<INTER>(p.table + cell * (2 * p.half), rl, p.half, f);
    if (p.k_weight) {
      float wt[8];
      load_weight8(p.k_weight, lane, wt);
      rms_row(x, wt, p.eps);
    }
    float o[8];
    rope_partners<INTER>(x, rl, o);
    if (p.k_weight) rope_row<INTER, false>(x, o, rl, f);
    else rope_row<INTER, true>(x, o, rl, f);
    if (BF16) bf16x8_to_f32(f32x8_to_bf16(x), x);           // rounded to K's type
    if (FMT == K8V4_FORMAT_Q4) {
      rotate_exact(x, lane, ts);
      quant_q4_store(x, lane, base, nullptr, r * 128, C.ks_off() + r * 16);
    } else {
      uint2 kc;
      const float s = quant_int8_half(x, kc);
      const float s_hi = __shfl_xor_sync(kQFull, s, 16);
      st2<uint2>(base, nullptr, r * 256 + 8 * lane, kc);
      if (lane == 0) st2(base, nullptr, C.ks_off() + r * 8, make_float2(s, s_hi));
    }
  }
  if (role != 0) {
    __syncwarp();
    append_v_row<BF16, FMT>(C, base, r, p.v, static_cast<int64_t>(tok) * p.v_stride + g * kD + 8 * lane, lane, ts);
  }
}

// Long appends of bf16 rows: the persistent structure of append_bf16_kernel (a
// warp steps through a contiguous run of (seq, token, head) items and loads the
// next item's K and V before it works on the current one).  The 16 cosines and
// sines of a lane are read when they are used (the next token's row is prefetched):
// held across the quantisers they leave room for two CTAs per SM only.
template <int FMT, bool INTER, bool NORM>
__global__ void __launch_bounds__(kWarps * 32, kBulkCtas) append_rope_bf16_kernel(const AppendRopeParams p) {
  __shared__ __align__(16) long long stage[kWarps][kRotScratch];
  __shared__ float scale_tab[128];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const CacheView& C = p.C;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long* ts = stage[w];
  fill_int8_scale_table(scale_tab);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t total = static_cast<uint32_t>(p.n_seqs) * static_cast<uint32_t>(p.n_tok) * static_cast<uint32_t>(C.H);
  const uint32_t n_warps = gridDim.x * kWarps;
  const uint32_t per = (total + n_warps - 1) / n_warps;
  uint32_t item = (blockIdx.x * kWarps + w) * per;
  const uint32_t item_end = min(item + per, total);
  if (item >= item_end) return;
  const uint32_t tok0 = p.div_h.div(item);
  int g = static_cast<int>(item - tok0 * static_cast<uint32_t>(C.H));
  uint32_t b = p.div_tok.div(tok0);
  int t = static_cast<int>(tok0 - b * static_cast<uint32_t>(p.n_tok));
  const int64_t cell_limit = min(p.max_pages * C.P, p.n_pos);
  int64_t cell = p.pos[b] + t;
  const uint16_t* kp = static_cast<const uint16_t*>(p.k) + static_cast<int64_t>(tok0) * p.k_stride + g * kD + 8 * lane;
  const uint16_t* vp = static_cast<const uint16_t*>(p.v) + static_cast<int64_t>(tok0) * p.v_stride + g * kD + 8 * lane;
  const int64_t k_next = p.k_stride - (C.H - 1) * kD, v_next = p.v_stride - (C.H - 1) * kD;   // last head -> next token
  const RopeLane rl = rope_lane<INTER>(lane, p.half);
  uint4 kr = __ldcs(reinterpret_cast<const uint4*>(kp)), vr = __ldcs(reinterpret_cast<const uint4*>(vp));
  auto prefetch_row = [&](int64_t c) {                   // the table row of a cell, towards L1
    if (rl.on && c >= 0 && c < cell_limit) {
      const float* row = p.table + c * (2 * p.half);
      if (INTER || lane * 8 < p.half) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + rl.at));
      if (INTER || lane * 8 >= p.half) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + p.half + rl.at));
    }
  };
  bool lookup = true;
  int cslot = 0;
  uint8_t* base = nullptr;
  for (; item < item_end; ++item) {
    const uint4 kc = kr, vc = vr;
    if (item + 1 < item_end) {
      const bool wrap = g + 1 == C.H;
      kp += wrap ? k_next : kD;
      vp += wrap ? v_next : kD;
      kr = __ldcs(reinterpret_cast<const uint4*>(kp));
      vr = __ldcs(reinterpret_cast<const uint4*>(vp));
    }
    const bool in_range = cell >= 0 && cell < cell_limit;
    if (in_range && lookup) {
      const uint32_t pidx = p.div_p.div(static_cast<uint32_t>(cell));
      cslot = static_cast<int>(static_cast<uint32_t>(cell) - pidx * static_cast<uint32_t>(C.P));
      const int64_t page = p.pt[static_cast<int64_t>(b) * p.max_pages + pidx];
      base = page >= 0 && page < C.n_pages ? C.pages + page * C.page_bytes : nullptr;
      lookup = false;
    }
    uint4 krot = kc;
    if (in_range) {
      float x[8];
      bf16x8_to_f32(kc, x);
      RopeFactors<INTER> f;
      rope_load<INTER>(p.table + cell * (2 * p.half), rl, p.half, f);
      if (NORM) {
        float wt[8];
        load_weight8(p.k_weight, lane, wt);
        rms_row(x, wt, p.eps);
      }
      float o[8];
      if (NORM) rope_partners<INTER>(x, rl, o);
      else rope_partners<INTER>(kc, rl, o);
      rope_row<INTER, !NORM>(x, o, rl, f);
      krot = f32x8_to_bf16(x);
    }
    const bool ok = in_range && base != nullptr;
    const int r = cslot * C.H + g;
    // the next item: head, then token (its cell), then sequence; its table row is
    // prefetched while this item is quantised
    if (++g == C.H) {
      g = 0;
      if (++t == p.n_tok) {
        t = 0;
        if (++b < static_cast<uint32_t>(p.n_seqs)) cell = p.pos[b];
        lookup = true;
      } else {
        ++cell;
        if (++cslot == C.P) lookup = true;
      }
      if (item + 1 < item_end) prefetch_row(cell);
    }
    if (!ok) {
      if (lane == 0) record_status(p.status, K8V4_ERANGE);
    } else {
      if (FMT == K8V4_FORMAT_Q4) rot_q4_row_bf16(krot, lane, ts, base, nullptr, r * 128, C.ks_off() + r * 16);
      else int8_row_bf16(krot, lane, scale_tab, base, nullptr, r * 256, C.ks_off() + r * 8);
      if (FMT == K8V4_FORMAT_INT8) int8_row_bf16(vc, lane, scale_tab, base, nullptr, C.v_off() + r * 256, C.vs_off() + r * 8);
      else rot_q4_row_bf16(vc, lane, ts, base, nullptr, C.v_off() + r * 128, C.vs_off() + r * 16);
    }
  }
}

template <int FMT, bool INTER>
int launch_fmt(const Launch& L, const AppendRopeParams& p, bool bf, int split, int64_t items) {
  const dim3 block(kWarps * 32);
  if (bf && !split) {
    const int64_t want = (items + kWarps - 1) / kWarps;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(L.num_sms) * kBulkCtas)));
    return launch_behind(L, p.k_weight ? append_rope_bf16_kernel<FMT, INTER, true> : append_rope_bf16_kernel<FMT, INTER, false>, grid, block, p);
  }
  const dim3 grid(static_cast<unsigned>(((split ? 2 : 1) * items + kWarps - 1) / kWarps));
  return launch_behind(L, bf ? append_rope_kernel<true, FMT, INTER> : append_rope_kernel<false, FMT, INTER>, grid, block, p, split);
}

}  // namespace

int launch_append_rope(const Launch& L, const CacheView& C, const int32_t* pt, int64_t max_pages, int n_seqs,
                       const int64_t* pos, int n_tok, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                       int dtype, const float* k_weight, float eps, const k8v4_rope& rope) {
  const int64_t items = static_cast<int64_t>(n_seqs) * n_tok * C.H;
  // K and V of an item by a warp each while all of those are resident at once (32 a SM):
  // 1,024 tokens of 2 heads take 5.9 us (fp32) and 5.8 (bf16) that way, 8.0 and 6.5 with a warp per
  // item; 1,536 tokens of 2 heads, where it would take two waves, 9.4 either way (bf16: 9.4 against 6.7)
  const int split = items * 2 <= static_cast<int64_t>(L.num_sms) * 32 ? 1 : 0;
  if ((split ? 2 : 1) * items >= (int64_t(1) << 31)) return K8V4_EINVAL;   // warp indices stay below 2^31
  AppendRopeParams p;
  p.C = C;
  p.pt = pt;
  p.max_pages = max_pages;
  p.pos = pos;
  p.n_seqs = n_seqs;
  p.n_tok = n_tok;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.k_weight = k_weight;
  p.eps = eps;
  p.table = rope.table;
  p.n_pos = rope.n_pos;
  p.half = rope.rot_dim / 2;
  p.div_h = FastDiv(static_cast<uint32_t>(C.H));
  p.div_tok = FastDiv(static_cast<uint32_t>(n_tok));
  p.div_p = FastDiv(static_cast<uint32_t>(C.P));
  p.status = L.status;
  const bool bf = dtype == K8V4_BF16;
  if (rope.interleaved) {
    if (C.fmt == K8V4_FORMAT_K8V4) return launch_fmt<K8V4_FORMAT_K8V4, true>(L, p, bf, split, items);
    if (C.fmt == K8V4_FORMAT_Q4) return launch_fmt<K8V4_FORMAT_Q4, true>(L, p, bf, split, items);
    return launch_fmt<K8V4_FORMAT_INT8, true>(L, p, bf, split, items);
  }
  if (C.fmt == K8V4_FORMAT_K8V4) return launch_fmt<K8V4_FORMAT_K8V4, false>(L, p, bf, split, items);
  if (C.fmt == K8V4_FORMAT_Q4) return launch_fmt<K8V4_FORMAT_Q4, false>(L, p, bf, split, items);
  return launch_fmt<K8V4_FORMAT_INT8, false>(L, p, bf, split, items);
}

}  // namespace k8v4
