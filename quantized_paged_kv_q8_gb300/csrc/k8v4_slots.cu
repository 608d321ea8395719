// kv_append_k8v4_slots: the append of a ragged batch's packed tokens, each to the
// cell that its slot names (page * P + slot), with no table and no uniform count per
// sequence.  The rows go through the append's row quantisers: the same bytes.
//
// What bounds it: the instructions of a row (the exact rotation and quantisation of V,
// as in the plain append).  Long bf16 appends take the plain append's persistent
// structure: a warp steps through a contiguous run of (token, head) items with the next
// item's rows, and the next token's slot, loaded before it works on the current one.
// 40 tokens of 2 heads 4.3 us; 20,011 bf16 tokens 28.2 us for 57 MB, 74% of the issue slots.
#include <algorithm>

#include "k8v4_ops.cuh"
#include "k8v4_quant.cuh"

namespace k8v4 {
namespace {

constexpr int kWarps = 8;
constexpr int kBulkCtas = 3;      // resident CTAs per SM of the bulk kernel (85 registers a thread)

struct SlotsParams {
  CacheView C;
  const int64_t* slots;
  int n_tok;
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;     // elements between tokens
  FastDiv div_h, div_p;
  int* status;
};

// The cell of a slot: its page (null: nothing is written) and its place in it.  Slots
// from 2^31 on (caches of more cells than that) take a 64-bit division.
__device__ __forceinline__ uint8_t* cell_of(const SlotsParams& p, int64_t slot, int lane, int& cslot) {
  const CacheView& C = p.C;
  cslot = 0;
  if (slot == -1) return nullptr;
  const int64_t page = slot < 0 ? -1 : slot < (int64_t(1) << 31) ? p.div_p.div(static_cast<uint32_t>(slot)) : slot / C.P;
  if (page < 0 || page >= C.n_pages) {
    if (lane == 0) record_status(p.status, K8V4_ERANGE);
    return nullptr;
  }
  cslot = static_cast<int>(slot - page * C.P);
  return C.pages + page * C.page_bytes;
}

// Short appends and fp32 rows: a warp per (token, head), or, for short ones, a warp
// pair (K half, V half), as append_kernel.
template <bool BF16, int FMT>
__global__ void __launch_bounds__(kWarps * 32) append_slots_kernel(const SlotsParams p, int split_kv) {
  __shared__ __align__(16) long long stage[kWarps][kRotScratch];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const CacheView& C = p.C;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t wi = static_cast<int64_t>(blockIdx.x) * kWarps + w;
  const int64_t total = static_cast<int64_t>(p.n_tok) * C.H;
  if (wi >= (split_kv ? 2 * total : total)) return;
  const int role = split_kv ? static_cast<int>(wi & 1) : 2;             // 0: K only, 1: V only, 2: both
  const uint32_t item = static_cast<uint32_t>(split_kv ? wi >> 1 : wi);  // (token, head)
  const uint32_t tok = p.div_h.div(item);
  const int g = static_cast<int>(item - tok * static_cast<uint32_t>(C.H));
  int cslot;
  uint8_t* base = cell_of(p, p.slots[tok], lane, cslot);
  if (base == nullptr) return;
  const int64_t r = static_cast<int64_t>(cslot) * C.H + g;
  if (role != 1) append_k_row<BF16, FMT>(C, base, r, p.k, static_cast<int64_t>(tok) * p.k_stride + g * kD + 8 * lane, lane, stage[w]);
  __syncwarp();                                             // both may use the warp's scratch
  if (role != 0) append_v_row<BF16, FMT>(C, base, r, p.v, static_cast<int64_t>(tok) * p.v_stride + g * kD + 8 * lane, lane, stage[w]);
}

// Long appends of bf16 rows
template <int FMT>
__global__ void __launch_bounds__(kWarps * 32, kBulkCtas) append_slots_bf16_kernel(const SlotsParams p) {
  __shared__ __align__(16) long long stage[kWarps][kRotScratch];
  __shared__ float scale_tab[128];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const CacheView& C = p.C;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  long long* ts = stage[w];
  fill_int8_scale_table(scale_tab);
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t total = static_cast<uint32_t>(p.n_tok) * static_cast<uint32_t>(C.H);
  const uint32_t n_warps = gridDim.x * kWarps;
  const uint32_t per = (total + n_warps - 1) / n_warps;
  uint32_t item = (blockIdx.x * kWarps + w) * per;
  const uint32_t item_end = min(item + per, total);
  if (item >= item_end) return;
  uint32_t tok = p.div_h.div(item);
  int g = static_cast<int>(item - tok * static_cast<uint32_t>(C.H));
  const uint16_t* kp = static_cast<const uint16_t*>(p.k) + static_cast<int64_t>(tok) * p.k_stride + g * kD + 8 * lane;
  const uint16_t* vp = static_cast<const uint16_t*>(p.v) + static_cast<int64_t>(tok) * p.v_stride + g * kD + 8 * lane;
  const int64_t k_next = p.k_stride - (C.H - 1) * kD, v_next = p.v_stride - (C.H - 1) * kD;   // last head -> next token
  uint4 kr = __ldcs(reinterpret_cast<const uint4*>(kp)), vr = __ldcs(reinterpret_cast<const uint4*>(vp));
  const uint32_t n_tok = static_cast<uint32_t>(p.n_tok);
  int64_t slot_next = tok + 1 < n_tok ? p.slots[tok + 1] : -1;
  int cslot;
  uint8_t* base = cell_of(p, p.slots[tok], lane, cslot);
  for (; item < item_end; ++item) {
    const uint4 kc = kr, vc = vr;
    if (item + 1 < item_end) {
      const bool wrap = g + 1 == C.H;
      kp += wrap ? k_next : kD;
      vp += wrap ? v_next : kD;
      kr = __ldcs(reinterpret_cast<const uint4*>(kp));
      vr = __ldcs(reinterpret_cast<const uint4*>(vp));
    }
    if (base != nullptr) {
      const int r = cslot * C.H + g;
      if (FMT == K8V4_FORMAT_Q4) rot_q4_row_bf16(kc, lane, ts, base, nullptr, r * 128, C.ks_off() + r * 16);
      else int8_row_bf16(kc, lane, scale_tab, base, nullptr, r * 256, C.ks_off() + r * 8);
      if (FMT == K8V4_FORMAT_INT8) int8_row_bf16(vc, lane, scale_tab, base, nullptr, C.v_off() + r * 256, C.vs_off() + r * 8);
      else rot_q4_row_bf16(vc, lane, ts, base, nullptr, C.v_off() + r * 128, C.vs_off() + r * 16);
    }
    if (++g == C.H) {                                       // the next token
      g = 0;
      if (item + 1 < item_end) base = cell_of(p, slot_next, lane, cslot);
      ++tok;
      slot_next = tok + 1 < n_tok ? p.slots[tok + 1] : -1;
    }
  }
}

template <int FMT>
int launch_fmt(const Launch& L, const SlotsParams& p, bool bf, int split, int64_t items) {
  const dim3 block(kWarps * 32);
  if (bf && !split) {
    const int64_t want = (items + kWarps - 1) / kWarps;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(want, static_cast<int64_t>(L.num_sms) * kBulkCtas)));
    return launch_behind(L, append_slots_bf16_kernel<FMT>, grid, block, p);
  }
  const dim3 grid(static_cast<unsigned>(((split ? 2 : 1) * items + kWarps - 1) / kWarps));
  return launch_behind(L, bf ? append_slots_kernel<true, FMT> : append_slots_kernel<false, FMT>, grid, block, p, split);
}

}  // namespace

int launch_append_slots(const Launch& L, const CacheView& C, const int64_t* slots, int n_tok, const void* k,
                        int64_t k_stride, const void* v, int64_t v_stride, int dtype) {
  const int64_t items = static_cast<int64_t>(n_tok) * C.H;
  // K and V of an item by a warp each while all of those are resident at once (32 a SM),
  // as in the rotating append
  const int split = items * 2 <= static_cast<int64_t>(L.num_sms) * 32 ? 1 : 0;
  SlotsParams p;
  p.C = C;
  p.slots = slots;
  p.n_tok = n_tok;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.div_h = FastDiv(static_cast<uint32_t>(C.H));
  p.div_p = FastDiv(static_cast<uint32_t>(C.P));
  p.status = L.status;
  const bool bf = dtype == K8V4_BF16;
  if (C.fmt == K8V4_FORMAT_K8V4) return launch_fmt<K8V4_FORMAT_K8V4>(L, p, bf, split, items);
  if (C.fmt == K8V4_FORMAT_Q4) return launch_fmt<K8V4_FORMAT_Q4>(L, p, bf, split, items);
  return launch_fmt<K8V4_FORMAT_INT8>(L, p, bf, split, items);
}

}  // namespace k8v4
