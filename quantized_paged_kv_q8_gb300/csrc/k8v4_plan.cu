// kv_plan_k8v4: the pages, block tables and slots of a step, from the sequences'
// lengths and requests, without a look at them on the host.
//
//   have_b = ceil(len_b / P),  need_b = ceil((len_b + new_b) / P) - have_b
//   stack' = stack ++ the pages of the finished sequences, in (sequence, entry) order
//   the k-th page handed out, counted over the sequences in order, is stack'[top - 1 - k];
//   a sequence gets its pages while its inclusive prefix of needs is at most top.
//
// The prefix of needs never falls, so once a sequence is refused every later one that
// needs a page is: those granted take a contiguous run from the top, and no decision waits
// for another.  Pages that are given back and handed out in the same call never pass
// through the stack's memory: the run read from it, [top - taken, n_free), and the run
// written to it, [n_free, top - taken), are disjoint (one of them is empty).
//
// What bounds it: latency and barriers (a few KB to a few MB move).  One launch: a cluster of eight
// CTAs, or one CTA for small steps.  Each CTA works the prefix sums of all sequences out for
// itself (three loads and 17 bytes of shared memory a sequence), and then takes its share
// of the tokens, handed-out pages and given-back pages as flat lists, finding each one's
// sequence by bisection.  The pages are handed out ahead of a barrier behind which the tokens read
// them from the table: a token that worked its page out again took a second bisection.
// 32 sequences with a token each 5.3 us; 600 sequences, 60 of them finished, 21,000
// tokens 16 us (19 with an item at a time; 59 in one CTA).
#include <algorithm>
#include <climits>

#include "k8v4_ops.cuh"

namespace k8v4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
constexpr int kRun = 4;                        // items of a long list that a thread has under way at a time
constexpr unsigned kFull = 0xffffffffu;

struct PlanParams {
  PlanArgs a;
  FastDiv div_p;
  int* status;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void set_remote(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  asm volatile("st.shared::cluster.u8 [%0], %1;" ::"r"(a), "r"(1u) : "memory");
}

// the sum of v over the threads ahead of this one, and over all of them
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* red, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();                                          // red may still be read
  if (lane == 31) red[warp] = s;
  __syncthreads();
  int64_t w = red[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kFull, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(kFull, w, 31);
  const int64_t ahead = __shfl_sync(kFull, w, max(warp - 1, 0));
  return s - v + (warp ? ahead : 0);
}

// the first of ends[0 .. n) (not decreasing) that is greater than v; n if none is
__device__ __forceinline__ int first_above(const int* ends, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > v) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// for the items 0 .. count of a flat list over the sequences (ends: inclusive prefixes), RUN at a time:
// each(items, their sequences), so that the chains of reads overlap.  A warp takes 32 RUN items in a row; in
// a long list the sequences of the first and the last bound the bisection of the others, most often to
// nothing.  Items behind the list come as -1.
template <int RUN, class F>
__device__ __forceinline__ void walk(const int* ends, int n, int count, int warp, int warps, F each) {
  const int lane = threadIdx.x & 31;
  for (int64_t c = warp; c * 32 * RUN < count; c += warps) {
    const int i0 = static_cast<int>(c * 32 * RUN), last = static_cast<int>(min(i0 + static_cast<int64_t>(32 * RUN), static_cast<int64_t>(count))) - 1;
    int from = 0, to = n;
    if (RUN > 1) {
      const int edge = first_above(ends, n, lane & 1 ? last : i0);
      from = __shfl_sync(kFull, edge, 0);
      to = __shfl_sync(kFull, edge, 1);
    }
    int item[RUN], b[RUN];
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      item[i] = last - i0 >= lane + 32 * i ? i0 + lane + 32 * i : -1;
      int lo = from, hi = item[i] < 0 ? from : to;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > item[i]) hi = mid;
        else lo = mid + 1;
      }
      b[i] = lo;
    }
    each(item, b);
  }
}

__global__ void __launch_bounds__(kThreads, 1) plan_kernel(const PlanParams p) {
  extern __shared__ int smem[];
  __shared__ int64_t red[32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PlanArgs& a = p.a;
  const int n = a.n_seqs, tid = threadIdx.x;
  const int rank = static_cast<int>(cluster_rank()), ctas = static_cast<int>(cluster_size());
  int* tok_end = smem;                                      // inclusive prefixes
  int* need_end = smem + n;
  int* back_end = smem + 2 * n;
  int* lens = smem + 3 * n;
  uint8_t* flag = reinterpret_cast<uint8_t*>(smem + 4 * n);  // bad finished row, then granted
  const int64_t cells_max = min(a.max_pages * a.P, static_cast<int64_t>(INT_MAX));      // new_lens holds no more
  const int flat = tid + kThreads * rank, stride = kThreads * ctas;
  auto pages_of = [&](int cells) -> int { return cells > 0 ? static_cast<int>(p.div_p.div(cells - 1u)) + 1 : 0; };
  auto len_ok = [&](int len) { return len >= 0 && len <= cells_max; };
  auto kept_of = [&](int b, int have) {                     // borrowed pages; -1: out of range
    const int k = a.n_borrowed ? a.n_borrowed[b] : 0;
    return k < 0 || k > have ? -1 : k;
  };
  int n_free = *a.n_free;
  if (n_free < 0 || n_free > a.n_pages) {
    if (flat == 0) record_status(p.status, K8V4_ERANGE);
    n_free = n_free < 0 ? 0 : static_cast<int>(a.n_pages);
  }

  const int warp = rank * (kThreads / 32) + (tid >> 5), warps = kThreads / 32 * ctas;
  const int per = (n + kThreads - 1) / kThreads;            // sequences of a thread, in a row
  const int b0 = min(n, tid * per), b1 = min(n, b0 + per);

  // ---- the rows of finished sequences: a page id out of range leaves the row alone
  int64_t backs = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = lens[b] = a.lens[b];
    flag[b] = 0;
    int bk = 0;
    if (a.n_new[b] == -1) {
      if (len_ok(len)) {
        const int have = pages_of(len), kept = kept_of(b, have);
        flag[b] = kept < 0;
        bk = kept < 0 ? 0 : have - kept;
        if (kept < 0) record_status(p.status, K8V4_ERANGE);
      }
    }
    backs += bk;
    back_end[b] = static_cast<int>(backs);
  }
  if (ctas > 1) cluster_arrive();                           // no flag is set remotely ahead of its zero
  const bool any_back = __syncthreads_or(backs > 0);        // the same in every CTA
  if (ctas > 1) cluster_wait();
  if (any_back) {
    int64_t all;
    const int ahead = static_cast<int>(block_scan(backs, red, &all));
    for (int b = b0; b < b1; ++b) back_end[b] += ahead;
    __syncthreads();
    auto check = [&](auto& item, auto& b) {
      constexpr int R = sizeof(item) / sizeof(int);
      int id[R];
#pragma unroll
      for (int i = 0; i < R; ++i) id[i] = item[i] < 0 ? 0 : a.pt[b[i] * a.max_pages + pages_of(lens[b[i]]) - (back_end[b[i]] - item[i])];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (id[i] >= 0 && id[i] < a.n_pages) continue;
        record_status(p.status, K8V4_ERANGE);
        for (int r = 0; r < ctas; ++r) set_remote(static_cast<uint32_t>(__cvta_generic_to_shared(flag + b[i])), r);
      }
    };
    if (all <= stride) walk<1>(back_end, n, static_cast<int>(all), warp, warps, check);
    else walk<kRun>(back_end, n, static_cast<int>(all), warp, warps, check);
    if (ctas > 1) cluster_barrier();
    else __syncthreads();
  }

  // ---- prefix sums over the sequences
  int64_t sum = 0, total;
  for (int b = b0; b < b1; ++b) sum += max(a.n_new[b], 0);
  int64_t at = block_scan(sum, red, &total);
  int need = 0, back = 0;
  bool bad = false, short_of = false;
  for (int b = b0; b < b1; ++b) {
    const int len = lens[b], want = a.n_new[b];
    const bool ok = len_ok(len);
    bad |= !ok || want < -1;
    at += max(want, 0);
    tok_end[b] = static_cast<int>(min(at, static_cast<int64_t>(INT_MAX)));
    int nd = 0, bk = 0, fits = 0;
    if (ok && want >= 0) {
      const int64_t len2 = static_cast<int64_t>(len) + want;
      bad |= len2 > cells_max;
      short_of |= at > a.max_tokens && want > 0;
      fits = len2 <= cells_max && (at <= a.max_tokens || want == 0);
      if (fits) nd = pages_of(static_cast<int>(len2)) - pages_of(len);
    } else if (ok && want == -1 && !flag[b]) {
      const int have = pages_of(len);
      bk = have - kept_of(b, have);
      fits = 2;                                             // given back
    }
    flag[b] = static_cast<uint8_t>(fits);
    need_end[b] = nd;
    back_end[b] = bk;
    need += nd;
    back += bk;
  }
  if (bad) record_status(p.status, K8V4_ERANGE);
  // needs and given-back pages are below n_seqs * max_pages < 2^31: one scan of both
  const int64_t both = block_scan(static_cast<int64_t>(need) << 32 | back, red, &total);
  int need_at = static_cast<int>(both >> 32), back_at = static_cast<int>(both & 0xffffffff);
  const int64_t top = n_free + (total & 0xffffffff);        // pages on the stack with those given back
  int taken = 0;
  for (int b = b0; b < b1; ++b) {
    const int nd = need_end[b];
    need_end[b] = need_at += nd;
    back_end[b] = back_at += back_end[b];
    if (flag[b] == 1 && nd > 0) {
      if (need_at <= top) taken = need_at;
      else flag[b] = 0, short_of = true;
    }
  }
  if (short_of) record_status(p.status, K8V4_ENOSPACE);
  __syncthreads();
  {
    const int w = __reduce_max_sync(kFull, taken);
    if ((tid & 31) == 0) red[tid >> 5] = w;
    __syncthreads();
    taken = __reduce_max_sync(kFull, static_cast<int>(red[tid & 31]));
  }

  // ---- the pages handed out and given back
  auto given = [&](int r) -> int {                          // the r-th page given back
    const int b = first_above(back_end, n, r);
    const int have = pages_of(lens[b]);
    return a.pt[b * a.max_pages + have - (back_end[b] - r)];
  };
  auto page_at = [&](int k) -> int {                        // the k-th page handed out
    const int64_t s = top - 1 - k;
    return s < n_free ? a.free_pages[s] : given(static_cast<int>(s - n_free));
  };
  auto need_of = [&](int b) { return need_end[b] - (b ? need_end[b - 1] : 0); };
  for (int k = flat; k < taken; k += stride) {
    const int b = first_above(need_end, n, k);
    const int col = pages_of(lens[b]) + k - (need_end[b] - need_of(b));
    const int id = page_at(k);
    if (id < 0 || id >= a.n_pages) record_status(p.status, K8V4_ERANGE);
    a.pt[b * a.max_pages + col] = id;
  }
  const int64_t left = top - taken;
  {
    const int count = static_cast<int>(max(left - n_free, static_cast<int64_t>(0)));
    auto put = [&](auto& item, auto& b) {
      constexpr int R = sizeof(item) / sizeof(int);
      int id[R];
#pragma unroll
      for (int i = 0; i < R; ++i) id[i] = item[i] < 0 ? 0 : a.pt[b[i] * a.max_pages + pages_of(lens[b[i]]) - (back_end[b[i]] - item[i])];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (item[i] < 0) continue;
        if (n_free + static_cast<int64_t>(item[i]) < a.n_pages) a.free_pages[n_free + static_cast<int64_t>(item[i])] = id[i];
        else record_status(p.status, K8V4_ERANGE);          // more pages than there are
      }
    };
    if (count <= stride) walk<1>(back_end, n, count, warp, warps, put);
    else walk<kRun>(back_end, n, count, warp, warps, put);
  }

  // ---- the tokens, once the pages are in the table
  if (ctas > 1) cluster_barrier();
  else __syncthreads();
  const int live = n ? min(tok_end[n - 1], a.max_tokens) : 0;
  auto place = [&](auto& item, auto& b) {
    constexpr int R = sizeof(item) / sizeof(int);
    int cell[R], j[R], id[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      cell[i] = -1;
      if (item[i] >= 0 && flag[b[i]] == 1) cell[i] = lens[b[i]] + (item[i] - (b[i] ? tok_end[b[i] - 1] : 0));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      id[i] = j[i] = 0;
      if (cell[i] < 0) continue;
      j[i] = static_cast<int>(p.div_p.div(static_cast<uint32_t>(cell[i])));
      id[i] = a.pt[b[i] * a.max_pages + j[i]];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (item[i] < 0) continue;
      int64_t slot = -1;
      if (cell[i] >= 0) {
        if (id[i] >= 0 && id[i] < a.n_pages) slot = static_cast<int64_t>(id[i]) * a.P + (cell[i] - j[i] * a.P);
        else record_status(p.status, K8V4_ERANGE);
      }
      a.positions[item[i]] = max(cell[i], 0);
      a.slots[item[i]] = slot;
    }
  };
  if (live <= stride) walk<1>(tok_end, n, live, warp, warps, place);
  else walk<kRun>(tok_end, n, live, warp, warps, place);
  for (int64_t t = live + static_cast<int64_t>(flat); t < a.max_tokens; t += stride) {
    a.positions[t] = 0;
    a.slots[t] = -1;
  }

  // ---- the sequences: every CTA has read what may be shared (new_lens may be seq_lens,
  // n_free_out n_free)
  for (int b = flat; b < n; b += stride) {
    const int len = lens[b], want = max(a.n_new[b], 0);
    a.offsets[b + 1] = min(tok_end[b], a.max_tokens);
    a.granted[b] = flag[b] == 1 ? want : 0;
    a.new_lens[b] = flag[b] == 1 ? len + want : flag[b] == 2 ? 0 : len;
  }
  if (flat == 0) {
    a.offsets[0] = 0;
    *a.n_free_out = static_cast<int>(min(left, a.n_pages));
  }
}

}  // namespace

int launch_plan(const Launch& L, const PlanArgs& a) {
  PlanParams p;
  p.a = a;
  p.div_p = FastDiv(static_cast<uint32_t>(a.P));
  p.status = L.status;
  const size_t smem = static_cast<size_t>(a.n_seqs) * 17;
  // (what a kernel has without asking, 48 KB, is for the 256 bytes of its own too)
  if (smem > 47 * 1024 &&
      cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanMaxSeqs * 17) != cudaSuccess)
    return K8V4_ECUDA;
  // one CTA where its threads have a few items each
  const unsigned ctas = a.max_tokens + 2 * static_cast<int64_t>(a.n_seqs) <= 4 * kThreads ? 1 : kCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, plan_kernel, p) != cudaSuccess) return K8V4_ECUDA;
  return cudaGetLastError() == cudaSuccess ? K8V4_OK : K8V4_ECUDA;
}

}  // namespace k8v4
