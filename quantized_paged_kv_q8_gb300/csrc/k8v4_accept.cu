// spec_accept_k8v4: drafted tokens accepted or replaced from the target's
// probabilities and given random numbers, the step after attn_k8v4_verify.
//
// With drafts x_0 .. x_{n-1}, target rows p_0 .. p_n and draft rows q_0 .. q_{n-1}
// (or none: drafts that were certain, q = 1 at the draft), draft i is accepted
// while u_i q_i(x_i) < p_i(x_i).  At the first draft a that is not, the token
// comes from w = max(p_a - q_a, 0); after n accepted drafts, from w = p_n: the
// smallest j whose running sum of w passes u W, W the whole sum.  The accepted
// tokens then have exactly the target's distribution.
//
// The running sums decide between tokens, and two summation orders in fp32 differ
// by more than a token's probability in a large vocabulary; they are therefore
// kept as pairs of fp32 numbers with the additions' errors carried (about 46
// bits, far below the spacing of the random numbers).
//
// What bounds it: reading the two rows (2 x 4 B a vocabulary entry; 64 sequences of
// 262,144 entries: 134 MB in 26.6 us, 5.0 TB/s), and for few sequences the latency of
// three dependent steps (drafts' probabilities, sums, search; 5.2 us in all, one
// sequence of 32,768).  One cluster of eight CTAs per sequence splits the vocabulary, so one
// sequence alone keeps eight SMs loading; CTA totals meet in distributed shared
// memory, and only the CTA that holds the token reads its part (from L2) again.
#include <algorithm>
#include <type_traits>

#include "k8v4_common.cuh"

namespace k8v4 {
namespace {

constexpr int kCluster = 8;
constexpr int kAccThreads = 512;
constexpr int kAccWarps = kAccThreads / 32;
constexpr int kUnroll = 8;        // loads of a thread in flight
constexpr int kUnrollFew = 16;    // of few sequences over a large vocabulary (launch_accept)

struct AcceptParams {
  const void* p;             // [n_seqs][max_drafts + 1][vocab]
  const void* q;             // [n_seqs][max_drafts][vocab], or null
  const int32_t* drafts;     // [n_seqs][max_drafts]
  const int32_t* n_drafts;   // [n_seqs], or null
  const float* u_accept;     // [n_seqs][max_drafts]
  const float* u_sample;     // [n_seqs]
  int max_drafts, vocab;
  int32_t* tokens;           // [n_seqs][max_drafts + 1]
  int32_t* n_accepted;       // [n_seqs]
  int* status;
};

template <bool BF16>
__device__ __forceinline__ float prob(const void* base, int64_t i) {
  if (BF16) return __uint_as_float(static_cast<uint32_t>(__ldca(static_cast<const uint16_t*>(base) + i)) << 16);
  return __ldca(static_cast<const float*>(base) + i);
}

// four entries from an index that is a multiple of four, in rows that begin at one
template <bool BF16>
__device__ __forceinline__ float4 prob4(const void* base, int64_t i) {
  if (!BF16) return __ldca(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i));
  const uint2 w = __ldca(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

// A sum as hi + lo, |lo| small beside hi: about 46 bits, no fp64 instruction (that
// unit takes 16 clocks a warp instruction here, and every warp would queue for it)
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ void add(Pair& s, float x) {      // the addition's error goes to lo
  const float t = __fadd_rn(s.hi, x);
  const float b = __fsub_rn(t, s.hi);
  s.lo = __fadd_rn(s.lo, __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(x, b)));
  s.hi = t;
}
__device__ __forceinline__ void add(Pair& s, const Pair& x) {
  add(s, x.hi);
  s.lo = __fadd_rn(s.lo, x.lo);
}
__device__ __forceinline__ bool greater(const Pair& a, const Pair& b) {
  return __fadd_rn(__fsub_rn(a.hi, b.hi), __fsub_rn(a.lo, b.lo)) > 0.0f;
}
__device__ __forceinline__ Pair shfl_xor(const Pair& s, int o) {
  return Pair{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)};
}
// inclusive sum over the warp's lanes
__device__ __forceinline__ Pair scan_warp(Pair s, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y{__shfl_up_sync(0xffffffffu, s.hi, o), __shfl_up_sync(0xffffffffu, s.lo, o)};
    if (lane >= o) add(s, y);
  }
  return s;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// store v at the same shared address of CTA `rank` of the cluster
__device__ __forceinline__ void store_remote(Pair* local, int rank, const Pair& v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.hi), "f"(v.lo) : "memory");
}

template <bool BF16, int UNROLL, bool WIDE>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kAccThreads, UNROLL == kUnrollFew ? 2 : 4)
    accept_kernel(const AcceptParams a) {
  __shared__ __align__(8) Pair cta_total[2][kCluster];   // every CTA's sums (w, then p alone), written by each to all
  __shared__ Pair warp_total[kAccWarps], s_ahead;
  __shared__ int s_acc, s_hit, s_last;
  cluster_arrive();                            // waited for before the first store to another CTA
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % kCluster;
  const int64_t b = blockIdx.x / kCluster;
  const int n_max = a.max_drafts, V = a.vocab;
  int n = n_max;
  if (a.n_drafts) {
    n = a.n_drafts[b];
    if (n < 0 || n > n_max) {
      if (rank == 0 && tid == 0) record_status(a.status, K8V4_ERANGE);
      n = n < 0 ? 0 : n_max;
    }
  }
  // ---- the accepted drafts (warp 0 of every CTA, one lane per draft; n <= 32)
  int draft = -1;
  if (warp == 0) {
    bool ok = false;
    if (lane < n) {
      draft = a.drafts[b * n_max + lane];
      if (draft >= 0 && draft < V) {
        const float pt = prob<BF16>(a.p, (b * (n_max + 1) + lane) * V + draft);
        const float qt = a.q ? prob<BF16>(a.q, (b * n_max + lane) * V + draft) : 1.0f;
        // u q < p decided exactly: the product has 48 bits
        ok = static_cast<double>(a.u_accept[b * n_max + lane]) * qt < static_cast<double>(pt);
      } else if (rank == 0) {
        record_status(a.status, K8V4_ERANGE);              // no such token: not accepted
      }
    }
    const unsigned no = ~__ballot_sync(0xffffffffu, ok);
    const int acc = no ? min(__ffs(no) - 1, n) : n;
    if (lane == 0) s_acc = acc;
    const int tok_at = __shfl_sync(0xffffffffu, draft, min(acc, 31));
    if (lane == 0) s_last = acc < n ? tok_at : -1;
    if (rank == 0) {
      if (lane == 0) a.n_accepted[b] = acc;
      if (lane <= n_max && lane != acc) a.tokens[b * (n_max + 1) + lane] = lane < acc ? draft : -1;
      if (lane == 0 && n_max == 32 && acc != 32) a.tokens[b * (n_max + 1) + 32] = -1;
    }
  }
  __syncthreads();
  const int acc = s_acc, refused = s_last;
  const int64_t p_row = (b * (n_max + 1) + acc) * V;
  const bool rejected = acc < n;
  const int64_t q_row = (b * n_max + acc) * V;
  const bool has_q = rejected && a.q != nullptr;
  // the token's weight: max(p - q, 0), or p with the certain draft left out (with
  // `refused` outside the row: p).  fmaxf also turns a NaN into 0.  Two loops below
  // rather than a test per entry: with the test every entry's loads would wait for the
  // one before
  auto weight = [&](int64_t j, auto with_q, int left_out) -> float {
    const float w = prob<BF16>(a.p, p_row + j);
    if constexpr (decltype(with_q)::value) return fmaxf(__fsub_rn(w, prob<BF16>(a.q, q_row + j)), 0.0f);
    else return j == left_out ? 0.0f : fmaxf(w, 0.0f);
  };
  const std::true_type kWithQ{};
  const std::false_type kAlone{};
  // ---- sums: CTA `rank` owns kAccWarps runs of the vocabulary, a warp each
  const int per_warp = ((V + kCluster * kAccWarps - 1) / (kCluster * kAccWarps) + 3) & ~3;
  auto run_begin = [&](int w) {
    return static_cast<int>(min(static_cast<int64_t>(V), static_cast<int64_t>(rank * kAccWarps + w) * per_warp));
  };
  const int w0 = run_begin(warp), w1 = min(V, w0 + per_warp);
  bool residual = rejected;
  Pair total{0.0f, 0.0f}, before{0.0f, 0.0f};
  cluster_wait();
  for (int pass = 0; pass < 2; ++pass) {
    Pair s{0.0f, 0.0f};
    // UNROLL entries of a lane from j on: consecutive fours 128 apart (a quarter of the
    // load instructions), or single ones 32 apart; guard: only those ahead of w1
    auto add_chunk = [&](int j, auto with_q, auto guard, int left_out) {
      float x[UNROLL];
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < UNROLL; i += 4) {
          const int at = j + 32 * i;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (!decltype(guard)::value || at < w1) {
            v = prob4<BF16>(a.p, p_row + at);
            if constexpr (decltype(with_q)::value) {
              const float4 q = prob4<BF16>(a.q, q_row + at);
              v = make_float4(__fsub_rn(v.x, q.x), __fsub_rn(v.y, q.y), __fsub_rn(v.z, q.z), __fsub_rn(v.w, q.w));
            } else {
              if (at == (left_out & ~3)) {
                const int k = left_out & 3;
                v = make_float4(k == 0 ? 0.0f : v.x, k == 1 ? 0.0f : v.y, k == 2 ? 0.0f : v.z, k == 3 ? 0.0f : v.w);
              }
            }
          }
          x[i] = fmaxf(v.x, 0.0f);
          x[i + 1] = fmaxf(v.y, 0.0f);
          x[i + 2] = fmaxf(v.z, 0.0f);
          x[i + 3] = fmaxf(v.w, 0.0f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
          x[i] = !decltype(guard)::value || j + 32 * i < w1 ? weight(j + 32 * i, with_q, left_out) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < UNROLL; ++i) add(s, x[i]);
    };
    auto sum_run = [&](auto with_q, int left_out) {
      int j = w0 + (WIDE ? 4 * lane : lane);
      constexpr int kLast = 32 * (UNROLL - (WIDE ? 4 : 1));
      for (; j + kLast < w1; j += 32 * UNROLL) add_chunk(j, with_q, std::false_type{}, left_out);
      if (j < w1) add_chunk(j, with_q, std::true_type{}, left_out);
    };
    if (residual && has_q) sum_run(kWithQ, -1);
    else sum_run(kAlone, residual ? refused : -1);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) add(s, shfl_xor(s, o));
    if (lane == 0) warp_total[warp] = s;
    __syncthreads();
    if (tid < kCluster) {
      Pair c{0.0f, 0.0f};
      for (int i = 0; i < kAccWarps; ++i) add(c, warp_total[i]);
      store_remote(&cta_total[pass][rank], tid, c);
    }
    cluster_arrive();
    cluster_wait();
    total = before = Pair{0.0f, 0.0f};
    for (int i = 0; i < kCluster; ++i) {
      if (i == rank) before = total;
      add(total, cta_total[pass][i]);
    }
    // nothing left of p - q (the two rows equal): the target itself.  Every CTA
    // adds the same sums in the same order, so all take the same branch
    if (total.hi > 0.0f || !residual) break;
    residual = false;
  }
  int32_t* const token = a.tokens + b * (n_max + 1) + acc;
  if (!(total.hi > 0.0f) || total.hi == INFINITY) {          // a row with no weight, or not a distribution
    if (rank == 0 && tid == 0) {
      record_status(a.status, K8V4_ERANGE);
      *token = -1;
    }
    return;
  }
  // ---- the smallest j whose running sum passes T = u W
  float u = a.u_sample[b];
  u = u >= 0.0f ? fminf(u, 0x1.fffffep-1f) : 0.0f;          // NaN and below 0: 0; from 1 on: below 1
  // Sums below 2^40 are compared times 2^80 (both exact): a residual may be a few units of
  // 2^-149, of which the product with u, and the error that T.lo carries, keep no bit
  const float up = total.hi < 0x1p40f ? 0x1p80f : 1.0f;
  auto scaled = [&](const Pair& s) { return Pair{__fmul_rn(s.hi, up), __fmul_rn(s.lo, up)}; };
  const Pair W = scaled(total);
  Pair T;
  T.hi = __fmul_rn(u, W.hi);
  T.lo = __fadd_rn(__fmaf_rn(u, W.hi, -T.hi), __fmul_rn(u, W.lo));
  auto passes = [&](const Pair& s) { return greater(scaled(s), T); };
  // before + this CTA's sum is, bit for bit, the next CTA's `before`: the first
  // CTA whose end passes T is the one that holds the token (the last one if none)
  Pair after = before;
  add(after, cta_total[residual == rejected ? 0 : 1][rank]);
  if (passes(before) || (!passes(after) && rank != kCluster - 1)) return;
  // the warp run that holds T, and the sum ahead of it
  if (warp == 0) {
    Pair s = lane < kAccWarps ? warp_total[lane] : Pair{0.0f, 0.0f};
    const bool some = s.hi > 0.0f;
    s = scan_warp(s, lane);
    Pair end = before;
    add(end, s);
    const unsigned past = __ballot_sync(0xffffffffu, some && passes(end));
    const unsigned any = __ballot_sync(0xffffffffu, some);
    const int hit = past ? __ffs(past) - 1 : any ? 31 - __clz(any) : 0;
    const Pair prev{__shfl_sync(0xffffffffu, end.hi, max(hit - 1, 0)), __shfl_sync(0xffffffffu, end.lo, max(hit - 1, 0))};
    if (lane == 0) {
      s_hit = hit;
      s_last = -1;
      s_ahead = hit > 0 ? prev : before;
    }
  }
  __syncthreads();
  Pair ahead = s_ahead;
  const int r0 = run_begin(s_hit), r1 = min(V, r0 + per_warp);
  // all threads search that run, kPerThread consecutive entries each per round
  constexpr int kPerThread = 4;
  for (int j0 = r0; j0 < r1; j0 += kAccThreads * kPerThread) {
    const int j = j0 + kPerThread * tid;
    float x[kPerThread];
    Pair s{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (residual && has_q) x[i] = j + i < r1 ? weight(j + i, kWithQ, -1) : 0.0f;
      else x[i] = j + i < r1 ? weight(j + i, kAlone, residual ? refused : -1) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) add(s, x[i]);
    const Pair incl = scan_warp(s, lane);
    __syncthreads();                                         // the last round's totals and s_hit are read
    if (lane == 31) warp_total[warp] = incl;
    if (tid == 0) s_hit = 0x7fffffff;
    __syncthreads();
    // the sum ahead of this warp, of this thread, then entry by entry
    Pair wsum = scan_warp(lane < kAccWarps ? warp_total[lane] : Pair{0.0f, 0.0f}, lane);
    Pair run = ahead;
    const int pl = max(warp - 1, 0);
    const Pair wprev{__shfl_sync(0xffffffffu, wsum.hi, pl), __shfl_sync(0xffffffffu, wsum.lo, pl)};
    if (warp > 0) add(run, wprev);
    const Pair tprev{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
    if (lane > 0) add(run, tprev);
    int found = 0x7fffffff, last = -1;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      add(run, x[i]);
      if (x[i] > 0.0f) {
        last = j + i;
        if (found == 0x7fffffff && passes(run)) found = j + i;
      }
    }
    if (found != 0x7fffffff) atomicMin(&s_hit, found);
    if (last >= 0) atomicMax(&s_last, last);                 // in case rounding leaves T unpassed
    __syncthreads();
    if (s_hit != 0x7fffffff) {
      if (tid == 0) *token = s_hit;
      return;
    }
    const Pair all{__shfl_sync(0xffffffffu, wsum.hi, kAccWarps - 1), __shfl_sync(0xffffffffu, wsum.lo, kAccWarps - 1)};
    add(ahead, all);
  }
  if (tid == 0) *token = s_last;
}

}  // namespace

int launch_accept(const Launch& L, const void* p, const void* q, int dtype, const int32_t* drafts,
                  const int32_t* n_drafts, const float* u_accept, const float* u_sample, int n_seqs, int max_drafts,
                  int vocab, int32_t* tokens, int32_t* n_accepted) {
  AcceptParams a;
  a.p = p;
  a.q = q;
  a.drafts = drafts;
  a.n_drafts = n_drafts;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.max_drafts = max_drafts;
  a.vocab = vocab;
  a.tokens = tokens;
  a.n_accepted = n_accepted;
  a.status = L.status;
  const dim3 grid(static_cast<unsigned>(n_seqs) * kCluster), block(kAccThreads);
  const bool bf = dtype == K8V4_BF16;
  // Few CTAs (all at once with two per SM) whose threads have more than kUnroll entries:
  // twice the loads in flight per thread.  24 sequences of 262,144 entries 15.4 -> 11.1 us,
  // 38 17.9 -> 17.3 (8.7 either way at 32,768); 64 sequences would lose (24.3 -> 25.0:
  // four CTAs of fewer registers per SM read more at a time).  Of those, rows that are whole and
  // aligned groups of four entries are read by fours: 24 of 262,144 11.0 -> 10.0 us, 38 17.1 -> 15.3
  // (at 32 registers that form spills: 64 of 32,768 entries 8.8 -> 10.0, so the others stay single)
  if (static_cast<int64_t>(n_seqs) * kCluster <= 2 * L.num_sms && vocab > kCluster * kAccThreads * kUnroll) {
    const uintptr_t four = dtype == K8V4_BF16 ? 8 : 16;
    const bool wide = vocab % 4 == 0 && reinterpret_cast<uintptr_t>(p) % four == 0 && reinterpret_cast<uintptr_t>(q) % four == 0;
    if (bf) return launch_behind(L, wide ? accept_kernel<true, kUnrollFew, true> : accept_kernel<true, kUnrollFew, false>, grid, block, a);
    return launch_behind(L, wide ? accept_kernel<false, kUnrollFew, true> : accept_kernel<false, kUnrollFew, false>, grid, block, a);
  }
  return launch_behind(L, bf ? accept_kernel<true, kUnroll, false> : accept_kernel<false, kUnroll, false>, grid, block, a);
}

}  // namespace k8v4
