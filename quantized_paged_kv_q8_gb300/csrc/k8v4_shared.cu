// Decode attention of a batch whose sequences share a prefix: the prefix part,
// scored once for all query rows on the 5th-generation tensor cores.
//
// The 8 n_seqs query rows of a KV head all see the same prefix cells, so their
// attention over it is a dense product with the cells read (and dequantised)
// once per 256 rows, where the per-sequence decode reads them once per sequence.
// The rows' partial results (o, m, l) go to the split combine together with those
// of each sequence's own cells.
//
// A CTA pair (tcgen05 cta_group::2, M = 256: 32 sequences x 8 heads, 128 rows
// per SM) sweeps a range of the prefix in tiles of 64 cells.  Per tile
//   S_h = Q_h K_h^T        two 128-lane halves (each has its own K scale), N = 64
//   P   = 2^(s - m) 2^7    online softmax in the log2 domain, two fp16 terms
//   O  += P1 V1 + P1 V2 + P2 V1    N = 256, V = (n - 8) d in two exact fp16 terms
// as in the chunked prefill, with these differences:
//  - each CTA of the pair dequantises half of every tile (32 of the 64 cells of K,
//    128 of the 256 dims of V): the pair reads both halves as one operand, so the
//    conversion and the shared-memory traffic per SM halve.  With one CTA per 128
//    rows the operand traffic alone (340 KB a tile at 128 B a clock) would take
//    longer than the products;
//  - warps have roles, handing over through mbarriers, so the tensor pipe, the
//    softmax and the conversion of neighbouring tiles overlap:
//      warps 0-7    rows: two threads per row (32 cells, and 128 of O's dims, each)
//      warps 8-11   conversion: global memory -> registers -> operand tiles
//      warp 12      (leader CTA) issues every product of the pair
//    The row warps hold O in fp32 registers (208 a thread, from the others' share);
//  - the reference maximum of a row moves only when a tile exceeds it by 2^8, and
//    then its O tile is rescaled in tensor memory, so the two CTAs need not agree;
//    every kChain tiles O is folded into the registers, in both CTAs at the same
//    tile, because the tensor core's accumulation is not rounded to nearest (2.9e-5
//    after 2,048 cells without the fold).
//
// Tensor memory (512 columns): S buffers [0,128), [128,256) (S0 | S1 each; the
// P terms overlay S0), O [256,512).  QK(i+2) overwrites P(i): its S1 half, which
// P does not touch, is issued behind PV(i) at once, its S0 half when PV(i) is done.
//
// Every mbarrier wait is bounded: on timeout the warp raises the CTA's failure
// word and leaves its loop (the row warps together, at their next vote); the
// kernel records an error, waits for its own products (bounded), frees its tensor
// memory and returns.
#include <algorithm>

#include "k8v4_tc.cuh"

namespace k8v4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPStride = 260;               // floats per partial row: o[256], m, l, 2 pad
constexpr int kRows = 128;                  // query rows per CTA (256 per pair)
constexpr int kPairSeqs = 2 * kRows / kGqa; // 32
constexpr int kTileN = 64;
constexpr int kThreads = 512;
constexpr int kRowThreads = 256, kConvWarp0 = 8, kIssueWarp = 12;
constexpr int kChain = 8;                   // tiles accumulated in one TMEM O tile
constexpr float kSlack = 8.0f;              // log2 headroom of P above its row's reference maximum
constexpr uint32_t kWaitDefaultNs = 1000000000u;
// registers per thread after the split; 2 * 208 + 72 + 24 = 4 * 128, what the block launches with
constexpr int kRowRegs = 208, kConvRegs = 72, kIssueRegs = 24;
static_assert(2 * kRowRegs + kConvRegs + kIssueRegs <= 4 * 128, "register split");

// shared memory (bytes); operand tiles 1024-byte aligned, the same in both CTAs
constexpr int kQOff = 0;                              // Q fp16 [4 chunks][128 rows][128 B]
constexpr int kKOff = kQOff + 65536;                  // K fp16, 2 buffers x [4 chunks][32 cells][128 B]
constexpr int kKBuf = 16384;
constexpr int kVOff = kKOff + 2 * kKBuf;              // V fp16, 2 buffers x 2 planes x [2 atoms][64 cells][128 B]
constexpr int kVPlane = 16384, kVBuf = 2 * kVPlane;
constexpr int kKsOff = kVOff + 2 * kVBuf;             // K scales, 4 tiles x [64][2] f32
constexpr int kRedOff = kKsOff + 4 * 512;             // [2][128] f32 exchange, [128] score factors
constexpr int kBarOff = kRedOff + 2 * 512 + 512;
constexpr int kCtlOff = kBarOff + 128;                // tmem slot, failure word, largest visible count, bad tiles
constexpr int kSmemBytes = kCtlOff + 64;
// the epilogue reuses the operand tiles as a fp32 [128][256] row buffer
static_assert(kKsOff - kQOff >= kRows * 256 * 4, "row buffer");
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// mbarriers, at kBarOff + 8 * index
enum { kBarKFull = 0, kBarVFull = 2, kBarPFull = 4, kBarSFull = 6, kBarODone = 8, kBarKsFull = 10, kBarDrain = 14 };

constexpr uint32_t kTmemCols = 512, kSBuf = 128, kS1Col = 64, kOCol = 256, kP2Col = 32;

struct SharedParams {
  CacheView C;
  const uint16_t* q;        // bf16 [n_seqs][HQ][256]
  const int32_t* pt;        // the first sequence's page table
  int64_t max_pages;
  const int32_t* lens;      // [n_seqs]
  int n_seqs, max_seq_len;
  int cells;                // prefix cells, a multiple of 16
  int splits, tiles_per_split;
  int ws_splits;            // partial rows per sequence in ws (this kernel writes the first `splits`)
  float sm_scale_log2;
  float* ws;
  int* status;
  uint32_t wait_ns;
  FastDiv page_div;
};

// ---------------------------------------------------------------- pair PTX
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void arrive_local(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_cluster(uint32_t bar, uint32_t parity, uint32_t sleep_ns) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(sleep_ns)
      : "memory");
  return done != 0;
}
// as mbar_wait, acquiring from both CTAs of the pair
__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity, uint32_t limit_ns) {
  if (try_cluster(bar, parity, 0)) return true;
  if (limit_ns < 1000u) return false;
  const uint64_t t0 = global_ns();
  for (;;) {
    if (global_ns() - t0 >= limit_ns) return false;
    if (try_cluster(bar, parity, 20000u)) return true;
  }
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_pair_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// completion of this thread's products so far -> the barrier at this offset of both CTAs
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  const uint16_t both = 3;
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(both)
      : "memory");
}
// a barrier over the row warps that also ORs a predicate
__device__ __forceinline__ bool rows_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void rows_barrier() { asm volatile("barrier.cta.sync 2, 256;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld8x2(uint32_t ta, uint32_t tb, float a[8], float b[8]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(r[8 + i]);
  }
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float v[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// ---------------------------------------------------------------- the kernel
// grid: x = 2 * (split * groups + group), y = KV head; clusters of two along x.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) shared_prefix_kernel(const SharedParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int g = blockIdx.y;
  const int groups = (p.n_seqs + kPairSeqs - 1) / kPairSeqs;
  const int unit = blockIdx.x >> 1;
  const int split = unit / groups;
  const int seq0 = (unit - split * groups) * kPairSeqs + static_cast<int>(rank) * (kRows / kGqa);   // this CTA's first sequence
  const CacheView& C = p.C;
  const int HQ = C.H * kGqa;
  const int row = tid & (kRows - 1), part = tid >> 7;
  const uint32_t bars = sb + kBarOff;
  volatile int* ctl = reinterpret_cast<volatile int*>(smem + kCtlOff);   // [0] tmem, [1] failed, [4..7] bad groups of 4 tiles
  float* red = reinterpret_cast<float*>(smem + kRedOff);                 // [2][128]
  float* fsc = red + 2 * kRows;                                          // [128]
  float* ksbuf = reinterpret_cast<float*>(smem + kKsOff);

  const int tile0 = split * p.tiles_per_split;
  const int n_tiles = min(p.tiles_per_split, (p.cells + kTileN - 1) / kTileN - tile0);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + 8 * (kBarKFull + i), 8);       // 4 conversion warps of both CTAs
      mbar_init(bars + 8 * (kBarVFull + i), 8);
      mbar_init(bars + 8 * (kBarPFull + i), 16);      // 8 row warps of both CTAs
      mbar_init(bars + 8 * (kBarSFull + i), 1);
      mbar_init(bars + 8 * (kBarODone + i), 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(bars + 8 * (kBarKsFull + i), 4);
    mbar_init(bars + 8 * kBarDrain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    ctl[1] = 0;
    for (int i = 4; i < 8; ++i) ctl[i] = 0;
  }
  if (warp == kIssueWarp) tmem_alloc_pair(sb + kCtlOff, kTmemCols);

  // ---- visibility of this thread's row
  int my_vis = 0;
  {
    const int s = seq0 + row / kGqa;
    if (s < p.n_seqs) {
      int v = p.lens[s];
      if (v < 0 || v > p.max_seq_len) {
        if (part == 0) record_status(p.status, K8V4_ERANGE);
        v = v < 0 ? 0 : p.max_seq_len;
      }
      my_vis = min(v, p.cells);
    }
  }
  // ---- Q rows -> fp16 with a per-row power-of-two scale, swizzled K-major; the
  // four parts of a row take dims [64 part, 64 part + 64)
  {
    const int s = seq0 + row / kGqa, h = row % kGqa;
    uint4 raw[8];
    if (s < p.n_seqs) {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(s) * HQ + g * kGqa + h) * kD + 64 * part);
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = src[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = make_uint4(0, 0, 0, 0);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        amax = fmaxf(amax, fabsf(__uint_as_float(w[u] << 16)));
        amax = fmaxf(amax, fabsf(__uint_as_float(w[u] & 0xffff0000u)));
      }
    }
    float* qmax = ksbuf;                                // [4][128]: the scale buffers are not in use yet
    qmax[part * kRows + row] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(qmax[row], qmax[kRows + row]), fmaxf(qmax[2 * kRows + row], qmax[3 * kRows + row]));
    const int ex = amax > 0.0f ? static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu) - 127 : 0;
    const int sh = max(-100, min(100, 14 - ex));
    const float up = ldexpf(1.0f, sh);
    if (part == 0) fsc[row] = p.sm_scale_log2 * ldexpf(1.0f, -sh);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t hv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const __half2 h2 = __floats2half2_rn(__fmul_rn(__uint_as_float(w[u] << 16), up),
                                             __fmul_rn(__uint_as_float(w[u] & 0xffff0000u), up));
        hv[u] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      sts128(sb + kQOff + part * 16384 + swz(row, i), hv[0], hv[1], hv[2], hv[3]);
    }
  }
  asm volatile("fence.proxy.async;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_barrier();          // barriers, tensor memory and Q of both CTAs are ready
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(ctl[0]);

  if (warp < 8) {
    // ================================================================ rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    const int half = part;                                 // cells [32 half, +32) of a tile, dims [128 half, +128) of O
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float my_f = fsc[row];
    const uint32_t p_full0 = map_to(bars + 8 * kBarPFull, 0);
    float o_run[128];
#pragma unroll
    for (int i = 0; i < 128; ++i) o_run[i] = 0.0f;
    float m_run = -INFINITY, l_part = 0.0f;
    bool failed = false;
    const uint32_t o_tile = tmem + lane_base + kOCol + 128 * half;
    auto fold = [&](float a) {                             // o_run = (o_run + O tile) * a
      const float2 a2 = make_float2(a, a);
#pragma unroll
      for (int h = 0; h < 16; ++h) {
        float o[8];
        tmem_ld8(o_tile + 8 * h, o);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 r = __fmul2_rn(__fadd2_rn(make_float2(o_run[8 * h + i], o_run[8 * h + i + 1]),
                                                 make_float2(o[i], o[i + 1])), a2);
          o_run[8 * h + i] = r.x;
          o_run[8 * h + i + 1] = r.y;
        }
      }
    };
    auto rescale = [&](float a) {                          // O tile *= a, o_run *= a
#pragma unroll
      for (int h = 0; h < 16; ++h) {
        float o[8];
        tmem_ld8(o_tile + 8 * h, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i] *= a;
          o_run[8 * h + i] *= a;
        }
        tmem_st8(o_tile + 8 * h, o);
      }
    };
    for (int i = 0; i < n_tiles; ++i) {
      const int buf = i & 1;
      const uint32_t parity = (i >> 1) & 1;
      if (!wait_pair(bars + 8 * (kBarSFull + buf), parity, p.wait_ns) ||
          !mbar_wait(bars + 8 * (kBarKsFull + (i & 3)), (i >> 2) & 1, p.wait_ns)) {
        failed = true;
        ctl[1] = 1;
      }
      tc_fence_after();
      const uint32_t sbase = tmem + lane_base + kSBuf * buf + 32 * half;
      const float* ks = ksbuf + 128 * (i & 3) + 64 * half;
      float sc[32];
      float mx = -INFINITY;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float a[8], b[8];
        tmem_ld8x2(sbase + 8 * h, sbase + kS1Col + 8 * h, a, b);
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          const float4 k2 = *reinterpret_cast<const float4*>(ks + 16 * h + 2 * c);
          sc[8 * h + c] = k2.x * a[c] + k2.y * b[c];
          sc[8 * h + c + 1] = k2.z * a[c + 1] + k2.w * b[c + 1];
        }
      }
      const int vis = my_vis - (tile0 + i) * kTileN - 32 * half;       // cells [0, vis) of this half
      const int bad = ctl[4 + (i & 3)];                                // 16-cell groups on a page out of range
      if (vis < 32 || bad) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c >= vis || ((bad >> (8 * half + (c >> 4))) & 1)) sc[c] = -INFINITY;
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) mx = fmaxf(mx, sc[c]);
      const float top = mx * my_f;
      tc_fence_before();
      // every thread's scores are in registers past this vote, so P may overlay S
      const bool any = rows_any(failed || top > m_run + kSlack);
      tc_fence_after();
      float alpha = 1.0f;
      if (any) {
        red[half * kRows + row] = top;
        // the row warps leave together: the failure word is read once, ahead of a vote
        if (rows_any(failed || ctl[1] != 0)) { failed = true; break; }
        const float mt = fmaxf(red[row], red[kRows + row]);
        if (mt > m_run + kSlack) {
          alpha = exp2f(m_run - mt);                                   // 0 on the first visible tile
          m_run = mt;
          l_part *= alpha;
        }
      }
      const bool folds = i > 0 && i % kChain == 0;
      if (i > 0 && (folds || any)) {
        if (folds || __any_sync(kFull, alpha != 1.0f)) {
          if (!wait_pair(bars + 8 * (kBarODone + (buf ^ 1)), ((i - 1) >> 1) & 1, p.wait_ns)) {
            failed = true;
            ctl[1] = 1;
          }
          tc_fence_after();
          if (folds) fold(alpha);
          else rescale(alpha);
        }
      }
      const float mu = (m_run == -INFINITY ? 0.0f : m_run) - 7.0f;
      float2 psum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float p1[8], p2[8];
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          const float a = ex2_ftz(fmaf(sc[16 * h + c], my_f, -mu)), b = ex2_ftz(fmaf(sc[16 * h + c + 1], my_f, -mu));
          const __half2 h1 = __floats2half2_rn(a, b);
          const float2 f1 = __half22float2(h1);
          const float2 r = __ffma2_rn(f1, make_float2(-1.0f, -1.0f), make_float2(a, b));   // exact
          const __half2 h2 = __floats2half2_rn(r.x, r.y);
          psum = __fadd2_rn(psum, make_float2(a, b));
          p1[c >> 1] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h1));
          p2[c >> 1] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h2));
        }
        const uint32_t pb = tmem + lane_base + kSBuf * buf + 16 * half + 8 * h;
        tmem_st8(pb, p1);
        tmem_st8(pb + kP2Col, p2);
      }
      l_part += psum.x + psum.y;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(p_full0 + 8 * buf);
    }
    // ---- the last O tile, then o / m / l of the rows
    if (!failed && n_tiles > 0) {
      if (wait_pair(bars + 8 * (kBarODone + ((n_tiles - 1) & 1)), ((n_tiles - 1) >> 1) & 1, p.wait_ns)) {
        tc_fence_after();
        fold(1.0f);
        tc_fence_before();
      } else {
        failed = true;
        ctl[1] = 1;
      }
    }
    // PV of the last tile is done in both CTAs (one commit covers the pair), and
    // with it every read of this CTA's operand tiles
    red[half * kRows + row] = l_part;
    const bool stop = rows_any(failed);
    if (!stop) {
      const float l = red[row] + red[kRows + row];
      float* rowbuf = reinterpret_cast<float*>(smem + kQOff);          // [128][256] fp32, rotated by 4 * row
#pragma unroll
      for (int i = 0; i < 128; i += 4) {
        const int d = 128 * half + i;
        *reinterpret_cast<float4*>(rowbuf + row * 256 + ((d + 4 * row) & 255)) =
            make_float4(o_run[i], o_run[i + 1], o_run[i + 2], o_run[i + 3]);
      }
      if (half == 0) {
        const int s = seq0 + row / kGqa;
        if (s < p.n_seqs) {
          float* dst = p.ws + ((static_cast<int64_t>(s) * p.ws_splits + split) * HQ + g * kGqa + row % kGqa) * kPStride;
          dst[256] = m_run - 7.0f;                                     // o and l are relative to 2^(m - 7)
          dst[257] = l;
        }
      }
      rows_barrier();
      for (int r = warp; r < kRows; r += 8) {
        const int s = seq0 + r / kGqa;
        if (s >= p.n_seqs) break;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 x = *reinterpret_cast<const float4*>(rowbuf + r * 256 + ((8 * lane + e + 4 * r) & 255));
          v[e] = x.x; v[e + 1] = x.y; v[e + 2] = x.z; v[e + 3] = x.w;
        }
#pragma unroll
        for (int hh = 1; hh < 8; hh <<= 1) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (e & hh) continue;
            const float a = v[e], b = v[e + hh];
            v[e] = a + b;
            v[e + hh] = a - b;
          }
        }
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const bool upper = (lane & m) != 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = __shfl_xor_sync(kFull, v[e], m);
            v[e] = upper ? x - v[e] : v[e] + x;
          }
        }
        float* dst = p.ws + ((static_cast<int64_t>(s) * p.ws_splits + split) * HQ + g * kGqa + r % kGqa) * kPStride + 8 * lane;
        reinterpret_cast<float4*>(dst)[0] = make_float4(v[0] * 0.0625f, v[1] * 0.0625f, v[2] * 0.0625f, v[3] * 0.0625f);
        reinterpret_cast<float4*>(dst)[1] = make_float4(v[4] * 0.0625f, v[5] * 0.0625f, v[6] * 0.0625f, v[7] * 0.0625f);
      }
    }
  } else if (warp < kIssueWarp) {
    // ================================================================ conversion
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    const int t = tid - 32 * kConvWarp0;                   // 0..127
    const int cw = t >> 5;
    // K: cell 32 rank + lane, dims [64 cw, +64); V: cell t & 63, blocks 4 rank + 2 (t >> 6) + {0, 1}
    const int kcell = 32 * static_cast<int>(rank) + lane, vcell = t & 63, vblk = 4 * static_cast<int>(rank) + 2 * (t >> 6);
    const uint32_t k_full0 = map_to(bars + 8 * kBarKFull, 0), v_full0 = map_to(bars + 8 * kBarVFull, 0);
    auto page_of = [&](int i, int cell) -> int {           // page id of a cell of tile i, -1 past the prefix, -2 if out of range
      const int c = (tile0 + i) * kTileN + cell;
      if (i >= n_tiles || c >= p.cells) return -1;
      const int64_t pidx = p.page_div.div(static_cast<uint32_t>(c));
      const int page = pidx < p.max_pages ? p.pt[pidx] : -2;
      return page >= 0 && page < C.n_pages ? page : -2;
    };
    auto slot_of = [&](int i, int cell) -> int {
      const int c = (tile0 + i) * kTileN + cell;
      return c - static_cast<int>(p.page_div.div(static_cast<uint32_t>(c))) * C.P;
    };
    uint4 kraw[4], vraw[2];
    uint32_t vd;
    float2 ksc;
    int kpage = page_of(0, kcell), vpage = page_of(0, vcell);
    bool kbad = false;                                     // (threads of the first two conversion warps) this cell's page
    auto load_k = [&](int i) {                             // K codes; the scales of cell vcell come with V's page
      if (kpage >= 0) {
        const uint8_t* src = C.pages + static_cast<int64_t>(kpage) * C.page_bytes +
                             (static_cast<int64_t>(slot_of(i, kcell)) * C.H + g) * 256 + 64 * cw;
#pragma unroll
        for (int u = 0; u < 4; ++u) kraw[u] = __ldg(reinterpret_cast<const uint4*>(src) + u);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) kraw[u] = make_uint4(0, 0, 0, 0);
      }
      kpage = page_of(i + 1, kcell);
    };
    auto load_v = [&](int i) {
      kbad = vpage == -2;
      ksc = make_float2(0.0f, 0.0f);
      if (vpage >= 0) {
        const int64_t r = static_cast<int64_t>(slot_of(i, vcell)) * C.H + g;
        const uint8_t* base = C.pages + static_cast<int64_t>(vpage) * C.page_bytes;
        const uint4* src = reinterpret_cast<const uint4*>(base + C.v_off() + r * 128 + 16 * vblk);
        vraw[0] = __ldg(src);
        vraw[1] = __ldg(src + 1);
        vd = __ldg(reinterpret_cast<const uint32_t*>(base + C.vs_off() + r * 16 + 2 * vblk));
        if (t < 64) ksc = __ldg(reinterpret_cast<const float2*>(base + C.ks_off() + r * 8));
      } else {
        vraw[0] = vraw[1] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
        vd = 0;
      }
      vpage = page_of(i + 1, vcell);
    };
    load_k(0);
    load_v(0);
    for (int i = 0; i < n_tiles; ++i) {
      const int buf = i & 1;
      const uint32_t last = ((i - 2) >> 1) & 1;            // phase of tile i - 2 on the buffers' barriers
      // ---- K(i) and its scales, once QK(i - 2) has read the buffer
      if (i >= 2 && !wait_pair(bars + 8 * (kBarSFull + buf), last, p.wait_ns)) { ctl[1] = 1; break; }
      {
        const uint32_t dst = sb + kKOff + buf * kKBuf + cw * 4096;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t h[8];
          i8x4_to_f16(kraw[u].x, h[0], h[1]);
          i8x4_to_f16(kraw[u].y, h[2], h[3]);
          i8x4_to_f16(kraw[u].z, h[4], h[5]);
          i8x4_to_f16(kraw[u].w, h[6], h[7]);
          sts128(dst + swz(lane, 2 * u), h[0], h[1], h[2], h[3]);
          sts128(dst + swz(lane, 2 * u + 1), h[4], h[5], h[6], h[7]);
        }
        if (t < 64) {
          reinterpret_cast<float2*>(ksbuf + 128 * (i & 3))[t] = ksc;
          const unsigned b = __ballot_sync(kFull, kbad);   // lanes 0 and 16 stand for their 16-cell groups
          if (b && lane == 0) record_status(p.status, K8V4_ERANGE);
          if (lane == 0) reinterpret_cast<volatile uint8_t*>(smem + kCtlOff + 16)[4 * (i & 3) + cw] =
              static_cast<uint8_t>((b & 1u) | ((b >> 15) & 2u));
        }
        asm volatile("fence.proxy.async;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          arrive_local(bars + 8 * (kBarKsFull + (i & 3)));
          arrive_cluster(k_full0 + 8 * buf);
        }
      }
      if (i + 1 < n_tiles) load_k(i + 1);
      // ---- V(i), once PV(i - 2) has read the buffer
      if (i >= 2 && !wait_pair(bars + 8 * (kBarODone + buf), last, p.wait_ns)) { ctl[1] = 1; break; }
      {
        const uint32_t dst = sb + kVOff + buf * kVBuf + (t >> 6) * 8192;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          const __half dh = __ushort_as_half(static_cast<unsigned short>(vd >> (16 * blk)));
          const __half2 d2 = __halves2half2(dh, dh);
          const uint32_t ws4[4] = {vraw[blk].x, vraw[blk].y, vraw[blk].z, vraw[blk].w};
#pragma unroll
          for (int hn = 0; hn < 2; ++hn) {                 // low nibbles: dims 0..15 of the block, high: 16..31
            uint32_t v1[8], v2[8];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              nib_vhat(prmt(ws4[q], 0u, 0x5140u), 4 * hn, d2, v1[2 * q], v2[2 * q]);
              nib_vhat(prmt(ws4[q], 0u, 0x5342u), 4 * hn, d2, v1[2 * q + 1], v2[2 * q + 1]);
            }
            const int u0 = 4 * blk + 2 * hn;
            sts128(dst + swz(vcell, u0), v1[0], v1[1], v1[2], v1[3]);
            sts128(dst + swz(vcell, u0 + 1), v1[4], v1[5], v1[6], v1[7]);
            sts128(dst + kVPlane + swz(vcell, u0), v2[0], v2[1], v2[2], v2[3]);
            sts128(dst + kVPlane + swz(vcell, u0 + 1), v2[4], v2[5], v2[6], v2[7]);
          }
        }
        asm volatile("fence.proxy.async;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_cluster(v_full0 + 8 * buf);
      }
      if (i + 1 < n_tiles) load_v(i + 1);
    }
  } else {
    // ================================================================ issue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == kIssueWarp && rank == 0 && lane == 0) {
      constexpr uint32_t idS = idesc_f16(256, 64, false, false);
      constexpr uint32_t idO = idesc_f16(256, 256, false, true);
      const uint64_t dq0 = smem_desc(sb + kQOff, 16, 1024);
      const uint64_t dk0 = smem_desc(sb + kKOff, 16, 1024);
      const uint64_t dv0 = smem_desc(sb + kVOff, 8192, 1024);
      auto qk_half = [&](int buf, int h) {                 // S[buf]_h = Q_h K_h^T
        uint64_t a = dq0 + ((h * 32768) >> 4), b = dk0 + ((buf * kKBuf + h * 8192) >> 4);
        const uint32_t d = tmem + kSBuf * buf + kS1Col * h;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {                      // 64-dim chunks of the half
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_pair(d, a + 2 * kk, b + 2 * kk, idS, (c | kk) ? 1u : 0u);
          a += 16384 >> 4;
          b += 4096 >> 4;
        }
      };
      bool ok = true;
      for (int i = 0; ok && i < min(2, n_tiles); ++i) {
        if (!wait_pair(bars + 8 * (kBarKFull + i), 0, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        qk_half(i, 1);
        qk_half(i, 0);
        commit_pair(bars + 8 * (kBarSFull + i));
      }
      for (int i = 0; ok && i < n_tiles; ++i) {
        const int buf = i & 1;
        const uint32_t parity = (i >> 1) & 1;
        if (!wait_pair(bars + 8 * (kBarVFull + buf), parity, p.wait_ns) ||
            !wait_pair(bars + 8 * (kBarPFull + buf), parity, p.wait_ns)) { ok = false; break; }
        tc_fence_after();
        const bool fresh = i % kChain == 0;
        uint32_t pa = tmem + kSBuf * buf;
        uint64_t v1 = dv0 + ((buf * kVBuf) >> 4);
#pragma unroll 1
        for (int kk = 0; kk < 4; ++kk) {                   // 16 cells = 8 TMEM columns of fp16 pairs
          mma_pair_ta(tmem + kOCol, pa, v1, idO, (kk > 0 || !fresh) ? 1u : 0u);
          mma_pair_ta(tmem + kOCol, pa, v1 + (kVPlane >> 4), idO, 1u);
          mma_pair_ta(tmem + kOCol, pa + kP2Col, v1, idO, 1u);
          pa += 8;
          v1 += 2048 >> 4;
        }
        commit_pair(bars + 8 * (kBarODone + buf));
        if (i + 2 < n_tiles) {
          if (!wait_pair(bars + 8 * (kBarKFull + buf), parity ^ 1, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          qk_half(buf, 1);
          if (!wait_pair(bars + 8 * (kBarODone + buf), parity, p.wait_ns)) { ok = false; break; }
          tc_fence_after();
          qk_half(buf, 0);
          commit_pair(bars + 8 * (kBarSFull + buf));
        }
      }
      if (!ok) ctl[1] = 1;
      // nothing of this thread's is in flight past here (after a failure too)
      commit_pair(bars + 8 * kBarDrain);
      (void)wait_pair(bars + 8 * kBarDrain, 0, kWaitDefaultNs);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && ctl[1]) record_status(p.status, K8V4_ECUDA);
  cluster_barrier();          // no product, commit or arrival of the pair is in flight
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace

// ---------------------------------------------------------------- host side
bool shared_prefix_supported(const CacheView& C) { return C.fmt == K8V4_FORMAT_K8V4; }

// The prefix cells that the pair kernel takes (0: none, every cell goes through
// the per-sequence decode) and its splits.
SharedPlan plan_shared(const CacheView& C, int n_seqs, int shared_len, int max_seq_len, int num_sms) {
  SharedPlan pl{};
  const int cells = std::min(shared_len, max_seq_len) / 16 * 16;
  if (!shared_prefix_supported(C) || n_seqs < 2 || cells < kTileN) return pl;
  pl.cells = cells;
  const int tiles = (cells + kTileN - 1) / kTileN;
  const int64_t units = static_cast<int64_t>((n_seqs + kPairSeqs - 1) / kPairSeqs) * C.H;
  const int slots = std::max(1, num_sms / 2);
  // one pair per two SMs at a time: the split count that minimises waves x (tiles
  // a pair sweeps + the fixed cost of a pair, worth about kFixedTiles tiles)
  constexpr int kFixedTiles = 10;
  int64_t best = INT64_MAX;
  for (int sp = 1; sp <= std::min(tiles, 256); ++sp) {
    const int tps = (tiles + sp - 1) / sp;
    const int64_t cost = (units * ((tiles + tps - 1) / tps) + slots - 1) / slots * (tps + kFixedTiles);
    if (cost < best) {
      best = cost;
      pl.tiles_per_split = tps;
    }
  }
  pl.splits = (tiles + pl.tiles_per_split - 1) / pl.tiles_per_split;
  return pl;
}

int launch_shared_prefix(const Launch& L, const CacheView& C, const SharedPlan& plan, const void* q, const int32_t* pt,
                         int64_t max_pages, const int32_t* lens, int n_seqs, int max_seq_len, float sm_scale, float* ws,
                         int ws_splits) {
  SharedParams p;
  p.C = C;
  p.q = static_cast<const uint16_t*>(q);
  p.pt = pt;
  p.max_pages = max_pages;
  p.lens = lens;
  p.n_seqs = n_seqs;
  p.max_seq_len = max_seq_len;
  p.cells = plan.cells;
  p.splits = plan.splits;
  p.tiles_per_split = plan.tiles_per_split;
  p.ws_splits = ws_splits;
  p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  p.ws = ws;
  p.status = L.status;
  p.wait_ns = wait_limit_ns() ? wait_limit_ns() : kWaitDefaultNs;
  p.page_div = FastDiv(static_cast<uint32_t>(C.P));
  // the register split needs the registers it hands out at launch
  static const int launch_regs = [] {
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, shared_prefix_kernel) == cudaSuccess ? attr.numRegs : 0;
  }();
  if (launch_regs * 4 < 2 * kRowRegs + kConvRegs + kIssueRegs) return K8V4_ECUDA;
  if (cudaFuncSetAttribute(shared_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
    return K8V4_ECUDA;
  const int groups = (n_seqs + kPairSeqs - 1) / kPairSeqs;
  const dim3 grid(2u * static_cast<unsigned>(groups) * static_cast<unsigned>(plan.splits), C.H);
  shared_prefix_kernel<<<grid, kThreads, kSmemBytes, L.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? K8V4_OK : K8V4_ECUDA;
}

}  // namespace k8v4
