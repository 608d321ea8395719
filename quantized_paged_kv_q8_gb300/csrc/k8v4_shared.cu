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
//      warps 0-15   rows: four threads per row (16 cells, and 64 of O's dims, each)
//      warps 16-19  conversion: raw tile -> registers -> operand tiles
//      warp 20      (leader CTA) issues every product of the pair
//      warp 21      copies the raw tiles (TMA)
//    With O in the registers of eight row warps (216 a thread) these were the slowest
//    part, two of them per scheduler with nothing to hide their latency behind;
//    sixteen leave no room for O, so the running O lives in global memory (L2),
//    where it goes every kChain tiles;
//  - the reference maximum of a row moves only when a tile exceeds it by 2^8, and
//    then its O tile is rescaled in tensor memory, so the two CTAs need not agree;
//    every kChain tiles O is added to the running O, in both CTAs at the same
//    tile, because the tensor core's accumulation is not rounded to nearest (2.9e-5
//    after 2,048 cells without that).
//
// Tensor memory (512 columns): S buffers [0,128), [128,256) (S0 | S1 each; a
// thread's P terms overlay its own columns of S0), O [256,512).  QK(i+2) overwrites
// P(i): its S1 half, which P does not touch, is issued behind PV(i) at once, its S0
// half when PV(i) is done.
//
// What bounds it: a tile takes about 2,450 clocks where its products take 2,050 at the
// full rate (QK does not run at it: qk below), the row warps beside the issuing warp
// being the last to finish; the running O adds about 200.  Measured (2 KV heads):
// 128 sequences on 118,784 cells 315 us of prefix (0.79 PFLOP/s of q K and p V, twice
// that of products, 1.89 being what a dense bf16 product reaches); 32 on 32,768, where
// set-up and the partial rows are a third of the time, 32 us.
//
// Every mbarrier wait is bounded: on timeout the warp raises the CTA's failure
// word and leaves its loop (the row warps together, at their next vote); the
// kernel records an error, waits for its own products (bounded), frees its tensor
// memory and returns.
#include <algorithm>
#include <mutex>

#include "k8v4_tc.cuh"
#include "k8v4_tma.cuh"

namespace k8v4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kPStride = 260;               // floats per partial row: o[256], m, l, 2 pad
constexpr int kRows = 128;                  // query rows per CTA (256 per pair)
constexpr int kPairSeqs = 2 * kRows / kGqa; // 32
constexpr int kTileN = 64;
constexpr int kRowWarps = 16, kRowThreads = 32 * kRowWarps;
constexpr int kThreads = kRowThreads + 256;
constexpr int kConvWarp0 = kRowWarps, kIssueWarp = kConvWarp0 + 4, kLoadWarp = kIssueWarp + 1;
// the register split waits for whole warpgroups: roles begin at multiples of four warps
static_assert(kConvWarp0 % 4 == 0 && kIssueWarp % 4 == 0 && kLoadWarp < kIssueWarp + 4 && kThreads == 32 * (kIssueWarp + 4), "roles");
constexpr int kChain = 16;                  // tiles accumulated in one TMEM O tile
constexpr float kSlack = 8.0f;              // log2 headroom of P above its row's reference maximum
constexpr uint32_t kWaitDefaultNs = 1000000000u;
// registers per thread after the split (16 row, 4 conversion and 4 other warps), out
// of the 80 of 24 warps that the block launches with
constexpr int kLaunchRegs = 80, kRowRegs = 96, kConvRegs = 72, kIssueRegs = 24;
static_assert(4 * kRowRegs + kConvRegs + kIssueRegs <= 6 * kLaunchRegs, "register split");

// shared memory (bytes); operand tiles 1024-byte aligned, the same in both CTAs
constexpr int kQOff = 0;                              // Q fp16 [4 chunks][128 rows][128 B]
constexpr int kKOff = kQOff + 65536;                  // K fp16, 2 buffers x [4 chunks][32 cells][128 B]
constexpr int kKBuf = 16384;
constexpr int kVOff = kKOff + 2 * kKBuf;              // V fp16, 2 buffers x 2 planes x [2 atoms][64 cells][128 B]
constexpr int kVPlane = 16384, kVBuf = 2 * kVPlane;
constexpr int kKsOff = kVOff + 2 * kVBuf;             // K scales, 4 tiles x [2][64] f32
constexpr int kRedOff = kKsOff + 4 * 512;             // [4][128] f32 exchange, [128] score factors
constexpr int kBarOff = kRedOff + 4 * 512 + 512;
constexpr int kCtlOff = kBarOff + 192;                // tmem slot, failure word, bad groups of 4 tiles, valid groups of the stages
constexpr int kRawOff = (kCtlOff + 64 + 1023) / 1024 * 1024;   // raw tiles, as many stages as fit (3, or 2 from 4 KV heads on)
constexpr int kSmemMax = 227 * 1024;
// a raw tile: K codes of the CTA's 32 cells (2 groups x 2 boxes of 16 cells x 128 B), V nibbles of the 64
// cells (4 boxes), and the runs of K and V scales of all heads (4 groups x 128 H and 256 H bytes)
constexpr int kRawV = 8192, kRawKs = 16384;
constexpr int raw_bytes(int H) { return (kRawKs + 1536 * H + 1023) / 1024 * 1024; }
constexpr int raw_stages(int H) { return (kSmemMax - kRawOff) / raw_bytes(H) < 3 ? (kSmemMax - kRawOff) / raw_bytes(H) : 3; }
static_assert(raw_stages(8) >= 2, "raw stages");
// the epilogue reuses the operand tiles as a fp32 [128][256] row buffer
static_assert(kKsOff - kQOff >= kRows * 256 * 4, "row buffer");

// mbarriers, at kBarOff + 8 * index
enum { kBarKFull = 0, kBarVFull = 2, kBarPFull = 4, kBarSFull = 6, kBarODone = 8, kBarKsFull = 10,
       kBarDrain = 14, kBarMost = 15, kBarRawFull = 16, kBarRawEmpty = 20 };

constexpr uint32_t kTmemCols = 512, kSBuf = 128, kS1Col = 64, kOCol = 256, kP2Col = 8;

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
  float* acc;               // [CTA][128 rows x 256] running O, for sweeps of more than kChain tiles
  int* status;
  uint32_t wait_ns;
  FastDiv page_div;
  int stages, stage_bytes;  // raw tiles in flight
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
// The arrivals that hand operand tiles to the products carry no wider release than
// the CTA's: what the tensor core reads is made visible by the proxy and tcgen05
// fences ahead of them, and a cluster-wide release would also wait for the
// global loads of the next tile (32 sequences on 32,768 cells: 107 us with it, 92
// without, when those were loads by thread).
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void arrive_local(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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
// completion of this thread's products so far -> the barrier at this offset of the CTAs
// in the mask: both, or the leader alone
constexpr uint16_t kBothCtas = 3, kLeaderCta = 1;
__device__ __forceinline__ void commit_to(uint32_t bar, uint16_t ctas) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(ctas)
      : "memory");
}
// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// the same over the four warps that share 32 rows (warps w, w + 4, w + 8, w + 12; w < 4)
__device__ __forceinline__ bool quad_any(int w, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(w + 3), "r"(pred ? 1u : 0u)
      : "memory");
  return r != 0;
}
// a barrier over the row warps that also ORs a predicate
__device__ __forceinline__ bool rows_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 512, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void rows_barrier() { asm volatile("barrier.cta.sync 2, 512;" ::: "memory"); }
// two runs of 16 fp32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, float a[16], float b[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(r[16 + i]);
  }
}
// two runs of 8 columns; the caller waits (tmem_wait_st)
__device__ __forceinline__ void tmem_st8x2(uint32_t ta, uint32_t tb, const float a[8], const float b[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%2,%3,%4,%5,%6,%7,%8,%9};\n\t"
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%1], {%10,%11,%12,%13,%14,%15,%16,%17};"
      ::"r"(ta), "r"(tb), "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
        "r"(__float_as_uint(a[3])), "r"(__float_as_uint(a[4])), "r"(__float_as_uint(a[5])), "r"(__float_as_uint(a[6])),
        "r"(__float_as_uint(a[7])), "r"(__float_as_uint(b[0])), "r"(__float_as_uint(b[1])), "r"(__float_as_uint(b[2])),
        "r"(__float_as_uint(b[3])), "r"(__float_as_uint(b[4])), "r"(__float_as_uint(b[5])), "r"(__float_as_uint(b[6])),
        "r"(__float_as_uint(b[7]))
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
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
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) shared_prefix_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                                            const __grid_constant__ CUtensorMap tm_v,
                                                                                            const SharedParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int g = blockIdx.y;
  const int groups = (p.n_seqs + kPairSeqs - 1) / kPairSeqs;
  const int unit = blockIdx.x >> 1;
  const int split = unit / groups;
  const int pair_seq0 = (unit - split * groups) * kPairSeqs;
  const int seq0 = pair_seq0 + static_cast<int>(rank) * (kRows / kGqa);   // this CTA's first sequence
  const CacheView& C = p.C;
  const int HQ = C.H * kGqa;
  const int row = tid & (kRows - 1), part = tid >> 7;      // (row warps) 16 cells of a tile and 64 dims of O per part
  const uint32_t bars = sb + kBarOff;
  volatile int* ctl = reinterpret_cast<volatile int*>(smem + kCtlOff);   // [0] tmem, [1] failed, [4..7] bad groups of 4 tiles
  float* red = reinterpret_cast<float*>(smem + kRedOff);                 // [4][128]
  float* fsc = red + 4 * kRows;                                          // [128]
  float* ksbuf = reinterpret_cast<float*>(smem + kKsOff);

  const int tile0 = split * p.tiles_per_split;
  // The prefix cells that any of the pair's sequences sees: those behind are neither
  // looked up nor read (their pages may be unwritten, their table entries padding), and
  // a range of nothing else still runs one tile, of no cells.  The same in both CTAs; the
  // load warp tells the others
  auto tiles_of = [&](int cells) { return max(1, min(p.tiles_per_split, (cells + kTileN - 1) / kTileN - tile0)); };
  int limit = 0;
  if (warp == kLoadWarp) {
    // one barrier per lane
    int count = 0;
    if (lane < kBarPFull) count = 8;                       // K, V tiles: 4 conversion warps of both CTAs
    else if (lane < kBarSFull) count = 2 * kRowWarps;      // P: the row warps of both CTAs
    else if (lane < kBarKsFull) count = 1;                 // S done, O done: one commit
    else if (lane < kBarDrain) count = 4;                  // K scales: the CTA's conversion warps
    else if (lane < kBarRawFull) count = 1;                // everything done, three quarters of PV: one commit
    else if (lane < kBarRawEmpty) count = 1;               // raw tile: the loader, and the bytes of its copies
    else if (lane < kBarRawEmpty + 4) count = 4;
    if (count) mbar_init(bars + 8 * lane, count);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (lane < 8) ctl[1 + lane] = 0;
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    }
  }
  if (warp == kIssueWarp) tmem_alloc_pair(sb + kCtlOff, kTmemCols);
  // Launched behind the splits of the sequences' own cells, this kernel takes its places
  // as their CTAs leave.  Lengths, page table, queries and pages come from the kernels
  // before that one, which only this wait makes visible here
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == kLoadWarp) {
    limit = pair_seq0 + lane < p.n_seqs ? __ldcg(p.lens + pair_seq0 + lane) : 0;
    limit = min(p.cells, min(p.max_seq_len, __reduce_max_sync(kFull, max(limit, 0))));
    if (lane == 0) {
      ctl[12] = limit;
      ctl[13] = tiles_of(limit);
    }
    __syncwarp();
  }

  // ---- the load warp's copies of tile i into a stage: raw tiles by TMA (per-thread
  // copies cost the conversion warps 870 clocks a tile: each touches 32 rows).  Page
  // ids of eight tiles, four 16-cell groups each, are held one per lane.
  int page_mine = INT32_MIN;
  auto load_tile = [&](int i, int stage, bool leader) {
    const int H = C.H;
    if ((i & 7) == 0) {
      const int c = (tile0 + i + (lane >> 2)) * kTileN + 16 * (lane & 3);
      const int64_t pidx = p.page_div.div(static_cast<uint32_t>(c));
      const int page = pidx < p.max_pages ? __ldcg(p.pt + pidx) : -1;
      page_mine = INT32_MIN;                               // behind the limit, or another range's
      if (i + (lane >> 2) < tiles_of(limit) && c < limit) page_mine = page >= 0 && page < C.n_pages ? page : -1;
    }
    const uint32_t dst = sb + kRawOff + stage * p.stage_bytes, bar = bars + 8 * (kBarRawFull + stage);
    const int my_group_page = __shfl_sync(kFull, page_mine, 4 * (i & 7) + (lane & 3));
    const unsigned good = __ballot_sync(kFull, my_group_page >= 0) & 15u;
    const unsigned bad = __ballot_sync(kFull, my_group_page == -1) & 15u;
    const unsigned kgood = (good >> (2 * rank)) & 3u;
    if (leader) {
      if (bad) record_status(p.status, K8V4_ERANGE);
      ctl[8 + stage] = static_cast<int>(good | (bad << 4));
      mbar_expect_tx(bar, __popc(good) * (2048u + 384u * H) + __popc(kgood) * 4096u);
    }
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      const int page = __shfl_sync(kFull, my_group_page, q);
      if (!leader || page < 0) continue;
      const int cell = (tile0 + i) * kTileN + 16 * q;
      const int slot = cell - static_cast<int>(p.page_div.div(static_cast<uint32_t>(cell))) * C.P;
      const int kq = q - 2 * static_cast<int>(rank);
      if (kq == 0 || kq == 1) {
        tma_load_4d(dst + kq * 4096, &tm_k, 0, g, slot, page, bar);
        tma_load_4d(dst + kq * 4096 + 2048, &tm_k, 128, g, slot, page, bar);
      }
      tma_load_4d(dst + kRawV + q * 2048, &tm_v, 0, g, slot, page, bar);
      const uint8_t* pg = C.pages + static_cast<int64_t>(page) * C.page_bytes;
      bulk_load(dst + kRawKs + q * 128 * H, pg + C.ks_off() + static_cast<int64_t>(slot) * 8 * H, 128 * H, bar);
      bulk_load(dst + kRawKs + 512 * H + q * 256 * H, pg + C.vs_off() + static_cast<int64_t>(slot) * 16 * H, 256 * H, bar);
    }
    __syncwarp();
  };
  // The first tile, while the others set Q up.  The next ones only behind that: all CTAs
  // begin at once, and their first copies would wait for everyone's second and third
  if (warp == kLoadWarp) load_tile(0, 0, elect_one());

  // ---- visibility of this thread's row
  int my_vis = 0;
  {
    const int s = seq0 + row / kGqa;
    if (warp < kRowWarps && s < p.n_seqs) {
      int v = __ldcg(p.lens + s);
      if (v < 0 || v > p.max_seq_len) {
        if (part == 0) record_status(p.status, K8V4_ERANGE);
        v = v < 0 ? 0 : p.max_seq_len;
      }
      my_vis = min(v, p.cells);
    }
  }
  // ---- Q rows -> fp16 with a per-row power-of-two scale, swizzled K-major: a warp
  // takes a row at a time (16 B a lane); the load warp starts on the raw tiles meanwhile
  if (warp < kLoadWarp) {
    constexpr int kPer = (kRows + kLoadWarp - 1) / kLoadWarp;
    uint4 raw[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int r = warp + kLoadWarp * j, s = seq0 + r / kGqa;
      raw[j] = make_uint4(0, 0, 0, 0);
      if (r < kRows && s < p.n_seqs)
        raw[j] = __ldcg(reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(s) * HQ + g * kGqa + r % kGqa) * kD) + lane);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int r = warp + kLoadWarp * j;
      if (r >= kRows) break;
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
      float amax = 0.0f;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[u] << 16)), fabsf(__uint_as_float(w[u] & 0xffff0000u))));
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
      const int ex = amax > 0.0f ? static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu) - 127 : 0;
      const int sh = min(100, 14 - ex);                    // from -114 on
      const float up = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);                       // 2^sh
      // above 0 also where the product underflows: a masked score is -inf times it
      if (lane == 0) fsc[r] = fmaxf(p.sm_scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23), 1.2e-38f);
      uint32_t hv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const __half2 h2 = __floats2half2_rn(__fmul_rn(__uint_as_float(w[u] << 16), up),
                                             __fmul_rn(__uint_as_float(w[u] & 0xffff0000u), up));
        hv[u] = *reinterpret_cast<const uint32_t*>(&h2);
      }
      // dims 8 lane .. +7: chunk lane / 8, unit lane % 8
      sts128(sb + kQOff + (lane >> 3) * 16384 + swz(r, lane & 7), hv[0], hv[1], hv[2], hv[3]);
    }
  }
  asm volatile("fence.proxy.async;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_barrier();          // barriers, tensor memory and Q of both CTAs are ready
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(ctl[0]);
  const int n_tiles = ctl[13];

  if (warp < kRowWarps) {
    // ================================================================ rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float my_f = fsc[row];
    const uint32_t p_full0 = map_to(bars + 8 * kBarPFull, 0);
    const uint32_t o_tile = tmem + lane_base + kOCol + 64 * part;
    // the running O of this thread's 64 dims: float4 number c at acc[512 c]
    float4* const acc = reinterpret_cast<float4*>(p.acc) +
                        (n_tiles > kChain ? (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * (kRows * 64) + tid : 0);
    float m_run = -INFINITY, l_part = 0.0f, acc_scale = 1.0f;          // acc counts times acc_scale
    bool failed = false, have_acc = false;
    for (int i = 0; i < n_tiles; ++i) {
      const int buf = i & 1;
      const uint32_t parity = (i >> 1) & 1;
      if (!mbar_wait(bars + 8 * (kBarSFull + buf), parity, p.wait_ns) ||
          !mbar_wait(bars + 8 * (kBarKsFull + (i & 3)), (i >> 2) & 1, p.wait_ns)) {
        failed = true;
        ctl[1] = 1;
      }
      tc_fence_after();
      // scores, unscaled (my_f > 0, so the maximum commutes with it); cell c of this part
      const uint32_t sbase = tmem + lane_base + kSBuf * buf + 16 * part;
      const float* ks = ksbuf + 128 * (i & 3) + 16 * part;             // s0 of the tile's cells, then s1
      float2 sc[8];
      {
        float a[16], b[16];
        tmem_ld16x2(sbase, sbase + kS1Col, a, b);
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          const float4 k0 = *reinterpret_cast<const float4*>(ks + c);
          const float4 k1 = *reinterpret_cast<const float4*>(ks + 64 + c);
          sc[c / 2] = __ffma2_rn(make_float2(k1.x, k1.y), make_float2(b[c], b[c + 1]),
                                 __fmul2_rn(make_float2(k0.x, k0.y), make_float2(a[c], a[c + 1])));
          sc[c / 2 + 1] = __ffma2_rn(make_float2(k1.z, k1.w), make_float2(b[c + 2], b[c + 3]),
                                     __fmul2_rn(make_float2(k0.z, k0.w), make_float2(a[c + 2], a[c + 3])));
        }
      }
      const int vis = my_vis - (tile0 + i) * kTileN - 16 * part;       // cells [0, vis) of this part
      const bool bad = (ctl[4 + (i & 3)] >> part) & 1;                 // its 16 cells are on a page out of range
      if (vis < 16 || bad) {
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
          if (c >= vis || bad) sc[c / 2].x = -INFINITY;
          if (c + 1 >= vis || bad) sc[c / 2].y = -INFINITY;
        }
      }
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        mx0 = fmaxf(mx0, fmaxf(sc[c].x, sc[c].y));
        mx1 = fmaxf(mx1, fmaxf(sc[c + 1].x, sc[c + 1].y));
      }
      const float top = fmaxf(mx0, mx1) * my_f;
      // the four threads of a row agree on its reference: a vote of their four warps
      const bool any = quad_any(warp & 3, failed || top > m_run + kSlack);
      float alpha = 1.0f;
      if (any) {
        red[part * kRows + row] = top;
        // the four leave together: the failure word is read once, ahead of a vote
        if (quad_any(warp & 3, failed || ctl[1] != 0)) { failed = true; break; }
        const float mt = fmaxf(fmaxf(red[row], red[kRows + row]), fmaxf(red[2 * kRows + row], red[3 * kRows + row]));
        if (mt > m_run + kSlack) {
          alpha = exp2f(m_run - mt);                                   // 0 on the first visible tile
          m_run = mt;
          l_part *= alpha;
        }
      }
      // P * 2^7 in two fp16 terms: the top 11 bits of p, and the rest of it rounded.
      // They overlay this thread's own S0 columns, P1 in the first 8, P2 behind it
      const float mu = (m_run == -INFINITY ? 0.0f : m_run) - 7.0f;
      const float2 f2 = make_float2(my_f, my_f), mu2 = make_float2(-mu, -mu);
      float2 psum = make_float2(0.0f, 0.0f);
      {
        float p1[8], p2[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float2 e = __ffma2_rn(sc[c], f2, mu2);
          const float2 q = make_float2(ex2_ftz(e.x), ex2_ftz(e.y));
          const float2 t = make_float2(__uint_as_float(__float_as_uint(q.x) & 0xffffe000u),
                                       __uint_as_float(__float_as_uint(q.y) & 0xffffe000u));
          const float2 r = __ffma2_rn(t, make_float2(-1.0f, -1.0f), q);   // q - t, exact
          const __half2 h1 = __floats2half2_rn(t.x, t.y), h2 = __floats2half2_rn(r.x, r.y);
          psum = __fadd2_rn(psum, q);
          p1[c] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h1));
          p2[c] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h2));
        }
        tmem_st8x2(sbase, sbase + kP2Col, p1, p2);
      }
      l_part += psum.x + psum.y;
      tmem_wait_st();
      // O of the tiles so far: into acc at every kChain-th tile (both CTAs), rescaled
      // in place where a reference moved in between
      const bool folds = i > 0 && i % kChain == 0;
      if (folds || (i > 0 && any && __any_sync(kFull, alpha != 1.0f))) {
        if (!mbar_wait(bars + 8 * (kBarODone + (buf ^ 1)), ((i - 1) >> 1) & 1, p.wait_ns)) {
          failed = true;
          ctl[1] = 1;
        }
        tc_fence_after();
        if (folds) {                                                   // acc = (acc + O) * alpha
          const float a = alpha * acc_scale;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            float4 old[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) old[c] = have_acc ? acc[512 * (4 * h + c)] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float o[16];
            tmem_ld16(o_tile + 16 * h, o);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              acc[512 * (4 * h + c)] = make_float4(old[c].x * a + o[4 * c] * alpha, old[c].y * a + o[4 * c + 1] * alpha,
                                                   old[c].z * a + o[4 * c + 2] * alpha, old[c].w * a + o[4 * c + 3] * alpha);
          }
          have_acc = true;
          acc_scale = 1.0f;
        } else {                                                       // O *= alpha
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            float o[8];
            tmem_ld8(o_tile + 8 * h, o);
#pragma unroll
            for (int c = 0; c < 8; ++c) o[c] *= alpha;
            tmem_st8(o_tile + 8 * h, o);
          }
          acc_scale *= alpha;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(p_full0 + 8 * buf);
    }
    // ---- the last O tile, then o / m / l of the rows
    float o[64];
    if (!failed) {
      if (mbar_wait(bars + 8 * (kBarODone + ((n_tiles - 1) & 1)), ((n_tiles - 1) >> 1) & 1, p.wait_ns)) {
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) tmem_ld32(o_tile + 32 * h, o + 32 * h);
        if (have_acc) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float4 old = acc[512 * c];
            o[4 * c] += old.x * acc_scale;
            o[4 * c + 1] += old.y * acc_scale;
            o[4 * c + 2] += old.z * acc_scale;
            o[4 * c + 3] += old.w * acc_scale;
          }
        }
        tc_fence_before();
      } else {
        failed = true;
        ctl[1] = 1;
      }
    }
    // PV of the last tile is done in both CTAs (one commit covers the pair), and
    // with it every read of this CTA's operand tiles
    red[part * kRows + row] = l_part;
    const bool stop = rows_any(failed);
    if (!stop) {
      const float l = (red[row] + red[kRows + row]) + (red[2 * kRows + row] + red[3 * kRows + row]);
      // inverse Walsh-Hadamard transform: six stages over the thread's own 64 dims in
      // registers, the last two (dims d + 64 k) as the rows are written
#pragma unroll
      for (int h = 1; h < 64; h <<= 1) {
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          if (i & h) continue;
          const float a = o[i], b = o[i + h];
          o[i] = a + b;
          o[i + h] = a - b;
        }
      }
      float* rowbuf = reinterpret_cast<float*>(smem + kQOff);          // [128][256] fp32, rotated by 4 * row
#pragma unroll
      for (int i = 0; i < 64; i += 4)
        *reinterpret_cast<float4*>(rowbuf + row * 256 + ((64 * part + i + 4 * row) & 255)) =
            make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      if (part == 0) {
        const int s = seq0 + row / kGqa;
        if (s < p.n_seqs) {
          float* dst = p.ws + ((static_cast<int64_t>(s) * p.ws_splits + split) * HQ + g * kGqa + row % kGqa) * kPStride;
          dst[256] = m_run - 7.0f;                                     // o and l are relative to 2^(m - 7)
          dst[257] = l;
        }
      }
      rows_barrier();
      for (int r = warp; r < kRows; r += kRowWarps) {
        const int s = seq0 + r / kGqa;
        if (s >= p.n_seqs) break;
        float2 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = *reinterpret_cast<const float2*>(rowbuf + r * 256 + ((64 * k + 2 * lane + 4 * r) & 255));
        float* dst = p.ws + ((static_cast<int64_t>(s) * p.ws_splits + split) * HQ + g * kGqa + r % kGqa) * kPStride + 2 * lane;
        const float2 s01 = make_float2(x[0].x + x[1].x, x[0].y + x[1].y), d01 = make_float2(x[0].x - x[1].x, x[0].y - x[1].y);
        const float2 s23 = make_float2(x[2].x + x[3].x, x[2].y + x[3].y), d23 = make_float2(x[2].x - x[3].x, x[2].y - x[3].y);
        constexpr float kInv = 0.0625f;
        *reinterpret_cast<float2*>(dst) = make_float2((s01.x + s23.x) * kInv, (s01.y + s23.y) * kInv);
        *reinterpret_cast<float2*>(dst + 64) = make_float2((d01.x + d23.x) * kInv, (d01.y + d23.y) * kInv);
        *reinterpret_cast<float2*>(dst + 128) = make_float2((s01.x - s23.x) * kInv, (s01.y - s23.y) * kInv);
        *reinterpret_cast<float2*>(dst + 192) = make_float2((d01.x - d23.x) * kInv, (d01.y - d23.y) * kInv);
      }
    }
  } else if (warp < kIssueWarp) {
    // ================================================================ conversion
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    const int t = tid - 32 * kConvWarp0;                   // 0..127
    const int cw = t >> 5;
    // K: cell 32 rank + lane, dims [64 cw, +64); V: cell t & 63, blocks 4 rank + 2 (t >> 6) + {0, 1}.
    // The copies put 16-byte unit u of a row at u ^ (row & 7) (128-byte swizzle).
    const int vcell = t & 63, vblk = 4 * static_cast<int>(rank) + 2 * (t >> 6), vrow = vcell & 15;
    const uint32_t k_full0 = map_to(bars + 8 * kBarKFull, 0), v_full0 = map_to(bars + 8 * kBarVFull, 0);
    const uint32_t kraw = (lane >> 4) * 4096 + (cw >> 1) * 2048 + (lane & 15) * 128;
    const uint32_t vraw = kRawV + (vcell >> 4) * 2048 + vrow * 128;
    const uint32_t ksraw = kRawKs + (vcell >> 4) * 128 * C.H + (vrow * C.H + g) * 8;
    const uint32_t vsraw = kRawKs + 512 * C.H + (vcell >> 4) * 256 * C.H + (vrow * C.H + g) * 16 + 2 * vblk;
    int stage = 0;
    uint32_t raw_phase = 0;
    for (int i = 0; i < n_tiles; ++i) {
      const int buf = i & 1;
      const uint32_t last = ((i - 2) >> 1) & 1;            // phase of tile i - 2 on the buffers' barriers
      const uint32_t raw = sb + kRawOff + stage * p.stage_bytes;
      if (!mbar_wait(bars + 8 * (kBarRawFull + stage), raw_phase, p.wait_ns)) { ctl[1] = 1; break; }
      const int valid = ctl[8 + stage];                    // the tile's 16-cell groups that were copied; bits 4..7: on a bad page
      // ---- K(i) and its scales, once QK(i - 2) has read the buffer
      if (i >= 2 && !mbar_wait(bars + 8 * (kBarSFull + buf), last, p.wait_ns)) { ctl[1] = 1; break; }
      {
        const uint32_t dst = sb + kKOff + buf * kKBuf + cw * 4096;
        uint4 kw[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) kw[u] = lds128(raw + kraw + (((4 * (cw & 1) + u) ^ (lane & 7)) << 4));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 w = kw[u];
          uint32_t h[8];
          i8x4_to_f16(w.x, h[0], h[1]);
          i8x4_to_f16(w.y, h[2], h[3]);
          i8x4_to_f16(w.z, h[4], h[5]);
          i8x4_to_f16(w.w, h[6], h[7]);
          sts128(dst + swz(lane, 2 * u), h[0], h[1], h[2], h[3]);
          sts128(dst + swz(lane, 2 * u + 1), h[4], h[5], h[6], h[7]);
        }
        if (t < 64) {
          float2 ksc;
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ksc.x), "=f"(ksc.y) : "r"(raw + ksraw));
          ksbuf[128 * (i & 3) + t] = ksc.x;
          ksbuf[128 * (i & 3) + 64 + t] = ksc.y;
          if (t == 0) ctl[4 + (i & 3)] = valid >> 4;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          arrive_local(bars + 8 * (kBarKsFull + (i & 3)));
          arrive_cluster(k_full0 + 8 * buf);
        }
      }
      // ---- V(i), once PV(i - 2) has read the buffer
      if (i >= 2 && !mbar_wait(bars + 8 * (kBarODone + buf), last, p.wait_ns)) { ctl[1] = 1; break; }
      {
        const uint32_t dst = sb + kVOff + buf * kVBuf + (t >> 6) * 8192;
        // a cell that was not copied, or that nobody sees, counts with V = 0 (its P is 0,
        // its bytes are anything)
        uint32_t vd;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vd) : "r"(raw + vsraw));
        const uint4 vw[2] = {lds128(raw + vraw + ((vblk ^ (vrow & 7)) << 4)), lds128(raw + vraw + (((vblk + 1) ^ (vrow & 7)) << 4))};
        if (!((valid >> (vcell >> 4)) & 1) || (tile0 + i) * kTileN + vcell >= ctl[12]) vd = 0;
        __syncwarp();
        if (lane == 0) arrive_local(bars + 8 * (kBarRawEmpty + stage));
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          const __half dh = __ushort_as_half(static_cast<unsigned short>(vd >> (16 * blk)));
          const __half2 d2 = __halves2half2(dh, dh);
          const uint4 w = vw[blk];
          const uint32_t ws4[4] = {w.x, w.y, w.z, w.w};
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
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive_cluster(v_full0 + 8 * buf);
      }
      if (++stage == p.stages) {
        stage = 0;
        raw_phase ^= 1;
      }
    }
  } else {
    // ================================================================ issue
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    // The whole warp runs the loop, and one elected lane executes the products:
    // with the control flow uniform the descriptors live in uniform registers,
    // where a lone thread's would be moved there one by one ahead of every product
    // (about 100 clocks each: 2,800 a tile, more than the products take).
    if (__shfl_sync(kFull, warp, 0) == kIssueWarp && rank == 0) {
      constexpr uint32_t idS = idesc_f16(256, 64, false, false);
      constexpr uint32_t idO = idesc_f16(256, 256, false, true);
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      const uint64_t dq0 = smem_desc(sb + kQOff, 16, 1024);
      const uint64_t dk0 = smem_desc(sb + kKOff, 16, 1024);
      const uint64_t dv0 = smem_desc(sb + kVOff, 8192, 1024);
      const bool leader = elect_one();
      auto ready = [&](int bar, uint32_t parity) -> bool {
        return __all_sync(kFull, mbar_wait(bars + 8 * bar, parity, p.wait_ns)) != 0;
      };
      // S[buf]_h += Q_h K_h^T over 16 dims, the two halves in turn.  Such a product takes
      // about 98 clocks (32 are its work): it reads 4 KB of Q for 64 columns
      auto qk = [&](int buf, int h, int kk) {
        const uint32_t off = (kk & 3) * 32;
        mma_pair(tm + kSBuf * buf + kS1Col * h, dq0 + (((2 * h + (kk >> 2)) * 16384 + off) >> 4),
                 dk0 + ((buf * kKBuf + (2 * h + (kk >> 2)) * 4096 + off) >> 4), idS, kk ? 1u : 0u);
      };
      constexpr int kAhead = 2;                            // products of the S1 half that go ahead
      bool ok = true;
      for (int i = 0; i < min(2, n_tiles); ++i) {
        if (!ready(kBarKFull + i, 0)) { ok = false; break; }
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            qk(i, 0, kk);
            qk(i, 1, kk);
          }
          commit_to(bars + 8 * (kBarSFull + i), kBothCtas);
        }
      }
      for (int i = 0; ok && i < n_tiles; ++i) {
        const int buf = i & 1;
        const uint32_t parity = (i >> 1) & 1;
        // Products are handed over a few at a time, the next ones when the last of the
        // ones ahead are still running: an instruction that finds the queue full holds
        // up the other warps of this scheduler (a row warp and a conversion warp).
        if (!ready(kBarVFull + buf, parity) || !ready(kBarPFull + buf, parity)) { ok = false; break; }
        tc_fence_after();
        const uint32_t more = i % kChain != 0 ? 1u : 0u;   // O of this chain so far is kept
        const uint32_t pa = tm + kSBuf * buf;
        const uint64_t v1 = dv0 + ((buf * kVBuf) >> 4);
        auto pv = [&](int kk, uint32_t acc) {              // 16 cells = 8 TMEM columns of fp16 pairs, of part kk
          const uint64_t v = v1 + ((kk * 2048) >> 4);
          const uint32_t p1 = pa + 16 * kk;
          mma_pair_ta(tm + kOCol, p1, v, idO, acc);
          mma_pair_ta(tm + kOCol, p1, v + (kVPlane >> 4), idO, 1u);
          mma_pair_ta(tm + kOCol, p1 + kP2Col, v, idO, 1u);
        };
        if (leader) pv(0, more);
        if (i + 1 < n_tiles && !ready(kBarSFull + (buf ^ 1), ((i + 1) >> 1) & 1)) { ok = false; break; }   // QK(i + 1)
        if (leader) {
          pv(1, 1u);
          pv(2, 1u);
          commit_to(bars + 8 * kBarMost, kLeaderCta);
          pv(3, 1u);
          commit_to(bars + 8 * (kBarODone + buf), kBothCtas);
        }
        if (i + 2 < n_tiles) {
          // QK(i + 2) overwrites P(i) with its S0 half; the S1 half begins behind PV(i)
          if (!ready(kBarKFull + buf, parity ^ 1) || !ready(kBarMost, i & 1)) { ok = false; break; }
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kAhead; ++kk) qk(buf, 1, kk);
          }
          if (!ready(kBarODone + buf, parity)) { ok = false; break; }
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              qk(buf, 0, kk);
              if (kk + kAhead < 8) qk(buf, 1, kk + kAhead);
            }
            commit_to(bars + 8 * (kBarSFull + buf), kBothCtas);
          }
        }
      }
      if (!ok) ctl[1] = 1;
      // all of this warp's products, waited for below (after a failure too)
      if (leader) commit_to(bars + 8 * kBarDrain, kBothCtas);
    } else if (__shfl_sync(kFull, warp, 0) == kLoadWarp) {
      // ============================================================== copies
      const bool leader = elect_one();
      int stage = 1, i = 1;
      uint32_t phase = 1;                                  // of the stage's last use, from its second on
      for (; i < n_tiles; ++i) {
        if (i >= p.stages && !__all_sync(kFull, mbar_wait(bars + 8 * (kBarRawEmpty + stage), phase, p.wait_ns))) { ctl[1] = 1; break; }
        load_tile(i, stage, leader);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // no copy is in flight past here (after a failure too): the last tiles' stages
      for (int j = max(0, i - p.stages); j < i; ++j)
        (void)mbar_wait(bars + 8 * (kBarRawFull + j % p.stages), (j / p.stages) & 1, kWaitDefaultNs);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // The commits arrive at the barriers of both CTAs, and each CTA waits for its own copies of
  // the last ones: shared memory that an arrival is still on its way to must not be given
  // to the next CTA.  (The row warps have waited for every S and the last O.)
  if (warp == kIssueWarp) {
    if (n_tiles > 1 && !ctl[1])
      (void)mbar_wait(bars + 8 * (kBarODone + (n_tiles & 1)), ((n_tiles - 2) >> 1) & 1, kWaitDefaultNs);
    (void)mbar_wait(bars + 8 * kBarDrain, 0, kWaitDefaultNs);
    __syncwarp();
  }
  if (tid == 0 && ctl[1]) record_status(p.status, K8V4_ECUDA);
  cluster_barrier();          // no product, commit or arrival of the pair is in flight
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace

// ---------------------------------------------------------------- host side
bool shared_prefix_supported(const CacheView& C) { return C.fmt == K8V4_FORMAT_K8V4 && decode_ws_supported(C); }

// Set-up of the kernel on the current device: its shared memory, its registers at launch
// (the split hands out that many) and the CTA pairs that the device runs at a time (an
// odd SM in a cluster's reach stays without a partner, so 152 SMs need not give 76).
// Kept once it has worked; a failure is not, and the next call tries again.
namespace {
std::mutex g_slots_mu;
int g_slots[64];
}  // namespace
int shared_prefix_slots() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  std::lock_guard<std::mutex> lock(g_slots_mu);
  if (g_slots[dev] > 0) return g_slots[dev];
  cudaFuncAttributes fa;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemMax;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int slots = 0;
  if (cudaFuncGetAttributes(&fa, shared_prefix_kernel) != cudaSuccess ||
      fa.numRegs * 6 < 4 * kRowRegs + kConvRegs + kIssueRegs ||
      cudaFuncSetAttribute(shared_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&slots, shared_prefix_kernel, &cfg) != cudaSuccess || slots < 1) {
    cudaGetLastError();                   // clear the error state that the failed call left
    return 0;
  }
  return g_slots[dev] = slots;
}

// The prefix cells that the pair kernel takes (0: none, every cell goes through
// the per-sequence decode) and its splits, for a device that runs `slots` CTA pairs at
// a time (0: its set-up failed, none).
SharedPlan plan_shared(const CacheView& C, int n_seqs, int shared_len, int max_seq_len, int slots) {
  SharedPlan pl{};
  const int cells = std::min(shared_len, max_seq_len) / 16 * 16;
  if (!shared_prefix_supported(C) || cells < kTileN || slots < 1) return pl;
  // Worth it where reading the prefix n_seqs times costs more than this kernel does.
  // Measured at 2 KV heads (64 own cells): the per-sequence decode takes 11 us + 0.23 us
  // per 1,000 cells of all sequences, this path 22 us + 0.72 us per 1,000 prefix
  // cells and 32 sequences.  At 8 sequences they meet between 8,192 cells (21.8 us
  // against 27.4) and 16,384 (34.8 against 32.2), at 32 between 1,024 (19.4, 24.0) and
  // 2,048 (26.9, 24.4), at 128 below 512 (43.2, 31.7); up to 3 sequences never.
  const int64_t groups = (n_seqs + kPairSeqs - 1) / kPairSeqs;
  if (static_cast<int64_t>(C.H) * cells * (23ll * n_seqs - 72ll * groups) <= 2200000ll) return pl;
  pl.cells = cells;
  const int tiles = (cells + kTileN - 1) / kTileN;
  const int64_t units = groups * C.H;
  // one pair per two SMs at a time: the split count that minimises waves x (tiles
  // a pair sweeps + the fixed cost of a pair, worth about kFixedTiles tiles) + the
  // partial rows of a split, written and read again (4,096 rows take a tile's time)
  constexpr int kFixedTiles = 9;
  const double rows = static_cast<double>(n_seqs) * C.H * kGqa;
  double best = 1e300;
  for (int sp = 1; sp <= std::min(tiles, kPrefixMaxSplits); ++sp) {
    const int tps = (tiles + sp - 1) / sp, real = (tiles + tps - 1) / tps;
    const double cost = static_cast<double>((units * real + slots - 1) / slots) * (tps + kFixedTiles) + real * rows / 4096.0;
    if (cost < best) {
      best = cost;
      pl.tiles_per_split = tps;
    }
  }
  pl.splits = (tiles + pl.tiles_per_split - 1) / pl.tiles_per_split;
  // the running O of each CTA, where a sweep is longer than a chain
  pl.acc_bytes = pl.tiles_per_split > kChain ? static_cast<size_t>(2 * units * pl.splits) * kRows * 256 * sizeof(float) : 0;
  return pl;
}

int launch_shared_prefix(const Launch& L, const CacheView& C, const SharedPlan& plan, const void* q, const int32_t* pt,
                         int64_t max_pages, const int32_t* lens, int n_seqs, int max_seq_len, float sm_scale, float* ws,
                         int ws_splits, float* acc, bool behind_splits) {
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
  p.acc = acc;
  p.status = L.status;
  p.wait_ns = wait_limit_ns() ? wait_limit_ns() : kWaitDefaultNs;
  p.page_div = FastDiv(static_cast<uint32_t>(C.P));
  p.stages = raw_stages(C.H);
  p.stage_bytes = raw_bytes(C.H);
  CUtensorMap mk, mv;
  if (!tensor_maps_of(C, &mk, &mv)) return K8V4_ECUDA;
  const int groups = (n_seqs + kPairSeqs - 1) / kPairSeqs;
  const dim3 grid(2u * static_cast<unsigned>(groups) * static_cast<unsigned>(plan.splits), C.H);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kRawOff + p.stages * p.stage_bytes;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = behind_splits ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, shared_prefix_kernel, mk, mv, p) != cudaSuccess) return K8V4_ECUDA;
  return cudaGetLastError() == cudaSuccess ? K8V4_OK : K8V4_ECUDA;
}

}  // namespace k8v4
