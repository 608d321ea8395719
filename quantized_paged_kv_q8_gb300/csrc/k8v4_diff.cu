// Differential attention of single queries over the k8v4 cache, split over the cells,
// and the combine of its partial rows:
//
//   x = A_1 V - lambda A_2 V,  A_m = softmax(scale q_m K_m^T) over lanes [128 m, 128 m + 128)
//   out = out_scale * x / sqrt(mean(x^2) + eps) * w        (bf16)
//
// The two maps of a head score the two halves of the same key rows and weigh the same
// values, so a cell's 408 bytes are read and converted once for both.  Each map has its
// own softmax statistics; they are known only at the end, so both products with V are kept
// (they share the converted V).  Per 16-cell tile a warp does
//   S_m^T = K_m q_m^T    8 + 8 products m16n8k16 (cells x 8 heads)
//   O_m^T += V^T P_m^T   16 + 16 products (dims x 8 heads), V converted once
// with K codes exact in fp16, q in fp16 (bf16 is exact after a power of two per row and
// map; fp32 takes two terms and twice the products of S, as in the decode kernel), P and V rounded to fp16 once each: 2^-11 of each term at most, against the 2^-8 of the
// bf16 result, where the plain decode carries both in two terms (48 products of V, not 32, and
// for one map).  V is (n - 8) d: a subnormal d is a multiple of fp16's least step, and so is
// (n - 8) d.  Only from d = 2^13 on does fp16 not hold it; a tile that has such a block (big_blocks)
// counts with V / 8 and 8 P, which is 3 added to its scores, and its values below 2^-11 to 2^-22.
//
// The worker warps are the decode kernel's: they take a range's tiles in turn, each with a ring of
// its own filled by TMA.  The ranges are not: the tiles of all (sequence, KV head) pairs, laid
// end to end, are cut into one equal piece for each SM, so that a ragged batch keeps every SM
// busy to the end.  A piece covers one pair's cells or the end of one and the beginning of others;
// each CTA finds its own from the lengths.
//
// What bounds it: the matrix instructions, about 6.8 clocks each on an SM (48 a tile: 32 us of one
// sequence of 237,568 cells), beside the conversions of the codes (about 980 instructions a tile in
// all); two warps a scheduler do not overlap them wholly.  That sequence, 2 KV heads: 58 us with the
// joining, 3.3 TB/s of the cache's 194 MB (fp32 queries, 64 products a tile: 62.5); 32 sequences of up to 8,192
// cells 41 us (44).  Two warps to a
// worker, each with a map's scores and half of V's dims (16 warps of 128 registers, weights handed
// over through shared memory): 63 us and 41.
#include <algorithm>
#include <climits>

#include "k8v4_diff.cuh"
#include "k8v4_tc.cuh"
#include "k8v4_tma.cuh"

namespace k8v4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxWorkers = 8;                // 255 registers a thread
constexpr int kStages = 2;
constexpr int kSmemCap = 227 * 1024;
constexpr uint32_t kWaitDefaultNs = 1000000000u;
constexpr int kBucketClamp = 1 << 24;
// a worker's partial in the epilogue: [8 heads x 2 maps][kHeadStride] floats of o, then
// 16 buckets and 16 sums (a stride of 4 mod 16 floats: conflict-free fragment stores)
constexpr int kHeadStride = 260;
constexpr int kPartBucket = 16 * kHeadStride;
constexpr int kPartSum = kPartBucket + 16;
constexpr int kPartFloats = kPartSum + 16;

struct Layout {
  int workers;
  int ksc_bytes, vsc_bytes, ksc_off, vsc_off;       // within a stage: K 4096, V 2048, K scales, V scales
  int stage_bytes, tx_bytes;
  int q_off, bar_off, ctl_off, total;
};
constexpr int kQTerm = 16 * 32 * 8;
constexpr int kVOff = 4096, kQBytes = 2 * kQTerm;  // q fragments [term][16 k-steps][32 lanes][2 words]

inline Layout layout_of(int H) {
  Layout L;
  L.ksc_bytes = 128 * H;
  L.vsc_bytes = 256 * H;
  L.ksc_off = kVOff + 2048;
  L.vsc_off = L.ksc_off + L.ksc_bytes;
  L.tx_bytes = L.vsc_off + L.vsc_bytes;
  L.stage_bytes = (std::max(L.tx_bytes, (kPartFloats * 4 + kStages - 1) / kStages) + 1023) & ~1023;
  for (L.workers = kMaxWorkers;; --L.workers) {
    L.q_off = L.workers * kStages * L.stage_bytes;
    L.bar_off = L.q_off + kQBytes;
    L.ctl_off = (L.bar_off + 8 * kStages * L.workers + 15) / 16 * 16;   // abort flag, the piece's sequence; sums of the warps
    L.total = L.ctl_off + 256 + 1024;
    if (L.total <= kSmemCap || L.workers == 1) break;
  }
  return L;
}

// The piece of CTA c of pair s has block c + s of the partial rows: along the line of tiles a block
// begins where a piece or a pair does.
constexpr int kMostCtas = kDiffMostRanges;
// What a CTA spends on a pair beside its tiles (query, first copies, the workers' merge), in tiles:
// each pair's tiles have that much empty line ahead of them, so that a piece with the end of one pair and
// the beginning of another is as long as the rest (one sequence of 237,568 cells, 2 heads: 64.7 us without)
constexpr int kPairTiles = 24;
__device__ __forceinline__ int64_t line_of(int tiles, int H) {         // of a sequence
  return tiles ? static_cast<int64_t>(H) * (tiles + kPairTiles) : 0;
}
// n / d for n, d >= 0, d > 0; the 64-bit routine only where it is needed
__device__ __forceinline__ int64_t quot(int64_t n, int64_t d) {
  if ((n | d) < (int64_t(1) << 31)) return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
  return n / d;
}

int ctas_of(int num_sms) { return std::min(num_sms, kMostCtas); }

struct DiffParams {
  CacheView C;
  const void* q;
  const int32_t* pt;
  int64_t max_pages;
  const int32_t* lens;        // visible cells of each query
  const int32_t* row_seq;     // a ragged batch's: the sequence and the packed token of each query, and their
  const int32_t* row_tok;     // number on the device; or null: query b is of sequence b, n_seqs of them
  const int32_t* count;
  int n_seqs, max_seq_len;
  float sm_scale_log2;
  DiffPieces ws;
  int* status;
  uint32_t wait_ns;
  FastDiv page_div;
  Layout L;
};

__device__ __forceinline__ void mma16(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float f16_lo(uint32_t h) { return __low2float(*reinterpret_cast<const __half2*>(&h)); }
__device__ __forceinline__ float f16_hi(uint32_t h) { return __high2float(*reinterpret_cast<const __half2*>(&h)); }
// 2^e exactly for e >= -126, 0 below
__device__ __forceinline__ float pow2i(int e) { return e < -126 ? 0.0f : __int_as_float((e + 127) << 23); }
// one word of nibble bytes b0..b3 -> four fp16x2 of n - 8, exact: {b0, b2} and {b1, b3}
// of the low nibbles, then of the high ones.  0x640n is 1024 + n and 0x64n0 is 1024 + 16 n in
// fp16; 1024 + n - 1032 and (1024 + 16 n) / 16 - 72 are both n - 8
__device__ __forceinline__ void nibs(uint32_t r, __half2 v[4]) {
  const uint32_t r8 = r >> 8;
  const __half2 m1032 = __halves2half2(__ushort_as_half(0xe408), __ushort_as_half(0xe408));     // -1032
  const __half2 c16th = __halves2half2(__ushort_as_half(0x2c00), __ushort_as_half(0x2c00));     // 1/16
  const __half2 m72 = __halves2half2(__ushort_as_half(0xd480), __ushort_as_half(0xd480));       // -72
  uint32_t t0 = (r & 0x000f000fu) | 0x64006400u, t1 = (r8 & 0x000f000fu) | 0x64006400u;
  uint32_t t2 = (r & 0x00f000f0u) | 0x64006400u, t3 = (r8 & 0x00f000f0u) | 0x64006400u;
  v[0] = __hadd2(*reinterpret_cast<__half2*>(&t0), m1032);
  v[1] = __hadd2(*reinterpret_cast<__half2*>(&t1), m1032);
  v[2] = __hfma2(*reinterpret_cast<__half2*>(&t2), c16th, m72);
  v[3] = __hfma2(*reinterpret_cast<__half2*>(&t3), c16th, m72);
}
__device__ __forceinline__ uint32_t times(__half2 a, uint32_t d) {
  const __half2 r = __hmul2(a, *reinterpret_cast<const __half2*>(&d));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// MMA row r (0..7) of a tile holds cell sigma(r), row r + 8 cell 8 + sigma(r): the two cells a
// quarter-warp reads in one 128-bit shared load then differ in bit 2, which the 128-byte
// swizzle turns into disjoint bank groups
__device__ __forceinline__ int sigma(int r) { return (r >> 1) | ((r & 1) << 2); }

// Wait for a phase: false once the bound has passed, or the CTA's abort flag is up
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, uint32_t limit_ns, const volatile int* abort) {
  if (mbar_test(bar, parity)) return true;
  if (limit_ns < 1000u) return false;
  const uint64_t t0 = global_ns();
  for (;;) {
    if (global_ns() - t0 >= limit_ns) return false;
    if (mbar_try(bar, parity, 20000u)) return true;
    if (*abort) return false;
  }
}

// ---------------------------------------------------------------- the split kernel
// grid: one CTA per SM
template <bool QF32>
__global__ void __launch_bounds__(32 * kMaxWorkers, 1)
    diff_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const DiffParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t sb = (raw_s + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (sb - raw_s);
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int W = blockDim.x >> 5;
  const Layout& LY = p.L;
  const uint32_t full = sb + LY.bar_off + 8 * kStages * w;               // this worker's stage barriers
  volatile int* ctl = reinterpret_cast<volatile int*>(sm + LY.ctl_off);  // [0] abort flag, [1] the piece's first sequence
  volatile int* abort_flag = ctl;
  if (threadIdx.x == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
    *abort_flag = 0;
  }
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(full + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const CacheView& C = p.C;
  const int H = C.H, HQ = H * kGqa;
  const int r0 = lane >> 2, c = lane & 3;
  auto len_of = [&](int b) { return min(max(p.lens[b], 0), p.max_seq_len); };
  // ---- this CTA's piece of the line of tiles
  int b = 0, g = 0;                          // sequence and KV head
  int64_t pos, end, per;                     // tiles of the line, [pos, end), and of a whole piece
  int64_t begin_b = 0;                       // the line's tile where sequence b begins
  {
    int64_t* sums = reinterpret_cast<int64_t*>(sm + LY.ctl_off + 32);    // of the warps
    int64_t* found = sums + kMaxWorkers;                                 // where the sequence of pos begins
    const int n_seqs = p.count ? *p.count : p.n_seqs;
    const int per_t = (n_seqs + blockDim.x - 1) / blockDim.x;
    const int s0 = min(n_seqs, static_cast<int>(threadIdx.x) * per_t), s1 = min(n_seqs, s0 + per_t);
    int64_t sum = 0;
    for (int i = s0; i < s1; ++i) {
      const int n = p.lens[i];
      if (blockIdx.x == 0 && (n < 0 || n > p.max_seq_len)) record_status(p.status, K8V4_ERANGE);
      sum += line_of((len_of(i) + 15) >> 4, H);
    }
    int64_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(kFull, scan, o);
      if (lane >= o) scan += u;
    }
    if (lane == 31) sums[w] = scan;
    __syncthreads();
    int64_t total = 0, ahead = scan - sum;
    for (int i = 0; i < W; ++i) {
      if (i < w) ahead += sums[i];
      total += sums[i];
    }
    per = max(quot(total + gridDim.x - 1, gridDim.x), static_cast<int64_t>(2 * W));   // at least two tiles a warp
    pos = min(blockIdx.x * per, total);
    end = min(pos + per, total);
    if (pos >= end) {                        // (the whole CTA)
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      return;
    }
    if (ahead <= pos && pos < ahead + sum) {
      int i = s0;
      for (;; ++i) {
        const int64_t n = line_of((len_of(i) + 15) >> 4, H);
        if (pos < ahead + n) break;
        ahead += n;
      }
      ctl[1] = i;
      *found = ahead;
    }
    __syncthreads();
    b = ctl[1];
    begin_b = *found;
    g = static_cast<int>(quot(pos - begin_b, ((len_of(b) + 15) >> 4) + kPairTiles));
  }
  int stage = 0;                             // of this worker's next tile, and its phase
  uint32_t phase = 0;
  bool aborted = false;                      // this warp left a loop with copies in flight
  const uint32_t ring = sb + w * kStages * LY.stage_bytes;
#pragma unroll 1
  while (pos < end) {
    // ---- a pair's part of the piece
    const int n_vis = len_of(b), pair_tiles = (n_vis + 15) >> 4;
    if (pair_tiles == 0) {                     // a sequence with nothing to see
      ++b;
      g = 0;
      continue;
    }
    const int64_t line0 = begin_b + static_cast<int64_t>(g) * (pair_tiles + kPairTiles) + kPairTiles;   // where its tiles begin
    pos = max(pos, line0);
    const int n_tiles = static_cast<int>(min(line0 + pair_tiles, end) - pos);
    if (n_tiles <= 0) break;                   // the piece ends ahead of them
    const int c_begin = 16 * static_cast<int>(pos - line0), c_end = min(c_begin + 16 * n_tiles, n_vis);
    const int pair = b * H + g;
    float* const rows = p.ws.rows + (static_cast<int64_t>(blockIdx.x) + pair) * 16 * kDiffRow;
    if (pos == line0 && threadIdx.x == 0) {
      const int first = static_cast<int>(quot(line0, per)), last = static_cast<int>(quot(line0 + pair_tiles - 1, per));
      p.ws.pairs[pair] = make_int2(first + pair, last - first + 1);
    }
    const int n_my = n_tiles > w ? (n_tiles - w + W - 1) / W : 0;          // tiles w + W u

    // ---- this worker's copies: local tile u -> the ring's next stage
    const int seq = p.row_seq ? p.row_seq[b] : b, tok = p.row_tok ? p.row_tok[b] : b;
    const int32_t* pt_row = p.pt + static_cast<int64_t>(seq) * p.max_pages;
    int win0 = -1000000, win_page = -1;
    auto page_of = [&](int u) -> int {         // warp-uniform u; all lanes call
      if (u < win0 || u >= win0 + 32) {
        win0 = u;
        const uint32_t cell = static_cast<uint32_t>(c_begin) + 16u * (w + W * (u + lane));     // (looked up only where it is one)
        const int64_t pidx = p.page_div.div(cell);
        win_page = (u + lane < n_my && pidx < p.max_pages) ? pt_row[pidx] : -1;
      }
      const int page = __shfl_sync(kFull, win_page, u - win0);
      return (page >= 0 && page < C.n_pages) ? page : -1;
    };
    // an out-of-range page issues no copy; its tile is skipped and recorded
    auto issue = [&](int u, int to, int page) {
      if (lane == 0) {
        const uint32_t st = ring + to * LY.stage_bytes, bar = full + 8 * to;
        if (page >= 0) {
          const int cell0 = c_begin + 16 * (w + W * u);
          const int slot0 = cell0 - static_cast<int>(p.page_div.div(static_cast<uint32_t>(cell0))) * C.P;
          mbar_expect_tx(bar, LY.tx_bytes);
          tma_load_4d(st, &tm_k, 0, g, slot0, page, bar);
          tma_load_4d(st + 2048, &tm_k, 128, g, slot0, page, bar);
          tma_load_4d(st + kVOff, &tm_v, 0, g, slot0, page, bar);
          const uint8_t* pg = C.pages + static_cast<int64_t>(page) * C.page_bytes;
          bulk_load(st + LY.ksc_off, pg + C.ks_off() + static_cast<int64_t>(slot0) * 8 * H, LY.ksc_bytes, bar);
          bulk_load(st + LY.vsc_off, pg + C.vs_off() + static_cast<int64_t>(slot0) * 16 * H, LY.vsc_bytes, bar);
        } else {
          record_status(p.status, K8V4_ERANGE);
          asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
        }
      }
    };
    const int stage0 = stage;
    int issued = 0;
    for (; issued < min(kStages, n_my); ++issued) issue(issued, (stage0 + issued) % kStages, page_of(issued));

    // ---- q fragments (B operand of S^T = K q^T) into shared memory: every warp works the factors out
    // for itself, warp 0 writes the fragments.  Lane (r0, c): head r0, dims 64 i + 16 c +
    // 4 j + e of k-step 4 i + j; k-steps 0..7 are map 0, 8..15 map 1, each with its own
    // power of two
    float f[2][2];                       // score factors: [map][heads 2c, 2c + 1]
    {
      const int64_t qrow = (static_cast<int64_t>(tok) * HQ + g * kGqa + r0) * kD;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float qv[32];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t e0 = qrow + 128 * m + 64 * i + 16 * c;
          if (QF32) {
            const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + e0);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const float4 v = src[t];
              qv[16 * i + 4 * t] = v.x; qv[16 * i + 4 * t + 1] = v.y;
              qv[16 * i + 4 * t + 2] = v.z; qv[16 * i + 4 * t + 3] = v.w;
            }
          } else {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + e0);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint4 v = src[t];
              const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                qv[16 * i + 8 * t + 2 * u] = __uint_as_float(wv[u] << 16);
                qv[16 * i + 8 * t + 2 * u + 1] = __uint_as_float(wv[u] & 0xffff0000u);
              }
            }
          }
        }
        float amax = 0.0f;
#pragma unroll
        for (int t = 0; t < 32; ++t) amax = fmaxf(amax, fabsf(qv[t]));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        const int ex = amax > 0.0f ? static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu) - 127 : 0;
        const int sh = max(-113, min(100, 14 - ex));              // amax * 2^sh in [2^14, 2^15)
        const float up = ldexpf(1.0f, sh);
        const float fscale = p.sm_scale_log2 * ldexpf(1.0f, -sh);
        if (w == 0) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const int o = 16 * (ks >> 2) + 4 * (ks & 3);
            const uint32_t h0 = pack_f16(qv[o] * up, qv[o + 1] * up), h1 = pack_f16(qv[o + 2] * up, qv[o + 3] * up);
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(sb + LY.q_off + ((8 * m + ks) * 32 + lane) * 8), "r"(h0), "r"(h1) : "memory");
            if (QF32) {
              const uint32_t l0 = pack_f16(qv[o] * up - f16_lo(h0), qv[o + 1] * up - f16_hi(h0));
              const uint32_t l1 = pack_f16(qv[o + 2] * up - f16_lo(h1), qv[o + 3] * up - f16_hi(h1));
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(sb + LY.q_off + kQTerm + ((8 * m + ks) * 32 + lane) * 8), "r"(l0), "r"(l1) : "memory");
            }
          }
        }
        f[m][0] = __shfl_sync(kFull, fscale, 8 * c);
        f[m][1] = __shfl_sync(kFull, fscale, 8 * c + 4);
      }
    }
    __syncthreads();

    // K fragment addresses within a stage (two 128-byte-swizzled [16][128] halves)
    const int rowA = sigma(r0), rowB = 8 + sigma(r0);
    uint32_t offA[2], offB[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      offA[i] = rowA * 128 + 16 * ((4 * i + c) ^ (rowA & 7));
      offB[i] = rowB * 128 + 16 * ((4 * i + c) ^ (rowB & 7));
    }
    const uint32_t ksA = LY.ksc_off + (rowA * H + g) * 8, ksB = LY.ksc_off + (rowB * H + g) * 8;
    // V fragment rows: matrix mi = lane >> 3 holds cells 8 (mi & 1) + sigma(0..7)
    const int mi = lane >> 3;
    const int vcell = 8 * (mi & 1) + sigma(lane & 7);
    const uint32_t vrow = kVOff + vcell * 128;
    const int vsw = vcell & 7;
    // the V scales of the fragment's four cells k = 2c, 2c+1, 2c+8, 2c+9
    const uint32_t soff0 = LY.vsc_off + (sigma(2 * c) * H + g) * 16, soff1 = LY.vsc_off + (sigma(2 * c + 1) * H + g) * 16;
    const uint32_t s8 = 8 * H * 16;
    const uint32_t half_row = LY.vsc_off + ((lane >> 1) * H + g) * 16 + 8 * (lane & 1);     // half of a cell's scales
    const uint32_t qf = sb + LY.q_off + 8 * lane;

    float o[2][16][4];                   // [map][16-dim m-tile][fragment]: heads 2c, 2c+1 of dims r0 (+8)
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int mt = 0; mt < 16; ++mt) o[m][mt][0] = o[m][mt][1] = o[m][mt][2] = o[m][mt][3] = 0.0f;
    int M[2][2] = {{INT_MIN, INT_MIN}, {INT_MIN, INT_MIN}};    // running buckets
    float l[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};

    int done = 0;
    for (int u = 0; u < n_my; ++u, ++done) {
      if (!__all_sync(kFull, wait_or_abort(full + 8 * stage, phase, p.wait_ns, abort_flag))) {
        if (lane == 0) {
          *abort_flag = 1;
          record_status(p.status, K8V4_ECUDA);
        }
        aborted = true;
        break;
      }
      const uint32_t st = ring + stage * LY.stage_bytes;
      if (page_of(u) >= 0) {
        const uint2 kAu = lds64(st + ksA), kBu = lds64(st + ksB);
        const int cell0 = c_begin + 16 * (w + W * u);
        const bool vA = cell0 + rowA < c_end, vB = cell0 + rowB < c_end;
        const uint2 dd = lds64(st + half_row);
        // a block that fp16 does not hold eight times over, of a cell that is seen
        const bool big = __any_sync(kFull, cell0 + (lane >> 1) < c_end && big_blocks(dd.x, dd.y));
        const bool odd = big || cell0 + 16 > c_end;
        const float more = big ? 3.0f : 0.0f, counts = big ? 0.125f : 1.0f;   // added to the scores, and what P counts in l
        uint32_t ph[2][2];
        // ---- S_m^T[cell][head] of both maps, two accumulators each
        float acc[2][2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int a4 = 0; a4 < 2; ++a4) acc[m][a4][0] = acc[m][a4][1] = acc[m][a4][2] = acc[m][a4][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint4 ka = lds128(st + 2048 * m + offA[i]);
            const uint4 kb = lds128(st + 2048 * m + offB[i]);
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t a[4];
              i8x4_to_f16(wa[j], a[0], a[2]);
              i8x4_to_f16(wb[j], a[1], a[3]);
              const uint2 qb = lds64(qf + (8 * m + 4 * i + j) * 256);
              mma16(acc[m][j & 1], a, qb.x, qb.y);
              if (QF32) {
                const uint2 ql = lds64(qf + kQTerm + (8 * m + 4 * i + j) * 256);
                mma16(acc[m][j & 1], a, ql.x, ql.y);
              }
            }
          }
        }
        float sc[2][4];
        bool up = false;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float kA = __uint_as_float(m ? kAu.y : kAu.x), kB = __uint_as_float(m ? kBu.y : kBu.x);
          sc[m][0] = vA ? fmaf(kA * (acc[m][0][0] + acc[m][1][0]), f[m][0], more) : -INFINITY;
          sc[m][1] = vA ? fmaf(kA * (acc[m][0][1] + acc[m][1][1]), f[m][1], more) : -INFINITY;
          sc[m][2] = vB ? fmaf(kB * (acc[m][0][2] + acc[m][1][2]), f[m][0], more) : -INFINITY;
          sc[m][3] = vB ? fmaf(kB * (acc[m][0][3] + acc[m][1][3]), f[m][1], more) : -INFINITY;
          up = up || sc[m][0] > 8.0f * M[m][0] || sc[m][2] > 8.0f * M[m][0] || sc[m][1] > 8.0f * M[m][1] || sc[m][3] > 8.0f * M[m][1];
        }
        // ---- softmax against the running bucket of each head (the decode kernel's), both maps at a time
        if (__any_sync(kFull, up)) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float t0 = fmaxf(sc[m][0], sc[m][2]), t1 = fmaxf(sc[m][1], sc[m][3]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              t0 = fmaxf(t0, __shfl_xor_sync(kFull, t0, off));
              t1 = fmaxf(t1, __shfl_xor_sync(kFull, t1, off));
            }
            const int nb0 = max(M[m][0], static_cast<int>(fminf(fmaxf(ceilf(t0 * 0.125f), -kBucketClamp), kBucketClamp)));
            const int nb1 = max(M[m][1], static_cast<int>(fminf(fmaxf(ceilf(t1 * 0.125f), -kBucketClamp), kBucketClamp)));
            const float g0 = M[m][0] == INT_MIN ? 0.0f : pow2i(8 * (M[m][0] - nb0));
            const float g1 = M[m][1] == INT_MIN ? 0.0f : pow2i(8 * (M[m][1] - nb1));
#pragma unroll
            for (int mt = 0; mt < 16; ++mt) {
              o[m][mt][0] *= g0; o[m][mt][2] *= g0;
              o[m][mt][1] *= g1; o[m][mt][3] *= g1;
            }
            l[m][0] *= g0;
            l[m][1] *= g1;
            M[m][0] = nb0;
            M[m][1] = nb1;
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const float rf0 = 8.0f * M[m][0] - 14.0f, rf1 = 8.0f * M[m][1] - 14.0f;
          const float p0 = ex2_ftz(sc[m][0] - rf0), p1 = ex2_ftz(sc[m][1] - rf1);      // p' = 2^(s - ref + 14) <= 2^14
          const float p2 = ex2_ftz(sc[m][2] - rf0), p3 = ex2_ftz(sc[m][3] - rf1);
          l[m][0] = fmaf(p0 + p2, counts, l[m][0]);
          l[m][1] = fmaf(p1 + p3, counts, l[m][1]);
          // to the B layout (head r0; cells 2c, 2c+1 | 2c+8, 2c+9)
          ph[m][0] = movmatrix_t(pack_f16(p0, p1));
          ph[m][1] = movmatrix_t(pack_f16(p2, p3));
        }
        // ---- PV of both maps in rotated space: V = RN((n - 8) d), m-tile 2 blk + hf = block
        // blk, dims 16 hf .. 16 hf + 15
#pragma unroll
        for (int bp = 0; bp < 4; ++bp) {
          uint32_t R[4];
          ldmatrix_x4_t(R, st + vrow + 16 * ((2 * bp + (mi >> 1)) ^ vsw));
          uint32_t w0 = lds32(st + soff0 + 4 * bp), w1 = lds32(st + soff1 + 4 * bp);
          uint32_t w2 = lds32(st + soff0 + s8 + 4 * bp), w3 = lds32(st + soff1 + s8 + 4 * bp);
          if (odd) {
            if (big) w0 = eighth_of(w0), w1 = eighth_of(w1), w2 = eighth_of(w2), w3 = eighth_of(w3);
            // cells that nobody sees count with V = 0: their bytes are anything
            if (cell0 + sigma(2 * c) >= c_end) w0 = 0;
            if (cell0 + sigma(2 * c + 1) >= c_end) w1 = 0;
            if (cell0 + 8 + sigma(2 * c) >= c_end) w2 = 0;
            if (cell0 + 8 + sigma(2 * c + 1) >= c_end) w3 = 0;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sel = h ? 0x7632u : 0x5410u;
            const uint32_t d01 = prmt(w0, w1, sel), d89 = prmt(w2, w3, sel);     // d of block 2bp+h, cell pairs
            __half2 xa[4], xb[4];
            nibs(R[2 * h], xa);
            nibs(R[2 * h + 1], xb);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t a[4] = {times(xa[2 * hf], d01), times(xa[2 * hf + 1], d01), times(xb[2 * hf], d89), times(xb[2 * hf + 1], d89)};
              mma16(o[0][2 * (2 * bp + h) + hf], a, ph[0][0], ph[0][1]);
              mma16(o[1][2 * (2 * bp + h) + hf], a, ph[1][0], ph[1][1]);
            }
          }
        }
      }
      __syncwarp();
      if (issued < n_my) {
        issue(issued, stage, page_of(issued));
        ++issued;
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        l[m][0] += __shfl_xor_sync(kFull, l[m][0], off);
        l[m][1] += __shfl_xor_sync(kFull, l[m][1], off);
      }
    }

    // ---------------------------------------------------------------- epilogue
    // a worker that left early first waits (bounded) for its copies in flight: the stages from its next one on
    if (aborted && lane == 0) {
      const int left = issued - done;
      for (int k = 0; k < left; ++k) {
        const uint32_t ph = stage + k >= kStages ? phase ^ 1 : phase;
        const uint64_t t0 = global_ns();
        while (!mbar_try(full + 8 * ((stage + k) % kStages), ph, 20000u) && global_ns() - t0 < kWaitDefaultNs) {
        }
      }
    }
    __syncwarp();
    float* mine = reinterpret_cast<float*>(sm + w * kStages * LY.stage_bytes);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const bool live0 = M[m][0] != INT_MIN, live1 = M[m][1] != INT_MIN;
      float* base = mine + 8 * m * kHeadStride;
#pragma unroll
      for (int mt = 0; mt < 16; ++mt) {
        const int d0 = 32 * (mt >> 1) + 16 * (mt & 1) + 2 * r0;
        *reinterpret_cast<float2*>(base + (2 * c) * kHeadStride + d0) =
            live0 ? make_float2(o[m][mt][0], o[m][mt][2]) : make_float2(0.0f, 0.0f);
        *reinterpret_cast<float2*>(base + (2 * c + 1) * kHeadStride + d0) =
            live1 ? make_float2(o[m][mt][1], o[m][mt][3]) : make_float2(0.0f, 0.0f);
      }
      if (r0 == 0) {
        reinterpret_cast<int*>(mine + kPartBucket)[8 * m + 2 * c] = M[m][0];
        reinterpret_cast<int*>(mine + kPartBucket)[8 * m + 2 * c + 1] = M[m][1];
        mine[kPartSum + 8 * m + 2 * c] = l[m][0];
        mine[kPartSum + 8 * m + 2 * c + 1] = l[m][1];
      }
    }
    __syncthreads();
    // a warp per (map, head): the workers' partials at the largest bucket, in rotated space
    for (int h = w; h < 16; h += W) {
      const float* mj_part = reinterpret_cast<const float*>(sm + min(lane, W - 1) * kStages * LY.stage_bytes);
      const int mj = lane < W ? reinterpret_cast<const int*>(mj_part + kPartBucket)[h] : INT_MIN;
      const float lj = lane < W ? mj_part[kPartSum + h] : 0.0f;
      const int Mx = __reduce_max_sync(kFull, mj);
      const float fj = mj == INT_MIN ? 0.0f : pow2i(8 * (mj - Mx));
      float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      float Ls = 0.0f;
#pragma unroll
      for (int j = 0; j < kMaxWorkers; ++j) {
        const float fw = __shfl_sync(kFull, fj, j), lw = __shfl_sync(kFull, lj, j);   // 0 for j >= W
        if (j < W) {
          const float* src = reinterpret_cast<const float*>(sm + j * kStages * LY.stage_bytes) + h * kHeadStride;
          const float4 x0 = *reinterpret_cast<const float4*>(src + 4 * lane);
          const float4 x1 = *reinterpret_cast<const float4*>(src + 128 + 4 * lane);
          v[0] += x0.x * fw; v[1] += x0.y * fw; v[2] += x0.z * fw; v[3] += x0.w * fw;
          v[4] += x1.x * fw; v[5] += x1.y * fw; v[6] += x1.z * fw; v[7] += x1.w * fw;
          Ls += lw * fw;
        }
      }
      constexpr float kInv = 1.0f / 16384.0f;    // 2^-14 of p'
      float* dst = rows + h * kDiffRow;
      reinterpret_cast<float4*>(dst)[lane] = make_float4(v[0] * kInv, v[1] * kInv, v[2] * kInv, v[3] * kInv);
      reinterpret_cast<float4*>(dst)[32 + lane] = make_float4(v[4] * kInv, v[5] * kInv, v[6] * kInv, v[7] * kInv);
      if (lane == 0) {
        dst[256] = Mx == INT_MIN ? -INFINITY : static_cast<float>(8 * Mx);
        dst[257] = Ls * (1.0f / 16384.0f);
      }
    }
    // the next pair's copies overwrite what the workers wrote and the merge read; after a failure the CTA leaves (its
    // other pieces' rows would be older ones: their blocks are marked empty)
    fence_async_smem();
    const bool stop = *abort_flag != 0;        // (the same in every warp: behind the barrier one may fail in the next pair already)
    __syncthreads();
    pos += n_tiles;
    if (++g == H) {
      g = 0;
      begin_b += line_of(pair_tiles, H);
      ++b;
    }
    if (stop) break;
  }
#pragma unroll 1
  while (pos < end) {                        // (only after a failure)
    const int pair_tiles = (len_of(b) + 15) >> 4;
    if (pair_tiles) {
      const int64_t line0 = begin_b + static_cast<int64_t>(g) * (pair_tiles + kPairTiles) + kPairTiles;
      const int pair = b * H + g;
      pos = max(pos, line0);
      if (pos >= end) break;
      float* const rows = p.ws.rows + (static_cast<int64_t>(blockIdx.x) + pair) * 16 * kDiffRow;
      if (threadIdx.x < 16) {
        rows[threadIdx.x * kDiffRow + 256] = -INFINITY;
        rows[threadIdx.x * kDiffRow + 257] = 0.0f;
      }
      if (pos == line0 && threadIdx.x == 0) {
        const int first = static_cast<int>(quot(line0, per)), last = static_cast<int>(quot(line0 + pair_tiles - 1, per));
        p.ws.pairs[pair] = make_int2(first + pair, last - first + 1);
      }
      pos = min(line0 + pair_tiles, end);
    }
    if (pair_tiles == 0 || ++g == H) {
      g = 0;
      begin_b += line_of(pair_tiles, H);
      ++b;
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------------- the combine
struct CombineParams {
  const float* ws;
  DiffRagged r;               // a ragged batch's rows
  DiffPieces pieces;          // those of single queries
  const int32_t* lens;        // and the cells that each sees, max_seq_len at most
  int max_seq_len, H, n_rows;              // rows: (sequence or token, query head)
  k8v4_diff d;
  uint16_t* out;
};
constexpr int kCombineThreads = 128;        // or 32 WARPS, where a row takes more

// a warp: the difference in rotated space (lane: dims 4 lane + e and 128 + 4 lane + e) brought
// back (linear, so once for both maps), normed, scaled, rounded and written
__device__ __forceinline__ void finish_row(float v[8], const k8v4_diff& d, int lane, uint16_t* out) {
#pragma unroll
  for (int hh = 1; hh < 8; hh <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e & hh) continue;
      const float a = v[e], bb = v[e + hh];
      v[e] = a + bb;
      v[e + hh] = a - bb;
    }
  }
#pragma unroll
  for (int mm = 1; mm < 32; mm <<= 1) {
    const float sign = (lane & mm) ? -1.0f : 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = fmaf(sign, v[e], __shfl_xor_sync(kFull, v[e], mm));       // (exactly the difference or the sum)
    }
  }
  float s2 = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] *= 0.0625f;
    s2 += v[e] * v[e];
  }
  if (d.norm_weight) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s2 += __shfl_xor_sync(kFull, s2, o);
    const bool seen = s2 != 0.0f;        // a row of zeros stays one where eps is 0
    const float scale = seen ? rsqrtf(s2 * (1.0f / kD) + d.eps) * d.out_scale : 0.0f;
    const float4 wa = reinterpret_cast<const float4*>(d.norm_weight)[lane], wb = reinterpret_cast<const float4*>(d.norm_weight)[32 + lane];
    v[0] *= scale * wa.x; v[1] *= scale * wa.y; v[2] *= scale * wa.z; v[3] *= scale * wa.w;
    v[4] *= scale * wb.x; v[5] *= scale * wb.y; v[6] *= scale * wb.z; v[7] *= scale * wb.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= d.out_scale;
  }
  auto two = [](float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&x);
  };
  uint2* dst = reinterpret_cast<uint2*>(out);
  dst[lane] = make_uint2(two(v[0], v[1]), two(v[2], v[3]));
  dst[32 + lane] = make_uint2(two(v[4], v[5]), two(v[6], v[7]));
}

// WARPS to a (row, query head): sixteen where a few rows have tens of ranges each (one sequence of
// 237,568 cells: 16 rows of 76, 10 us cold), one where there are thousands of rows of a few (11,700 CTAs
// of four rows, 97 MB of partial rows and 24 MB of results, bound by its instructions: 40 registers for
// twelve CTAs an SM, the lambdas worked out ahead), four between.  Sixteen on more rows than SMs wait in line (78 registers: one row an SM): 256 rows of five
// ranges 13 us, with four 8.8.
template <int WARPS, bool RAGGED>
__global__ void __launch_bounds__(WARPS > 4 ? 32 * WARPS : kCombineThreads, WARPS == 1 ? 12 : 1) diff_combine_kernel(const CombineParams p) {
  constexpr int kRowsCta = WARPS > 4 ? 1 : kCombineThreads / 32 / WARPS;
  constexpr int kMost = kDiffMostRanges;
  __shared__ float wt[kRowsCta][2][kMost];
  __shared__ float red[kRowsCta][2][2][WARPS];
  __shared__ float4 part[WARPS > 1 ? kRowsCta : 1][2][WARPS][64];
  __shared__ float lam_s[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, slot = (threadIdx.x >> 5) / WARPS, warp = (threadIdx.x >> 5) % WARPS;
  const int t = warp * 32 + lane;                       // of the row's threads
  const int rr = blockIdx.x * kRowsCta + slot;
  if (rr >= p.n_rows) return;
  const int HQ = p.H * kGqa;
  const int row = rr / HQ, hq = rr - row * HQ;
  const int g = hq / kGqa, h = hq % kGqa;
  const float* base;                                    // range s of map m: base + m * m_stride + s * s_stride
  int64_t m_stride, s_stride;
  int splits;
  const int i = RAGGED ? p.r.tok_tile[row] : -2 - row;
  if (i == -1) return;                                  // no sequence's: left as it is
  if (RAGGED && i >= 0) {
    const int32_t* tile = p.r.tiles + 8 * static_cast<int64_t>(i);
    splits = min(tile[3], kMost);
    s_stride = 256 * kDiffRow;
    m_stride = s_stride * splits;
    base = p.ws + (static_cast<int64_t>(tile[4]) + 2 * g * splits) * s_stride + ((row - tile[1]) * kGqa + h) * kDiffRow;
  } else {
    const int len = min(p.lens[-2 - i], p.max_seq_len);
    int2 at = p.pieces.pairs[static_cast<int64_t>(-2 - i) * p.H + g];      // not written where there is nothing to see
    if (len <= 0 || at.x < 0 || at.y < 0 || at.x > p.pieces.blocks - at.y) at = make_int2(0, 0);   // (nor behind a failed wait)
    splits = min(at.y, kMost);
    m_stride = kGqa * kDiffRow;
    s_stride = 2 * m_stride;
    base = p.pieces.rows + at.x * s_stride + h * kDiffRow;
  }
  auto sync = [] {
    if (WARPS == 1) __syncwarp();
    else __syncthreads();
  };
  // one range, as most rows of a long batch have: no weights to work out, every load at once
  if (WARPS == 1 && splits == 1) {
    float4 x[2][2];
    float l[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const float4* src = reinterpret_cast<const float4*>(base + m * m_stride);
      x[m][0] = __ldcs(src + lane);
      x[m][1] = __ldcs(src + 32 + lane);
      l[m] = base[m * m_stride + 257];
    }
    const float lambda = p.r.lambdas[hq];               // (only ragged batches have a warp to a row)
    const float f0 = l[0] > 0.0f ? 1.0f / l[0] : 0.0f, f1 = l[1] > 0.0f ? -lambda / l[1] : 0.0f;
    // (what a range in which the row sees nothing left in o counts with 0)
    float v[8];
    auto join = [&](float a, float b) { return (f0 != 0.0f ? a * f0 : 0.0f) + (f1 != 0.0f ? b * f1 : 0.0f); };
    v[0] = join(x[0][0].x, x[1][0].x); v[1] = join(x[0][0].y, x[1][0].y);
    v[2] = join(x[0][0].z, x[1][0].z); v[3] = join(x[0][0].w, x[1][0].w);
    v[4] = join(x[0][1].x, x[1][1].x); v[5] = join(x[0][1].y, x[1][1].y);
    v[6] = join(x[0][1].z, x[1][1].z); v[7] = join(x[0][1].w, x[1][1].w);
    finish_row(v, p.d, lane, p.out + static_cast<int64_t>(rr) * kD);
    return;
  }
  float Mx[2], L[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    Mx[m] = -INFINITY;
    for (int s = t; s < splits; s += 32 * WARPS) {
      const float v = base[m * m_stride + s * s_stride + 256];
      wt[slot][m][s] = v;
      Mx[m] = fmaxf(Mx[m], v);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) Mx[m] = fmaxf(Mx[m], __shfl_xor_sync(kFull, Mx[m], o));
    if (WARPS > 1 && lane == 0) red[slot][0][m][warp] = Mx[m];
  }
  float term[2] = {0.0f, 0.0f};
  if (!RAGGED && warp < 2) {
    const float e = diff_lambda_term(p.d, hq, warp, lane);
    if (lane == 0) lam_s[warp] = e;
  }
  sync();
#pragma unroll
  for (int m = 0; m < 2; ++m) {
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
      if (WARPS > 1) Mx[m] = fmaxf(Mx[m], red[slot][0][m][w]);
    L[m] = 0.0f;
    for (int s = t; s < splits; s += 32 * WARPS) {
      const float v = wt[slot][m][s], w = v == -INFINITY ? 0.0f : exp2f(v - Mx[m]);
      if (w != 0.0f) L[m] += w * base[m * m_stride + s * s_stride + 257];
      wt[slot][m][s] = w;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) L[m] += __shfl_xor_sync(kFull, L[m], o);
    if (WARPS > 1 && lane == 0) red[slot][1][m][warp] = L[m];
  }
  sync();
  float acc[2][8];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[m][e] = 0.0f;
    constexpr int kUnroll = WARPS == 1 ? 1 : 4;
    for (int s0 = warp; s0 < splits; s0 += WARPS * kUnroll) {
      float4 x[kUnroll][2];
      float w[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int s = s0 + WARPS * k;
        w[k] = s < splits ? wt[slot][m][s] : 0.0f;
        if (w[k] != 0.0f) {                             // a range with nothing seen has no o either
          const float4* src = reinterpret_cast<const float4*>(base + m * m_stride + s * s_stride);
          x[k][0] = src[lane];
          x[k][1] = src[32 + lane];
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (w[k] == 0.0f) continue;
        acc[m][0] += x[k][0].x * w[k]; acc[m][1] += x[k][0].y * w[k]; acc[m][2] += x[k][0].z * w[k]; acc[m][3] += x[k][0].w * w[k];
        acc[m][4] += x[k][1].x * w[k]; acc[m][5] += x[k][1].y * w[k]; acc[m][6] += x[k][1].z * w[k]; acc[m][7] += x[k][1].w * w[k];
      }
    }
    if (WARPS > 1) {
      part[slot][m][warp][lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
      part[slot][m][warp][32 + lane] = make_float4(acc[m][4], acc[m][5], acc[m][6], acc[m][7]);
    }
  }
  if (WARPS > 1) {
    __syncthreads();
    if (warp) return;
    if (!RAGGED) {
      term[0] = lam_s[0];
      term[1] = lam_s[1];
    }
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      L[m] = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        L[m] += red[slot][1][m][w];
        if (w == 0) continue;
        const float4 a = part[slot][m][w][lane], b = part[slot][m][w][32 + lane];
        acc[m][0] += a.x; acc[m][1] += a.y; acc[m][2] += a.z; acc[m][3] += a.w;
        acc[m][4] += b.x; acc[m][5] += b.y; acc[m][6] += b.z; acc[m][7] += b.w;
      }
    }
  }
  const float lambda = RAGGED ? p.r.lambdas[hq] : p.d.lambda_q1 ? term[0] - term[1] + p.d.lambda_init : p.d.lambda_init;
  const float f0 = L[0] > 0.0f ? 1.0f / L[0] : 0.0f, f1 = L[1] > 0.0f ? -lambda / L[1] : 0.0f;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = acc[0][e] * f0 + acc[1][e] * f1;
  finish_row(v, p.d, lane, p.out + static_cast<int64_t>(rr) * kD);
}

}  // namespace

// ---------------------------------------------------------------- host side
bool diff_supported(const CacheView& C) {
  return C.fmt == K8V4_FORMAT_K8V4 && C.n_pages < (int64_t(1) << 31) && C.page_bytes < (int64_t(1) << 39);
}

size_t place_pieces(DiffPieces* p, uint8_t* ws, int64_t n_pairs, int num_sms) {
  const size_t head = (static_cast<size_t>(n_pairs) * sizeof(int2) + 255) / 256 * 256;
  if (p) {
    p->pairs = reinterpret_cast<int2*>(ws);
    p->rows = reinterpret_cast<float*>(ws + head);
    p->blocks = static_cast<int>(n_pairs) + ctas_of(num_sms);
  }
  return head + (static_cast<size_t>(n_pairs) + ctas_of(num_sms)) * 16 * kDiffRow * sizeof(float);
}
size_t diff_decode_ws_bytes(const CacheView& C, int n_seqs, int num_sms) {
  return place_pieces(nullptr, nullptr, static_cast<int64_t>(n_seqs) * C.H, num_sms);
}

int launch_diff_combine_ragged(const Launch& L, const float* ws, const DiffRagged& r, const DiffPieces& pieces,
                               const int32_t* lens, int n_tok, int H, bool few, const k8v4_diff& diff, void* out) {
  CombineParams p;
  p.ws = ws;
  p.r = r;
  p.pieces = pieces;
  p.lens = lens;
  p.max_seq_len = INT_MAX;                              // (the schedule's are clipped)
  p.H = H;
  p.n_rows = n_tok * H * kGqa;                          // below 2^30
  p.d = diff;
  p.out = static_cast<uint16_t*>(out);
  // (16 warps' registers leave an SM one row at a time)
  if (few && p.n_rows <= L.num_sms) return launch_behind(L, diff_combine_kernel<16, true>, dim3(p.n_rows), dim3(512), p);
  if (few) return launch_behind(L, diff_combine_kernel<4, true>, dim3(p.n_rows), dim3(kCombineThreads), p);
  return launch_behind(L, diff_combine_kernel<1, true>, dim3((p.n_rows + 3) / 4), dim3(kCombineThreads), p);
}

int launch_diff_split(const Launch& L, const CacheView& C, const void* q, int q_dtype, const int32_t* pt, int64_t max_pages,
                      const int32_t* lens, const DiffQueries& rows, int n_seqs, int max_seq_len, float sm_scale,
                      const DiffPieces& ws) {
  DiffParams p;
  p.C = C;
  p.q = q;
  p.pt = pt;
  p.max_pages = max_pages;
  p.lens = lens;
  p.row_seq = rows.seq;
  p.row_tok = rows.tok;
  p.count = rows.count;
  p.n_seqs = n_seqs;
  p.max_seq_len = max_seq_len;
  p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  p.ws = ws;
  p.status = L.status;
  p.wait_ns = wait_limit_ns() ? wait_limit_ns() : kWaitDefaultNs;
  p.page_div = FastDiv(static_cast<uint32_t>(C.P));
  p.L = layout_of(C.H);
  CUtensorMap mk, mv;
  if (!tensor_maps_of(C, &mk, &mv)) return K8V4_ECUDA;
  const auto kernel = q_dtype == K8V4_F32 ? diff_split_kernel<true> : diff_split_kernel<false>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, p.L.total) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
    return K8V4_ECUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas_of(L.num_sms));
  cfg.blockDim = dim3(32 * p.L.workers);
  cfg.dynamicSmemBytes = p.L.total;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, mk, mv, p) != cudaSuccess) return K8V4_ECUDA;
  return cudaGetLastError() == cudaSuccess ? K8V4_OK : K8V4_ECUDA;
}

int launch_diff_decode(const Launch& L, const CacheView& C, const void* q, int q_dtype, const int32_t* pt, int64_t max_pages,
                       const int32_t* lens, int n_seqs, int max_seq_len, float sm_scale, const k8v4_diff& diff, void* out,
                       void* ws) {
  DiffPieces pieces;
  place_pieces(&pieces, static_cast<uint8_t*>(ws), static_cast<int64_t>(n_seqs) * C.H, L.num_sms);
  const int rc = launch_diff_split(L, C, q, q_dtype, pt, max_pages, lens, DiffQueries{}, n_seqs, max_seq_len, sm_scale, pieces);
  if (rc) return rc;
  CombineParams c;
  c.ws = nullptr;
  c.r = DiffRagged{nullptr, nullptr, nullptr};
  c.pieces = pieces;
  c.lens = lens;
  c.max_seq_len = max_seq_len;
  c.H = C.H;
  c.n_rows = n_seqs * C.H * kGqa;
  c.d = diff;
  c.out = static_cast<uint16_t*>(out);
  // the pieces are one to an SM: few pairs have many each
  if (n_seqs * C.H * 8 <= ctas_of(L.num_sms)) return launch_behind(L, diff_combine_kernel<16, false>, dim3(c.n_rows), dim3(512), c);
  return launch_behind(L, diff_combine_kernel<4, false>, dim3(c.n_rows), dim3(kCombineThreads), c);
}

}  // namespace k8v4
