// qk_norm_rope_k8v4: the per-head RMS norm of queries and keys (optional) and
// the position rotation, in one pass over the rows that the projection left.
//
//   x' = x / sqrt(mean(x^2) + eps) * w          (per head, w optional)
//   (y1, y2) = (x1 c - x2 s, x2 c + x1 s)       (pairs of the first rot_dim)
//
// What bounds it: memory.  A row is read once and written once (2 x 512 B in
// bf16) next to one table row per token, which all heads of the token share.  A
// warp owns a row (16 B a lane in bf16), so the norm is one butterfly and the
// partner of a pair one shuffle away; a warp takes `per` heads of one token, so
// that the table row and the norm weight are loaded once for them, and issues
// the loads of all of them before it uses the first.  Measured: 8,192 tokens of
// 16 + 2 heads in bf16, normed, out of a packed projection (153 MB): 27.3 us, 5.6 TB/s;
// a copy of as many bytes takes 26.2.  One token: 2.8 us, the latency of a launch and
// two dependent reads.
#include <algorithm>

#include "k8v4_quant.cuh"
#include "k8v4_rope.cuh"

namespace k8v4 {
namespace {

constexpr int kRopeWarps = 2;     // per CTA (8,192 tokens x 18 heads, us: 8 28.9, 4 27.8, 2 27.3)
constexpr int kRopeCtas = 16;     // per SM: 64 registers a thread

struct RopeParams {
  const void* q;
  const void* k;
  int64_t q_stride, k_stride;    // elements between tokens
  int n_q, n_k;                  // heads
  const float* q_weight;         // fp32 [256], or null
  const float* k_weight;
  float eps;
  const int64_t* pos;            // [n_seqs]
  int64_t n_tokens;              // n_seqs * n_tok
  const float* table;
  int64_t n_pos;
  int half;
  void* q_out;
  void* k_out;
  int units_q, units;            // warps per token: of the queries, of both
  FastDiv div_units, div_tok;
  int* status;
};

// PER: heads of one token that a warp takes
template <bool BF16, bool INTER, int PER>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeCtas) norm_rope_kernel(const RopeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t wi = static_cast<int64_t>(blockIdx.x) * kRopeWarps + w;
  if (wi >= p.n_tokens * p.units) return;
  const uint32_t item = static_cast<uint32_t>(wi);          // the host keeps warp indices below 2^31
  const uint32_t tok = p.div_units.div(item);
  int unit = static_cast<int>(item - tok * static_cast<uint32_t>(p.units));
  const uint32_t b = p.div_tok.div(tok);
  const bool is_k = unit >= p.units_q;
  if (is_k) unit -= p.units_q;
  const int heads = is_k ? p.n_k : p.n_q, h0 = unit * PER;
  const int64_t stride = is_k ? p.k_stride : p.q_stride;
  const void* src = is_k ? p.k : p.q;
  void* dst = is_k ? p.k_out : p.q_out;
  const float* weight = is_k ? p.k_weight : p.q_weight;
  const int64_t in0 = static_cast<int64_t>(tok) * stride + h0 * kD;
  const int64_t out0 = (static_cast<int64_t>(tok) * heads + h0) * kD;
  const RopeLane rl = rope_lane<INTER>(lane, p.half);

  uint4 raw[PER][BF16 ? 1 : 2];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (h0 + i < heads) {
      if (BF16) {
        raw[i][0] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + in0 + i * kD) + lane);
      } else {
        const uint4* r = reinterpret_cast<const uint4*>(static_cast<const float*>(src) + in0 + i * kD) + 2 * lane;
        raw[i][0] = __ldcs(r);
        raw[i][BF16 ? 0 : 1] = __ldcs(r + 1);
      }
    }
  }
  const int64_t at = p.pos[b] + (tok - static_cast<int64_t>(b) * p.div_tok.d);
  if (at < 0 || at >= p.n_pos) {                            // no table row: the token's output rows stay as they are
    if (lane == 0) record_status(p.status, K8V4_ERANGE);
    return;
  }
  RopeFactors<INTER> f;
  rope_load<INTER>(p.table + at * (2 * p.half), rl, p.half, f);
  float wt[8];
  if (weight) load_weight8(weight, lane, wt);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (h0 + i >= heads) break;
    float x[8];
    if (BF16) {
      bf16x8_to_f32(raw[i][0], x);
    } else {
      const uint4 a = raw[i][0], c = raw[i][BF16 ? 0 : 1];
      x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y); x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
      x[4] = __uint_as_float(c.x); x[5] = __uint_as_float(c.y); x[6] = __uint_as_float(c.z); x[7] = __uint_as_float(c.w);
    }
    float o[8];
    if (weight) {                                           // the same for the warp
      rms_row(x, wt, p.eps);
      rope_partners<INTER>(x, rl, o);
      rope_row<INTER, false>(x, o, rl, f);
    } else {
      if (BF16) rope_partners<INTER>(raw[i][0], rl, o);
      else rope_partners<INTER>(x, rl, o);
      rope_row<INTER, true>(x, o, rl, f);
    }
    if (BF16) {
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + out0 + i * kD)[lane] = f32x8_to_bf16(x);
    } else {
      float4* to = reinterpret_cast<float4*>(static_cast<float*>(dst) + out0 + i * kD) + 2 * lane;
      to[0] = make_float4(x[0], x[1], x[2], x[3]);
      to[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

template <bool BF16, bool INTER>
int launch_per(const Launch& L, RopeParams p, int per, int64_t warps) {
  const dim3 grid(static_cast<unsigned>((warps + kRopeWarps - 1) / kRopeWarps)), block(kRopeWarps * 32);
  return launch_behind(L, per == 1 ? norm_rope_kernel<BF16, INTER, 1> : norm_rope_kernel<BF16, INTER, BF16 ? 4 : 2>, grid, block, p);
}

}  // namespace

int launch_norm_rope(const Launch& L, const void* q, int64_t q_stride, int n_q, const void* k, int64_t k_stride,
                     int n_k, int dtype, const float* q_weight, const float* k_weight, float eps, const int64_t* pos,
                     int n_seqs, int n_tok, const k8v4_rope& rope, void* q_out, void* k_out) {
  RopeParams p;
  p.q = q;
  p.k = k;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.n_q = n_q;
  p.n_k = n_k;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.pos = pos;
  p.n_tokens = static_cast<int64_t>(n_seqs) * n_tok;
  p.table = rope.table;
  p.n_pos = rope.n_pos;
  p.half = rope.rot_dim / 2;
  p.q_out = q_out;
  p.k_out = k_out;
  p.status = L.status;
  // one head per warp while the rows leave SMs idle (latency), else several
  const int64_t rows = p.n_tokens * (n_q + n_k);
  const int per = rows <= static_cast<int64_t>(L.num_sms) * 32 ? 1 : dtype == K8V4_BF16 ? 4 : 2;
  p.units_q = (n_q + per - 1) / per;
  p.units = p.units_q + (n_k + per - 1) / per;
  p.div_units = FastDiv(static_cast<uint32_t>(p.units));
  p.div_tok = FastDiv(static_cast<uint32_t>(n_tok));
  const int64_t warps = p.n_tokens * p.units;
  if (warps >= (int64_t(1) << 31)) return K8V4_EINVAL;
  if (dtype == K8V4_BF16)
    return rope.interleaved ? launch_per<true, true>(L, p, per, warps) : launch_per<true, false>(L, p, per, warps);
  return rope.interleaved ? launch_per<false, true>(L, p, per, warps) : launch_per<false, false>(L, p, per, warps);
}

}  // namespace k8v4
