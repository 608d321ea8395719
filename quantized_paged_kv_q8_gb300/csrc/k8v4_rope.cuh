// Device helpers of the position rotation: one 256-element row of a query or
// key head held by a warp, 8 elements per lane (element 8 * lane + r), with the
// optional RMS norm ahead of the rotation.  Shared by the norm-and-rotate kernel
// and the rotating append, so both give the same bits.
//
// For a pair (x1, x2) at angle a the rotation gives
//   y1 = x1 cos a - x2 sin a,   y2 = x2 cos a + x1 sin a,
// the cosine and sine being fp32 entries of the caller's table.  The pairs are
// the elements (i, i + rot_dim / 2) or (2i, 2i + 1) of the first rot_dim
// elements; the others pass through.
//
// Rounding: without a norm, y is the exact x1 c - x2 s rounded to fp32 (to 2^-46 of
// the larger product before that rounding), then to the row's type.  The stored K
// codes are rints of quotients of these values, so one fp32 unit here moves a
// code now and then; with the products' errors carried, the result does not
// depend on how a compiler fuses the multiply and the subtraction.  Behind a norm,
// whose own result is a few fp32 units off, one product is rounded and the other
// fused (2 packed instructions where the carried form takes 13).
#pragma once

#include "k8v4_common.cuh"

namespace k8v4 {
namespace {

// x c + o s for two elements (the packed fp32 instructions), the error terms of
// both products and of their sum carried: p - npe = x c and q - nqe = o s exactly,
// d + de = p + q exactly.  Differences are fused multiplies by -1: the packed
// forms negate no operand.
__device__ __forceinline__ float2 dot2_carried(float2 x, float2 c, float2 o, float2 s) {
  const float2 m1 = make_float2(-1.0f, -1.0f);
  const float2 p = __fmul2_rn(x, c), q = __fmul2_rn(o, s);
  const float2 npe = __ffma2_rn(__fmul2_rn(x, m1), c, p), nqe = __ffma2_rn(__fmul2_rn(o, m1), s, q);
  const float2 d = __fadd2_rn(p, q);
  const float2 bb = __ffma2_rn(p, m1, d);
  const float2 de = __fadd2_rn(__ffma2_rn(__ffma2_rn(bb, m1, d), m1, p), __ffma2_rn(bb, m1, q));
  return __fadd2_rn(d, __ffma2_rn(__fadd2_rn(npe, nqe), m1, de));
}

// the same with one product rounded
__device__ __forceinline__ float2 dot2_plain(float2 x, float2 c, float2 o, float2 s) {
  return __ffma2_rn(x, c, __fmul2_rn(o, s));
}

// Where a lane's 8 elements get their cosines and sines from, and which lane
// holds their partners.  half = rot_dim / 2, a multiple of 8.
struct RopeLane {
  bool on;        // this lane's elements rotate
  int at;         // first table column of the cosines
  int partner;    // lane of the partners (the lane itself for adjacent pairs)
  float sign;     // of the sine: -1 for the first half of split pairs
};
template <bool INTER>
__device__ __forceinline__ RopeLane rope_lane(int lane, int half) {
  RopeLane r;
  r.on = 8 * lane < 2 * half;
  if (INTER) {
    r.at = 4 * lane;
    r.partner = lane;
    r.sign = 1.0f;
  } else {
    const bool first = 8 * lane < half;
    r.at = first ? 8 * lane : 8 * lane - half;
    r.partner = !r.on ? lane : first ? lane + (half >> 3) : lane - (half >> 3);
    r.sign = first ? -1.0f : 1.0f;
  }
  return r;
}

// The lane's cosines and signed sines of one table row: 8 of each for split
// pairs, 4 of each for adjacent ones.
template <bool INTER>
struct RopeFactors {
  float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
};
template <bool INTER>
__device__ __forceinline__ void rope_load(const float* row, const RopeLane& rl, int half,
                                          RopeFactors<INTER>& f) {
  if (!rl.on) return;
  const float4* c4 = reinterpret_cast<const float4*>(row + rl.at);
  const float4* s4 = reinterpret_cast<const float4*>(row + half + rl.at);
#pragma unroll
  for (int i = 0; i < (INTER ? 1 : 2); ++i) {
    const float4 a = __ldca(c4 + i), b = __ldca(s4 + i);
    f.c[4 * i] = a.x; f.c[4 * i + 1] = a.y; f.c[4 * i + 2] = a.z; f.c[4 * i + 3] = a.w;
    f.s[4 * i] = rl.sign * b.x; f.s[4 * i + 1] = rl.sign * b.y; f.s[4 * i + 2] = rl.sign * b.z; f.s[4 * i + 3] = rl.sign * b.w;
  }
}

// Rotate the row in place (all lanes call; lanes past rot_dim keep their values).
// o: the partners' values (split pairs; adjacent ones are the lane's own).
template <bool INTER, bool CARRIED>
__device__ __forceinline__ void rope_row(float x[8], const float o[8], const RopeLane& rl, const RopeFactors<INTER>& f) {
  auto dot2 = [](float2 v, float2 c, float2 w, float2 s) { return CARRIED ? dot2_carried(v, c, w, s) : dot2_plain(v, c, w, s); };
  if (!rl.on) return;
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = make_float2(x[2 * i], x[2 * i + 1]);
      const float2 y = dot2(v, make_float2(f.c[i], f.c[i]), make_float2(v.y, v.x), make_float2(-f.s[i], f.s[i]));
      x[2 * i] = y.x;
      x[2 * i + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int r = 0; r < 8; r += 2) {
      const float2 y = dot2(make_float2(x[r], x[r + 1]), make_float2(f.c[r], f.c[r + 1]), make_float2(o[r], o[r + 1]),
                            make_float2(f.s[r], f.s[r + 1]));
      x[r] = y.x;
      x[r + 1] = y.y;
    }
  }
}
// the partners of split pairs: by value, or (bf16 rows as they were loaded) two to a word
template <bool INTER>
__device__ __forceinline__ void rope_partners(const float x[8], const RopeLane& rl, float o[8]) {
#pragma unroll
  for (int r = 0; r < 8; ++r) o[r] = INTER ? 0.0f : __shfl_sync(0xffffffffu, x[r], rl.partner);
}
template <bool INTER>
__device__ __forceinline__ void rope_partners(const uint4& raw, const RopeLane& rl, float o[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t y = INTER ? 0u : __shfl_sync(0xffffffffu, w[i], rl.partner);
    o[2 * i] = __uint_as_float(y << 16);
    o[2 * i + 1] = __uint_as_float(y & 0xffff0000u);
  }
}

// x * rsqrt(mean(x^2) + eps) * w over the row's 256 elements, fp32 throughout
// (the squares summed 8 to a lane, then by a butterfly: the same order for every
// caller)
__device__ __forceinline__ void rms_row(float x[8], const float w[8], float eps) {
  constexpr unsigned kAll = 0xffffffffu;
  float2 s2 = __fmul2_rn(make_float2(x[0], x[1]), make_float2(x[0], x[1]));
#pragma unroll
  for (int r = 2; r < 8; r += 2) s2 = __ffma2_rn(make_float2(x[r], x[r + 1]), make_float2(x[r], x[r + 1]), s2);
  float s = __fadd_rn(s2.x, s2.y);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(kAll, s, o));
  const float inv = rsqrtf(__fmaf_rn(s, 1.0f / kD, eps));
#pragma unroll
  for (int r = 0; r < 8; r += 2) {
    const float2 y = __fmul2_rn(__fmul2_rn(make_float2(x[r], x[r + 1]), make_float2(inv, inv)), make_float2(w[r], w[r + 1]));
    x[r] = y.x;
    x[r + 1] = y.y;
  }
}

__device__ __forceinline__ void load_weight8(const float* w, int lane, float out[8]) {
  const float4 a = __ldca(reinterpret_cast<const float4*>(w) + 2 * lane), b = __ldca(reinterpret_cast<const float4*>(w) + 2 * lane + 1);
  out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
  out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
}

// 8 fp32 -> 8 bf16, round to nearest even (word i holds elements 2i low, 2i + 1 high)
__device__ __forceinline__ uint4 f32x8_to_bf16(const float x[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace
}  // namespace k8v4
