// block_norm_k8v4: what stands between two blocks of a layer, one pass over the rows:
//
//   a = y / sqrt(mean(y^2) + eps) * w_post     (norm optional)
//   a = a * act(gate)                          (gate optional)
//   h = residual + alpha * a                   (residual optional; stored)
//   n = h / sqrt(mean(h^2) + eps) * w_pre      (optional; of h as stored)
//
// What bounds it: memory.  A row is read once and written once or twice; it stays in
// registers between the two norms, so each of its elements is one lane's from load to
// store.  The loads of a thread's first chunks are issued before the row's first reduction.
// 8,192 rows of 4,096 dims with every part (fp32 y, bf16 gate, residual and outputs): 403 MB
// in 68.6 us, 5.9 TB/s.
#include <algorithm>

#include "k8v4_ops.cuh"

namespace k8v4 {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct NormParams {
  const void* y;
  const void* gate;
  const void* residual;
  const float* post_weight;
  const float* pre_weight;
  void* h_out;
  void* n_out;
  int64_t y_stride, gate_stride;
  int n_tok, dim, gate_act;
  float alpha, eps, inv_dim;
};

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// VEC consecutive elements of a row, as they are stored: 8 (16-byte loads) or 1
template <bool F32, int VEC>
struct Raw {
  uint4 w[F32 && VEC == 8 ? 2 : 1];
  __device__ __forceinline__ void load(const void* row, int64_t at) {
    if (VEC == 8) {
      const uint4* src = F32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(row) + at)
                             : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + at);
      w[0] = src[0];
      if (F32) w[F32 && VEC == 8 ? 1 : 0] = src[1];
    } else {
      w[0].x = F32 ? static_cast<const uint32_t*>(row)[at] : static_cast<uint32_t>(static_cast<const uint16_t*>(row)[at]) << 16;
    }
  }
  __device__ __forceinline__ void zero() { w[0] = w[F32 && VEC == 8 ? 1 : 0] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float at(int e) const {
    if (VEC == 1) return __uint_as_float(w[0].x);
    const uint4 q = w[F32 ? e >> 2 : 0];
    if (F32) return __uint_as_float((e & 3) == 0 ? q.x : (e & 3) == 1 ? q.y : (e & 3) == 2 ? q.z : q.w);
    const uint32_t v = (e >> 1) == 0 ? q.x : (e >> 1) == 1 ? q.y : (e >> 1) == 2 ? q.z : q.w;
    return e & 1 ? bf_hi(v) : bf_lo(v);
  }
};
template <int VEC>
__device__ __forceinline__ void load_weight(const float* w, int64_t at, float x[VEC]) {
  if (VEC == 8) {
    const float4 a = *reinterpret_cast<const float4*>(w + at), b = *reinterpret_cast<const float4*>(w + at + 4);
    x[0] = a.x; x[1 % VEC] = a.y; x[2 % VEC] = a.z; x[3 % VEC] = a.w;
    x[4 % VEC] = b.x; x[5 % VEC] = b.y; x[6 % VEC] = b.z; x[7 % VEC] = b.w;
  } else {
    x[0] = w[at];
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// store VEC elements rounded to the type; x becomes what was stored
template <bool F32, int VEC>
__device__ __forceinline__ void store(void* row, int64_t at, float x[VEC]) {
  if (F32) {
    float* dst = static_cast<float*>(row) + at;
    if (VEC == 8) {
      reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1 % VEC], x[2 % VEC], x[3 % VEC]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(x[4 % VEC], x[5 % VEC], x[6 % VEC], x[7 % VEC]);
    } else {
      *dst = x[0];
    }
    return;
  }
  uint16_t* dst = static_cast<uint16_t*>(row) + at;
  if (VEC == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16(x[(2 * i) % VEC], x[(2 * i + 1) % VEC]);
      x[(2 * i) % VEC] = bf_lo(w[i]);
      x[(2 * i + 1) % VEC] = bf_hi(w[i]);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    const uint32_t w = pack_bf16(x[0], 0.0f);
    *dst = static_cast<uint16_t>(w);
    x[0] = bf_lo(w);
  }
}

// the sum over the threads of a row (blockDim.x of them; a warp, or the CTA's)
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if (blockDim.x == 32) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < warps ? red[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// grid: blockDim.y rows a CTA; a row's elements in chunks of VEC, chunk x + blockDim.x * i a
// thread's i-th.  One row of threads larger than a warp: blockDim.y is 1.
template <bool YF32, bool F32, int VEC, int NV>
__global__ void __launch_bounds__(1024, NV == 1 && !F32 ? 2 : 1) block_norm_kernel(const NormParams p) {
  __shared__ float red[2][32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= p.n_tok) return;                        // (a whole warp, where a row is one)
  const void* y = YF32 ? static_cast<const void*>(static_cast<const float*>(p.y) + row * p.y_stride)
                       : static_cast<const void*>(static_cast<const uint16_t*>(p.y) + row * p.y_stride);
  const int64_t rest = row * p.dim;
  // one chunk a thread: the loads of the gate and the residual go out with the first.
  // With more chunks they would not fit the registers of 1,024 threads; the row's y does
  constexpr bool kAhead = NV == 1;
  Raw<F32, VEC> g0, r0;
  float x[NV][VEC];
  {
    Raw<YF32, VEC> yr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = VEC * (threadIdx.x + blockDim.x * i);
      yr[i].zero();
      if (at < p.dim) yr[i].load(y, at);
    }
    if (kAhead) {
      const int at = VEC * threadIdx.x;
      g0.zero();
      r0.zero();
      if (at < p.dim && p.gate) g0.load(p.gate, row * p.gate_stride + at);
      if (at < p.dim && p.residual) r0.load(p.residual, rest + at);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[i][e] = yr[i].at(e);
  }
  float scale = 1.0f;
  if (p.post_weight) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += x[i][e] * x[i][e];
    scale = rsqrtf(row_sum(s, red[0]) * p.inv_dim + p.eps);
  }
  float s2 = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = VEC * (threadIdx.x + blockDim.x * i);
    if (at >= p.dim) continue;
    if (!kAhead && p.gate) g0.load(p.gate, row * p.gate_stride + at);
    if (!kAhead && p.residual) r0.load(p.residual, rest + at);
    if (p.post_weight) {
      float w[VEC];
      load_weight<VEC>(p.post_weight, at, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[i][e] *= scale * w[e];
    }
    if (p.gate) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float z = g0.at(e);
        float f = z;
        if (p.gate_act != K8V4_GATE_NONE) {
          // (the short exponential is off by |z| units or so of fp32, which bf16 results do not see)
          const float u = 1.0f / (1.0f + (F32 ? expf(-z) : __expf(-z)));
          f = p.gate_act == K8V4_GATE_SILU ? z * u : u;
        }
        x[i][e] *= f;
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[i][e] = p.residual ? fmaf(p.alpha, x[i][e], r0.at(e)) : p.alpha * x[i][e];
    store<F32, VEC>(p.h_out, rest + at, x[i]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s2 += x[i][e] * x[i][e];
  }
  if (!p.pre_weight) return;
  const float scale2 = rsqrtf(row_sum(s2, red[1]) * p.inv_dim + p.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = VEC * (threadIdx.x + blockDim.x * i);
    if (at >= p.dim) continue;
    float w[VEC];
    load_weight<VEC>(p.pre_weight, at, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] *= x[i][e] * scale2;
    store<F32, VEC>(p.n_out, rest + at, w);
  }
}

template <bool YF32, bool F32>
int launch_types(const Launch& L, const NormParams& p, bool wide) {
  const int chunks = wide ? p.dim / 8 : p.dim;
  // chunks a thread holds, and the threads of a row: a warp for short rows, so that a
  // norm needs no barrier.  bf16 rows of a chunk a thread fill the SM with 2,048 threads of 32
  // registers: 8,192 rows of 4,096 dims 68.6 us, 73 with 38 registers, 81 with two chunks a thread, 83
  // where the CTAs stay and fetch the next row during this one's sums.  fp32 rows would spill there
  // (20,000 x 1,000: 68 us, 61 with 48 registers) and past 4,096 dims take two chunks (4,000 x 8,192: 112 us, 136).
  const int hold = wide ? (chunks <= (F32 ? 512 : 1024) ? 1 : chunks <= 2048 ? 2 : 4) : (chunks <= 4096 ? 4 : chunks <= 16384 ? 16 : 32);
  const int threads = std::max(32, ((chunks + hold - 1) / hold + 31) & ~31);
  const int rows = threads == 32 ? 4 : 1;
  const dim3 block(threads, rows), grid(static_cast<unsigned>((static_cast<int64_t>(p.n_tok) + rows - 1) / rows));
  if (wide && hold == 1) return launch_behind(L, block_norm_kernel<YF32, F32, 8, 1>, grid, block, p);
  if (wide && hold == 2) return launch_behind(L, block_norm_kernel<YF32, F32, 8, 2>, grid, block, p);
  if (wide) return launch_behind(L, block_norm_kernel<YF32, F32, 8, 4>, grid, block, p);
  if (hold == 4) return launch_behind(L, block_norm_kernel<YF32, F32, 1, 4>, grid, block, p);
  if (hold == 16) return launch_behind(L, block_norm_kernel<YF32, F32, 1, 16>, grid, block, p);
  return launch_behind(L, block_norm_kernel<YF32, F32, 1, 32>, grid, block, p);
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

int launch_block_norm(const Launch& L, const BlockNormArgs& a, int y_dtype, int dtype) {
  NormParams p;
  p.y = a.y;
  p.gate = a.gate;
  p.residual = a.residual;
  p.post_weight = a.post_weight;
  p.pre_weight = a.pre_weight;
  p.h_out = a.h_out;
  p.n_out = a.n_out;
  p.y_stride = a.y_stride;
  p.gate_stride = a.gate_stride;
  p.n_tok = a.n_tok;
  p.dim = a.dim;
  p.gate_act = a.gate_act;
  p.alpha = a.residual_scale;
  p.eps = a.eps;
  p.inv_dim = 1.0f / static_cast<float>(a.dim);
  // rows in 16-byte pieces of every array, where all of them allow it
  const int ye = y_dtype == K8V4_F32 ? 4 : 8, te = dtype == K8V4_F32 ? 4 : 8;
  const bool wide = a.dim % 8 == 0 && a.y_stride % ye == 0 && on16(a.y) && on16(a.h_out) && on16(a.post_weight) &&
                    on16(a.pre_weight) && on16(a.residual) && (!a.pre_weight || on16(a.n_out)) &&
                    (!a.gate || (on16(a.gate) && a.gate_stride % te == 0));
  if (y_dtype == K8V4_F32)
    return dtype == K8V4_F32 ? launch_types<true, true>(L, p, wide) : launch_types<true, false>(L, p, wide);
  return dtype == K8V4_F32 ? launch_types<false, true>(L, p, wide) : launch_types<false, false>(L, p, wide);
}

}  // namespace k8v4
