// Residual add with the norms on either side of it, for sm_100a.
//
//   u = y                                        (y: a block's output, bf16)
//   u = (y * w_post) * rsqrt(mean(y^2) + eps)    with a norm behind the block
//   u = u * gate                                 with a gate a channel or a token and channel
//   h = residual + a * u                         the residual stream, stored as bf16
//   x = (h * w_pre) * rsqrt(mean(h^2) + eps)     the next block's input
// x leaves as bf16, or as the per-token codes and scale that the FP8 GEMM
// reads (s = amax|x| / 448, code = E4M3(x / s)).  Everything between the
// loads and the stores is fp32: x is computed from h before h is rounded to
// bf16, and the codes from x itself, so each output is rounded once.
//
// Bound by DRAM: 7 bytes an element (y, residual, h, code), 8 with bf16 x, 2
// more with a gate a token.  A row is read once and stays in registers (8 V
// values a thread, P threads a row), so that the two or three reductions cost
// no second pass; the weights are the same for every row and come from L1.
// The norm and the row's scale need one reduction, not two: with z = h *
// w_pre, x = RN(z * r) for one r > 0, and rounding is monotone, so max|x| =
// RN(max|z| * r) and (sum h^2, max|z|) are reduced together.
#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "quant_math.cuh"

namespace ptpc {

namespace {

struct NormArgs {
  const uint4 *y, *r, *g, *wpost, *wpre;  // rows of 16-byte vectors (8 bf16)
  int64_t ldy, ldr, ldg, ldh;             // row pitches in vectors
  uint4 *h, *x;
  uint8_t *xq;
  float *xs;
  int T, nvec, P;
  float count, eps, a;
};

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// Sum and maximum over the P threads of a row (P a multiple of 32); `red` has
// a slot for each warp of the CTA, and another call uses another one.
__device__ __forceinline__ float2 row_reduce(float sum, float top, int P, int row_in_cta, float2 *red) {
  #pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  const int warps = P >> 5;
  if (warps > 1) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(sum, top);
    __syncthreads();
    // every warp adds the row's warps in the same order: one value for the row
    const int lane = threadIdx.x & 31;
    const float2 v = lane < warps ? red[row_in_cta * warps + lane] : make_float2(0.0f, 0.0f);
    sum = v.x;
    top = v.y;
    #pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
  }
  return make_float2(sum, top);
}

__device__ __forceinline__ float rstd_of(float sum, const NormArgs &p) {
  return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, p.count), p.eps));
}

// The scale of a row whose largest |x| is amax: amax / 448; 1 and zero codes
// where that is 0 (an all-zero row, or one below the smallest float times 448).
__device__ __forceinline__ GroupScale group_scale_f32(float amax) {
  GroupScale g;
  g.s = __fdiv_rn(amax, 448.0f);
  g.mode = g.s >= kFastPathMinScale ? kFast : kSlow;
  if (g.s == 0.0f) {
    g.s = 1.0f;
    g.mode = kZeroGroup;
  }
  g.r = __frcp_rn(g.s);
  return g;
}

__device__ __forceinline__ uint2 quant8(const float (&x)[8], const GroupScale &g) {
  if (g.mode == kZeroGroup) return make_uint2(0u, 0u);
  uint32_t c[4];
  if (g.mode == kFast) {
    const uint64_t s2 = pack2(g.s), nr2 = pack2(-g.r);
    #pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = quant_nx2_fast(__float_as_uint(x[2 * i]) ^ 0x80000000u, __float_as_uint(x[2 * i + 1]) ^ 0x80000000u, s2,
                            nr2);
  } else {
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 q;
      q.x = quotient(x[2 * i], g);
      q.y = quotient(x[2 * i + 1], g);
      c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// What comes in between y and h, for 8 values: u = y (* w_post * rstd) (* gate),
// h = residual + a * u.
__device__ __forceinline__ void add_block(const NormArgs &p, const uint4 yv, const uint4 rv, const uint4 gv, int j,
                                          float rstd_y, float (&h)[8]) {
  unpack8(rv, h);
  if (p.y == nullptr) return;
  float u[8], w[8];
  unpack8(yv, u);
  if (p.wpost != nullptr) {
    unpack8(__ldg(p.wpost + j), w);
    #pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = __fmul_rn(__fmul_rn(u[e], w[e]), rstd_y);
  }
  if (p.g != nullptr) {
    unpack8(gv, w);
    #pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = __fmul_rn(u[e], w[e]);
  }
  #pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = __fadd_rn(h[e], __fmul_rn(p.a, u[e]));
}

template <int V, bool QUANT>
__global__ void __launch_bounds__(V <= 2 ? 1024 : 512) residual_norm_kernel(const NormArgs p) {
  __shared__ float2 red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int rl = threadIdx.x / p.P, lt = threadIdx.x - rl * p.P;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / p.P) + rl;
  const bool active = row < p.T;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  // a gate's vectors are loaded with the others, but not with 8 vectors a
  // thread, where they would not fit in registers
  constexpr bool kGateFirst = V < 8;
  auto load_gate = [&](int j, bool in) -> uint4 {
    return in && p.g != nullptr ? (p.ldg != 0 ? ld_stream(p.g + row * p.ldg + j) : __ldg(p.g + j)) : zero;
  };
  uint4 yv[V], rv[V], gv[V];
  #pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = lt + i * p.P;
    const bool in = active && j < p.nvec;
    yv[i] = in && p.y != nullptr ? ld_stream(p.y + row * p.ldy + j) : zero;
    rv[i] = in ? ld_stream(p.r + row * p.ldr + j) : zero;
    if (kGateFirst) gv[i] = load_gate(j, in);
  }
  float rstd_y = 1.0f;
  if (p.wpost != nullptr) {
    float sum = 0.0f;
    #pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      unpack8(yv[i], f);
      float part = 0.0f;
      #pragma unroll
      for (int e = 0; e < 8; ++e) part = fmaf(f[e], f[e], part);
      sum += part;
    }
    rstd_y = rstd_of(row_reduce(sum, 0.0f, p.P, rl, red[0]).x, p);
  }
  float z[V][8];
  float sum = 0.0f, top = 0.0f;
  #pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = lt + i * p.P;
    const bool in = active && j < p.nvec;
    add_block(p, yv[i], rv[i], kGateFirst ? gv[i] : load_gate(j, in), in ? j : 0, rstd_y, z[i]);
    if (in && p.h != nullptr) p.h[row * p.ldh + j] = pack8(z[i]);
    float w[8];
    unpack8(__ldg(p.wpre + (in ? j : 0)), w);
    float part = 0.0f;
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      part = fmaf(z[i][e], z[i][e], part);
      z[i][e] = __fmul_rn(z[i][e], w[e]);
      if (QUANT) top = fmaxf(top, fabsf(z[i][e]));
    }
    sum += part;
  }
  const float2 both = row_reduce(sum, top, p.P, rl, red[1]);
  const float rstd = rstd_of(both.x, p);
  GroupScale g;
  if (QUANT) {
    g = group_scale_f32(__fmul_rn(both.y, rstd));
    if (active && lt == 0) p.xs[row] = g.s;
  }
  #pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = lt + i * p.P;
    if (!active || j >= p.nvec) continue;
    #pragma unroll
    for (int e = 0; e < 8; ++e) z[i][e] = __fmul_rn(z[i][e], rstd);
    if (QUANT)
      reinterpret_cast<uint2 *>(p.xq)[row * p.nvec + j] = quant8(z[i], g);
    else
      p.x[row * p.nvec + j] = pack8(z[i]);
  }
}

// Rows too long for registers (more than 32768 columns): a CTA a row, which
// is read again for each reduction (from L2).  h is written in the last pass,
// each vector by the thread that read it, so h may be the residual's buffer.
template <bool QUANT>
__global__ void __launch_bounds__(1024) residual_norm_long_kernel(const NormArgs p) {
  __shared__ float2 red[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float rstd_y = 1.0f;
  if (p.wpost != nullptr) {
    float sum = 0.0f;
    for (int j = threadIdx.x; j < p.nvec; j += 1024) {
      float f[8];
      unpack8(p.y[row * p.ldy + j], f);
      float part = 0.0f;
      #pragma unroll
      for (int e = 0; e < 8; ++e) part = fmaf(f[e], f[e], part);
      sum += part;
    }
    rstd_y = rstd_of(row_reduce(sum, 0.0f, 1024, 0, red[0]).x, p);
  }
  auto load = [&](int j, float (&h)[8]) {
    add_block(p, p.y != nullptr ? p.y[row * p.ldy + j] : zero, p.r[row * p.ldr + j],
              p.g != nullptr ? p.g[row * p.ldg + j] : zero, j, rstd_y, h);
  };
  float sum = 0.0f, top = 0.0f;
  for (int j = threadIdx.x; j < p.nvec; j += 1024) {
    float h[8], w[8];
    load(j, h);
    unpack8(__ldg(p.wpre + j), w);
    float part = 0.0f;
    #pragma unroll
    for (int e = 0; e < 8; ++e) {
      part = fmaf(h[e], h[e], part);
      top = fmaxf(top, fabsf(__fmul_rn(h[e], w[e])));
    }
    sum += part;
  }
  const float2 both = row_reduce(sum, top, 1024, 0, red[1]);
  const float rstd = rstd_of(both.x, p);
  GroupScale g;
  if (QUANT) {
    g = group_scale_f32(__fmul_rn(both.y, rstd));
    if (threadIdx.x == 0) p.xs[row] = g.s;
  }
  for (int j = threadIdx.x; j < p.nvec; j += 1024) {
    float h[8], w[8];
    load(j, h);
    unpack8(__ldg(p.wpre + j), w);
    if (p.h != nullptr) p.h[row * p.ldh + j] = pack8(h);
    #pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = __fmul_rn(__fmul_rn(h[e], w[e]), rstd);
    if (QUANT)
      reinterpret_cast<uint2 *>(p.xq)[row * p.nvec + j] = quant8(h, g);
    else
      p.x[row * p.nvec + j] = pack8(h);
  }
}

template <int V>
cudaError_t launch_v(const NormArgs &p, int grid, int block, bool quant, cudaStream_t st) {
  return quant ? launch_pdl(residual_norm_kernel<V, true>, grid, block, st, p)
               : launch_pdl(residual_norm_kernel<V, false>, grid, block, st, p);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNorm &a, cudaStream_t st) {
  NormArgs p = {};
  p.y = static_cast<const uint4 *>(a.y);
  p.r = static_cast<const uint4 *>(a.residual);
  p.g = static_cast<const uint4 *>(a.gate);
  p.wpost = static_cast<const uint4 *>(a.post_w);
  p.wpre = static_cast<const uint4 *>(a.pre_w);
  p.ldy = a.ldy / 8;
  p.ldr = a.ldr / 8;
  p.ldg = a.ldg / 8;
  p.ldh = a.ldh / 8;
  p.h = static_cast<uint4 *>(a.h);
  p.x = static_cast<uint4 *>(a.x);
  p.xq = a.xq;
  p.xs = a.xs;
  p.T = a.T;
  p.nvec = a.C / 8;
  p.count = (float)a.C;
  p.eps = a.eps;
  p.a = a.residual_scale;
  const bool quant = a.xq != nullptr;
  // Vectors a thread: with rows enough to fill the GPU, 4 (all of a row's
  // loads are in flight at once, few threads meet at each reduction); with
  // fewer rows than SMs a row is spread over as many threads as it has
  // vectors, up to 1024.
  auto threads = [&](int V) { return (p.nvec + 32 * V - 1) / (32 * V) * 32; };
  int V = p.T < num_sms() ? 1 : 4;
  while (V < 8 && threads(V) > (V <= 2 ? 1024 : 512)) V *= 2;
  p.P = threads(V);
  if (p.P > 512 && V == 8) {
    return quant ? launch_pdl(residual_norm_long_kernel<true>, p.T, 1024, st, p)
                 : launch_pdl(residual_norm_long_kernel<false>, p.T, 1024, st, p);
  }
  const int rows = std::max(1, 256 / p.P);
  const int grid = (p.T + rows - 1) / rows;
  switch (V) {
    case 1: return launch_v<1>(p, grid, rows * p.P, quant, st);
    case 2: return launch_v<2>(p, grid, rows * p.P, quant, st);
    case 4: return launch_v<4>(p, grid, rows * p.P, quant, st);
    default: return launch_v<8>(p, grid, rows * p.P, quant, st);
  }
}

}  // namespace ptpc
