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
// no second pass.  The norm and the row's scale need one reduction, not two:
// with z = h * w_pre, x = RN(z * r) for one r > 0, and rounding is monotone, so
// max|x| = RN(max|z| * r) and (sum h^2, max|z|) are reduced together.
// What keeps it from the floor is issue: 28 instructions a value (a CTA a row 34),
// a fifth of them the row's reductions and scale in every thread; hence packed
// fp32 arithmetic and, with many rows, factors kept in shared memory.
// Measured in a graph: 8192 tokens of 8192 columns with both norms, a channel gate
// and codes 92.5 us (5.1 TB/s, 0.77 of the copy rate; a CTA a row 101; repeated
// calls on changing rows 96.7, 0.74), 4000 of
// 16384 101 (136), 8192 of 4096 without the norm behind 42.7 (44.8), 3001 of
// 5136 with a token gate and bf16 out 31.3 (34.6), 2048 of 4096 10.5 (in L2), one
// token of 8192 2.7.
// Copies of the rows ahead into shared memory (cp.async, two or three stages)
// were slower: 120 to 140 us on the first of these.
#include <algorithm>
#include <atomic>
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

// Sum and (TOP) maximum over the P threads of a row (P a multiple of 32);
// `red` has a slot for each warp of the CTA, and the next call uses another one.
template <bool TOP>
__device__ __forceinline__ float2 row_reduce(float sum, float top, int P, int row_in_cta, float2 *red) {
  #pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (TOP) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
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
      if (TOP) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
  }
  return make_float2(sum, top);
}

__device__ __forceinline__ float rstd_of(float sum, const NormArgs &p) {
  return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, p.count), p.eps));
}

// Added to `sum`: the squares of eight values.
__device__ __forceinline__ uint64_t squares(const uint64_t (&f)[4], uint64_t sum) {
  #pragma unroll
  for (int i = 0; i < 4; ++i) sum = fma2(f[i], f[i], sum);
  return sum;
}

__device__ __forceinline__ float total(uint64_t sum) {
  const float2 v = halves(sum);
  return v.x + v.y;
}

// What comes in between y and h, for 8 values: u = y (* w_post * rstd) (* gate),
// h = residual + a * u.
__device__ __forceinline__ void add_block(const NormArgs &p, const uint4 yv, const uint4 rv, const uint4 gv, int j,
                                          float rstd_y, uint64_t (&h)[4]) {
  unpack8(rv, h);
  if (p.y == nullptr) return;
  uint64_t u[4], w[4];
  unpack8(yv, u);
  if (p.wpost != nullptr) {
    unpack8(__ldg(p.wpost + j), w);
    const uint64_t rstd2 = pack2(rstd_y);
    #pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = mul2(mul2(u[i], w[i]), rstd2);
  }
  if (p.g != nullptr) {
    unpack8(gv, w);
    #pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = mul2(u[i], w[i]);
  }
  const uint64_t a2 = pack2(p.a);
  #pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = fma2(a2, u[i], h[i]);
}

// h -> z = h * w_pre, and what the row's sums take of it.
template <bool QUANT>
__device__ __forceinline__ void weigh(const NormArgs &p, int j, uint64_t (&z)[4], uint64_t &sum, float &top) {
  uint64_t w[4];
  unpack8(__ldg(p.wpre + j), w);
  sum = squares(z, sum);
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[i] = mul2(z[i], w[i]);
    if (QUANT) {
      const float2 v = halves(z[i]);
      top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
  }
}

// z -> x and out; nrstd: -rstd for codes (they are taken of -x), rstd for bf16.
template <bool QUANT>
__device__ __forceinline__ void finish(const NormArgs &p, int64_t row, int j, uint64_t (&z)[4], float rstd,
                                       const GroupScale &g) {
  const uint64_t r2 = pack2(QUANT ? -rstd : rstd);
  #pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = mul2(z[i], r2);
  if (QUANT)
    reinterpret_cast<uint2 *>(p.xq)[row * p.nvec + j] = quant8_negated(z, g);
  else
    p.x[row * p.nvec + j] = pack8(z);
}

// The sums and the scale that a row ends with.
template <bool QUANT>
__device__ __forceinline__ float row_end(const NormArgs &p, const float2 both, int64_t row, bool writes, GroupScale &g) {
  const float rstd = rstd_of(both.x, p);
  if (QUANT) {
    g = group_scale_f32(__fmul_rn(both.y, rstd));
    if (writes) p.xs[row] = g.s;
  }
  return rstd;
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
    uint64_t sum = 0;
    #pragma unroll
    for (int i = 0; i < V; ++i) {
      uint64_t f[4];
      unpack8(yv[i], f);
      sum = squares(f, sum);
    }
    rstd_y = rstd_of(row_reduce<false>(total(sum), 0.0f, p.P, rl, red[0]).x, p);
  }
  uint64_t z[V][4], sum = 0;
  float top = 0.0f;
  #pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = lt + i * p.P;
    const bool in = active && j < p.nvec;
    add_block(p, yv[i], rv[i], kGateFirst ? gv[i] : load_gate(j, in), in ? j : 0, rstd_y, z[i]);
    if (in && p.h != nullptr) p.h[row * p.ldh + j] = pack8(z[i]);
    weigh<QUANT>(p, in ? j : 0, z[i], sum, top);
  }
  GroupScale g;
  const float rstd = row_end<QUANT>(p, row_reduce<QUANT>(total(sum), top, p.P, rl, red[1]), row, active && lt == 0, g);
  #pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = lt + i * p.P;
    if (active && j < p.nvec) finish<QUANT>(p, row, j, z[i], rstd, g);
  }
}

// Rows enough for several a CTA: CTAs that stay, with what is the same for
// every row kept in shared memory as fp32, F = w_post * (the channels'
// gate) * a and w_pre.  A vector of both takes 4 loads in place of 3, and 36
// instructions less.  The next row's loads are issued as soon as this one's
// registers are free, ahead of its second reduction.
constexpr int kStayV = 4;

template <bool QUANT, bool GATE>
__global__ void __launch_bounds__(512) residual_norm_stay_kernel(const NormArgs p) {
  extern __shared__ uint4 factors[];   // [F low, F high, w_pre low, w_pre high][nvec]: halves of 8 values
  __shared__ float2 red[4][32];
  griddep_launch_dependents();
  griddep_wait();
  const int rl = threadIdx.x / p.P, lt = threadIdx.x - rl * p.P, rows = blockDim.x / p.P;
  const bool has_f = p.y != nullptr && (p.wpost != nullptr || (!GATE && p.g != nullptr) || p.a != 1.0f);
  for (int j = threadIdx.x; j < p.nvec; j += blockDim.x) {
    uint64_t f[4], w[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pack2(1.0f);
    if (p.wpost != nullptr) {
      unpack8(__ldg(p.wpost + j), w);
      #pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], w[i]);
    }
    if (!GATE && p.g != nullptr) {
      unpack8(__ldg(p.g + j), w);
      #pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], w[i]);
    }
    #pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(f[i], pack2(p.a));
    ulonglong2 *to = reinterpret_cast<ulonglong2 *>(factors) + j;
    to[0] = make_ulonglong2(f[0], f[1]);
    to[p.nvec] = make_ulonglong2(f[2], f[3]);
    unpack8(__ldg(p.wpre + j), w);
    to[2 * p.nvec] = make_ulonglong2(w[0], w[1]);
    to[3 * p.nvec] = make_ulonglong2(w[2], w[3]);
  }
  __syncthreads();
  auto factor = [&](int which, int j, uint64_t (&w)[4]) {
    const ulonglong2 *from = reinterpret_cast<const ulonglong2 *>(factors) + 2 * which * p.nvec + j;
    const ulonglong2 lo = from[0], hi = from[p.nvec];
    w[0] = lo.x, w[1] = lo.y, w[2] = hi.x, w[3] = hi.y;
  };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 yv[kStayV], rv[kStayV], gv[GATE ? kStayV : 1];
  auto load = [&](int64_t row) {
    #pragma unroll
    for (int i = 0; i < kStayV; ++i) {
      const int j = lt + i * p.P;
      const bool in = row < p.T && j < p.nvec;
      yv[i] = in && p.y != nullptr ? ld_stream(p.y + row * p.ldy + j) : zero;
      rv[i] = in ? ld_stream(p.r + row * p.ldr + j) : zero;
      if (GATE) gv[i] = in ? ld_stream(p.g + row * p.ldg + j) : zero;
    }
  };
  const int64_t step = (int64_t)gridDim.x * rows;
  int64_t row = (int64_t)blockIdx.x * rows + rl;
  load(row);
  int turn = 0;   // the row's slots for its sums: not those of the row before
  #pragma unroll 1
  for (; row - rl < p.T; row += step, turn ^= 2) {
    float rstd_y = 1.0f;
    if (p.wpost != nullptr) {
      uint64_t sum = 0;
      #pragma unroll
      for (int i = 0; i < kStayV; ++i) {
        uint64_t f[4];
        unpack8(yv[i], f);
        sum = squares(f, sum);
      }
      rstd_y = rstd_of(row_reduce<false>(total(sum), 0.0f, p.P, rl, red[turn]).x, p);
    }
    const uint64_t rstd2 = pack2(rstd_y);
    uint64_t z[kStayV][4], sum = 0;
    float top = 0.0f;
    #pragma unroll
    for (int i = 0; i < kStayV; ++i) {
      const int j = lt + i * p.P;
      if (j < p.nvec) {
        uint64_t u[4], w[4];
        unpack8(rv[i], z[i]);
        if (p.y != nullptr) {
          unpack8(yv[i], u);
          if (has_f) {
            factor(0, j, w);
            #pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = mul2(u[e], w[e]);
          }
          if (GATE) {
            unpack8(gv[i], w);
            #pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = mul2(u[e], w[e]);
          }
          #pragma unroll
          for (int e = 0; e < 4; ++e) z[i][e] = fma2(u[e], rstd2, z[i][e]);
        }
        if (row < p.T && p.h != nullptr) p.h[row * p.ldh + j] = pack8(z[i]);
        factor(1, j, w);
        sum = squares(z[i], sum);
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
          z[i][e] = mul2(z[i][e], w[e]);
          if (QUANT) {
            const float2 v = halves(z[i][e]);
            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        }
      }
    }
    load(row + step);
    GroupScale g;
    const float rstd = row_end<QUANT>(p, row_reduce<QUANT>(total(sum), top, p.P, rl, red[turn + 1]), row,
                                      row < p.T && lt == 0, g);
    #pragma unroll
    for (int i = 0; i < kStayV; ++i) {
      const int j = lt + i * p.P;
      if (row < p.T && j < p.nvec) finish<QUANT>(p, row, j, z[i], rstd, g);
    }
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
    uint64_t sum = 0;
    for (int j = threadIdx.x; j < p.nvec; j += 1024) {
      uint64_t f[4];
      unpack8(p.y[row * p.ldy + j], f);
      sum = squares(f, sum);
    }
    rstd_y = rstd_of(row_reduce<false>(total(sum), 0.0f, 1024, 0, red[0]).x, p);
  }
  auto load = [&](int j, uint64_t (&h)[4]) {
    add_block(p, p.y != nullptr ? p.y[row * p.ldy + j] : zero, p.r[row * p.ldr + j],
              p.g != nullptr ? p.g[row * p.ldg + j] : zero, j, rstd_y, h);
  };
  uint64_t sum = 0;
  float top = 0.0f;
  for (int j = threadIdx.x; j < p.nvec; j += 1024) {
    uint64_t h[4];
    load(j, h);
    weigh<QUANT>(p, j, h, sum, top);
  }
  GroupScale g;
  const float rstd = row_end<QUANT>(p, row_reduce<QUANT>(total(sum), top, 1024, 0, red[1]), row, threadIdx.x == 0, g);
  for (int j = threadIdx.x; j < p.nvec; j += 1024) {
    uint64_t h[4], none = 0;
    float unused = 0.0f;
    load(j, h);
    if (p.h != nullptr) p.h[row * p.ldh + j] = pack8(h);
    weigh<QUANT>(p, j, h, none, unused);
    finish<QUANT>(p, row, j, h, rstd, g);
  }
}

template <int V>
cudaError_t launch_v(const NormArgs &p, int grid, int block, bool quant, cudaStream_t st) {
  return quant ? launch_pdl(residual_norm_kernel<V, true>, grid, block, st, p)
               : launch_pdl(residual_norm_kernel<V, false>, grid, block, st, p);
}

constexpr int kStaySmem = 224 * 1024;   // of an SM, 1 KB a CTA and the static part besides

template <bool QUANT, bool GATE>
cudaError_t launch_stay(const NormArgs &p, int grid, int block, size_t smem, cudaStream_t st) {
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t a = cudaFuncSetAttribute(residual_norm_stay_kernel<QUANT, GATE>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kStaySmem);
    if (a != cudaSuccess) return a;
    attr_set[dev].store(true, std::memory_order_release);
  }
  return launch_pdl_smem(residual_norm_stay_kernel<QUANT, GATE>, dim3(grid), block, smem, st, p);
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
  auto threads = [&](int V) { return (p.nvec + 32 * V - 1) / (32 * V) * 32; };
  // CTAs that stay, where at least four rows come to each (each lays out the
  // factors first: at two rows 20.0 us against 19.4 on 1300 tokens of 8192)
  // and their threads nearly fill the registers (3001 rows of 5136 columns,
  // 384 threads an SM: 41 us against 39).
  p.P = threads(kStayV);
  if (p.P <= 512) {
    const bool gate = p.g != nullptr && p.ldg != 0;
    const int rows = std::max(1, 256 / p.P), block = rows * p.P, tiles = (p.T + rows - 1) / rows;
    const size_t smem = (size_t)p.nvec * 64;
    const int per_sm = std::min(512 / block, (int)(kStaySmem / (smem + 2048))), grid = num_sms() * per_sm;
    if (per_sm * block >= 448 && tiles >= 4 * grid) {
      if (gate)
        return quant ? launch_stay<true, true>(p, grid, block, smem, st) : launch_stay<false, true>(p, grid, block, smem, st);
      return quant ? launch_stay<true, false>(p, grid, block, smem, st) : launch_stay<false, false>(p, grid, block, smem, st);
    }
  }
  // Vectors a thread: with rows enough to fill the GPU, 4 (all of a row's
  // loads are in flight at once, few threads meet at each reduction); with
  // fewer rows than SMs a row is spread over as many threads as it has
  // vectors, up to 1024.
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
