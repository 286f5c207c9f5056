// Device arithmetic that the quantising kernels share: the scale of a group
// from its largest magnitude, the quotient x / scale without a divide, E4M3
// codes, and 16-byte streaming loads.  The method and what it guarantees are
// described at the top of quant.cu.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

namespace ptpc {

namespace {

constexpr float kFastPathMinScale = 0x1p-100f;

// Division mode shared by every element of a row / column.
enum : int { kZeroGroup = 0, kFast = 1, kSlow = 2 };

struct GroupScale {
  float s;     // dequantisation scale
  float r;     // RN(1/s) (fast mode only)
  int mode;
};

// Scale of a group from its largest magnitude (bf16 bits): amax / fmax, the
// format's largest finite value (448 for E4M3).
__device__ __forceinline__ GroupScale group_scale_from_amax_bits(uint32_t amax_bits16, float fmax = 448.0f) {
  GroupScale g;
  const float amax = __uint_as_float(amax_bits16 << 16);
  if (amax == 0.0f) {
    g.s = 1.0f;
    g.r = 1.0f;
    g.mode = kZeroGroup;
  } else {
    g.s = __fdiv_rn(amax, fmax);
    g.r = __frcp_rn(g.s);
    g.mode = g.s >= kFastPathMinScale ? kFast : kSlow;
  }
  return g;
}

__device__ __forceinline__ float quotient(float x, const GroupScale &g) {
  if (g.mode == kFast) {
    const float q0 = __fmul_rn(x, g.r);
    const float e = __fmaf_rn(q0, g.s, -x);
    return __fmaf_rn(-e, g.r, q0);
  }
  return __fdiv_rn(x, g.s);
}

// Two bf16 (low half = first element) -> two E4M3 codes (low byte = first).
__device__ __forceinline__ uint32_t quant_pair(uint32_t w, const GroupScale &g) {
  const float lo = __uint_as_float(w << 16);
  const float hi = __uint_as_float(w & 0xFFFF0000u);
  float2 q;
  q.x = quotient(lo, g);
  q.y = quotient(hi, g);
  return (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
}

// Fast path for two bf16 of one 32-bit word, with Blackwell's packed fp32x2
// arithmetic: the same three IEEE operations as quotient(), two lanes per
// instruction.  nx = -x is built during unpacking, so that
//   q0 = RN((-x) * (-r)) = RN(x * r),  e = RN(q0 * s + (-x)),  q = RN(e * (-r) + q0)
// (the residual form that keeps -0 as -0).  Returns the two E4M3 codes,
// first element in the low byte.
__device__ __forceinline__ uint32_t quant_nx2_fast(uint32_t nlo, uint32_t nhi, uint64_t s2, uint64_t nr2);

__device__ __forceinline__ uint32_t quant_pair_fast(uint32_t w, uint64_t s2, uint64_t nr2) {
  const uint32_t nlo = (w << 16) ^ 0x80000000u;       // -x of the first element
  const uint32_t nhi = (w & 0xFFFF0000u) ^ 0x80000000u;  // -x of the second element
  return quant_nx2_fast(nlo, nhi, s2, nr2);
}

// The fast-path arithmetic of quant_pair_fast on two elements given as the
// fp32 bits of their negations (first element -> low byte of the result).
__device__ __forceinline__ uint32_t quant_nx2_fast(uint32_t nlo, uint32_t nhi, uint64_t s2, uint64_t nr2) {
  uint64_t nx2, q0, e, q;
  asm("mov.b64 %0, {%1, %2};" : "=l"(nx2) : "r"(nlo), "r"(nhi));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q0) : "l"(nx2), "l"(nr2));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(q0), "l"(s2), "l"(nx2));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(e), "l"(nr2), "l"(q0));
  uint32_t qlo, qhi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(qlo), "=r"(qhi) : "l"(q));
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "r"(qhi), "r"(qlo));
  return (uint32_t)c;
}

// Eight bf16 (16 bytes) -> eight codes (8 bytes), fast path.
__device__ __forceinline__ uint2 quant_vec_fast(const uint4 v, uint64_t s2, uint64_t nr2) {
  uint2 o;
  o.x = quant_pair_fast(v.x, s2, nr2) | (quant_pair_fast(v.y, s2, nr2) << 16);
  o.y = quant_pair_fast(v.z, s2, nr2) | (quant_pair_fast(v.w, s2, nr2) << 16);
  return o;
}

// The fast path on x as it is: with -r in place of r the three steps give
// -q exactly (signed zeros included: checked against the form above for every
// (bf16 amax, bf16 x) pair with s >= 2^-100), so the codes come out with
// their sign bits flipped, which one XOR per four codes undoes.  This saves
// building -x for every element.
__device__ __forceinline__ uint32_t quant_x2_negated(uint32_t w, uint64_t s2, uint64_t nr2) {
  const uint32_t lo = w << 16, hi = w & 0xFFFF0000u;
  uint64_t x2, nq0, e, nq;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x2) : "r"(lo), "r"(hi));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(nq0) : "l"(x2), "l"(nr2));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(nq0), "l"(s2), "l"(x2));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(nq) : "l"(e), "l"(nr2), "l"(nq0));
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(nq));
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "r"(b), "r"(a));
  return (uint32_t)c;
}

__device__ __forceinline__ uint2 quant_vec_fast_flip(const uint4 v, uint64_t s2, uint64_t nr2) {
  uint2 o;
  o.x = (quant_x2_negated(v.x, s2, nr2) | (quant_x2_negated(v.y, s2, nr2) << 16)) ^ 0x80808080u;
  o.y = (quant_x2_negated(v.z, s2, nr2) | (quant_x2_negated(v.w, s2, nr2) << 16)) ^ 0x80808080u;
  return o;
}

// Eight bf16 (16 bytes) -> eight codes (8 bytes), any mode.
__device__ __forceinline__ uint2 quant_vec(const uint4 v, const GroupScale &g) {
  if (g.mode == kZeroGroup) return make_uint2(0u, 0u);
  uint2 o;
  o.x = quant_pair(v.x, g) | (quant_pair(v.y, g) << 16);
  o.y = quant_pair(v.z, g) | (quant_pair(v.w, g) << 16);
  return o;
}

__device__ __forceinline__ uint64_t pack2(float a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "r"(__float_as_uint(a)));
  return r;
}

// Two fp32 values in a register pair: each operation rounds as the scalar one.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float2 halves(uint64_t a) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(a));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}

__device__ __forceinline__ uint64_t join2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(__float_as_uint(lo)), "r"(__float_as_uint(hi)));
  return r;
}

// Eight bf16 -> four pairs of fp32, and back with one rounding.
__device__ __forceinline__ void unpack8(const uint4 v, uint64_t (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = join2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
  uint32_t w[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = halves(f[i]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The scale of fp32 values whose largest magnitude is amax: amax / 448; 1 and
// zero codes where that is 0 (all zero, or below the smallest float times 448).
__device__ __forceinline__ GroupScale group_scale_f32(float amax) {
  GroupScale g;
  g.s = __fdiv_rn(amax, 448.0f);
  g.mode = g.s >= kFastPathMinScale && g.s < __uint_as_float(0x7F800000u) ? kFast : kSlow;
  if (g.s == 0.0f) {
    g.s = 1.0f;
    g.mode = kZeroGroup;
  }
  g.r = __frcp_rn(g.s);
  return g;
}

// The codes of eight values given as their negations.
__device__ __forceinline__ uint2 quant8_negated(const uint64_t (&nx)[4], const GroupScale &g) {
  if (g.mode == kZeroGroup) return make_uint2(0u, 0u);
  uint32_t c[4];
  if (g.mode == kFast) {
    const uint64_t s2 = pack2(g.s), nr2 = pack2(-g.r);
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = halves(nx[i]);
      c[i] = quant_nx2_fast(__float_as_uint(v.x), __float_as_uint(v.y), s2, nr2);
    }
  } else {
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = halves(nx[i]);
      const float2 q = make_float2(quotient(-v.x, g), quotient(-v.y, g));
      c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
    }
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Quantises n vectors src[j0], src[j0 + step], ... of one group into
// dst[j] (8 codes each), choosing the arithmetic once for the whole run.
template <typename Src>
__device__ __forceinline__ void quant_run(Src src, uint2 *dst, int j0, int n, int step, const GroupScale &g) {
  if (g.mode == kFast) {
    const uint64_t s2 = pack2(g.s), nr2 = pack2(-g.r);
    for (int j = j0; j < n; j += step) dst[j] = quant_vec_fast(src(j), s2, nr2);
  } else if (g.mode == kSlow) {
    for (int j = j0; j < n; j += step) dst[j] = quant_vec(src(j), g);
  } else {
    for (int j = j0; j < n; j += step) dst[j] = make_uint2(0u, 0u);
  }
}

// max(|bf16|) of a 16-byte vector folded into acc (bf16x2 magnitudes; the
// sign bits of acc are meaningless).  One max.xorsign.abs per two elements.
__device__ __forceinline__ uint32_t absmax_bits(uint32_t acc, uint4 v) {
  asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(acc) : "r"(v.x));
  asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(acc) : "r"(v.y));
  asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(acc) : "r"(v.z));
  asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(acc) : "r"(v.w));
  return acc;
}

// Larger of the two 16-bit magnitudes of a folded accumulator.
__device__ __forceinline__ uint32_t fold_halves(uint32_t m) {
  m &= 0x7FFF7FFFu;
  return max(m & 0xFFFFu, m >> 16);
}

__device__ __forceinline__ uint4 ld_stream(const uint4 *p) { return __ldcs(p); }

}  // namespace

}  // namespace ptpc
