// Rotary position embedding of queries and keys, fused with the append of
// keys and values to the FP8 (E4M3) paged cache, for sm_100a.
//
// The first `rot` values of each head of q and k are turned in pairs (a, b)
// by the token's angles, taken from a table [max_position, rot] that holds
// rot / 2 cosines, then rot / 2 sines, for each position:
//   (a, b) -> (RN(RN(a c) - RN(b s)), RN(RN(b c) + RN(a s)))    fp32
// with pairs (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved.  q leaves
// as bf16; k (not rounded to bf16 in between) and v are quantised as the
// plain append does, per (token, KV head): scale = amax / 448, code =
// E4M3(x / scale).  The products and sums are not contracted and the quotient
// is the IEEE one, so codes and scales are functions of the inputs alone.
//
// Bound by DRAM: 4 bytes a value of q, 3 a value of k and v.  A head's vector
// belongs to D / 8 lanes, 16 bytes a lane; a lane gets the other half of its
// pairs by a shuffle.  A group of lanes takes N heads of one token (N = 4
// where there are tokens enough: four loads in flight a lane, and the token's
// angles, 64 bytes a lane, read once for the four; N = 1 otherwise).
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "quant_math.cuh"

namespace ptpc {

namespace {

constexpr int kRopeThreads = 128;

struct RopeArgs {
  const uint4 *q, *k, *v;              // token t, head h at [t * ld + h * D / 8] (vectors of 8)
  int64_t ldq, ldk, ldv, ldo;
  const float *cos_sin;
  int64_t max_position, num_slots;
  const int64_t *positions, *slots;
  int T, Hq, Hkv, rot;
  uint4 *q_out;
  uint8_t *kc, *vc;
  float *ks, *vs;
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// Codes of 8 values whose vector (L lanes) has the scale of its largest
// magnitude; every lane of the warp takes part.
template <int L>
__device__ __forceinline__ uint2 quantise_vector(const float (&x)[8], float &scale) {
  float amax = 0.0f;
  #pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
  #pragma unroll
  for (int o = L / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  scale = __fdiv_rn(amax, 448.0f);
  uint32_t c[4];
  // an all-zero vector, or one whose scale underflows: scale 1, codes 0
  const bool none = scale == 0.0f;
  if (none) scale = 1.0f;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
    c[i] = none ? 0u : (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int D, int N, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs p) {
  constexpr int L = D / 8;                    // lanes a head
  constexpr int kGroups = kRopeThreads / L;   // groups of lanes a CTA
  griddep_launch_dependents();
  griddep_wait();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % L, e0 = lane * 8;
  const int heads = p.Hq + 2 * p.Hkv;
  // this group's heads: h0, h0 + kGroups, ... (neighbouring groups read neighbouring heads)
  const int h0 = blockIdx.y * (kGroups * N) + threadIdx.x / L;
  const int64_t pos = p.positions[t], slot = p.slots[t];
  if (pos < 0 || pos >= p.max_position) return;   // the whole CTA: one token
  const bool keep = slot >= 0 && slot < p.num_slots;
  uint4 raw[N];
  #pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = h0 + i * kGroups;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (h < p.Hq)
      raw[i] = ld_stream(p.q + t * p.ldq + (int64_t)h * L + lane);
    else if (h < p.Hq + p.Hkv)
      raw[i] = ld_stream(p.k + t * p.ldk + (int64_t)(h - p.Hq) * L + lane);
    else if (h < heads)
      raw[i] = ld_stream(p.v + t * p.ldv + (int64_t)(h - p.Hq - p.Hkv) * L + lane);
  }
  // the angles of this lane's pairs: 8 (one half of each pair is here), or 4
  // when interleaved (both halves are)
  constexpr int A = INTERLEAVED ? 4 : 8;
  const int half = p.rot / 2;
  const bool turns = e0 < p.rot;
  const bool upper = !INTERLEAVED && e0 >= half;   // holds the pairs' second halves
  float c[A], s[A];
  if (turns) {
    const int first = INTERLEAVED ? e0 / 2 : e0 - (upper ? half : 0);
    const float4 *cs = reinterpret_cast<const float4 *>(p.cos_sin + pos * p.rot + first);
    const float4 *sn = reinterpret_cast<const float4 *>(p.cos_sin + pos * p.rot + half + first);
    #pragma unroll
    for (int i = 0; i < A / 4; ++i) {
      const float4 a = __ldg(cs + i), b = __ldg(sn + i);
      c[4 * i] = a.x; c[4 * i + 1] = a.y; c[4 * i + 2] = a.z; c[4 * i + 3] = a.w;
      s[4 * i] = b.x; s[4 * i + 1] = b.y; s[4 * i + 2] = b.z; s[4 * i + 3] = b.w;
    }
  }
  // the lane that holds the other halves of this lane's pairs (itself where nothing turns)
  const int other = INTERLEAVED || !turns ? threadIdx.x & 31
                                          : (threadIdx.x & 31) + (upper ? -(half / 8) : half / 8);
  #pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = h0 + i * kGroups;
    float x[8];
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
    uint32_t o[4] = {0u, 0u, 0u, 0u};
    if (!INTERLEAVED) {
      #pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __shfl_sync(0xffffffffu, w[j], other);
    }
    if (turns && h < p.Hq + p.Hkv) {
      if (INTERLEAVED) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = x[2 * j], b = x[2 * j + 1];
          x[2 * j] = __fsub_rn(__fmul_rn(a, c[j]), __fmul_rn(b, s[j]));
          x[2 * j + 1] = __fadd_rn(__fmul_rn(b, c[j]), __fmul_rn(a, s[j]));
        }
      } else {
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float y = e % 2 == 0 ? __uint_as_float(o[e / 2] << 16) : __uint_as_float(o[e / 2] & 0xFFFF0000u);
          const float own = __fmul_rn(x[e], c[e % A]), mix = __fmul_rn(y, s[e % A]);
          x[e] = upper ? __fadd_rn(own, mix) : __fsub_rn(own, mix);
        }
      }
    }
    // the groups of a warp may hold heads of different kinds, and their
    // shuffles are the warp's: decided for the warp as a whole
    const bool stores_codes = h >= p.Hq && h < heads;
    if (h < p.Hq)
      p.q_out[t * p.ldo + (int64_t)h * L + lane] =
          make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
    if (__any_sync(0xffffffffu, stores_codes)) {
      float scale;
      const uint2 code = quantise_vector<L>(x, scale);
      if (stores_codes && keep) {
        const bool is_v = h >= p.Hq + p.Hkv;
        const int64_t at = slot * p.Hkv + (h - p.Hq - (is_v ? p.Hkv : 0));
        reinterpret_cast<uint2 *>((is_v ? p.vc : p.kc) + at * D)[lane] = code;
        if (lane == 0) (is_v ? p.vs : p.ks)[at] = scale;
      }
    }
  }
}

template <int D, int N>
cudaError_t launch_n(const RopeArgs &p, bool interleaved, cudaStream_t st) {
  const int per_cta = kRopeThreads / (D / 8) * N;
  const dim3 grid(p.T, (p.Hq + 2 * p.Hkv + per_cta - 1) / per_cta);
  return interleaved ? launch_pdl(rope_append_kernel<D, N, true>, grid, kRopeThreads, st, p)
                     : launch_pdl(rope_append_kernel<D, N, false>, grid, kRopeThreads, st, p);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppend &a, cudaStream_t st) {
  RopeArgs p = {};
  p.q = static_cast<const uint4 *>(a.q);
  p.k = static_cast<const uint4 *>(a.k);
  p.v = static_cast<const uint4 *>(a.v);
  p.ldq = a.ldq / 8;
  p.ldk = a.ldk / 8;
  p.ldv = a.ldv / 8;
  p.ldo = a.ldo / 8;
  p.cos_sin = a.cos_sin;
  p.max_position = a.max_position;
  p.num_slots = a.num_slots;
  p.positions = a.positions;
  p.slots = a.slots;
  p.T = a.T;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.rot = a.rot;
  p.q_out = static_cast<uint4 *>(a.q_out);
  p.kc = a.kc;
  p.vc = a.vc;
  p.ks = a.ks;
  p.vs = a.vs;
  const int64_t lanes = (int64_t)a.T * (a.Hq + 2 * a.Hkv) * (a.D / 8);
  const bool many = lanes >= (int64_t)num_sms() * 2048 * 2;  // fills the GPU's threads with 4 heads a group
  if (a.D == 64) return many ? launch_n<64, 4>(p, a.interleaved, st) : launch_n<64, 1>(p, a.interleaved, st);
  return many ? launch_n<128, 4>(p, a.interleaved, st) : launch_n<128, 1>(p, a.interleaved, st);
}

}  // namespace ptpc
