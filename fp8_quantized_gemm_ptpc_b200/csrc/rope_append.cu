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
// pairs by a shuffle.  A group of lanes takes N heads of one token: N = 4 where
// there are tokens enough (four loads in flight a lane, and the token's angles,
// 64 bytes a lane, read once for the four), N = 1 otherwise.  Groups fill the
// CTAs one behind the other, whatever the number of heads.  Measured in a graph:
// 8192 tokens of 64 + 16 heads of 128 62.9 us (5.2 TB/s, 0.78 of the copy rate; N =
// 2 75.9, N = 5 63.5; repeated calls 65.5, 0.75), of 32 + 16 heads 40.4; 3001 of 12 + 24 heads of 64, half
// turned, 8.1; 32 tokens 2.6.  Issue is next: two cycles of three.
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

template <int D, int N, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs p) {
  constexpr int L = D / 8;                    // lanes a head
  constexpr int kGroups = kRopeThreads / L;   // groups of lanes a CTA
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x % L, e0 = lane * 8;
  const int heads = p.Hq + 2 * p.Hkv, per_token = (heads + N - 1) / N;   // groups of lanes a token
  const uint32_t group = blockIdx.x * kGroups + threadIdx.x / L;
  const int64_t t = group / (uint32_t)per_token;
  // this group's heads: h0, h0 + per_token, ... (neighbouring groups read neighbouring heads)
  const int h0 = (int)(group - (uint32_t)t * per_token);
  const bool token = t < p.T;
  const int64_t pos = token ? p.positions[t] : -1, slot = token ? p.slots[t] : -1;
  const bool active = pos >= 0 && pos < p.max_position, keep = slot >= 0 && slot < p.num_slots;
  uint4 raw[N];
  #pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = h0 + i * per_token;
    const bool is_q = h < p.Hq, is_k = h < p.Hq + p.Hkv;
    const uint4 *from = is_q ? p.q + t * p.ldq : is_k ? p.k + t * p.ldk : p.v + t * p.ldv;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (active && h < heads) raw[i] = ld_stream(from + (int64_t)(h - (is_q ? 0 : is_k ? p.Hq : p.Hq + p.Hkv)) * L + lane);
  }
  // the angles of this lane's pairs: 8 (one half of each pair is here), or 4
  // when interleaved (both halves are)
  constexpr int A = INTERLEAVED ? 4 : 8;
  const int half = p.rot / 2;
  const bool turns = active && e0 < p.rot;
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
  // first halves take a c - b s, second ones b c + a s: a - is a negated sine
  uint64_t c2[4], s2[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTERLEAVED) {
      c2[i] = pack2(c[i % A]);
      s2[i] = join2(-s[i % A], s[i % A]);
    } else {
      c2[i] = join2(c[(2 * i) % A], c[(2 * i + 1) % A]);
      s2[i] = upper ? join2(s[(2 * i) % A], s[(2 * i + 1) % A]) : join2(-s[(2 * i) % A], -s[(2 * i + 1) % A]);
    }
  }
  // the lane that holds the other halves of this lane's pairs (itself where nothing turns)
  const int self = threadIdx.x & 31;
  const int other = INTERLEAVED || e0 >= p.rot ? self : self + (upper ? -(half / 8) : half / 8);
  #pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = h0 + i * per_token;
    uint4 mate = raw[i];
    if (!INTERLEAVED) {
      mate.x = __shfl_sync(0xffffffffu, raw[i].x, other);
      mate.y = __shfl_sync(0xffffffffu, raw[i].y, other);
      mate.z = __shfl_sync(0xffffffffu, raw[i].z, other);
      mate.w = __shfl_sync(0xffffffffu, raw[i].w, other);
    }
    uint64_t x[4];
    unpack8(raw[i], x);
    if (turns && h < p.Hq + p.Hkv) {
      uint64_t y[4];
      unpack8(mate, y);
      #pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (INTERLEAVED) {
          const float2 v = halves(x[e]);
          y[e] = join2(v.y, v.x);
        }
        // scalar sums: the compiler makes one fused operation of a packed product and a packed sum
        const float2 own = halves(mul2(x[e], c2[e])), mix = halves(mul2(y[e], s2[e]));
        x[e] = join2(__fadd_rn(own.x, mix.x), __fadd_rn(own.y, mix.y));
      }
    }
    // the groups of a warp may hold heads of different kinds, and their
    // shuffles are the warp's: decided for the warp as a whole
    const bool is_kv = active && h >= p.Hq && h < heads;
    if (active && h < p.Hq) p.q_out[t * p.ldo + (int64_t)h * L + lane] = pack8(x);
    if (__any_sync(0xffffffffu, is_kv)) {
      float amax = 0.0f;
      #pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = halves(x[e]);
        amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
      #pragma unroll
      for (int o = L / 2; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (is_kv && keep) {
        const GroupScale g = group_scale_f32(amax);
        const uint64_t minus = pack2(-1.0f);
        #pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = mul2(x[e], minus);
        const bool is_v = h >= p.Hq + p.Hkv;
        const int64_t at = slot * p.Hkv + (h - p.Hq - (is_v ? p.Hkv : 0));
        reinterpret_cast<uint2 *>((is_v ? p.vc : p.kc) + at * D)[lane] = quant8_negated(x, g);
        if (lane == 0) (is_v ? p.vs : p.ks)[at] = g.s;
      }
    }
  }
}

template <int D, int N>
cudaError_t launch_n(const RopeArgs &p, bool interleaved, cudaStream_t st) {
  const int64_t groups = (int64_t)p.T * ((p.Hq + 2 * p.Hkv + N - 1) / N);
  constexpr int kGroups = kRopeThreads / (D / 8);
  // groups are counted in 32 bits: more are more than the memory of a GPU holds
  if (groups > 0xFFFFFF00ll) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)((groups + kGroups - 1) / kGroups));
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
