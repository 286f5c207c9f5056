// Causal attention of each sequence's newest tokens over its FP8 (E4M3) paged
// cache, on the fifth-generation tensor cores (tcgen05).
//
// A sequence has n new tokens at the end of a context of m positions; token i
// sees positions 0 .. m - n + i.  A KV head's G query heads share its keys, so
// the rows of the products are (token, head of the group) pairs, row R = i * G
// + g: a CTA takes 256 rows of one sequence and KV head as two streams of 128,
// and walks the context in tiles of 128 positions with the running maximum and
// sum of a softmax.
//
// Warps 8-11 read the codes (16 bytes a lane; any block size; a tile ahead, in
// registers), turn them into f16 and lay them out in shared memory for the
// MMAs.  The scales go in here, relative to a reference of each 32 positions
// (a warp's rows):  K' = code * ks / kref,  V' = code * vs / vref, so that the
// softmax has one factor for 32 columns instead of one a column.  kref is the
// largest key scale; the product is formed as code * hi + code * lo with the
// ratio split in two f16, so K' is rounded once.  vref is 2^-6 of a power of
// two at least the largest value scale: V' reaches 448 * 64, near f16's largest
// value, so that the ratio keeps f16's 11 bits down to 2^-20 of the largest
// scale.  A key's error is 2^-12 of its value, spread over D products; a
// value's at most 2^-11.
// Warp 12 issues S = Q K'^T (kind::f16, q as f16 after a power-of-two scale a
// row, exact) and O += P V' with P from tensor memory.
// Warps 0-3 and 4-7 (a stream each, a thread a row) do the softmax in base 2.
// With t = S * kref * qscale * log2 e, a weight is P' = 2^(t + log2 vref - r):
// the reference r follows the largest t + log2 vref, so the f16 P' stays near
// 1 however the value scales spread, and the sum of 2^(t - r) is that of P' /
// vref.  r moves (and O, in tensor memory, is rescaled) only when a tile
// exceeds it by more than 8, so P' < 2^8.  P' overwrites S in place.
// While one stream is in the softmax the other's products run.  A CTA with 128
// rows or fewer gives both streams the same rows and every other tile each,
// and joins them at the end.
//
// With few rows the context is split over CTAs whose partial results a second
// kernel joins (plan_chunk).  Every wait is bounded; a timeout sets a bit in
// the status word at the front of the workspace.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "sm100.cuh"

namespace ptpc {

namespace {

constexpr int kCaThreads = 416;   // warps 0-7 softmax, 8-11 converters, 12 MMA issuer
constexpr int kCaRows = 128;      // rows a stream
constexpr int kCaTile = 128;      // positions a tile
constexpr int kCaStages = 2;      // stages of the K ring and of the V ring
constexpr int kCaMeta = 8;        // tiles whose scales are kept (more than the stages ahead of the softmax)
constexpr uint32_t kStatusTimeoutChunk = 1u << 4;
constexpr float kCaLazy = 8.0f;   // r moves when a row's maximum exceeds it by this
constexpr int kCaMaxSplits = 64;

// What the softmax needs of a tile, for each 32 positions.
struct TileMeta {
  float kref[4];
  float lv[4];        // log2 vref
  float inv_vref[4];
  uint32_t valid[4];  // bit i: the position is in the cache
  uint32_t nan[4];    // bit i: the position's value vector is not finite (diagonal tiles only)
};

struct ChunkArgs {
  const __nv_bfloat16 *q;       // [total_q, Hq, D], token pitch ldq
  int64_t ldq;
  const uint8_t *kc, *vc;       // [num_slots, Hkv, D]
  const float *ks, *vs;         // [num_slots, Hkv]
  const int32_t *block_tables;  // [B, max_blocks]
  const int32_t *context_lens, *cu_q;
  int B, Hq, Hkv, G, total_q;
  int block_size, max_blocks, max_context;
  uint64_t bs_magic;            // ceil(2^64 / block_size)
  int64_t num_slots;
  int splits, split_tiles;
  float scale_log2;
  float *part_ml, *part_acc;
  __nv_bfloat16 *out;           // [total_q, Hq, D]
  uint32_t *status;
};

template <int D>
struct CaSmem {
  static constexpr int kOperand = kCaRows * D * 2;          // a 128 x D f16 tile
  static constexpr int Q = 0;                               // [stream]
  static constexpr int K = Q + 2 * kOperand;                // [stage]
  static constexpr int V = K + kCaStages * kOperand;        // [stage]
  static constexpr int META = V + kCaStages * kOperand;
  static constexpr int ML = META + kCaMeta * (int)sizeof(TileMeta);  // [row]: r and l of stream 1 when joined
  static constexpr int BARS = ML + kCaRows * 8;
  static constexpr int kBars = 4 * kCaStages + 3 * 2 + 1;
  static constexpr int BYTES = 1024 + BARS + kBars * 8 + 16;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes (low byte first) as f16, exact.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// D[tmem] (+)= A[smem] * B[smem], kind::f16 -> fp32.
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// The same with A in tensor memory (two f16 along K a column, a row a lane).
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Instruction descriptor: dense kind::f16, f16 operands, fp32 accumulation,
// M = 128; B K-major, or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kCaRows >> 4) << 24);
}

// MN-major operand with the 128-byte swizzle: rows of 128 bytes (64 f16 along
// N), one per K index, 8-row atoms 1024 bytes apart along K; the next 64
// values of N start `atom_bytes` further.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t atom_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(atom_bytes >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Byte offset of 16-byte piece c (0 .. D / 8 - 1) of row r in an operand tile:
// atoms of 64 f16 (128-byte swizzled rows), 16 KB apart.
__device__ __forceinline__ int piece_off(int r, int c) {
  return (c >> 3) * (kCaRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// What a CTA works on.
struct Work {
  int b, row0, rows;      // sequence, first row of the CTA in it (row = token * G + head), rows
  int first_q, n, m;      // the sequence's first token in q, its new tokens, its context
  int t0, tiles;          // first tile of the CTA's part of the context, tiles in it
  int tiles0;             // tiles that stream 0 needs (two streams of rows), <= tiles
  int kv_end;             // positions past this are not read
};

__device__ __forceinline__ int seq_tokens(const ChunkArgs &p, int b, int &first) {
  const int a = min(max(__ldg(p.cu_q + b), 0), p.total_q);
  const int e = min(max(__ldg(p.cu_q + b + 1), a), p.total_q);
  first = a;
  return e - a;
}

// The sequence and rows of the w-th row tile, counted over the sequences (a
// warp's scan; the same in every warp).  A sequence's last tile, which sees
// most, comes first.  false: there is no such tile.
__device__ __forceinline__ bool find_work(const ChunkArgs &p, int w, Work &k) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = 0; base < p.B; base += 32) {
    const int b = base + lane;
    int first = 0, n = 0;
    if (b < p.B) n = seq_tokens(p, b, first);
    const int mine = (int)(((int64_t)n * p.G + 2 * kCaRows - 1) / (2 * kCaRows));
    int upto = mine;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > w);
    if (past != 0) {
      const int at = __ffs(past) - 1;
      const int tiles = __shfl_sync(0xffffffffu, mine, at);
      const int start = before + __shfl_sync(0xffffffffu, upto, at) - tiles;
      k.b = base + at;
      k.n = __shfl_sync(0xffffffffu, n, at);
      k.first_q = __shfl_sync(0xffffffffu, first, at);
      const int tile = tiles - 1 - (w - start);
      k.row0 = tile * 2 * kCaRows;
      k.rows = (int)min((int64_t)2 * kCaRows, (int64_t)k.n * p.G - k.row0);
      k.m = max(__ldg(p.context_lens + k.b), 0);
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

template <int D>
__global__ void __launch_bounds__(kCaThreads, 1) chunk_attn_kernel(const ChunkArgs p) {
  using S = CaSmem<D>;
  extern __shared__ uint8_t ca_smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(ca_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::BARS);
  uint64_t *k_full = bars;                  // [stage] K' of a tile is in shared memory (4 warps)
  uint64_t *k_empty = k_full + kCaStages;   // [stage] its products are done
  uint64_t *v_full = k_empty + kCaStages;
  uint64_t *v_empty = v_full + kCaStages;
  uint64_t *s_full = v_empty + kCaStages;   // [stream] S is in tensor memory, and the products before it are done
  uint64_t *p_full = s_full + 2;            // [stream] P' written, O rescaled (128)
  uint64_t *o_done = p_full + 2;            // [stream] the stream's last product
  uint64_t *drain = o_done + 2;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
  TileMeta *meta = reinterpret_cast<TileMeta *>(sm + S::META);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.x % p.Hkv, split = blockIdx.y;
  Work k;
  if (!find_work(p, blockIdx.x / p.Hkv, k)) return;   // the same in every thread
  {
    // positions that the CTA's last row sees, and stream 0's
    const int seen = min(k.m, p.max_context);
    const int i_last = (k.row0 + k.rows - 1) / p.G, i_last0 = (k.row0 + kCaRows - 1) / p.G;
    k.kv_end = max(0, min(seen, k.m - k.n + i_last + 1));
    const int end0 = max(0, min(seen, k.m - k.n + i_last0 + 1));
    const int all = (k.kv_end + kCaTile - 1) / kCaTile, all0 = (end0 + kCaTile - 1) / kCaTile;
    k.t0 = split * p.split_tiles;
    k.tiles = max(0, min(all - k.t0, p.split_tiles));
    k.tiles0 = max(0, min(all0 - k.t0, k.tiles));
  }
  // the first position that not every row of the CTA sees
  const int all_see = k.m - k.n + k.row0 / p.G + 1;
  const bool two = k.rows > kCaRows;   // two streams of rows; otherwise both take the same rows, every other tile each

  // ---- this thread's row (softmax warps)
  const int stream = warp >> 2;        // 0, 1: softmax; 2: converters; 3: the MMA issuer
  const int lrow = threadIdx.x & 127;
  const int trow = (two && stream == 1 ? kCaRows : 0) + lrow;   // row in the CTA
  const int R = k.row0 + trow;
  const int tok = R / p.G, head = R - tok * p.G;
  const bool has_row = stream < 2 && trow < k.rows;

  if (k.tiles == 0) {
    // nothing to see (in this part of the context): zeros, or an empty part
    if (has_row && !(stream == 1 && !two)) {
      const int64_t oh = (int64_t)(k.first_q + tok) * p.Hq + kvh * p.G + head;
      if (p.splits == 1) {
        uint4 *o = reinterpret_cast<uint4 *>(p.out + oh * D);
        #pragma unroll
        for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
      } else {
        const int64_t idx = oh * p.splits + split;
        p.part_ml[idx * 2] = -INFINITY;
        p.part_ml[idx * 2 + 1] = 0.0f;
      }
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < kCaStages; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], kCaRows);
      mbar_init(&o_done[s], 1);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }

  // ---- q as f16 (a power-of-two scale a row brings its largest value to
  // [1, 2): exact, but for values 2^-24 of the largest and below)
  float rowfac = 0.0f;
  if (stream < 2) {
    uint4 w[D / 8];
    uint32_t amax = 0;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (int64_t)(k.first_q + tok) * p.ldq +
                                                       (int64_t)(kvh * p.G + head) * D);
    #pragma unroll
    for (int c = 0; c < D / 8; ++c) w[c] = has_row ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
    #pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
      #pragma unroll
      for (int i = 0; i < 4; ++i) amax = max(amax, max((v[i] << 16) & 0x7FFFFFFFu, v[i] & 0x7FFF0000u));
    }
    // 2^e, e the exponent of the largest magnitude, kept where 2^-e is a normal number too
    const uint32_t ex = min(max(amax >> 23, 1u), 253u);
    const float up = __uint_as_float((254u - ex) << 23);
    rowfac = __uint_as_float(ex << 23) * p.scale_log2;
    if (two || stream == 0) {
      uint8_t *qs = sm + S::Q + (two ? stream : 0) * S::kOperand;
      #pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
        uint32_t h[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i)
          h[i] = f16_pair(__uint_as_float(v[i] << 16) * up, __uint_as_float(v[i] & 0xFFFF0000u) * up);
        *reinterpret_cast<uint4 *>(qs + piece_off(lrow, c)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
      fence_async_shared();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (stream == 2) {
    // ------------------------------------------------------------ converters
    constexpr int LPR = D / 16;           // lanes a row, 16 codes a lane
    constexpr int RP = 32 / LPR;          // rows a load instruction
    constexpr int STEPS = 32 / RP;
    const int cw = warp - 8;
    const int piece = lane % LPR;
    const int32_t *table = p.block_tables + (int64_t)k.b * p.max_blocks;
    // the slot of this lane's position of local tile j (-1: not read)
    auto slot_of = [&](int j) -> int {
      if (j >= k.tiles) return -1;
      const int pos = (k.t0 + j) * kCaTile + 32 * cw + lane;
      if (pos >= k.kv_end) return -1;
      const int bi = (int)__umul64hi((uint64_t)pos, p.bs_magic);
      if (bi >= p.max_blocks) return -1;
      const int blk = __ldg(table + bi);
      const int64_t sl = (int64_t)blk * p.block_size + (pos - bi * p.block_size);
      return blk < 0 || sl >= p.num_slots ? -1 : (int)sl;
    };
    auto load_codes = [&](const uint8_t *cache, int slot, uint4 (&r)[STEPS]) {
      #pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int s = __shfl_sync(0xffffffffu, slot, i * RP + lane / LPR);
        r[i] = s >= 0 ? __ldg(reinterpret_cast<const uint4 *>(cache + ((int64_t)s * p.Hkv + kvh) * D) + piece)
                      : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    auto load_scale = [&](const float *scales, int slot) {
      return slot >= 0 ? __ldg(scales + (int64_t)slot * p.Hkv + kvh) : 0.0f;
    };
    // bits of a positive finite scale, 0 otherwise
    auto usable = [](float s) -> uint32_t { return s > 0.0f && s < INFINITY ? __float_as_uint(s) : 0u; };
    // A zero vector has scale 1 whatever its neighbours': taken as 0, or its
    // 32 positions' weights would crowd out the others'.  Only a scale of
    // exactly 1 makes the warp look (a wait for memory, but a rare one).
    auto drop_zero = [&](float scale, int slot) -> float {
      const bool one = slot >= 0 && scale == 1.0f;
      if (!__any_sync(0xffffffffu, one)) return scale;
      uint32_t any = 0;
      if (one) {
        const uint4 *row = reinterpret_cast<const uint4 *>(p.vc + ((int64_t)slot * p.Hkv + kvh) * D);
        #pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          const uint4 v = __ldg(row + c);
          any |= v.x | v.y | v.z | v.w;
        }
      }
      return one && (any & 0x7F7F7F7Fu) == 0 ? 0.0f : scale;
    };
    // 16 codes of row r as f16: two 16-byte pieces.  Lanes of the second half
    // of a row store their odd piece first, so that the 8 lanes of a row meet
    // 8 different banks.
    auto store = [&](uint8_t *dst, int r, const uint32_t (&h)[8]) {
      const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), b = make_uint4(h[4], h[5], h[6], h[7]);
      const bool odd = D == 128 && piece >= 4;
      *reinterpret_cast<uint4 *>(dst + piece_off(r, 2 * piece + (odd ? 1 : 0))) = odd ? b : a;
      *reinterpret_cast<uint4 *>(dst + piece_off(r, 2 * piece + (odd ? 0 : 1))) = odd ? a : b;
    };
    // the value scales' reference: 2^-6 of a power of two >= the largest
    // usable one, in [2^-90, 2^120] (1: none)
    auto value_ref = [](uint32_t top) -> uint32_t {
      const uint32_t up = (top + 0x007FFFFFu) & 0x7F800000u;
      return top != 0 ? min(max(up, 43u << 23) - (6u << 23), 247u << 23) : 127u << 23;
    };
    // K' of tile j, and what the softmax needs of the tile's scales
    auto put_k = [&](int j, const uint4 (&r)[STEPS], float scale, float v_scale, int slot) -> bool {
      const int s = j % kCaStages;
      const uint32_t top = __reduce_max_sync(0xffffffffu, usable(scale));
      const float kref = top != 0 ? __uint_as_float(top) : 1.0f;
      const float ratio = __fdiv_rn(scale, kref);
      const float hi = __half2float(__float2half_rn(ratio));
      const uint32_t split2 = f16_pair(hi, ratio - hi);   // infinite scales: NaN, in their column alone
      const uint32_t valid = __ballot_sync(0xffffffffu, slot >= 0);
      const uint32_t vb = value_ref(__reduce_max_sync(0xffffffffu, usable(v_scale)));
      const bool w = j < kCaStages || mbar_wait(&k_empty[s], (uint32_t)(j / kCaStages - 1) & 1u);
      if (!__all_sync(0xffffffffu, w)) return false;
      if (lane == 0) {
        TileMeta &t = meta[j % kCaMeta];
        t.kref[cw] = kref;
        t.valid[cw] = valid;
        t.lv[cw] = (float)((int)(vb >> 23) - 127);
        t.inv_vref[cw] = __uint_as_float((254u << 23) - vb);
      }
      uint8_t *dst = sm + S::K + s * S::kOperand;
      #pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int row = i * RP + lane / LPR;
        const uint32_t f = __shfl_sync(0xffffffffu, split2, row);
        const uint32_t hi2 = __byte_perm(f, f, 0x1010), lo2 = __byte_perm(f, f, 0x3232);
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
        uint32_t h[8];
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t c = e4m3_f16x2(w[e >> 1] >> (16 * (e & 1)));
          h[e] = fma_f16x2(c, hi2, mul_f16x2(c, lo2));
        }
        store(dst, 32 * cw + row, h);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[s]);
      return true;
    };
    auto put_v = [&](int j, uint4 (&r)[STEPS], float scale) -> bool {
      const int s = j % kCaStages;
      const float inv = __uint_as_float((254u << 23) - value_ref(__reduce_max_sync(0xffffffffu, usable(scale))));
      const uint32_t ratio = f16_pair(scale * inv, scale * inv);
      // tiles that some rows see in part: P' = 0 must cancel a value that is
      // not finite, so its vector is zeroed and marked for the rows that see it
      const bool partial = (k.t0 + j + 1) * kCaTile > all_see;
      uint32_t nan = 0;
      if (partial) {
        nan = __ballot_sync(0xffffffffu, !(scale < INFINITY));
        #pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
          bool bad = (nan >> (i * RP + lane / LPR)) & 1u;
          #pragma unroll
          for (int e = 0; e < 4; ++e) bad = bad || (((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
          const uint32_t lanes = __ballot_sync(0xffffffffu, bad);
          if (bad) r[i] = make_uint4(0u, 0u, 0u, 0u);
          #pragma unroll
          for (int g = 0; g < RP; ++g)
            if ((lanes >> (g * LPR)) & ((1u << LPR) - 1u)) nan |= 1u << (i * RP + g);
        }
      }
      const bool w = j < kCaStages || mbar_wait(&v_empty[s], (uint32_t)(j / kCaStages - 1) & 1u);
      if (!__all_sync(0xffffffffu, w)) return false;
      if (partial && lane == 0) meta[j % kCaMeta].nan[cw] = nan;
      uint8_t *dst = sm + S::V + s * S::kOperand;
      #pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int row = i * RP + lane / LPR;
        uint32_t f = __shfl_sync(0xffffffffu, ratio, row);
        if (partial && ((nan >> row) & 1u)) f = 0u;
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
        uint32_t h[8];
        #pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = mul_f16x2(e4m3_f16x2(w[e >> 1] >> (16 * (e & 1))), f);
        store(dst, 32 * cw + row, h);
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[s]);
      return true;
    };
    uint4 kr[STEPS], vr[STEPS];
    int s0 = slot_of(0), s1 = slot_of(1), s2 = slot_of(2);
    load_codes(p.kc, s0, kr);
    float ksc = load_scale(p.ks, s0), vsc = load_scale(p.vs, s0), vsc1 = load_scale(p.vs, s1);
    load_codes(p.vc, s0, vr);
    vsc = drop_zero(vsc, s0);
    bool ok = put_k(0, kr, ksc, vsc, s0);
    ksc = load_scale(p.ks, s1);
    load_codes(p.kc, s1, kr);
    #pragma unroll 1
    for (int j = 0; j < k.tiles && ok; ++j) {
      // here: s0, s1, s2 the slots of tiles j, j + 1, j + 2; kr, ksc of j + 1; vr, vsc of j; vsc1 of j + 1
      const int s3 = slot_of(j + 3);
      if (j + 1 < k.tiles) {
        vsc1 = drop_zero(vsc1, s1);
        ok = put_k(j + 1, kr, ksc, vsc1, s1);
        if (!ok) break;
        ksc = load_scale(p.ks, s2);
        load_codes(p.kc, s2, kr);
      }
      ok = put_v(j, vr, vsc);
      if (!ok) break;
      vsc = vsc1;
      vsc1 = load_scale(p.vs, s2);
      load_codes(p.vc, s1, vr);
      s1 = s2;
      s2 = s3;
    }
    if (!ok && lane == 0) atomicOr(p.status, kStatusTimeoutChunk);
  } else if (stream == 3) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      constexpr uint32_t idesc_qk = idesc_f16(kCaTile, false);
      constexpr uint32_t idesc_pv = idesc_f16(D, true);
      bool ok = true;
      auto wait_full = [&](uint64_t *bar, int j) {
        return mbar_wait(&bar[j % kCaStages], (uint32_t)(j / kCaStages) & 1u);
      };
      // S of stream s for tile j: behind the stream's product before it, whose
      // P' it overwrites (products of one thread run in order)
      auto qk = [&](int s, int j) {
        const uint32_t qb = smem_u32(sm + S::Q + (two ? s : 0) * S::kOperand);
        const uint32_t kb = smem_u32(sm + S::K + (j % kCaStages) * S::kOperand);
        #pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (kCaRows * 128) + (kk & 3) * 32;
          mma_f16_ss(tmem_base + s * 128, sw128_kmajor_desc(qb + off), sw128_kmajor_desc(kb + off), idesc_qk,
                     kk > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[s]);
      };
      auto pv = [&](int s, int j, bool first) {
        const uint32_t vb = smem_u32(sm + S::V + (j % kCaStages) * S::kOperand);
        #pragma unroll
        for (int kk = 0; kk < kCaTile / 16; ++kk)
          mma_f16_ts(tmem_base + 256 + s * D, tmem_base + s * 128 + kk * 8,
                     sw128_mn_desc(vb + kk * 16 * 128, kCaRows * 128), idesc_pv, !first || kk > 0 ? 1u : 0u);
      };
      if (two) {
        ok = wait_full(k_full, 0);
        if (ok) {
          tc_fence_after();
          if (k.tiles0 > 0) qk(0, 0);
          qk(1, 0);
          mma_commit(&k_empty[0]);
        }
        for (int j = 0; j < k.tiles && ok; ++j) {
          for (int s = j < k.tiles0 ? 0 : 1; s < 2 && ok; ++s) {
            ok = wait_full(v_full, j) && mbar_wait(&p_full[s], (uint32_t)j & 1u);
            if (!ok) break;
            tc_fence_after();
            pv(s, j, j == 0);
            const int mine = s == 0 ? k.tiles0 : k.tiles;
            if (j + 1 == mine) mma_commit(&o_done[s]);
            if (s == 1) mma_commit(&v_empty[j % kCaStages]);
            if (j + 1 < mine) {
              ok = wait_full(k_full, j + 1);
              if (!ok) break;
              tc_fence_after();
              qk(s, j + 1);
              if (s == 1) mma_commit(&k_empty[(j + 1) % kCaStages]);
            }
          }
        }
      } else {
        for (int j = 0; j < min(2, k.tiles) && ok; ++j) {
          ok = wait_full(k_full, j);
          if (!ok) break;
          tc_fence_after();
          qk(j, j);
          mma_commit(&k_empty[j % kCaStages]);
        }
        for (int j = 0; j < k.tiles && ok; ++j) {
          const int s = j & 1;
          ok = wait_full(v_full, j) && mbar_wait(&p_full[s], (uint32_t)(j >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          pv(s, j, j < 2);
          mma_commit(&v_empty[j % kCaStages]);
          if (j + 2 >= k.tiles) mma_commit(&o_done[s]);
          if (j + 2 < k.tiles) {
            ok = wait_full(k_full, j + 2);
            if (!ok) break;
            tc_fence_after();
            qk(s, j + 2);
            mma_commit(&k_empty[(j + 2) % kCaStages]);
          }
        }
      }
      if (!ok) atomicOr(p.status, kStatusTimeoutChunk);
      // every product issued has completed before the CTA ends
      mma_commit(drain);
      mbar_wait(drain, 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem_base + lane_addr + stream * 128;        // S, then P'
    const uint32_t to = tmem_base + lane_addr + 256 + stream * D;    // O
    const int count = two ? (stream == 0 ? k.tiles0 : k.tiles) : (k.tiles + 1 - stream) >> 1;
    // positions that this row sees; rows of no token see all (nothing to mask), and are not written
    const int sees = has_row ? k.m - k.n + tok + 1 : 0x7FFFFFFF;
    float r = -INFINITY, l = 0.0f;
    bool ok = true;
    #pragma unroll 1
    for (int it = 0; it < count; ++it) {
      const int j = two ? it : 2 * it + stream;
      const bool arrived = mbar_wait(&s_full[stream], (uint32_t)it & 1u);
      ok = __all_sync(0xffffffffu, arrived);
      if (!ok) break;
      tc_fence_after();
      const TileMeta &tm = meta[j % kCaMeta];
      uint32_t mask[4];
      bool full = true;
      #pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = sees - ((k.t0 + j) * kCaTile + 32 * c);
        const uint32_t causal = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
        mask[c] = tm.valid[c] & causal;
        full = full && mask[c] == 0xffffffffu;
      }
      full = __all_sync(0xffffffffu, full);
      float cf[4];
      #pragma unroll
      for (int c = 0; c < 4; ++c) cf[c] = tm.kref[c] * rowfac;
      // the tile's largest t + log2 vref
      float top = -INFINITY;
      #pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        tmem_ld_32x32b_x32(ts + 32 * c, x);
        tmem_wait_ld();
        float m0 = -INFINITY, m1 = -INFINITY;
        if (full) {
          #pragma unroll
          for (int i = 0; i < 32; i += 4) {
            m0 = fmaxf(fmaxf(m0, __uint_as_float(x[i])), __uint_as_float(x[i + 1]));
            m1 = fmaxf(fmaxf(m1, __uint_as_float(x[i + 2])), __uint_as_float(x[i + 3]));
          }
          top = fmaxf(top, fmaf(fmaxf(m0, m1), cf[c], tm.lv[c]));
        } else {
          #pragma unroll
          for (int i = 0; i < 32; ++i)
            m0 = fmaxf(m0, (mask[c] >> i) & 1u ? __uint_as_float(x[i]) * cf[c] : -INFINITY);
          top = fmaxf(top, m0 + tm.lv[c]);
        }
      }
      const bool need = top > r + kCaLazy;
      if (__any_sync(0xffffffffu, need)) {
        const float f = need && r != -INFINITY ? ex2(r - top) : 1.0f;
        if (need) r = top;
        l *= f;
        if (it > 0) {
          #pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t x[32];
            tmem_ld_32x32b_x32(to + 32 * c, x);
            tmem_wait_ld();
            #pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
            tmem_st_32x32b_x32(to + 32 * c, x);
          }
        }
      }
      const float rs = r == -INFINITY ? 0.0f : r;
      #pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32], y[16];
        tmem_ld_32x32b_x32(ts + 32 * c, x);
        tmem_wait_ld();
        const float bias = tm.lv[c] - rs;
        const uint64_t cf2 = pack_f32x2(cf[c], cf[c]), b2 = pack_f32x2(bias, bias);
        uint64_t sum0 = 0, sum1 = 0;
        #pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 t = unpack_f32x2(
              fma_f32x2(pack_f32x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), cf2, b2));
          float a = ex2(t.x), b = ex2(t.y);
          if (!full) {
            a = (mask[c] >> (2 * i)) & 1u ? a : 0.0f;
            b = (mask[c] >> (2 * i + 1)) & 1u ? b : 0.0f;
          }
          y[i] = f16_pair(a, b);
          if (i & 1) sum1 = add_f32x2(sum1, pack_f32x2(a, b));
          else sum0 = add_f32x2(sum0, pack_f32x2(a, b));
        }
        const float2 sm2 = unpack_f32x2(add_f32x2(sum0, sum1));
        l = fmaf(sm2.x + sm2.y, tm.inv_vref[c], l);
        tmem_st_32x32b_x16(ts + 16 * c, y);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[stream]);
    }
    if (ok && count > 0) ok = mbar_wait(&o_done[stream], 0);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) atomicOr(p.status, kStatusTimeoutChunk);
    tc_fence_after();
    if (!ok) l = 0.0f;
    float f0 = l == 0.0f ? 0.0f : 1.0f;   // factor of this stream's O
    float f1 = 0.0f;                      // factor of the other stream's, when the two are joined
    float *joined = reinterpret_cast<float *>(sm + S::K);   // [D][128], in the K ring: every S is done
    float2 *ml1 = reinterpret_cast<float2 *>(sm + S::ML);
    if (!two) {
      if (stream == 1) {
        if (l != 0.0f || count > 0) {
          #pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t x[32];
            tmem_ld_32x32b_x32(to + 32 * c, x);
            tmem_wait_ld();
            #pragma unroll
            for (int i = 0; i < 32; ++i) joined[(32 * c + i) * kCaRows + lrow] = __uint_as_float(x[i]);
          }
        }
        ml1[lrow] = make_float2(r, l);
        __threadfence_block();
        asm volatile("bar.arrive 1, 256;" ::: "memory");
      } else {
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const float2 o = ml1[lrow];
        if (o.y != 0.0f) {   // NaN too
          const float rn = fmaxf(r, o.x);
          f0 = l == 0.0f ? 0.0f : ex2(r - rn);
          f1 = ex2(o.x - rn);
          l = l * f0 + o.y * f1;
          r = rn;
        }
      }
    }
    if (two || stream == 0) {
      // a value vector that is not finite: in a tile that every row sees it
      // came through the product; in the others (the last three at most) it
      // was left out of the product and reaches the rows that see it here
      for (int j = max(0, k.tiles - 3); j < k.tiles; ++j) {
        if ((k.t0 + j + 1) * kCaTile <= all_see) continue;
        const TileMeta &tm = meta[j % kCaMeta];
        #pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int n = sees - ((k.t0 + j) * kCaTile + 32 * c);
          const uint32_t causal = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
          if (tm.nan[c] & tm.valid[c] & causal) l = __uint_as_float(0x7FC00000u);
        }
      }
      const int64_t oh = (int64_t)(k.first_q + tok) * p.Hq + kvh * p.G + head;
      const int64_t part = oh * p.splits + split;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      if (has_row && p.splits > 1) {
        p.part_ml[part * 2] = l == 0.0f ? -INFINITY : r;
        p.part_ml[part * 2 + 1] = l;
      }
      #pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        __syncwarp();
        tmem_ld_32x32b_x32(to + 32 * c, x);   // stale where no product was issued: f0 is 0 there
        tmem_wait_ld();
        float o[32];
        #pragma unroll
        for (int i = 0; i < 32; ++i) {
          o[i] = f0 == 0.0f ? 0.0f : __uint_as_float(x[i]) * f0;
          if (f1 != 0.0f) o[i] = fmaf(joined[(32 * c + i) * kCaRows + lrow], f1, o[i]);
        }
        if (has_row && p.splits > 1) {
          float4 *dst = reinterpret_cast<float4 *>(p.part_acc + part * D + 32 * c);
          #pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else if (has_row) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.out + oh * D + 32 * c);
          #pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(bf16_pair(o[8 * i] * inv, o[8 * i + 1] * inv),
                                bf16_pair(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                bf16_pair(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                bf16_pair(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Joins the partial results of a context split over CTAs: a warp a (token,
// head), D / 32 values a lane.
template <int D>
__global__ void __launch_bounds__(256) chunk_attn_combine_kernel(const ChunkArgs p) {
  griddep_wait();
  const int64_t oh = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (oh >= (int64_t)p.total_q * p.Hq) return;
  const int row = (int)(oh / p.Hq);
  if (row < __ldg(p.cu_q) || row >= __ldg(p.cu_q + p.B)) return;   // rows of no sequence are left as they were
  const float *ml = p.part_ml + oh * p.splits * 2;
  float top = -INFINITY;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, ml[2 * s]);
  constexpr int N = D / 32;
  float acc[N];
  #pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  float l = 0.0f;
  for (int s = 0; s < p.splits; ++s) {
    if (ml[2 * s + 1] == 0.0f) continue;
    const float w = ex2(ml[2 * s] - top);
    l = fmaf(ml[2 * s + 1], w, l);
    const float *a = p.part_acc + (oh * p.splits + s) * D + lane * N;
    #pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = *reinterpret_cast<const float2 *>(a + i);
      acc[i] = fmaf(v.x, w, acc[i]);
      acc[i + 1] = fmaf(v.y, w, acc[i + 1]);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t *o = reinterpret_cast<uint32_t *>(p.out + oh * D + lane * N);
  #pragma unroll
  for (int i = 0; i < N; i += 2) o[i / 2] = bf16_pair(acc[i] * inv, acc[i + 1] * inv);
}

struct ChunkPlan {
  int64_t row_tiles;   // at least the row tiles of all sequences
  int splits, split_tiles;
};

// Row tiles, and the CTAs that share a context.  A part costs its tiles and a
// start and end worth kFixed tiles; the parts of the last wave leave SMs idle,
// so the split with the least (waves x cost) is taken.
ChunkPlan plan_chunk(int64_t total_q, int64_t B, int Hkv, int G, int64_t max_q, int64_t max_context) {
  constexpr int64_t kFixed = 6;
  ChunkPlan c;
  c.row_tiles = std::min(total_q * G / (2 * kCaRows) + B, B * ((max_q * G + 2 * kCaRows - 1) / (2 * kCaRows)));
  const int64_t tiles = std::max<int64_t>(1, (max_context + kCaTile - 1) / kCaTile);
  const int64_t ctas = c.row_tiles * Hkv, sms = num_sms();
  int64_t best = -1;
  c.splits = 1;
  c.split_tiles = (int)tiles;
  for (int64_t s = 1; s <= kCaMaxSplits; ++s) {
    const int64_t each = (tiles + s - 1) / s;
    if (s > 1 && (each < 4 || ctas * s > 4 * sms)) break;
    const int64_t parts = (tiles + each - 1) / each;
    if (parts != s) continue;
    const int64_t cost = (ctas * s + sms - 1) / sms * (each + kFixed) + (s > 1 ? kFixed : 0);
    if (best < 0 || cost < best) {
      best = cost;
      c.splits = (int)s;
      c.split_tiles = (int)each;
    }
  }
  return c;
}

size_t part_ml_bytes(int64_t total_q, int Hq, int splits) {
  return ((size_t)total_q * Hq * splits * 2 * sizeof(float) + 255) / 256 * 256;
}

constexpr size_t kStatusBytes = 256;

template <int D>
cudaError_t launch_chunk(const ChunkArgs &p, const ChunkPlan &c, cudaStream_t st) {
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t a =
        cudaFuncSetAttribute(chunk_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, CaSmem<D>::BYTES);
    if (a != cudaSuccess) return a;
    attr_set[dev].store(true, std::memory_order_release);
  }
  const dim3 grid((unsigned)(c.row_tiles * p.Hkv), (unsigned)c.splits);
  chunk_attn_kernel<D><<<grid, kCaThreads, CaSmem<D>::BYTES, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || c.splits == 1) return e;
  return launch_pdl(chunk_attn_combine_kernel<D>, dim3((unsigned)(((int64_t)p.total_q * p.Hq + 7) / 8)), 256, st, p);
}

}  // namespace

int chunk_attn_splits(int64_t total_q, int64_t B, int Hq, int Hkv, int64_t max_q, int64_t max_context) {
  return plan_chunk(total_q, B, Hkv, Hq / Hkv, max_q, max_context).splits;
}

int64_t chunk_attn_ctas(int64_t total_q, int64_t B, int Hq, int Hkv, int64_t max_q, int64_t max_context) {
  return plan_chunk(total_q, B, Hkv, Hq / Hkv, max_q, max_context).row_tiles * Hkv;
}

size_t chunk_attn_workspace_bytes(int64_t total_q, int64_t B, int Hq, int Hkv, int D, int64_t max_q,
                                  int64_t max_context) {
  const int splits = chunk_attn_splits(total_q, B, Hq, Hkv, max_q, max_context);
  if (splits == 1) return kStatusBytes;
  return kStatusBytes + part_ml_bytes(total_q, Hq, splits) + (size_t)total_q * Hq * splits * D * sizeof(float);
}

cudaError_t launch_chunk_attention(const ChunkAttention &a, cudaStream_t st) {
  const ChunkPlan c = plan_chunk(a.total_q, a.B, a.Hkv, a.Hq / a.Hkv, a.max_q, a.max_context);
  ChunkArgs p = {};
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.ldq = a.ldq;
  p.kc = a.kc;
  p.vc = a.vc;
  p.ks = a.ks;
  p.vs = a.vs;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.cu_q = a.cu_q;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.total_q = a.total_q;
  p.block_size = a.block_size;
  p.max_blocks = a.max_blocks;
  p.max_context = a.max_context;
  // the high word of pos * ceil(2^64 / block_size) is pos / block_size for
  // every pos < 2^32: the product exceeds pos / block_size by less than 2^-32
  p.bs_magic = ~0ull / (uint64_t)a.block_size + 1;
  p.num_slots = a.num_slots;
  p.splits = c.splits;
  p.split_tiles = c.split_tiles;
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.status = static_cast<uint32_t *>(a.ws);
  p.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + kStatusBytes);
  p.part_acc = p.part_ml + part_ml_bytes(a.total_q, a.Hq, c.splits) / sizeof(float);
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  return a.D == 64 ? launch_chunk<64>(p, c, st) : launch_chunk<128>(p, c, st);
}

}  // namespace ptpc
