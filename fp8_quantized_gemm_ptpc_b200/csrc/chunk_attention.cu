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
// Warps 8-11 (K) and 12-15 (V) read the codes (16 bytes a lane; any block size;
// a tile ahead, in registers), turn them into f16 and lay them out in shared
// memory for the MMAs.  The scales go in here, relative to a reference of each
// 32 positions (a warp's rows):  K' = code * ks / kref,  V' = code * vs / vref,
// so that the softmax has one factor for 32 columns instead of one a column.
// kref is a power of two at least the largest key scale; the product is formed
// as code * hi + code * lo with the ratio split in two f16, so K' is rounded
// once.  vref is 2^-6 of such a power for the value scales: V' reaches 448 *
// 64, near f16's largest value.  An error is at most 2^-11 of the key or value
// itself.
// Scales go by a common reference only where they lie within 2^6 of the largest
// of the 32 (kCaSpread).  Otherwise one position would take f16's range, for P'
// as for K' and V', from the others: a zero vector, which has scale 1, or a
// large one that a row does not even see.  Such 32 positions keep their codes as
// they are (V's times 64) and have factors of their own, which the softmax takes
// from COLS, unit by unit of 64 positions and a good deal slower (apart_unit); a
// zero value weighs in the sum alone.  Where all are such, 2048 tokens on 30,720
// take 5.4 ms, with a zero vector every 512 positions 2.9.  Keeping that code out of the loop that
// other units take matters: in one body with it they were 3.5% slower, and now
// 1% (2048 tokens on 30,720; the converters' tests of the scales, most of it).
// Warps 16 and 17 (a stream each) issue S = Q K'^T (kind::f16, q as f16 after a
// power-of-two scale a row, exact) and O += P' V' with P' from tensor memory.
// Warps 0-3 and 4-7 (a stream each, a thread a row) do the softmax in base 2.
// With t = S * kref * qscale * log2 e, a weight is P' = 2^(t + log2 vref - r):
// the reference r follows the largest t + log2 vref, so the f16 P' stays near
// 1 whatever the values' size, and the sum of 2^(t - r) is that of P' /
// vref.  r moves (and O, in tensor memory, is rescaled) only when the weights
// of 64 positions, taken with the r of before, sum to 2^15 or more, which also
// keeps each below f16's largest value: the common case needs no maximum at
// all.  A row's first r is the maximum of its first 64 positions.  P'
// overwrites S in place.
// A tile goes through in halves of 64 positions, each with scores of its own in
// tensor memory: a stream's products of one half run while its softmax works on
// the other.  A CTA with 128 rows or fewer gives both streams the same rows and
// every other tile each, and joins them at the end.
//
// With few rows the context is split over CTAs whose partial results a second
// kernel joins (plan_chunk).  Every wait is bounded; a timeout sets a bit in
// the status word at the front of the workspace, and the rows are NaN.
//
// What bounds it (B200, heads of 128).  64 positions of both streams take about
// 1,900 cycles of an SM, in which the products need 620 (the MMAs of 64 columns
// read shared memory for 49 cycles each, 16 columns of depth a time) and the
// exponentials' unit is busy for 1,024; the schedulers issue in 57% of the
// cycles, the rest is latency.  With 128 rows or fewer the conversions bound it:
// 3,100 cycles for 128 positions.  A CTA's start and end cost about 17,000
// cycles (its places 1,200, the first codes and q 7,000, the first scores, its
// last product and output 6,500, the next CTA's launch 2,500), which is why a
// context is split only where SMs would idle.  Heads of 64 take the same 1,900
// cycles for half the products.  With 64 + 8 heads, 2048 tokens on 30,720 more
// take 2.01 ms (0.64 of the measured bf16 rate) a few calls at a time and 2.29 ms
// (0.56) one behind the other, where the board's power limit holds the clock at
// 1.5 GHz; with 32 + 8, eight prompts of 300 to 4000 tokens 566 and 595 us (0.46,
// 0.43; 1.63 GHz).  A step of single tokens is decode_attention's: 32 on 4096
// positions, 64 + 8 heads, 134 us here and 54 there.
// Measured and dropped: scores of 128 columns (the MMAs of both streams then
// collide, and shared memory answers the converters late), one S buffer and two
// of P' a stream, four softmax warpgroups, the next scores' loads ahead of P'
// (all slower); converter code apart for whole tiles, a polynomial for one
// exponential in sixteen (no gain), for more (slower); L2 prefetches two tiles
// ahead (8% faster for single tokens, 2% slower for chunks) or by the spare
// warps (6% faster, drafts 2% slower); with few rows a third stage of V, the
// kernel as a programmatic dependent, tensor memory ahead of the search (no gain).
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

// Warpgroups: 0, 1 the softmax of a stream each, 2 converts K, 3 converts V,
// 4 issues the products (its first two warps, a stream each).
constexpr int kCaThreads = 640;
// Registers a thread once the roles part (the softmax keeps 64 of a row's
// scores): 2 x 136 + 2 x 80 + 48 = 5 x 96, what the CTA is launched with.
constexpr int kCaRegsSoftmax = 136, kCaRegsConvert = 80, kCaRegsIssuer = 48;
constexpr int kCaRows = 128;      // rows a stream
constexpr int kCaTile = 128;      // positions a tile
constexpr int kCaStages = 2;      // stages of the K ring and of the V ring
constexpr int kCaMeta = 8;        // tiles whose scales are kept (more than the stages ahead of the softmax)
constexpr uint32_t kStatusTimeoutChunk = 1u << 4;
constexpr float kCaMost = 32768.0f;   // r is looked at again when a row's weights of 64 positions reach this sum,
constexpr float kCaLazy = 8.0f;       // and moves where the largest exceeds it by this (64 * 2^8 < kCaMost)
constexpr int kCaMaxSplits = 64;
constexpr uint32_t kCaSpread = 6u << 23;    // scales share a reference within 2^6 of the largest (float bits),
constexpr uint32_t kCaLeast = 53u << 23;    // and from 2^-74 on
constexpr float kCaNear = -100.0f;          // 2^this and sums times it are normal numbers
constexpr float kCaNoValue = -88.0f;        // what log2 of a value's scale counts as in r, at least

// What the softmax needs of a tile: for each of its two halves of 64 positions
// and the 32-position parts of a half
struct TileMeta {
  struct Half {
    float kref[2], lv[2];                   // lv = log2 vref; NaN: a position has factors of its own (CaSmem::COLS)
    float inv_vref[2];
    uint32_t valid[2];                      // bit i: the position is in the cache
  } half[2];
  uint32_t nan[4];                          // bit i: the position's value vector is not finite (diagonal tiles only)
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
  uint32_t num_blocks;
  int tile_blocks, tile_rest;    // kCaTile = tile_blocks * block_size + tile_rest
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
  static constexpr int COLS = ML + kCaRows * 8;             // [tile of kCaMeta][position]: what kref and lv are for it alone
  static constexpr int BARS = COLS + kCaMeta * kCaTile * 8;
  static constexpr int kBars = 4 * kCaStages + 3 * 4 + 3;
  static constexpr int BYTES = 1024 + BARS + kBars * 8 + 16;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// l 2^by, by <= 0.  A sum l may reach 2^88 a position: some of it is left where
// the factor itself is below fp32's smallest number.
__device__ __forceinline__ float times_2to(float l, float by) {
  return by > kCaNear ? l * ex2(by) : l * ex2(0.5f * by) * ex2(0.5f * by);
}

__device__ __forceinline__ void ex2_in_order(float &x) { asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(x)); }

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
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ void add_f32x2_in_order(uint64_t &a, uint64_t b) {
  asm volatile("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
}

__device__ __forceinline__ uint32_t f16_pair_in_order(float lo, float hi) {
  uint32_t r;
  asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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
// Four E4M3 codes (lowest byte first) as two pairs of f16, exact.
__device__ __forceinline__ void e4m3_f16x4(uint32_t four, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
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

// The upper halves of the operands' shared-memory descriptors; the lower half
// is (address >> 4) | (byte offset between atoms along M or N >> 4) << 16, and
// a step inside a tile adds to it, so the issuing thread spends an addition a
// product.
constexpr uint32_t kDescHi = (1024u >> 4)    // 8-row atoms 1024 bytes apart
                             | 1u << 14      // descriptor version (tcgen05)
                             | 2u << 29;     // 128-byte swizzle
// K-major tile: rows of 64 f16 along K (128 bytes).
__device__ __forceinline__ uint32_t desc_k_major(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4 | 1u << 16; }
// MN-major tile: rows of 64 f16 along N, one per K index; the next 64 values
// of N start kCaRows * 128 bytes further.
__device__ __forceinline__ uint32_t desc_mn_major(uint32_t saddr) {
  return (saddr & 0x3FFFFu) >> 4 | (uint32_t)(kCaRows * 128 >> 4) << 16;
}

// D[tmem] (+)= A[smem] * B[smem], kind::f16 -> fp32.
template <bool ACC>
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%1, %4};\n\tmov.b64 y, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "n"(ACC ? 1 : 0)
      : "memory");
}
// The same with A in tensor memory (two f16 along K a column, a row a lane).
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(kDescHi), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_32x32b_x4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
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

// Loads that stay where they are written, so that a tile's are in flight
// while the tile before it is converted.
__device__ __forceinline__ uint4 ld_codes(const uint8_t *ptr) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(ptr));
  return v;
}
__device__ __forceinline__ float ld_scale(const float *ptr) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(ptr));
  return v;
}

// Waits for a phase, in few instructions; false after some seconds (a failed
// try takes from tens to some thousand cycles).
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity) {
  uint32_t left = 1u << 20;
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "AGAIN%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%2], %3;\n\t"
      "@p bra THERE%=;\n\t"
      "sub.u32 %1, %1, 1;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "@q bra AGAIN%=;\n\t"
      "THERE%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done), "+r"(left)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// Of a stream's units, where it has every other tile, those that lie whole
// within the first `seen` positions.
__device__ __forceinline__ int plain_units(int seen, int stream) {
  const int all = max(seen, 0) >> 6;              // units of both streams
  const int tiles = all >> 1;                     // whole tiles, then perhaps half of one
  const int mine = (tiles + 1 - stream) >> 1;
  return 2 * mine + ((all & 1) && (tiles & 1) == stream ? 1 : 0);
}

// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool bar_test(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// Ties loaded registers to the wait before: nothing that reads them moves above it.
__device__ __forceinline__ void arrived32(uint32_t (&r)[32]) {
  #pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                 "+r"(r[i + 6]), "+r"(r[i + 7]));
}

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Instruction descriptor: dense kind::f16, f16 operands, fp32 accumulation,
// M = 128; B K-major, or MN-major.
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kCaRows >> 4) << 24);
}

// Byte offset of 16-byte piece c (0 .. D / 8 - 1) of row r in an operand tile:
// atoms of 64 f16 (128-byte swizzled rows), 16 KB apart.
__device__ __forceinline__ int piece_off(int r, int c) {
  return (c >> 3) * (kCaRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Shared memory by its own addresses (a pointer made from an aligned base would
// be a generic one).
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t at, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ float2 lds64(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t at, uint32_t a) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(a) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
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
    int first = 0, n = 0, m = 0;
    if (b < p.B) {
      m = max(__ldg(p.context_lens + b), 0);
      n = seq_tokens(p, b, first);
    }
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
      k.m = __shfl_sync(0xffffffffu, m, at);
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// 16 bytes from memory into shared memory, asynchronously; zeros where `in` is
// false (nothing is read then).
__device__ __forceinline__ void copy16_or_zero(uint32_t to, const void *from, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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
  uint64_t *s_full = v_empty + kCaStages;   // [stream][half] S of 64 positions is in tensor memory
  uint64_t *p_full = s_full + 4;            // [stream][half] their P' is written, O rescaled (4 warps)
  uint64_t *o_done = p_full + 4;            // [stream][half] their product is done
  uint64_t *q_full = o_done + 4;            // q is in shared memory (its rows' threads)
  uint64_t *drain = q_full + 1;             // [stream] its issuer's last commit
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 2);
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
  const int stream = warp >> 2;        // the warpgroup: 0, 1: softmax streams
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
    const uint32_t users = two ? 2 : 1;   // streams that use a tile
    for (int s = 0; s < kCaStages; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], users);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], users);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4);
      mbar_init(&o_done[s], 1);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    mbar_init(q_full, two ? 2 * kCaRows : kCaRows);
    fence_barrier_init();
  }
  if (warp == 16) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }

  // The barriers and tensor memory are ready: each role passes here once its
  // first loads are on their way.
  auto all_set = [&]() -> uint32_t {
    tc_fence_before();
    asm volatile("bar.sync 4, %0;" ::"n"(kCaThreads) : "memory");
    tc_fence_after();
    return *reinterpret_cast<volatile uint32_t *>(tmem_holder);
  };
  uint32_t tmem_base;

  if (stream == 2 || stream == 3) {
    // ------------------------------------------------------------ converters
    regs_down<kCaRegsConvert>();
    constexpr int LPR = D / 16;           // lanes a row, 16 codes a lane
    constexpr int RP = 32 / LPR;          // rows a load instruction
    constexpr int STEPS = 32 / RP;
    const bool is_k = stream == 2;
    const int cw = warp & 3;
    // this lane's row of RP and its 16 codes of the row.  8 neighbouring lanes
    // hold the same half of an even and an odd row: their 16-byte stores, two
    // pieces apart in a row, meet 8 different banks under the swizzle.
    const int row_in = D == 128 ? (lane >> 4) * 2 + ((lane >> 2) & 1) : lane >> 2;
    const int piece = D == 128 ? ((lane >> 3) & 1) * 4 + (lane & 3) : lane & 3;
    const int32_t *table = p.block_tables + (int64_t)k.b * p.max_blocks;
    // This lane's position of each tile, walked tile by tile: its block in the
    // table and its place in it.  fetch() loads the block of the next tile;
    // slot() says where that is, -1 where nothing is read.  A tile lies
    // between the two, so that nothing waits for the table.
    int pos = k.t0 * kCaTile + 32 * cw + lane;
    int bi = (int)__umul64hi((uint64_t)pos, p.bs_magic), in_block = pos - bi * p.block_size;
    int blk = 0, at = 0;
    bool there = false;
    auto fetch = [&]() {
      there = pos < k.kv_end && bi < p.max_blocks;
      blk = __ldg(table + min(bi, p.max_blocks - 1));
      at = in_block;
      pos += kCaTile;
      bi += p.tile_blocks;
      in_block += p.tile_rest;
      if (in_block >= p.block_size) {
        in_block -= p.block_size;
        ++bi;
      }
    };
    auto slot_of = [&]() -> int { return there && (uint32_t)blk < p.num_blocks ? blk * p.block_size + at : -1; };
    const uint8_t *codes = (is_k ? p.kc : p.vc) + kvh * D + piece * 16;
    const uint32_t row_bytes = (uint32_t)(p.Hkv * D);
    // A position that is not in the cache reads slot 0 instead (a load with no
    // condition: a select behind it would wait for it).  Its key is masked by
    // the softmax whatever it holds, its value is zeroed, its scales are
    // dropped where they are used.
    auto load_step = [&](int slot, int i) {   // the codes of step i; slot >= 0
      return ld_codes(codes + (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, slot, i * RP + row_in) * row_bytes);
    };
    auto load_scale = [&](const float *scales, int slot) {
      return ld_scale(scales + (int64_t)max(slot, 0) * p.Hkv + kvh);
    };
    // bits of a finite scale's magnitude, 0 otherwise
    auto usable = [](float s) -> uint32_t { return fabsf(s) < INFINITY ? __float_as_uint(fabsf(s)) : 0u; };
    // The value scale that counts: 0 where there is none.  A zero vector has
    // scale 1 whatever its neighbours': taken as 0 too, or its weight would
    // crowd out the others'.  Only a scale of exactly 1 makes the warp look (a
    // wait for memory, but a rare one).
    auto value_scale = [&](float scale, int slot) -> float {
      const bool one = slot >= 0 && scale == 1.0f;
      if (!__any_sync(0xffffffffu, one)) return slot >= 0 ? scale : 0.0f;
      uint32_t any = 0;
      if (one) {
        const uint4 *row = reinterpret_cast<const uint4 *>(p.vc + ((int64_t)slot * p.Hkv + kvh) * D);
        #pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          const uint4 v = __ldg(row + c);
          any |= v.x | v.y | v.z | v.w;
        }
      }
      return slot < 0 || (one && (any & 0x7F7F7F7Fu) == 0) ? 0.0f : scale;
    };
    // The reference of 32 scales: a power of two >= the largest usable one,
    // less `below` powers, in [2^-90, 2^120] (1: there is none); as bits.
    // apart: not all of the positions in the cache can go by it.
    auto reference = [&](float scale, int slot, uint32_t below, bool &apart) -> uint32_t {
      const uint32_t mine = usable(scale), top = __reduce_max_sync(0xffffffffu, mine);
      const uint32_t up = (top + 0x007FFFFFu) & 0x7F800000u;
      apart = __any_sync(0xffffffffu, slot >= 0 && (mine < kCaLeast || top - mine > kCaSpread));
      return top != 0 ? min(max(up, 43u << 23) - (below << 23), 247u << 23) : 127u << 23;
    };
    // 2^-x of a power of two 2^x
    auto inverse = [](uint32_t bits) { return __uint_as_float((254u << 23) - bits); };
    // Where this lane's two 16-byte pieces of its row of step i go, relative to
    // the warp's rows of a stage: the step's rows are whole 8-row groups on
    // (D = 64), or half ones (D = 128: the swizzle's bit 2 alternates).
    uint32_t put[2][2];
    #pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      #pragma unroll
      for (int c = 0; c < 2; ++c)
        put[odd][c] = (uint32_t)piece_off(32 * cw + row_in + odd * RP, 2 * piece + c) - odd * RP * 128;
    }
    auto store = [&](uint32_t stage, int i, const uint32_t (&h)[8]) {
      const uint32_t to = stage + i * RP * 128;
      sts128(to + put[i & 1][0], h[0], h[1], h[2], h[3]);
      sts128(to + put[i & 1][1], h[4], h[5], h[6], h[7]);
    };
    // stage j % kCaStages is free (its products of kCaStages tiles ago are done)
    auto wait_free = [&](uint64_t *empty, int j) -> bool {
      const bool w = j < kCaStages || bar_wait(&empty[j % kCaStages], (uint32_t)(j / kCaStages - 1) & 1u);
      return __all_sync(0xffffffffu, w);
    };
    auto publish = [&](uint64_t *full, int j) {
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[j % kCaStages]);
    };

    // One loop for both, so that the roles' code stays within the instruction
    // cache (32 KB: beyond it, they run at half the rate).
    uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
    const uint32_t ring = smem_u32(sm + (is_k ? S::K : S::V));
    uint4 r[STEPS];
    fetch();
    int slot = slot_of();
    fetch();
    float ksc = load_scale(p.ks, slot), vsc = load_scale(p.vs, slot);
    #pragma unroll
    for (int i = 0; i < STEPS; ++i) r[i] = load_step(max(slot, 0), i);
    tmem_base = all_set();
    bool ok = true;
    #pragma unroll 1
    for (int j = 0; j < k.tiles; ++j) {
      // the next tile's scales, and below its codes as soon as their registers
      // are free: memory has a whole tile's time to answer
      const int next = slot_of(), next0 = max(next, 0);
      fetch();
      const float next_ksc = load_scale(p.ks, next), next_vsc = load_scale(p.vs, next);
      const float v_scale = value_scale(vsc, slot);
      const float scale = is_k ? (slot >= 0 ? ksc : 0.0f) : v_scale;
      bool v_apart, k_apart = false;
      const uint32_t vb = reference(v_scale, slot, 6, v_apart), ref = is_k ? reference(scale, slot, 0, k_apart) : vb;
      const uint32_t valid = __ballot_sync(0xffffffffu, slot >= 0);
      // x' = code * scale / ref, the ratio as a sum of two f16
      const float ratio = scale * inverse(ref);
      const float hi = __half2float(__float2half_rn(ratio));
      uint32_t split2 = f16_pair(hi, ratio - hi);   // of an infinite scale: NaN (K: in its column alone)
      // scales apart: the codes as they are, V's times 64, exact
      if (__builtin_expect(is_k ? k_apart : v_apart, 0))
        split2 = is_k ? f16_pair(1.0f, 0.0f) : f16_pair(scale - scale + copysignf(64.0f, scale), 0.0f);
      uint32_t nan = 0;
      // tiles that some rows see in part: P' = 0 must cancel a value that is
      // not finite, so its vector is zeroed and marked for the rows that see it
      const bool partial = !is_k && (k.t0 + j + 1) * kCaTile > all_see;
      if (__builtin_expect(partial || (!is_k && valid != 0xffffffffu), 0)) {
        nan = __ballot_sync(0xffffffffu, !(scale < INFINITY));
        #pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
          const int row = i * RP + row_in;
          bool bad = false;
          #pragma unroll
          for (int e = 0; e < 4; ++e) bad = bad || (((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
          const bool there = (valid >> row) & 1u;
          bad = bad && partial && there;
          if (bad || !there) r[i] = make_uint4(0u, 0u, 0u, 0u);
          nan |= __reduce_or_sync(0xffffffffu, bad ? 1u << row : 0u);
        }
        if (partial && ((nan >> lane) & 1u)) split2 = 0u;
      }
      ok = wait_free(empty, j);
      if (!ok) break;
      const float lv = (float)((int)(vb >> 23) - 127);
      if (is_k) {
        // each position's own factors, which one with its scale apart goes by
        // (and the 64 positions that go through the softmax with it)
        const float kf = k_apart ? scale - scale + scale : __uint_as_float(ref);
        const float vf = v_apart ? (usable(v_scale) != 0 ? __log2f(fabsf(v_scale)) - 6.0f : -INFINITY) : lv;
        sts64(smem_u32(sm + S::COLS) + ((j % kCaMeta) * kCaTile + 32 * cw + lane) * 8, kf, vf);
      }
      if (lane == 0) {
        if (is_k) {
          const uint32_t m = smem_u32(&meta[j % kCaMeta].half[cw >> 1]) + (cw & 1) * 4;
          sts32(m, ref);
          sts32(m + 8, v_apart || k_apart ? 0x7FC00000u : __float_as_uint(lv));
          sts32(m + 16, __float_as_uint(inverse(vb)));
          sts32(m + 24, valid);
        } else if (partial) {
          meta[j % kCaMeta].nan[cw] = nan;
        }
      }
      const uint32_t stage = ring + (j % kCaStages) * S::kOperand;
      #pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const uint32_t f = __shfl_sync(0xffffffffu, split2, i * RP + row_in);
        const uint32_t hi2 = __byte_perm(f, f, 0x1010), lo2 = __byte_perm(f, f, 0x3232);
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
        uint32_t h[8];
        #pragma unroll
        for (int e = 0; e < 8; e += 2) {
          uint32_t a, b;
          e4m3_f16x4(w[e >> 1], a, b);
          h[e] = fma_f16x2(a, hi2, mul_f16x2(a, lo2));
          h[e + 1] = fma_f16x2(b, hi2, mul_f16x2(b, lo2));
        }
        store(stage, i, h);
        r[i] = load_step(next0, i);
      }
      publish(full, j);
      slot = next;
      ksc = next_ksc;
      vsc = next_vsc;
    }
    if (!ok && lane == 0) atomicOr(p.status, kStatusTimeoutChunk);
  } else if (stream == 4) {
    // ------------------------------------------------------------ MMA issuers
    // A warp a stream, so that a stream's products wait for its own softmax alone.
    regs_down<kCaRegsIssuer>();
    tmem_base = all_set();
    if (warp < 18 && elect_one()) {
      constexpr uint32_t idesc_qk = idesc_f16(kCaTile / 2, false);
      constexpr uint32_t idesc_pv = idesc_f16(D, true);
      const int s = warp - 16;
      const int count = two ? (s == 0 ? k.tiles0 : k.tiles) : (k.tiles + 1 - s) >> 1;
      auto wait_full = [&](uint64_t *bar, int j) {
        return bar_wait(&bar[j % kCaStages], (uint32_t)(j / kCaStages) & 1u);
      };
      const uint32_t q_desc = desc_k_major(smem_u32(sm + S::Q)) + (two ? s : 0) * (S::kOperand >> 4);
      const uint32_t k_desc = desc_k_major(smem_u32(sm + S::K)), v_desc = desc_mn_major(smem_u32(sm + S::V));
      const uint32_t ts = tmem_base + s * 128, to = tmem_base + 256 + s * D;
      // S of half h of tile j: behind the half's product before it, whose P'
      // it overwrites (products of one thread run in order)
      auto qk = [&](int j, int h) {
        const uint32_t b = k_desc + (j % kCaStages) * (S::kOperand >> 4) + h * (64 * 128 >> 4);
        mma_f16_ss<false>(ts + h * 64, q_desc, b, idesc_qk);
        #pragma unroll
        for (int kk = 1; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * (kCaRows * 128) + (kk & 3) * 32) >> 4;
          mma_f16_ss<true>(ts + h * 64, q_desc + off, b + off, idesc_qk);
        }
        mma_commit(&s_full[2 * s + h]);
        if (h == 1) mma_commit(&k_empty[j % kCaStages]);
      };
      // O += P' V' of half h of tile j
      auto pv = [&](int j, int h, bool first) {
        const uint32_t b = v_desc + (j % kCaStages) * (S::kOperand >> 4) + h * (64 * 128 >> 4);
        #pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_ts(to, ts + h * 64 + kk * 8, b + kk * (16 * 128 >> 4), idesc_pv, kk > 0 || !first ? 1u : 0u);
        mma_commit(&o_done[2 * s + h]);
        if (h == 1) mma_commit(&v_empty[j % kCaStages]);
      };
      auto tile = [&](int it) { return two ? it : 2 * it + s; };
      bool ok = bar_wait(q_full, 0);
      if (ok && count > 0) {
        ok = wait_full(k_full, tile(0));
        tc_fence_after();
        if (ok) {
          qk(tile(0), 0);
          qk(tile(0), 1);
        }
      }
      for (int it = 0; it < count && ok; ++it) {
        const int j = tile(it), next = it + 1 < count ? tile(it + 1) : -1;
        ok = wait_full(v_full, j);
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
          ok = ok && bar_wait(&p_full[2 * s + h], (uint32_t)it & 1u);
          if (!ok) break;
          tc_fence_after();
          pv(j, h, it + h == 0);
          if (next >= 0) {
            ok = h == 1 || wait_full(k_full, next);
            if (!ok) break;
            tc_fence_after();
            qk(next, h);
          }
        }
      }
      // tiles that only the other stream needs: this one's share of freeing them
      for (int j = count; two && j < k.tiles && ok; ++j) {
        ok = wait_full(k_full, j);
        if (ok) mbar_arrive(&k_empty[j % kCaStages]);
        ok = ok && wait_full(v_full, j);
        if (ok) mbar_arrive(&v_empty[j % kCaStages]);
      }
      if (!ok) atomicOr(p.status, kStatusTimeoutChunk);
      // every product issued has completed before the CTA ends
      mma_commit(&drain[s]);
      bar_wait(&drain[s], 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    regs_up<kCaRegsSoftmax>();
    // A row's q, its output and its partial results are whole lines of memory:
    // the warp moves them a row or more at a time, D / 8 lanes of 16 bytes a
    // row, through its rows' place in shared memory.  What runs once a CTA is
    // kept small, in loops: it comes from beyond the instruction cache.
    constexpr int CH = D / 8, RPI = 32 / CH;
    const int in_row = lane % CH;
    const uint32_t qs = smem_u32(sm + S::Q) + stream * S::kOperand;
    {
      const int64_t from = has_row ? (int64_t)(k.first_q + tok) * p.ldq + (int64_t)(kvh * p.G + head) * D : -1;
      #pragma unroll 2
      for (int i = 0; i < 32; i += RPI) {
        const int64_t at = __shfl_sync(0xffffffffu, from, i + lane / CH);
        copy16_or_zero(qs + piece_off((warp & 3) * 32 + i + lane / CH, in_row), p.q + max(at, (int64_t)0) + in_row * 8, at >= 0);
      }
    }
    tmem_base = all_set();
    copies_done();
    __syncwarp();
    // q as f16 (a power-of-two scale a row brings its largest value to [1, 2):
    // exact, but for values 2^-24 of the largest and below), in place
    constexpr int kAtOnce = 4;
    uint32_t tops = 0;   // the largest magnitudes of the row's even and odd values, as bits
    uint4 qv[kAtOnce];
    auto take_q = [&](int c) {
      #pragma unroll
      for (int i = 0; i < kAtOnce; ++i) qv[i] = lds128(qs + piece_off(lrow, c + i));
    };
    #pragma unroll 1
    for (int c = 0; c < CH; c += kAtOnce) {
      take_q(c);
      #pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
        #pragma unroll
        for (int e = 0; e < 4; ++e) tops = __vmaxu2(tops, w[e] & 0x7FFF7FFFu);
      }
    }
    // 2^e, e the exponent of the largest magnitude, kept where 2^-e is a normal number too
    const uint32_t ex = min(max(max(tops >> 16, tops & 0xFFFFu) >> 7, 1u), 253u);
    const float up = __uint_as_float((254u - ex) << 23);
    const uint64_t up2 = pack_f32x2(up, up);
    #pragma unroll 1
    for (int c = 0; c < CH; c += kAtOnce) {
      take_q(c);
      #pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
        uint32_t h[4];
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack_f32x2(mul_f32x2(
              pack_f32x2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u)), up2));
          h[e] = f16_pair(f.x, f.y);
        }
        sts128(qs + piece_off(lrow, c + i), h[0], h[1], h[2], h[3]);
      }
    }
    fence_async_shared();
    if (two || stream == 0) mbar_arrive(q_full);
    const float rowfac = __uint_as_float(ex << 23) * p.scale_log2;
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem_base + lane_addr + stream * 128;        // S, then P'
    const uint32_t to = tmem_base + lane_addr + 256 + stream * D;    // O
    const int count = two ? (stream == 0 ? k.tiles0 : k.tiles) : (k.tiles + 1 - stream) >> 1;
    // positions that this row sees; rows of no token see all (nothing to mask), and are not written
    const int sees = has_row ? k.m - k.n + tok + 1 : 0x7FFFFFFF;
    float r = -INFINITY, l = 0.0f;
    bool ok = true;
    const int units = 2 * count;   // of 64 positions, two a tile
    auto tile = [&](int u) { return two ? u >> 1 : (u & ~1) + stream; };
    auto wait_scores = [&](int u) {
      return __all_sync(0xffffffffu, bar_wait(&s_full[2 * stream + (u & 1)], (uint32_t)(u >> 1) & 1u));
    };
    uint32_t x[2][32], y[2][16];
    uint4 m0, m1;
    float cf[2], lv[2], over[2], sum[2];
    uint32_t valid[2];
    // a unit's scores and what belongs to them, on their way
    auto start = [&](int u) {
      const uint32_t m = smem_u32(&meta[tile(u) % kCaMeta].half[u & 1]);
      tmem_ld_32x32b_x32(ts + 64 * (u & 1), x[0]);
      tmem_ld_32x32b_x32(ts + 64 * (u & 1) + 32, x[1]);
      m0 = lds128(m);
      m1 = lds128(m + 16);
    };
    // and here
    auto arrive = [&]() {
      // t = S * cf: cf at least the smallest normal number, so that a masked -inf stays one
      cf[0] = fmaxf(__uint_as_float(m0.x) * rowfac, 0x1p-126f);
      cf[1] = fmaxf(__uint_as_float(m0.y) * rowfac, 0x1p-126f);
      lv[0] = __uint_as_float(m0.z);
      lv[1] = __uint_as_float(m0.w);
      over[0] = __uint_as_float(m1.x);
      over[1] = __uint_as_float(m1.y);
      valid[0] = m1.z;
      valid[1] = m1.w;
      tmem_wait_ld();
      arrived32(x[0]);
      arrived32(x[1]);
    };
    // its weights with the reference as it is, and their sums by 32 positions
    auto weights = [&]() {
      const float rs = r == -INFINITY ? 0.0f : r;
      #pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float bias = lv[c] - rs;
        const uint64_t cf2 = pack_f32x2(cf[c], cf[c]), b2 = pack_f32x2(bias, bias);
        uint64_t sum0 = 0, sum1 = 0;
        // pair i's exponentials, then what pair i - 3 is for: written down in
        // this order, since a warp issues in order and waits for each result
        constexpr int kLag = 3;
        float2 w[16];
        #pragma unroll
        for (int i = 0; i < 16 + kLag; ++i) {
          if (i < 16) {
            w[i] = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])), cf2, b2));
            ex2_in_order(w[i].x);
            ex2_in_order(w[i].y);
          }
          if (i >= kLag) {
            const float2 v = w[i - kLag];
            y[c][i - kLag] = f16_pair_in_order(v.x, v.y);
            add_f32x2_in_order(i & 1 ? sum1 : sum0, pack_f32x2(v.x, v.y));
          }
        }
        const float2 both = unpack_f32x2(add_f32x2(sum0, sum1));
        sum[c] = both.x + both.y;
      }
    };
    auto give = [&](int u) {
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[2 * stream + (u & 1)]);
    };
    auto hand_over = [&](int u) {
      tmem_st_32x32b_x16(ts + 64 * (u & 1), y[0]);
      tmem_st_32x32b_x16(ts + 64 * (u & 1) + 16, y[1]);
      give(u);
    };
    // Where the row's reference moves to `high`: l follows here, the factor for
    // O is returned.
    auto factor = [&](bool move, float high) -> float {
      const float by = move && r != -INFINITY ? r - high : 0.0f;
      if (move) r = high;
      l = times_2to(l, by);
      return ex2(by);
    };
    // Whether a position of a unit has factors of its own, and such a unit as a
    // whole: seldom, so few scores at a time in little code.
    auto is_apart = [&](int u) -> bool {
      const uint4 m = lds128(smem_u32(&meta[tile(u) % kCaMeta].half[u & 1]));
      return !(__uint_as_float(m.z) + __uint_as_float(m.w) < INFINITY);
    };
    auto apart_unit = [&](int u) -> bool {
      constexpr int kFew = 8;
      const uint4 m = lds128(smem_u32(&meta[tile(u) % kCaMeta].half[u & 1]) + 16);
      const uint32_t own = smem_u32(sm + S::COLS) + ((tile(u) % kCaMeta) * kCaTile + 64 * (u & 1)) * 8;
      const int before = sees - ((k.t0 + tile(u)) * kCaTile + 64 * (u & 1));
      // f(i, score less `from`, log2 of the value's scale) of a few positions
      auto few = [&](int at, float from, auto f) {
        uint32_t sc[kFew];
        tmem_ld_32x32b_x8(ts + 64 * (u & 1) + at, sc);
        tmem_wait_ld();
        const uint32_t there = (at & 32 ? m.w : m.z) >> (at & 31);
        #pragma unroll
        for (int i = 0; i < kFew; ++i) {
          const float2 f_own = lds64(own + (at + i) * 8);
          const float t = fmaf(__uint_as_float(sc[i]), f_own.x * rowfac, -from);
          f(i, ((there >> i) & 1u) != 0 && at + i < before ? t : -INFINITY, f_own.y);
        }
      };
      float high = -INFINITY;
      #pragma unroll 1
      for (int at = 0; at < 64; at += kFew)
        few(at, 0.0f, [&](int, float t, float v) { high = fmaxf(high, t + fmaxf(v, kCaNoValue)); });
      const bool move = high > r + kCaLazy;
      if (__any_sync(0xffffffffu, move)) {
        const float f = factor(move, high);
        if (u > 0) {
          if (!__all_sync(0xffffffffu, bar_wait(&o_done[2 * stream + ((u - 1) & 1)], (uint32_t)((u - 1) >> 1) & 1u)))
            return false;
          tc_fence_after();
          #pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(to + c, o);
            tmem_wait_ld();
            #pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st_32x32b_x16(to + c, o);
          }
        }
      }
      const float rs = r == -INFINITY ? 0.0f : r;
      #pragma unroll 1
      for (int at = 0; at < 64; at += kFew) {
        float w[kFew];
        few(at, rs, [&](int i, float t, float v) {
          l += ex2(t);
          w[i] = ex2(t + v);
        });
        uint32_t half[kFew / 2];
        #pragma unroll
        for (int i = 0; i < kFew; i += 2) half[i / 2] = f16_pair(w[i], w[i + 1]);
        // over scores that have been taken: half as many columns
        tmem_st_32x32b_x4(ts + 64 * (u & 1) + at / 2, half);
      }
      give(u);
      return true;
    };
    if (!__any_sync(0xffffffffu, has_row)) {
      // none of the warp's rows is a token's: their weights are never used
      for (int u = 0; u < units && ok; ++u) {
        ok = wait_scores(u);
        if (ok && lane == 0) mbar_arrive(&p_full[2 * stream + (u & 1)]);
      }
    } else {
      // units whose positions every row of the warp sees, by their place
      const int plain = min(units, __reduce_min_sync(0xffffffffu, two ? (sees - k.t0 * kCaTile) >> 6
                                                                      : plain_units(sees - k.t0 * kCaTile, stream)));
      int u = 0;
      #pragma unroll 1
      while (u < units && ok) {
        // A unit that may need anything: a mask, a first reference or another one.
        ok = wait_scores(u);
        if (!ok) break;
        tc_fence_after();
        if (is_apart(u)) {
          ok = apart_unit(u);
          if (!ok) break;
          ++u;
          continue;
        }
        start(u);
        arrive();
        const int before = sees - ((k.t0 + tile(u)) * kCaTile + 64 * (u & 1));   // positions of it that the row sees
        float high = -INFINITY;
        #pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int n = before - 32 * c;
          const uint32_t mask = valid[c] & (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u);
          float top = -INFINITY;
          #pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[c][i] = (mask >> i) & 1u ? x[c][i] : 0xFF800000u;
            top = fmaxf(top, __uint_as_float(x[c][i]));
          }
          high = fmaxf(high, fmaf(top, cf[c], lv[c]));
        }
        const bool move = high > r + kCaLazy;
        if (__any_sync(0xffffffffu, move)) {
          const float f = factor(move, high);
          if (u > 0) {
            // O follows, once the product of the unit before is done
            ok = __all_sync(0xffffffffu, bar_wait(&o_done[2 * stream + ((u - 1) & 1)], (uint32_t)((u - 1) >> 1) & 1u));
            if (!ok) break;
            tc_fence_after();
            #pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              tmem_ld_32x32b_x16(to + 32 * c, y[0]);
              tmem_ld_32x32b_x16(to + 32 * c + 16, y[1]);
              tmem_wait_ld();
              #pragma unroll
              for (int i = 0; i < 16; ++i) {
                y[0][i] = __float_as_uint(__uint_as_float(y[0][i]) * f);
                y[1][i] = __float_as_uint(__uint_as_float(y[1][i]) * f);
              }
              tmem_st_32x32b_x16(to + 32 * c, y[0]);
              tmem_st_32x32b_x16(to + 32 * c + 16, y[1]);
            }
          }
        }
        weights();
        l = fmaf(sum[0], over[0], fmaf(sum[1], over[1], l));
        hand_over(u);
        ++u;
        // Units that need nothing, in a loop of their own: little code without
        // jumps.  Whether a unit was one shows when its weights are there; one
        // that was not (a row without a reference, weights too large for the
        // reference or NaN, a position that is not in the cache) goes back.
        // The next unit's scores are mostly there by then: their barrier is
        // tested (150 cycles) behind the exponentials, and they are fetched
        // while P' is stored.
        if (u >= plain) continue;
        ok = wait_scores(u);
        if (!ok) break;
        tc_fence_after();
        start(u);
        #pragma unroll 1
        while (true) {
          arrive();
          weights();
          const bool more = u + 1 < plain;
          const bool there = !more || bar_test(&s_full[2 * stream + ((u + 1) & 1)], (uint32_t)((u + 1) >> 1) & 1u);
          const bool odd = r == -INFINITY || !(sum[0] + sum[1] < kCaMost) || (valid[0] & valid[1]) != 0xffffffffu;
          if (__any_sync(0xffffffffu, odd || !there)) {
            if (__any_sync(0xffffffffu, odd)) break;
            ok = wait_scores(u + 1);
            if (!ok) break;
          }
          l = fmaf(sum[0], over[0], fmaf(sum[1], over[1], l));
          hand_over(u);
          ++u;
          if (!more) break;
          tc_fence_after();
          start(u);
        }
      }
    }
    // the last product is that of the last tile's second half
    if (ok && count > 0) ok = bar_wait(&o_done[2 * stream + 1], (uint32_t)(count - 1) & 1u);
    // stream 1 hands its O over in the K ring: the other stream's products have
    // to be done too (drain has one phase; o_done may be phases behind)
    if (ok && !two && stream == 1 && count > 0) ok = bar_wait(&drain[0], 0);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) atomicOr(p.status, kStatusTimeoutChunk);
    tc_fence_after();
    if (!ok) l = __uint_as_float(0x7FC00000u);   // a wait ran out: NaN, not a part of the sum
    float f0 = l == 0.0f ? 0.0f : 1.0f;   // factor of this stream's O
    float f1 = 0.0f;                      // factor of the other stream's, when the two are joined
    float *joined = reinterpret_cast<float *>(sm + S::K);   // [D][128], in the K ring
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
          l = l == 0.0f ? times_2to(o.y, o.x - rn) : fminf(r, o.x) - rn > kCaNear
              ? l * f0 + o.y * f1 : times_2to(l, r - rn) + times_2to(o.y, o.x - rn);
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
        if ((tm.nan[0] | tm.nan[1] | tm.nan[2] | tm.nan[3]) == 0) continue;
        #pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int n = sees - ((k.t0 + j) * kCaTile + 32 * c);
          const uint32_t causal = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
          if (tm.nan[c] & tm.half[c >> 1].valid[c & 1] & causal) l = __uint_as_float(0x7FC00000u);
        }
      }
      // the row's place again: not kept in registers through the units
      uint32_t tid;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
      const int again = (two && stream == 1 ? kCaRows : 0) + (int)(tid & 127), R = k.row0 + again;
      const bool has_row = again < k.rows;
      const int tok = R / p.G, head = R - tok * p.G;
      const int64_t oh = (int64_t)(k.first_q + tok) * p.Hq + kvh * p.G + head;
      const int64_t part = oh * p.splits + split;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      if (has_row && p.splits > 1) {
        p.part_ml[part * 2] = l == 0.0f ? -INFINITY : r;
        p.part_ml[part * 2 + 1] = l;
      }
      // Through this warp's part of the q area, whose products are done: 32
      // rows of D * 2 bytes, the outputs or half of the partial sums.
      const uint32_t area = qs + (warp & 3) * (32 * D * 2);
      auto place = [&](int row, int c) { return area + row * (D * 2) + ((c ^ (row & (CH - 1))) << 4); };
      const int64_t row_at = !has_row ? -1 : p.splits > 1 ? part * (D * 4) : oh * (D * 2);
      uint8_t *base = p.splits > 1 ? reinterpret_cast<uint8_t *>(p.part_acc) : reinterpret_cast<uint8_t *>(p.out);
      const float f = p.splits > 1 ? f0 : f0 * inv, fj = p.splits > 1 ? f1 : f1 * inv;
      const uint64_t ff = pack_f32x2(f, f);
      #pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld_32x32b_x32(to + 32 * c, v);   // stale where no product was issued: f0 is 0 there
        tmem_wait_ld();
        arrived32(v);
        #pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 w = unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), ff));
          v[i] = __float_as_uint(w.x);
          v[i + 1] = __float_as_uint(w.y);
        }
        if (f0 == 0.0f) {
          #pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        if (f1 != 0.0f) {
          #pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = __float_as_uint(fmaf(joined[(32 * c + i) * kCaRows + lrow], fj, __uint_as_float(v[i])));
        }
        const bool halved = p.splits > 1;
        if (halved) {
          #pragma unroll
          for (int i = 0; i < 8; ++i)
            sts128(place(lane, (8 * c + i) & (CH - 1)), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
          #pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = bf16_pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
          #pragma unroll
          for (int i = 0; i < 4; ++i)
            sts128(place(lane, 4 * c + i), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        if (c != D / 32 - 1 && !(halved && c == D / 64 - 1)) continue;
        // the area is full: its rows, each to a place of its own
        __syncwarp();
        uint8_t *to_half = base + (halved && c == D / 32 - 1 ? D * 2 : 0) + in_row * 16;
        #pragma unroll 4
        for (int i = 0; i < 32; i += RPI) {
          const int64_t at = __shfl_sync(0xffffffffu, row_at, i + lane / CH);
          const uint4 w = lds128(place(i + lane / CH, in_row));
          if (at >= 0) *reinterpret_cast<uint4 *>(to_half + at) = w;
        }
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
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
    l = ml[2 * s] - top > kCaNear ? fmaf(ml[2 * s + 1], w, l) : l + times_2to(ml[2 * s + 1], ml[2 * s] - top);
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
// start and end worth kFixed tiles, and the parts of the last wave leave SMs
// idle: the split with the least (waves x cost) is taken, where a split also
// pays for the second kernel and its partial results (kRowsATile rows a part
// take it about a tile's time).  The launch has room for the most row tiles that
// the bounds allow; the waves are counted for the middle between those and the
// fewest, which would put a sequence of one row tile more into a second wave (72
// -> 92 us).  Over 26 shapes, called one behind the other (geometric means): 52.1
// us, never split 71.1, each shape's best split 49.4; the farthest from its best
// is three sequences of 43 to 248 tokens on 10,133 to 15,681 positions, 24 + 3
// heads: 108.4 us in 3 parts, 86.9 in 4, since every part is priced by
// max_context and by tiles that a shorter sequence does not have.
ChunkPlan plan_chunk(int64_t total_q, int64_t B, int Hkv, int G, int64_t max_q, int64_t max_context) {
  constexpr int64_t kFixed = 3, kRowsATile = 12000;
  ChunkPlan c;
  c.row_tiles = std::min(total_q * G / (2 * kCaRows) + B, B * ((max_q * G + 2 * kCaRows - 1) / (2 * kCaRows)));
  const int64_t tiles = std::max<int64_t>(1, (max_context + kCaTile - 1) / kCaTile);
  const int64_t sms = num_sms(), rows = total_q * G * Hkv;
  const int64_t fewest = std::max(B, (total_q * G + 2 * kCaRows - 1) / (2 * kCaRows));
  const int64_t ctas = std::max<int64_t>(1, (std::min(fewest, c.row_tiles) + c.row_tiles) / 2) * Hkv;
  int64_t best = -1;
  c.splits = 1;
  c.split_tiles = (int)tiles;
  for (int64_t s = 1; s <= kCaMaxSplits; ++s) {
    const int64_t each = (tiles + s - 1) / s;
    if (s > 1 && (each < 2 || ctas * s > 8 * sms)) break;
    const int64_t parts = (tiles + each - 1) / each;
    if (parts != s) continue;
    const int64_t cost = (ctas * s + sms - 1) / sms * (each + kFixed) + (s > 1 ? kFixed + rows * s / kRowsATile : 0);
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
  p.num_blocks = (uint32_t)(a.num_slots / a.block_size);
  p.tile_blocks = kCaTile / a.block_size;
  p.tile_rest = kCaTile % a.block_size;
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
