// attn_decode_kernel.cuh -- attention of few query rows over long keys, for B200 (sm_100a): single
// (or a few drafted) tokens over a paged key/value cache, the same behind a shared prefix, and few
// rows of cross attention over contiguous keys.
//
//   S_ij = scale q_i . k_j,   O_i = sum_j softmax(S_i)_j v_j,   LSE_i = ln sum_j exp(S_ij)
//
// A "sequence" is one set of keys; the rows that see it are the R = group * T query rows of a KV
// head (T tokens of the `group` query heads sharing it) or, for a shared prefix, those of the whole
// batch.  Every key and value is used by R rows only, R * 2 operations a byte (bf16) or R * 4
// (E4M3): the kernel is bound by HBM, and is built to keep loads in flight and to touch each byte
// once:
//
//  * Keys and values reach shared memory by TMA (128-byte swizzled rows) through rings of 8 KB
//    stages, eight stages a CTA and three CTAs an SM: about 100 KB in flight while as much is
//    computed on.  (Loads straight into registers, a first version, held 340 us for the 550 MB of
//    B64 Hq32 Hkv8 N<=8192 D128 E4M3, the warps waiting for memory 70 % of the time.)
//  * The products are transposed, S^T = K Q^T and O^T = V^T P^T, so that the rows are the N = 8 index of
//    the tensor-core instruction (m16n8k16): few rows are few columns, and none of the work is for
//    rows that are not there (with rows as M = 16, half of it was at the usual 8 rows or fewer).  P
//    goes from the first product's layout to the second's by a register transposition of each 8 x 8.
//  * A lane reads its operands as they lie: the K = 16 index of K Q^T may be any permutation of D as
//    long as Q uses the same one, so a lane takes 16 contiguous bytes of its key's row for several K
//    steps (pieces 2t, 2t+1 of a swizzled row: no bank conflicts); likewise the M = 16 index of V^T P^T
//    is any permutation of the output columns, so a lane takes 16 bytes of the four value rows that it
//    holds as K index, and pairs two rows with one byte permutation per operand register.
//  * E4M3 codes are converted two at a time to f16, exactly (moving the bits to bf16 by integer
//    instructions took twice the arithmetic pipe's time, which then bounded the kernel).  The f16
//    operands on the other side keep the products exact enough:
//      Q    each row is multiplied by the power of two that brings its largest magnitude to 2^13, so
//           that a bf16 number keeps all its bits down to 2^-27 of the row's largest, and loses at
//           most 2^-38 of that below; the power is taken back from the scores in fp32.
//      P    a token's V exponent multiplies its probability: P' = p 2^13 2^(ev - E) with E the
//           largest exponent that the warp has met, 11 bits down to 2^-27 of the largest (2^-17 at
//           ev = E - 10).  When E grows, O is scaled by a power of two; tokens more than 10 below E
//           get passes of their own.
//  * The running maximum moves only when some row of the warp grew by more than 8 (E4M3: 2), so the
//    usual step needs one vote and no shuffle, and O is rarely rescaled.
//
// Schedule.  The work is counted in blocks of 64 keys of one (sequence, KV head, row block) unit,
// and two more for each unit, all in one line.  Each of the grid's CTAs takes an equal, contiguous range of that line,
// found from the lengths on the device, so uneven batches stay balanced and a captured launch serves
// any lengths.  A range covers whole units (written out directly) and at most two partial ones
// (written as unnormalised O, maximum and sum in fp32 to the CTA's two slots of the workspace); a
// second kernel joins the parts of each split unit in key order.  No atomics, no state in the
// workspace: results depend on the inputs alone.
//
// kWarp: many short sequences (one row tile).  Each warp takes whole units of its own, with its own
// ring; nothing is joined between warps, and a shared prefix's result (computed by the many-row
// kernel) is joined in registers as the unit is written.  Sharing such units among a CTA's warps took
// three times as long (B128 Hkv8 N<=256 behind a prefix: 37 us), most of it between units.
//
// Measured (B200; one call after another, and in brackets with L2 flushed before each): B64 Hq32 Hkv8
// N<=8192 D128 E4M3 (550 MB) 104 us (116), 5.3 TB/s; B3 T4 N<=100001 bf16 (820 MB) 145 us (159), 5.7 TB/s:
// 0.8 and 0.87 of a copy's rate.  What is left is the steps' own latency (conversion, products and
// exponentials in turn, three warps a scheduler) and the ends of the units; short calls are launches, the
// look-up of the schedule and one step's latency after another (B1 N500: 15 us a call, 12 on the GPU).
//
// Registers: 168, for three CTAs an SM.  At that, ptxas spills (bytes stored / loaded): 16 rows at D = 128 12 / 12
// (bf16) and 360 / 248 (E4M3), at D = 96 24 / 36 and 108 / 116, at D = 64 E4M3 40 / 88; 8 rows of E4M3 60 / 124 at
// D = 128, 20 / 40 at D = 96; the others nothing.
//
// A CTA's four warps take `row_tiles` tiles of 16 rows (1, 2 or 4; or one of 8) and share the keys 4 / row_tiles
// ways; the warps of one way share its ring (a stage is refilled once all of them have left it).
// Their results are joined in shared memory, in the ring's place.  Every wait is bounded.
#pragma once

#include <cuda_bf16.h>

#include "attn_cache_kernel.cuh"

namespace attn {

constexpr int kDecThreads = 128;
constexpr int kDecBlock = 64;       // keys per block of the schedule
// Stages of all the CTA's rings together: eight, with three CTAs an SM; the warp form, which has fewer
// warps with work, twelve and two CTAs.
__host__ __device__ constexpr int dec_stages(bool warps) { return warps ? 12 : 8; }
constexpr int kDecStageBytes = 8192;

enum : unsigned {
  kSiteDecodeFull = 51,
  kSiteDecodeEmpty = 52,
};

struct DecParams {
  const __nv_bfloat16* q;    // [B][Hkv][GT][D]
  const uint8_t* ks;         // E4M3: exponents [num_pages][Hkv][page]
  const uint8_t* vs;
  const __nv_bfloat16* v;    // bf16: the values once more, for those that are not finite
  const int* table;          // [B][max_pages], or null: sequence b is page b
  const int* lens;           // [B], or null: len_all
  long long cap;             // max_pages * page: no sequence is longer
  int len_all, max_pages, num_pages, page, Hkv, B;
  FastDiv div_page;
  int GT, T;                 // rows of a sequence and KV head; tokens (row i is token i % T)
  int causal;                // token t sees keys up to len - T + t
  FastDiv div_gt;
  int row_tiles, unit_rows;             // of a CTA: tiles of rows, and their rows together
  int row_blocks;                       // of a sequence
  int box;                              // key rows of a TMA box: the step, or 16
  // shared prefix handled here (prefix_len > 0): an extra first sequence with all rows of the batch
  const int* prefix_table;
  int prefix_len, prefix_row_blocks;
  int whole_units;           // 1: units are not split (each stands in the line as one block)
  int min_share;             // places a CTA takes at least
  float c;                   // scale * log2(e)
  __nv_bfloat16* o;          // [B][Hkv][GT][D]
  float* lse;                // [B][Hkv][GT]
  // workspace
  float* slot_o;             // [2 * grid][unit_rows][D]
  float2* slot_ml;           // [2 * grid][unit_rows]
  // shared prefix: whole units go here instead of o, lse, indexed like o: [0] own keys, [1] prefix
  float* area_o[2];
  float2* area_ml[2];
  // the prefix's results from the many-row kernel (tiles > 0): slots of 128 rows, two a CTA for parts of
  // units and then a unit's own; a unit is a tile of a head, of `places` places in that kernel's line, the
  // first `over` of them without blocks
  struct {
    const float* o;
    const float2* ml;
    int tiles, seqs, seq_tiles, places, over;
    long long share, ctas;
  } many;
};

__device__ __forceinline__ int dec_len(const DecParams& p, int b) {
  const long long n = p.lens != nullptr ? (long long)p.lens[b] : (long long)p.len_all;
  return (int)max(0LL, min(n, p.cap));
}

// (Lengths go up to 2^31 - 1: sums with one that may pass it are in 64 bits or unsigned.)
__device__ __forceinline__ int dec_key_blocks(int len) { return (int)(((long long)len + kDecBlock - 1) / kDecBlock); }
__device__ __forceinline__ int dec_blocks(const DecParams& p, int len) {
  return p.whole_units ? 1 : max(1, dec_key_blocks(len));
}

// Weight of a result with running maximum ml.x and sum ml.y against maximum m (none: 0; NaN stays).
__device__ __forceinline__ float dec_weight(float2 ml, float m) {
  return ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2_approx(ml.x - m);
}

// LSE of a row from its maximum (base 2) and sum.
__device__ __forceinline__ float dec_lse(float m, float l) {
  return l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * 0.69314718055994530942f;
}

// The many-row kernel's results for row i of sequence b and head h: n of them, rows `at(k)` of
// p.many.o and p.many.ml.
struct DecParts {
  int n;
  long long f, first_slot, row, whole;
  __device__ __forceinline__ long long at(int k) const {
    return (whole >= 0 ? whole : k == 0 ? first_slot : 2 * (f + k)) * 128 + row;
  }
};
__device__ __forceinline__ DecParts dec_prefix_parts(const DecParams& p, int b, int h, int i) {
  DecParts r;
  const int tile = p.many.seq_tiles > 1 ? b * p.many.seq_tiles + i / 128 : b / p.many.seqs;
  r.row = p.many.seq_tiles > 1 ? i % 128 : b % p.many.seqs * p.GT + i;
  const long long unit = (long long)h * p.many.tiles + tile, u0 = unit * p.many.places;
  r.f = (u0 + p.many.over) / p.many.share;
  const long long e = (u0 + p.many.places - 1) / p.many.share;
  r.n = (int)(e - r.f) + 1;
  r.whole = r.n == 1 ? 2 * p.many.ctas + unit : -1;
  r.first_slot = 2 * r.f + (u0 > r.f * p.many.share ? 1 : 0);
  return r;
}

// The line of work: the prefix's units first, then sequence by sequence; within a sequence KV head by
// KV head, row block by row block.  A unit takes kDecOver places for its start and end (about 4 us of
// a CTA, a block 1.3 us at full load), then one for each of its blocks.
constexpr int kDecOver = 2;
__device__ __forceinline__ int dec_places(int blocks) { return blocks + kDecOver; }
// Blocks of a unit before place `p` of it.
__device__ __forceinline__ int dec_block_at(int p) { return p > kDecOver ? p - kDecOver : 0; }

struct DecLine {
  long long prefix;   // places of the prefix's units together
  long long total;
  long long share;    // places of a CTA
};

// Whole block (kDecThreads threads): the line's length, and the sequence that holds position `x`
// of it (seq, and the line position of its first block) -- or, with find_seq >= 0, the position of
// that sequence.  `sh` is shared scratch of 16 long longs.
__device__ __forceinline__ DecLine dec_locate(const DecParams& p, unsigned ctas, long long cta, int find_seq,
                                              long long* sh, int& seq, long long& first) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long per_seq = (long long)p.Hkv * p.row_blocks;
  const int per = (p.B + kDecThreads - 1) / kDecThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += dec_places(dec_blocks(p, dec_len(p, b)));
  mine *= per_seq;
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  DecLine ln;
  ln.prefix = p.prefix_len > 0 ? (long long)p.Hkv * p.prefix_row_blocks * dec_places(dec_key_blocks(p.prefix_len)) : 0;
  long long before = ln.prefix, total = ln.prefix;
#pragma unroll
  for (int w = 0; w < kDecThreads / 32; ++w) {
    if (w < warp) before += sh[w];
    total += sh[w];
  }
  ln.total = total;
  ln.share = max((long long)p.min_share, (total + ctas - 1) / ctas);
  const long long x = cta * ln.share;
  long long at = before + incl - mine;   // line position of this thread's first sequence
  if (find_seq >= 0 ? (find_seq >= b0 && find_seq < b1) : (x >= at && x < at + mine)) {
    int b = b0;
    for (; b < b1; ++b) {
      const long long n = per_seq * dec_places(dec_blocks(p, dec_len(p, b)));
      if (find_seq >= 0 ? b == find_seq : x < at + n) break;
      at += n;
    }
    sh[8] = b;
    sh[9] = at;
  }
  if (tid == 0 && find_seq < 0 && (x < ln.prefix || x >= total)) {
    sh[8] = x < ln.prefix ? -1 : p.B;
    sh[9] = 0;
  }
  __syncthreads();
  seq = (int)sh[8];
  first = sh[9];
  __syncthreads();
  return ln;
}

// D += A B, m16n8k16, bf16 (f16) operands and fp32 accumulators in registers.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two E4M3 codes (the low or the high half of w) -> an f16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3_lo_to_f16(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi_to_f16(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Two floats -> packed f16x2 (nearest even); `lo` in bits 0-15.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A power of two from its exponent field (0 < e < 255: 2^(e - 127); 255: infinity; 0: 0).
__device__ __forceinline__ float pow2_field(int e) { return __uint_as_float((uint32_t)e << 23); }

template <int D, bool kF8>
struct DecCfg {
  static constexpr int kElem = kF8 ? 1 : 2;
  static constexpr int kChunks = (D * kElem + 127) / 128;   // 128-byte pieces of a row
  static constexpr int kGroups = 2 / kChunks;               // 16-key groups per step
  static constexpr int kStep = 16 * kGroups;
  static constexpr int kChunkBytes = kStep * 128;
  static constexpr int kVOff = kChunks * kChunkBytes;       // V behind K in a stage
  static_assert(2 * kVOff == kDecStageBytes, "a stage holds one step");
  static constexpr float kLazy = kF8 ? 2.f : kRescaleLog2;  // growth of a row's maximum that is let go
  static constexpr float kLift = kF8 ? 13.f : 0.f;          // P is 2^kLift times the probability
  static constexpr int kWindow = 10;                        // V exponents of one pass
  static constexpr int kKWords = D * kElem / 16;            // 32-bit words of a key a lane holds (1/4 of it)
  static constexpr int kVWords = D * kElem / 32;            // of a value row (1/8 of it)
  static constexpr int kRowStride = D + 4;                  // floats, of a row of the join
  static constexpr int kJoinBytes = 4 * 16 * kRowStride * 4;
  static_assert(kJoinBytes <= dec_stages(false) * kDecStageBytes, "the join takes the rings' place");
};
// E4M3: a stage's exponents, K's then V's (32 keys at most), behind all the stages; slack for
// 1024-byte alignment
constexpr int kDecExpBytes = 64;
__host__ __device__ constexpr int dec_smem(bool warps) {
  return dec_stages(warps) * (kDecStageBytes + kDecExpBytes) + 1024;
}

// Byte `b` of row `r` in a tile of 128-byte rows as TMA swizzles it.
__device__ __forceinline__ uint32_t dec_sw(uint32_t r, uint32_t b) { return r * 128 + (b ^ ((r & 7) << 4)); }

// First element of K step s's four in D that lane t holds: 16-byte pieces 2t, 2t+1 of a full
// 128-byte row piece, piece t of half of one, 8-byte pieces where E4M3 rows are neither.
template <int D, bool kF8>
__device__ __forceinline__ constexpr int dec_koff(int s, int t) {
  if (kF8 && D == 128) return 16 * (2 * t + s / 4) + 4 * (s % 4);
  if (kF8 && D == 64) return 16 * t + 4 * s;
  if (kF8) return 32 * (s / 2) + 8 * t + 4 * (s % 2);
  const int i = s / 2, c = i / 2;   // 16-byte pieces of 8 elements, two to a lane and 64-element chunk
  return (64 * c + 64 <= D) ? 64 * c + 8 * (2 * t + i % 2) + 4 * (s % 2) : 64 * c + 8 * t + 4 * (s % 2);
}

// Output column number `ct` (0 <= ct < D/8) of lane group n (0..7): the columns a lane loads
// contiguously.  Two of them are M indices g and g + 8 of one product.
template <int D, bool kF8>
__device__ __forceinline__ constexpr int dec_col(int ct, int n) {
  if (kF8 && D == 128) return 16 * n + ct;
  return ct < 8 * (D / 64) ? 64 * (ct / 8) + 8 * n + ct % 8 : 64 * (D / 64) + 4 * n + (ct - 8 * (D / 64));
}

__device__ __forceinline__ void lds16(uint32_t* w, uint32_t addr) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ void lds8(uint32_t* w, uint32_t addr) {
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}
__device__ __forceinline__ int lds1(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr));
  return (int)r;
}
__device__ __forceinline__ void lds4(uint32_t* w, uint32_t addr) {
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

// Lane t's words of key row r in the K tile at `tile`: word order as dec_koff's steps.
template <int D, bool kF8>
__device__ __forceinline__ void dec_load_k(uint32_t (&w)[DecCfg<D, kF8>::kKWords], uint32_t tile, uint32_t r, uint32_t t) {
  constexpr int kChunkBytes = DecCfg<D, kF8>::kChunkBytes;
  if constexpr (kF8 && D % 64 != 0) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) lds8(w + 2 * i, tile + dec_sw(r, 32 * i + 8 * t));
  } else {
    constexpr int kRowBytes = D * DecCfg<D, kF8>::kElem;
#pragma unroll
    for (int c = 0; c < kRowBytes / 128; ++c) {
      lds16(w + 8 * c, tile + c * kChunkBytes + dec_sw(r, 32 * t));
      lds16(w + 8 * c + 4, tile + c * kChunkBytes + dec_sw(r, 32 * t + 16));
    }
    if constexpr (kRowBytes % 128 != 0)
      lds16(w + 8 * (kRowBytes / 128), tile + (kRowBytes / 128) * kChunkBytes + dec_sw(r, 16 * t));
  }
}

// Lane group g's words of value row r in the V tile at `tile`.
template <int D, bool kF8>
__device__ __forceinline__ void dec_load_v(uint32_t (&w)[DecCfg<D, kF8>::kVWords], uint32_t tile, uint32_t r, uint32_t g) {
  constexpr int kChunkBytes = DecCfg<D, kF8>::kChunkBytes;
  if constexpr (kF8 && D == 128) {
    lds16(w, tile + dec_sw(r, 16 * g));
  } else if constexpr (kF8) {
    if constexpr (D >= 64) lds8(w, tile + dec_sw(r, 8 * g));
    if constexpr (D % 64 != 0) lds4(w + 2 * (D / 64), tile + dec_sw(r, 64 * (D / 64) + 4 * g));
  } else {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) lds16(w + 4 * c, tile + c * kChunkBytes + dec_sw(r, 16 * g));
    if constexpr (D % 64 != 0) lds8(w + 4 * (D / 64), tile + (D / 64) * kChunkBytes + dec_sw(r, 8 * g));
  }
}

// An 8 x 8 matrix of 16-bit values, transposed across the warp: lane (g, t) gives row g, columns 2t and
// 2t + 1, and gets row g of the transpose.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Column ct (of a lane's contiguous ones) of two value rows as a pair, an A operand of V^T P^T: bf16 as
// they are, E4M3 as f16 (the byte permutation serves two columns).
template <bool kF8>
__device__ __forceinline__ uint32_t dec_pair(const uint32_t* r0, const uint32_t* r1, int ct) {
  if constexpr (kF8) {
    const uint32_t x = __byte_perm(r0[ct / 4], r1[ct / 4], (ct & 2) ? 0x7362u : 0x5140u);
    return (ct & 1) ? e4m3_hi_to_f16(x) : e4m3_lo_to_f16(x);
  } else {
    return __byte_perm(r0[ct / 2], r1[ct / 2], (ct & 1) ? 0x7632u : 0x5410u);
  }
}

// kN: tiles of 8 rows a warp takes (1: units of at most 8 rows; else 2).
template <int D, bool kF8, int kN, bool kWarp>
__global__ void __launch_bounds__(kDecThreads, kWarp ? 2 : 3)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const DecParams p) {
  using Cfg = DecCfg<D, kF8>;
  constexpr int G = Cfg::kGroups, KW = Cfg::kKWords, VW = Cfg::kVWords;
  constexpr int kTile = 8 * kN;   // rows of a warp
  constexpr int kDecStages = dec_stages(kWarp);
  extern __shared__ uint8_t smem_raw[];
  __shared__ float2 sml[4][16];
  __shared__ long long scratch[16];
  __shared__ uint64_t full[kDecStages], empty[kDecStages];
  __shared__ uint32_t abort_word;
  __shared__ uint32_t odd_words[4];   // this warp's way met values that are not finite (see the step)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  auto so = reinterpret_cast<float(*)[16][Cfg::kRowStride]>(smem);
  volatile uint32_t* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int row_tiles = p.row_tiles;
  const int kg = warp / row_tiles, rt = warp - kg * row_tiles, ways = 4 / row_tiles;
  const int stages = kDecStages / ways;                 // of this way's ring
  const uint32_t ring = smem_u32(smem) + kg * stages * kDecStageBytes;
  uint8_t* const exps = smem + kDecStages * kDecStageBytes + kg * stages * kDecExpBytes;
  volatile uint32_t* odd = &odd_words[kg];   // (one way: its row tiles' warps share the stages, and this)
  uint64_t* ring_full = full + kg * stages;
  uint64_t* ring_empty = empty + kg * stages;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDecStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], row_tiles);
    }
    *abort_flag = 0u;
    for (int i = 0; i < 4; ++i) odd_words[i] = 0u;
    fence_mbar_init();
    if (p.cap > 0 || p.prefix_len > 0) {   // (without any key there are no tensor maps)
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
    }
  }

  launch_dependents();
  int seq = 0;
  long long first = 0, begin, end;
  if constexpr (kWarp) {
    __syncthreads();
    begin = (long long)blockIdx.x * 4 + warp;
    end = (long long)p.B * p.Hkv;
  } else {
    const DecLine ln = dec_locate(p, gridDim.x, blockIdx.x, -1, scratch, seq, first);   // (its barriers order the above)
    begin = (long long)blockIdx.x * ln.share;
    end = min(ln.total, begin + ln.share);
  }
  // ring positions (stage, parity of its use) of the next issue (the way's first warp) and of the
  // next step, over all units; uses of the ring before its first refill need no wait
  uint32_t i_stage = 0u, i_phase = 0u, i_count = 0u, stage = 0u, phase = 0u;
  const uint64_t policy = l2_policy_evict_first();   // each key and value is read once
  const int no_plane = p.num_pages * p.Hkv;          // outside the tensor maps: zeros
  bool ok = true;

  for (long long x = begin; x < end && ok;) {
    // ---- the unit at line position x, and the part of it in this CTA's range (kWarp: unit x)
    if constexpr (kWarp) seq = (int)(x / p.Hkv);
    const bool prefix = !kWarp && seq < 0;
    const int len = prefix ? p.prefix_len : dec_len(p, seq);
    const int nblk = kWarp ? 1 : prefix ? dec_key_blocks(len) : dec_blocks(p, len);
    const int row_blocks = prefix ? p.prefix_row_blocks : p.row_blocks;
    const int rows = prefix ? p.B * p.GT : p.GT;
    const int places = dec_places(nblk);
    const int unit = kWarp ? 0 : (int)((x - first) / places);
    const int p0 = kWarp ? 0 : (int)((x - first) - (long long)unit * places);
    const int p1 = kWarp ? 1 : (int)min((long long)places, p0 + (end - x));
    const int blk0 = kWarp ? 0 : dec_block_at(p0), blk1 = kWarp ? 1 : dec_block_at(p1);
    // the next unit of the line
    auto move_on = [&](int row_blocks_) {
      x += p1 - p0;
      const long long seq_places = (long long)p.Hkv * row_blocks_ * places;
      if (x >= first + seq_places) {
        first += seq_places;
        ++seq;
      }
    };
    if (!kWarp && blk0 == blk1) {   // only places of its start: the next CTA has the unit
      move_on(row_blocks);
      continue;
    }
    const int h = kWarp ? (int)(x - (long long)seq * p.Hkv) : unit / row_blocks, rb = kWarp ? 0 : unit - h * row_blocks;
    const int* table = prefix ? p.prefix_table : (p.table ? p.table + (size_t)seq * p.max_pages : nullptr);
    const int i0 = (rb * row_tiles + rt) * kTile;   // first row of this warp's tile
    const int key_begin = blk0 * kDecBlock;   // (of a unit that is not split: 0)
    const int key_end = (kWarp || p.whole_units) ? len : (int)min((long long)len, (long long)blk1 * kDecBlock);

    // row i of the unit -> its index in q, o, lse
    auto row_index = [&](int i) -> long long {
      if (!prefix) return ((long long)seq * p.Hkv + h) * p.GT + i;
      const uint32_t b = fast_div((uint32_t)i, p.div_gt);
      return ((long long)b * p.Hkv + h) * p.GT + (i - (int)b * p.GT);
    };
    // this way's steps: keys key_begin + (kg + ways * n) * kStep
    const int stride = kWarp ? Cfg::kStep : ways * Cfg::kStep;
    const int k_first = kWarp ? 0 : key_begin + kg * Cfg::kStep;
    const int steps = (uint32_t)k_first < (uint32_t)key_end
                          ? (int)(((uint32_t)(key_end - k_first) + (uint32_t)stride - 1u) / (uint32_t)stride) : 0;
    // page pg of the unit -> its plane in the tensor maps
    auto plane_of = [&](int pg) -> int {
      const int id = table ? __ldg(table + pg) : seq;
      return (unsigned)id < (unsigned)p.num_pages ? id * p.Hkv + h : no_plane;
    };
    // A position walking along the steps: page and row in it.
    struct Walk {
      int pg, row;
    };
    auto walk_at = [&](int k) -> Walk {
      const int pg = (int)fast_div((uint32_t)k, p.div_page);
      return Walk{pg, k - pg * p.page};
    };
    auto walk_on = [&](Walk& w, int by) {
      for (w.row += by; w.row >= p.page; w.row -= p.page) ++w.pg;
    };
    // The loads of a step: boxes with a key only.  The planes were looked up a step before.
    constexpr int kMaxBoxes = G;
    const int boxes_per_step = Cfg::kStep / p.box;
    Walk iw[kMaxBoxes];
    int iplane[kMaxBoxes];
    auto look_up = [&](int n) {   // planes of step n's boxes (where it has keys), iw standing at that step
#pragma unroll
      for (int i = 0; i < kMaxBoxes; ++i)
        iplane[i] = (i < boxes_per_step && n < steps && k_first + n * stride + i * p.box < key_end) ? plane_of(iw[i].pg) : -1;
    };
    auto issue = [&](int n) -> bool {   // one lane; moves iw and the planes on to step n + 1
      if (i_count >= (uint32_t)stages &&
          !wait_phase(&ring_empty[i_stage], i_phase ^ 1u, abort_flag, kSiteDecodeEmpty))
        return false;
      uint32_t bytes = 0u;
#pragma unroll
      for (int i = 0; i < kMaxBoxes; ++i) {
        if (iplane[i] < 0) continue;
        bytes += (uint32_t)(2 * Cfg::kChunks * p.box * 128);
        if constexpr (kF8) {
          if (iplane[i] != no_plane) {
            bytes += 2u * (uint32_t)p.box;
          } else {   // zero codes: any exponent does, but those of the stage's last use may be NaN
            for (int q = 0; q < p.box; q += 16) {
              uint4* dst = reinterpret_cast<uint4*>(exps + i_stage * kDecExpBytes + i * p.box + q);
              dst[0] = dst[2] = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
            }
            fence_proxy_async_smem();
          }
        }
      }
      mbar_arrive_expect_tx(&ring_full[i_stage], bytes);
#pragma unroll
      for (int i = 0; i < kMaxBoxes; ++i) {
        if (iplane[i] < 0) continue;
        if constexpr (kF8) {
          if (iplane[i] != no_plane) {
            const long long at = (long long)iplane[i] * p.page + iw[i].row;
            uint8_t* dst = exps + i_stage * kDecExpBytes + i * p.box;
            bulk_load_1d(dst, p.ks + at, (uint32_t)p.box, &ring_full[i_stage]);
            bulk_load_1d(dst + 32, p.vs + at, (uint32_t)p.box, &ring_full[i_stage]);
          }
        }
#pragma unroll
        for (int c = 0; c < Cfg::kChunks; ++c) {
          uint8_t* dst = smem + (kg * stages + i_stage) * kDecStageBytes + c * Cfg::kChunkBytes + i * p.box * 128;
          tma_load_3d(dst, &tmap_k, &ring_full[i_stage], c * (128 / Cfg::kElem), iw[i].row, iplane[i], policy);
          tma_load_3d(dst + Cfg::kVOff, &tmap_v, &ring_full[i_stage], c * (128 / Cfg::kElem), iw[i].row, iplane[i],
                      policy);
        }
      }
      ++i_count;
      if (++i_stage == (uint32_t)stages) {
        i_stage = 0u;
        i_phase ^= 1u;
      }
#pragma unroll
      for (int i = 0; i < kMaxBoxes; ++i) walk_on(iw[i], stride);
      look_up(n + 1);
      return true;
    };
    const bool issuer = rt == 0 && lane == 0;
    if (issuer) {
#pragma unroll
      for (int i = 0; i < kMaxBoxes; ++i) iw[i] = walk_at(k_first + i * p.box);
      look_up(0);
      for (int n = 0; n < min(stages - 1, steps) && ok; ++n) ok = issue(n);
    }
    ok = __all_sync(0xffffffffu, ok);

    // O^T: [row tile][pair of columns 2c, 2c+1]: rows 2t, 2t+1 of column 2c, then of 2c+1
    float o[kN][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < kN; ++nt)
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][c][e] = 0.f;
    // per row 8 nt + 2t + e of the tile: running maximum, this lane's part of the sum, the factor of
    // its scores, and the first key that it does not see
    float m[kN][2], l[kN][2], cf[kN][2];
    int lim[kN][2], lim_min = len;
    const bool active = i0 < rows;   // (a tile past the rows only keeps the ring going)

    // Q as the B operand of K Q^T: words 2s, 2s+1 of row 8 nt + g are K step s
    uint32_t qw[kN][2 * (D / 16)];
#pragma unroll
    for (int nt = 0; nt < kN; ++nt) {
      const int i = i0 + 8 * nt + g;
      const __nv_bfloat16* qr = p.q + (i < rows ? row_index(i) : 0) * D;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const uint2 a = i < rows ? __ldg(reinterpret_cast<const uint2*>(qr + dec_koff<D, kF8>(s, t4))) : make_uint2(0u, 0u);
        qw[nt][2 * s] = a.x, qw[nt][2 * s + 1] = a.y;
      }
      float back = 1.f;
      if constexpr (kF8) {
        // bf16 -> f16 times 2^sh, which brings the row's largest magnitude to [2^13, 2^14)
        uint32_t top = 0u;
#pragma unroll
        for (int w = 0; w < 2 * (D / 16); ++w) top = max(top, max(qw[nt][w] & 0x7fffu, (qw[nt][w] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int sh = min(126, 140 - (int)(top >> 7));
        const float mul = pow2_field(127 + sh);
        back = pow2_field(127 - sh);
#pragma unroll
        for (int w = 0; w < 2 * (D / 16); ++w)
          qw[nt][w] = pack_f16x2(__uint_as_float(qw[nt][w] << 16) * mul, __uint_as_float(qw[nt][w] & 0xffff0000u) * mul);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.f;
        cf[nt][e] = p.c * __shfl_sync(0xffffffffu, back, 4 * (2 * t4 + e));   // from the lane of that row
        lim[nt][e] = (p.causal && !prefix) ? len - p.T + 1 + (i0 + 8 * nt + 2 * t4 + e) % p.T : len;
      }
    }
    if (p.causal && !prefix) lim_min = len - p.T + 1;
    int top_e = 0;   // E4M3: the largest V exponent so far (0: none yet)

    for (int n = 0; n < steps && ok; ++n) {
      const int k = k_first + n * stride;
      // the stage of the step before last is free once the way's warps have left it
      if (issuer && n + stages - 1 < steps) ok = issue(n + stages - 1);
      ok = wait_phase(&ring_full[stage], phase, abort_flag, kSiteDecodeFull) && ok;
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      // Keys that a later token of the call sees and an earlier one does not: a value there that is not finite
      // would reach the earlier one as 0 * NaN.  It is taken out of the stage (E4M3: its mark is), and put in for
      // the rows that see it behind the last step.  (Done here, where few registers are in use: left to the products'
      // operands it cost 16 rows 5 to 12 %.  In shared memory, B64 T4 N<=8192 E4M3 takes 206 us instead of 248, B20 T4
      // N<=2000 bf16 35 instead of 40, the 16-row forms spilling less; T1 B20 N<=2000 E4M3 26.5 instead of 25.8.)
      if (p.T > 1 && lim_min - k < Cfg::kStep) {
        const int r0 = max(0, lim_min - k), r1 = min(Cfg::kStep, key_end - k);
        bool found = false;
        if constexpr (kF8) {
          uint8_t* e = exps + stage * kDecExpBytes + 32 + lane;
          if (lane >= r0 && lane < r1 && *e == kE8Nan) {
            found = true;
            *e = 0;   // (codes of 0: any exponent does, and this one is no maximum)
          }
        } else {
          // 16 bytes a lane: an exponent of all ones carries into the sign's place
          const uint32_t tile = ring + stage * kDecStageBytes + Cfg::kVOff;
          uint32_t carry = 0u;
          for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
#pragma unroll
            for (int c = 0; c < Cfg::kChunks; ++c) {
              uint32_t w[4];
              lds16(w, tile + c * Cfg::kChunkBytes + i * 16);
#pragma unroll
              for (int e = 0; e < 4; ++e) carry |= (w[e] & 0x7f807f80u) + 0x00800080u;
            }
          found = (carry & 0x80008000u) != 0u;
          if (__any_sync(0xffffffffu, found)) {
            uint16_t* x = reinterpret_cast<uint16_t*>(smem + (kg * stages + stage) * kDecStageBytes + Cfg::kVOff);
            for (int c = 0; c < Cfg::kChunks; ++c)
              for (int i = r0 * 64 + lane; i < r1 * 64; i += 32)
                if ((x[c * (Cfg::kChunkBytes / 2) + i] & 0x7f80u) == 0x7f80u) x[c * (Cfg::kChunkBytes / 2) + i] = 0;
            found = true;
          }
        }
        if (found) {
          *odd = 1u;
          fence_proxy_async_smem();   // the stage's next load follows
        }
        __syncwarp();
      }
      if (active) {
        const uint32_t tile_k = ring + stage * kDecStageBytes, tile_v = tile_k + Cfg::kVOff;
        // S^T = K Q^T: keys g and g + 8 of each group, rows 2t and 2t + 1 of each tile.  Even and odd K
        // steps add to sums of their own and the groups alternate: a lone chain of D / 16 products is
        // most of a step's latency.
        float s[G][kN][4];
        {
          float odd[G][kN][4];
          uint32_t ka[G][KW], kb[G][KW];
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            dec_load_k<D, kF8>(ka[gr], tile_k, 16 * gr + g, t4);
            dec_load_k<D, kF8>(kb[gr], tile_k, 16 * gr + 8 + g, t4);
#pragma unroll
            for (int nt = 0; nt < kN; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[gr][nt][e] = odd[gr][nt][e] = 0.f;
          }
#pragma unroll
          for (int q = 0; q < D / 16; ++q)
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
              if constexpr (kF8) {
                const uint32_t a[4] = {e4m3_lo_to_f16(ka[gr][q]), e4m3_lo_to_f16(kb[gr][q]), e4m3_hi_to_f16(ka[gr][q]),
                                       e4m3_hi_to_f16(kb[gr][q])};
#pragma unroll
                for (int nt = 0; nt < kN; ++nt)
                  mma_16816_f16(q & 1 ? odd[gr][nt] : s[gr][nt], a, qw[nt][2 * q], qw[nt][2 * q + 1]);
              } else {
                const uint32_t a[4] = {ka[gr][2 * q], kb[gr][2 * q], ka[gr][2 * q + 1], kb[gr][2 * q + 1]};
#pragma unroll
                for (int nt = 0; nt < kN; ++nt)
                  mma_16816(q & 1 ? odd[gr][nt] : s[gr][nt], a, qw[nt][2 * q], qw[nt][2 * q + 1]);
              }
            }
#pragma unroll
          for (int gr = 0; gr < G; ++gr)
#pragma unroll
            for (int nt = 0; nt < kN; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[gr][nt][e] += odd[gr][nt][e];
        }
        int ev[G][2];   // E4M3: V exponents of keys g, g + 8
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          float kf[2] = {1.f, 1.f};
          if constexpr (kF8) {
            // (a marked row has codes 0: 0 * infinity is the NaN it stands for)
            const uint32_t at = smem_u32(exps) + stage * kDecExpBytes + 16 * gr + g;
            kf[0] = pow2_field(lds1(at));
            kf[1] = pow2_field(lds1(at + 8));
            ev[gr][0] = lds1(at + 32);
            ev[gr][1] = lds1(at + 40);
          }
#pragma unroll
          for (int nt = 0; nt < kN; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[gr][nt][e] *= cf[nt][e & 1];
              if constexpr (kF8) s[gr][nt][e] *= kf[e >> 1];
            }
        }
        const bool tail = (uint32_t)k + Cfg::kStep > (uint32_t)key_end;
        if (tail || k + Cfg::kStep > lim_min) {
#pragma unroll
          for (int gr = 0; gr < G; ++gr)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int key = k + 16 * gr + 8 * j + g;
#pragma unroll
              for (int nt = 0; nt < kN; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (key >= min(lim[nt][e], key_end)) s[gr][nt][2 * j + e] = -INFINITY;
              if (kF8 && key >= key_end) ev[gr][j] = top_e;   // not a key: any exponent does
            }
        }
        auto scale_o = [&](int nt, float a0, float a1) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            o[nt][c][0] *= a0;
            o[nt][c][1] *= a1;
            o[nt][c][2] *= a0;
            o[nt][c][3] *= a1;
          }
        };
        float mx[kN][2];
        bool grew = false;
#pragma unroll
        for (int nt = 0; nt < kN; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[nt][e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
            for (int gr = 1; gr < G; ++gr) mx[nt][e] = fmaxf(mx[nt][e], fmaxf(s[gr][nt][e], s[gr][nt][2 + e]));
            grew = grew || mx[nt][e] > m[nt][e] + Cfg::kLazy;
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int nt = 0; nt < kN; ++nt) {
            float a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = mx[nt][e];
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
              x = fmaxf(x, m[nt][e]);
              a[e] = x == m[nt][e] ? 1.f : ex2_approx(m[nt][e] - x);
              m[nt][e] = x;
              l[nt][e] *= a[e];
            }
            scale_o(nt, a[0], a[1]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < kN; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = (m[nt][e] == -INFINITY ? 0.f : m[nt][e]) - Cfg::kLift;
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float& x = s[gr][nt][2 * j + e];
                x = ex2_approx(x - ref);
                l[nt][e] += x;
              }
          }
        // The four value rows of group gr that this lane holds as K index.
        auto load_v = [&](uint32_t (&vr)[4][VW], int gr) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 16 * gr + 2 * t4 + (e & 1) + 8 * (e >> 1);
            dec_load_v<D, kF8>(vr[e], tile_v, j, g);
            if (tail && k + j >= key_end) {   // not a key: its row may hold anything, and 0 * NaN would stay
#pragma unroll
              for (int w = 0; w < VW; ++w) vr[e][w] = 0u;
            }
          }
        };
        // P of group gr and row tile nt as the B operand, its keys' factors f0 (key g) and f1 (key g + 8)
        auto operand_p = [&](int gr, int nt, float f0, float f1, uint32_t& b0, uint32_t& b1) {
          const float(&x)[4] = s[gr][nt];
          if constexpr (kF8) {
            b0 = transpose8x8(pack_f16x2(x[0] * f0, x[1] * f0));
            b1 = transpose8x8(pack_f16x2(x[2] * f1, x[3] * f1));
          } else {
            b0 = transpose8x8(pack_bf16x2(x[0], x[1]));
            b1 = transpose8x8(pack_bf16x2(x[2], x[3]));
          }
        };
        bool wide = false;
        if constexpr (kF8) {
          // are all of the step's V exponents in [top_e - kWindow, top_e]?
          auto outside = [&]() -> bool {
            uint32_t far = 0u;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) far = max(far, max((uint32_t)(top_e - ev[gr][0]), (uint32_t)(top_e - ev[gr][1])));
            return __any_sync(0xffffffffu, far > (uint32_t)Cfg::kWindow);
          };
          if (outside()) {
            int top = top_e;
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (ev[gr][j] != kE8Nan) top = max(top, ev[gr][j]);
            top = __reduce_max_sync(0xffffffffu, top);
            if (top > top_e && top_e > 0) {
              const float a = pow2_field(max(0, 127 - (top - top_e)));
#pragma unroll
              for (int nt = 0; nt < kN; ++nt) scale_o(nt, a, a);
            }
            top_e = top;
            if (tail) {
#pragma unroll
              for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if (k + 16 * gr + 8 * j + g >= key_end) ev[gr][j] = top_e;
            }
            wide = outside();
          }
        }
        if (!wide) {
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            uint32_t b0[kN], b1[kN], vr[4][VW];
#pragma unroll
            for (int nt = 0; nt < kN; ++nt)
              operand_p(gr, nt, kF8 ? pow2_field(127 + ev[gr][0] - top_e) : 1.f,
                        kF8 ? pow2_field(127 + ev[gr][1] - top_e) : 1.f, b0[nt], b1[nt]);
            load_v(vr, gr);
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const uint32_t a[4] = {dec_pair<kF8>(vr[0], vr[1], 2 * c), dec_pair<kF8>(vr[0], vr[1], 2 * c + 1),
                                     dec_pair<kF8>(vr[2], vr[3], 2 * c), dec_pair<kF8>(vr[2], vr[3], 2 * c + 1)};
#pragma unroll
              for (int nt = 0; nt < kN; ++nt) {
                if constexpr (kF8)
                  mma_16816_f16(o[nt][c], a, b0[nt], b1[nt]);
                else
                  mma_16816(o[nt][c], a, b0[nt], b1[nt]);
              }
            }
          }
        } else if constexpr (kF8) {
          // Exponents too far apart for one pass: the largest of those left, and what is within the
          // window below it, pass by pass (a marked row's factor is NaN, in the first).
          uint32_t left = (1u << (2 * G)) - 1u;   // this lane's keys not yet added
          for (bool first_pass = true; __any_sync(0xffffffffu, left != 0u); first_pass = false) {
            int top = 0;
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if ((left >> (2 * gr + j) & 1u) && ev[gr][j] != kE8Nan) top = max(top, ev[gr][j]);
            top = __reduce_max_sync(0xffffffffu, top);
            const float back = pow2_field(max(0, 127 - (top_e - top)));
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
              float f[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const bool marked = ev[gr][j] == kE8Nan;
                const bool now = (left >> (2 * gr + j) & 1u) && (marked ? first_pass : top - ev[gr][j] <= Cfg::kWindow);
                f[j] = !now ? 0.f : marked ? __uint_as_float(0x7fffffffu) : pow2_field(127 + ev[gr][j] - top);
                if (now) left &= ~(1u << (2 * gr + j));
              }
              uint32_t vr[4][VW];
              load_v(vr, gr);
#pragma unroll
              for (int nt = 0; nt < kN; ++nt) {
                uint32_t b0, b1;
                operand_p(gr, nt, f[0], f[1], b0, b1);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                  const uint32_t a[4] = {dec_pair<kF8>(vr[0], vr[1], 2 * c), dec_pair<kF8>(vr[0], vr[1], 2 * c + 1),
                                         dec_pair<kF8>(vr[2], vr[3], 2 * c), dec_pair<kF8>(vr[2], vr[3], 2 * c + 1)};
                  float t[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_16816_f16(t, a, b0, b1);
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[nt][c][e] = fmaf(t[e], back, o[nt][c][e]);
                }
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring_empty[stage]);   // this warp has left the stage
      if (++stage == (uint32_t)stages) {
        stage = 0u;
        phase ^= 1u;
      }
    }
    if (!kWarp && __syncthreads_or(!ok)) ok = false;   // all rings are empty (or a wait gave up)
    if (p.T > 1 && *odd != 0u) {   // rare: the values that were taken out, from the cache
#pragma unroll 1
      for (int key = max(key_begin, lim_min); key < key_end; ++key) {
        if (!kWarp && (key - key_begin) / Cfg::kStep % ways != kg) continue;
        const Walk at = walk_at(key);
        const int plane = plane_of(at.pg);
        if (plane == no_plane) continue;
        const long long row = (long long)plane * p.page + at.row;
        if (kF8 && p.vs[row] != kE8Nan) continue;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const float x = kF8 ? __uint_as_float(0x7fffffffu) : __bfloat162float(p.v[row * D + dec_col<D, kF8>(c, g)]);
          if (fabsf(x) < INFINITY) continue;
#pragma unroll
          for (int nt = 0; nt < kN; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (key < lim[nt][e]) o[nt][c / 2][2 * (c & 1) + e] += x;
        }
      }
      if (kWarp) {   // (else before the next unit, below)
        __syncwarp();
        if (lane == 0) *odd = 0u;
        __syncwarp();
      }
    }
#pragma unroll
    for (int nt = 0; nt < kN; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
        // P was 2^kLift times the probability
        if constexpr (kF8) l[nt][e] *= pow2_field(127 - (int)Cfg::kLift);
      }
    if constexpr (kF8) {
      // and O is in units of the largest V exponent
      const float a = pow2_field(127 - (int)Cfg::kLift), b = pow2_field(top_e);
#pragma unroll
      for (int nt = 0; nt < kN; ++nt)
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][c][e] = o[nt][c][e] * a * b;
    }
    if constexpr (kWarp) {
      if (!ok) break;
      // ---- write the unit: lane (g, t) has rows 2t, 2t + 1 of each tile and the columns of group g
      if (p.many.tiles > 0) wait_for_previous();   // the prefix's results, from the kernel before
#pragma unroll
      for (int nt = 0; nt < kN; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 8 * nt + 2 * t4 + e;
          if (i >= rows) continue;
          const long long row = row_index(i);
          float mt = m[nt][e], lt = l[nt][e];
          float acc[D / 8];
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            acc[2 * c] = o[nt][c][e];
            acc[2 * c + 1] = o[nt][c][2 + e];
          }
          if (p.many.tiles > 0) {
            // the prefix's parts, four at a time: their sums, then their rows, all loads before any use
            constexpr int kAhead = 4;
            const DecParts pt = dec_prefix_parts(p, seq, h, i);
            for (int k0 = 0; k0 < pt.n; k0 += kAhead) {
              float2 ml[kAhead];
              float4 v[kAhead][D / 32];
#pragma unroll
              for (int k = 0; k < kAhead; ++k) {
                const long long at = pt.at(min(k0 + k, pt.n - 1));
                ml[k] = p.many.ml[at];
#pragma unroll
                for (int ct = 0; ct < D / 8; ct += 4)
                  v[k][ct / 4] = *reinterpret_cast<const float4*>(p.many.o + at * D + dec_col<D, kF8>(ct, g));
              }
              float mn = mt;
#pragma unroll
              for (int k = 0; k < kAhead; ++k) mn = fmaxf(mn, ml[k].x);
              const float a = dec_weight(make_float2(mt, lt), mn);
              mt = mn;
              lt *= a;
#pragma unroll
              for (int ct = 0; ct < D / 8; ++ct) acc[ct] *= a;
#pragma unroll
              for (int k = 0; k < kAhead; ++k) {
                const float w = k0 + k < pt.n ? dec_weight(ml[k], mn) : 0.f;
                lt = fmaf(ml[k].y, w, lt);
#pragma unroll
                for (int ct = 0; ct < D / 8; ct += 4) {
                  acc[ct] = fmaf(v[k][ct / 4].x, w, acc[ct]);
                  acc[ct + 1] = fmaf(v[k][ct / 4].y, w, acc[ct + 1]);
                  acc[ct + 2] = fmaf(v[k][ct / 4].z, w, acc[ct + 2]);
                  acc[ct + 3] = fmaf(v[k][ct / 4].w, w, acc[ct + 3]);
                }
              }
            }
          }
          const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
          for (int ct = 0; ct < D / 8; ct += 4)
            *reinterpret_cast<uint2*>(p.o + row * D + dec_col<D, kF8>(ct, g)) =
                make_uint2(pack_bf16x2(acc[ct] * inv, acc[ct + 1] * inv), pack_bf16x2(acc[ct + 2] * inv, acc[ct + 3] * inv));
          if (g == 0) p.lse[row] = dec_lse(mt, lt);
        }
      x += (long long)gridDim.x * 4;
      continue;
    }
    if (!ok) break;

    // ---- join the warps' results, and write the unit out or its part to a slot
#pragma unroll
    for (int nt = 0; nt < kN; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * t4 + e;
        if (g == 0) sml[warp][r] = make_float2(m[nt][e], l[nt][e]);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          so[warp][r][dec_col<D, kF8>(2 * c, g)] = o[nt][c][e];
          so[warp][r][dec_col<D, kF8>(2 * c + 1, g)] = o[nt][c][2 + e];
        }
      }
    __syncthreads();
    if (rt == 0 && lane == 0) *odd = 0u;   // (all warps have read it; the next steps follow the barrier below)
    const bool whole = blk0 == 0 && blk1 == nblk;
    const long long slot = 2LL * blockIdx.x + (x == begin ? 0 : 1);
    const int unit_row = rb * row_tiles * kTile;
    const int unit_rows = min(row_tiles * kTile, rows - unit_row);
    for (int idx = threadIdx.x; idx < unit_rows * (D / 4); idx += kDecThreads) {
      const int r = idx / (D / 4), d = (idx - r * (D / 4)) * 4;
      const int tile = r / kTile, rr = r % kTile;
      float mt = -INFINITY;
      for (int w = 0; w < ways; ++w) mt = fmaxf(mt, sml[tile + w * row_tiles][rr].x);
      float lt = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < ways; ++w) {
        const float2 ml = sml[tile + w * row_tiles][rr];
        const float a = dec_weight(ml, mt);
        const float4 ov = *reinterpret_cast<const float4*>(&so[tile + w * row_tiles][rr][d]);
        lt = fmaf(ml.y, a, lt);
        acc.x = fmaf(ov.x, a, acc.x);
        acc.y = fmaf(ov.y, a, acc.y);
        acc.z = fmaf(ov.z, a, acc.z);
        acc.w = fmaf(ov.w, a, acc.w);
      }
      if (whole && p.area_o[0] == nullptr) {
        const long long row = row_index(unit_row + r);
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        *reinterpret_cast<uint2*>(p.o + row * D + d) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (d == 0) p.lse[row] = dec_lse(mt, lt);
      } else {
        const long long at = whole ? row_index(unit_row + r) : slot * p.unit_rows + r;
        float* dst = whole ? p.area_o[prefix] : p.slot_o;
        *reinterpret_cast<float4*>(dst + at * D + d) = acc;
        if (d == 0) (whole ? p.area_ml[prefix] : p.slot_ml)[at] = make_float2(mt, lt);
      }
    }
    fence_proxy_async_smem();   // the next unit's copies follow these accesses
    __syncthreads();

    move_on(row_blocks);
  }
  if (!kWarp && p.many.tiles > 0) wait_for_previous();   // the joining kernel relies on the one before, too
  // Drain after a wait gave up: every issued copy lands before the CTA exits.
  if (!ok && rt == 0 && lane == 0)
    for (int i = 0; i < min(stages, (int)i_count); ++i) {
      i_phase ^= i_stage == 0u ? 1u : 0u;
      i_stage = i_stage == 0u ? (uint32_t)stages - 1u : i_stage - 1u;
      drain_phase(&ring_full[i_stage], i_phase, abort_flag);
    }
}

// Joins the parts of every split unit in key order, and, behind a shared prefix (area_o set), the
// prefix's results with each row's own.  Block (unit, y): a warp for each of four rows of the unit.
// Lane k takes part k's maximum, sum and place (32 at a time), then the warp adds the parts' rows.
// Bound by launch and three dependent reads (lengths, sums, rows; the parts are in L2).
template <int D>
__global__ void __launch_bounds__(kDecThreads) attn_decode_join_kernel(const DecParams p, unsigned ctas) {
  __shared__ long long scratch[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned unit = blockIdx.x;
  const unsigned per_seq = (unsigned)p.Hkv * (unsigned)p.row_blocks;
  const int b = (int)(unit / per_seq);
  const int hr = (int)(unit - (unsigned)b * per_seq);
  const int h = hr / p.row_blocks, rb = hr - h * p.row_blocks;
  int seq;
  long long first;
  const DecLine ln = dec_locate(p, ctas, 0, b, scratch, seq, first);
  // what follows in the stream waits for this kernel alone, so some block always waits for the one before
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) wait_for_previous();
  const int places = dec_places(dec_blocks(p, dec_len(p, b)));
  const long long u0 = first + (long long)hr * places, u1 = u0 + places;
  const bool shared = p.area_o[0] != nullptr;
  if (!shared && (u0 + kDecOver) / ln.share == (u1 - 1) / ln.share) return;   // written by the one CTA that had it
  const int r = (int)blockIdx.y * 4 + warp, i = rb * p.unit_rows + r;
  if (r >= p.unit_rows || i >= p.GT) return;
  const long long row = ((long long)b * p.Hkv + h) * p.GT + i;
  wait_for_previous();

  float m = -INFINITY, l = 0.f;
  float acc[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) acc[c] = 0.f;
  // n results at rows at(k) of po, pml
  auto add = [&](int n, const float* po, const float2* pml, auto at) {
    for (int k0 = 0; k0 < n; k0 += 32) {
      const bool mine = k0 + lane < n;
      const long long place = mine ? at(k0 + lane) : 0;
      const float2 ml = mine ? pml[place] : make_float2(-INFINITY, 0.f);
      float mn = ml.x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
      mn = fmaxf(m, mn);
      const float a = dec_weight(make_float2(m, l), mn), w = dec_weight(ml, mn);
      float sum = ml.y * w;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      m = mn;
      l = fmaf(l, a, sum);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) acc[c] *= a;
      const int here = min(32, n - k0);
#pragma unroll 8
      for (int k = 0; k < here; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        const long long pk = __shfl_sync(0xffffffffu, place, k);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(po[pk * D + 32 * c + lane], wk, acc[c]);
      }
    }
  };
  // the parts [a0, a1) of the line, of a unit whose rows start at `slot_row`'s of a slot; whole: an area's row
  auto add_unit = [&](long long a0, long long a1, int part, int slot_row) {
    const long long f = (a0 + kDecOver) / ln.share, e = (a1 - 1) / ln.share;
    if (f == e)
      add(1, p.area_o[part], p.area_ml[part], [&](int) { return row; });
    else
      add((int)(e - f) + 1, p.slot_o, p.slot_ml, [&](int k) {
        return (2 * (f + k) + ((k == 0 && a0 > f * ln.share) ? 1 : 0)) * p.unit_rows + slot_row;
      });
  };
  if (p.prefix_len > 0) {   // few rows: computed by the same kernel
    const int pre = dec_places(dec_key_blocks(p.prefix_len));
    const int pr = b * p.GT + i;
    const long long a0 = ((long long)h * p.prefix_row_blocks + pr / p.unit_rows) * pre;
    add_unit(a0, a0 + pre, 1, pr % p.unit_rows);
  }
  if (p.many.tiles > 0) {
    const DecParts pt = dec_prefix_parts(p, b, h, i);
    add(pt.n, p.many.o, p.many.ml, [&](int k) { return pt.at(k); });
  }
  add_unit(u0, u1, 0, r);
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) p.o[row * D + 32 * c + lane] = __float2bfloat16_rn(acc[c] * inv);
  if (lane == 0) p.lse[row] = dec_lse(m, l);
}

}  // namespace attn
