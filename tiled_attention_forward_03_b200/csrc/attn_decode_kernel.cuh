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
//  * A lane reads its operands of the tensor-core instruction (m16n8k16, 16 query rows) as they lie:
//    the K = 16 index of Q K^T may be any permutation of D as long as Q uses the same one, so a lane
//    takes 16 contiguous bytes of its key's row for several K steps (pieces 2t, 2t+1 of a swizzled
//    row: no bank conflicts); likewise the N = 8 index of P V is any permutation of the output
//    columns, so a lane takes 16 bytes of the four value rows that it holds as K index, and pairs two
//    rows with one byte permutation per operand register.  Nothing is transposed.
//  * E4M3 codes become bf16 by moving their bits (sign, then exponent and mantissa 4 bits down: the
//    value times 2^-120, exact for subnormal codes too) and one exact multiplication by 2^120.  A
//    token's K exponent multiplies its scores in fp32, its V exponent its probability before that is
//    rounded to bf16: both are powers of two and round nothing.
//  * The running maximum moves only when some row of the warp grew by more than 8 (2^8 in P), so the
//    usual step needs one vote and no shuffle, and O is rarely rescaled.
//
// Schedule.  The work is counted in blocks of 64 keys of one (sequence, KV head, row block) unit,
// all units in one line.  Each of the grid's CTAs takes an equal, contiguous range of that line,
// found from the lengths on the device, so uneven batches stay balanced and a captured launch serves
// any lengths.  A range covers whole units (written out directly) and at most two partial ones
// (written as unnormalised O, maximum and sum in fp32 to the CTA's two slots of the workspace); a
// second kernel joins the parts of each split unit in key order.  No atomics, no state in the
// workspace: results depend on the inputs alone.
//
// A CTA's four warps take `row_tiles` tiles of 16 rows (1, 2 or 4) and share the keys 4 / row_tiles
// ways; the warps of one way share its ring (a stage is refilled once all of them have left it).
// Their results are joined in shared memory, in the ring's place.  Every wait is bounded.
#pragma once

#include <cuda_bf16.h>

#include "attn_cache_kernel.cuh"

namespace attn {

constexpr int kDecThreads = 128;
constexpr int kDecBlock = 64;       // keys per block of the schedule
constexpr int kDecStages = 8;       // of all the CTA's rings together
constexpr int kDecStageBytes = 8192;

enum : unsigned {
  kSiteDecodeFull = 51,
  kSiteDecodeEmpty = 52,
};

struct DecParams {
  const __nv_bfloat16* q;    // [B][Hkv][GT][D]
  const uint8_t* ks;         // E4M3: exponents [num_pages][Hkv][page]
  const uint8_t* vs;
  const int* table;          // [B][max_pages], or null: sequence b is page b
  const int* lens;           // [B], or null: len_all
  long long cap;             // max_pages * page: no sequence is longer
  int len_all, max_pages, num_pages, page, Hkv, B;
  FastDiv div_page;
  int GT, T;                 // rows of a sequence and KV head; tokens (row i is token i % T)
  int causal;                // token t sees keys up to len - T + t
  FastDiv div_gt;
  int row_tiles;                        // of a CTA
  int row_blocks;                       // of a sequence
  int box;                              // key rows of a TMA box: the step, or 16
  // shared prefix handled here (prefix_len > 0): an extra first sequence with all rows of the batch
  const int* prefix_table;
  int prefix_len, prefix_row_blocks;
  int whole_units;           // 1: CTAs take whole units only (every sequence is short)
  int min_share;             // blocks a CTA takes at least
  float c;                   // scale * log2(e)
  __nv_bfloat16* o;          // [B][Hkv][GT][D]
  float* lse;                // [B][Hkv][GT]
  // workspace
  float* slot_o;             // [2 * grid][slot_rows][D]
  float2* slot_ml;           // [2 * grid][slot_rows]
  int slot_rows;
  // shared prefix: whole units go here instead of o, lse, indexed like o: [0] own keys, [1] prefix
  float* area_o[2];
  float2* area_ml[2];
  // partial results of the prefix from the tensor-core kernel: [prefix_splits][B*Hkv*GT]
  int prefix_splits;
  const float* split_o;
  const float2* split_ml;
};

__device__ __forceinline__ int dec_len(const DecParams& p, int b) {
  const long long n = p.lens != nullptr ? (long long)p.lens[b] : (long long)p.len_all;
  return (int)max(0LL, min(n, p.cap));
}

__device__ __forceinline__ int dec_blocks(const DecParams& p, int len) {
  return p.whole_units ? 1 : max(1, (int)(((long long)len + kDecBlock - 1) / kDecBlock));
}

// The line of blocks: the prefix's first, then sequence by sequence; within a sequence KV head by
// KV head, row block by row block.
struct DecLine {
  long long prefix;   // blocks of the prefix's units together
  long long total;
  long long share;    // blocks of a CTA
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
  for (int b = b0; b < b1; ++b) mine += dec_blocks(p, dec_len(p, b));
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
  ln.prefix = p.prefix_len > 0 ? (long long)p.Hkv * p.prefix_row_blocks *
                                     (p.whole_units ? 1 : (p.prefix_len + kDecBlock - 1) / kDecBlock)
                               : 0;
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
      const long long n = per_seq * dec_blocks(p, dec_len(p, b));
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

// D += A B, m16n8k16, bf16 operands and fp32 accumulators in registers.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool kF8>
struct DecCfg {
  static constexpr int kElem = kF8 ? 1 : 2;
  static constexpr int kChunks = (D * kElem + 127) / 128;   // 128-byte pieces of a row
  static constexpr int kGroups = 2 / kChunks;               // 16-key groups per step
  static constexpr int kStep = 16 * kGroups;
  static constexpr int kChunkBytes = kStep * 128;
  static constexpr int kVOff = kChunks * kChunkBytes;       // V behind K in a stage
  static_assert(2 * kVOff == kDecStageBytes, "a stage holds one step");
  static constexpr int kKWords = D * kElem / 16;            // 32-bit words of a key a lane holds (1/4 of it)
  static constexpr int kVWords = D * kElem / 32;            // of a value row (1/8 of it)
  static constexpr int kRowStride = D + 4;                  // floats, of a row of the join
  static constexpr int kJoinBytes = 4 * 16 * kRowStride * 4;
  static_assert(kJoinBytes <= kDecStages * kDecStageBytes, "the join takes the rings' place");
};
constexpr int kDecSmem = kDecStages * kDecStageBytes + 1024;   // slack for 1024-byte alignment

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

// Output column of operand register `ct` of P V (0 <= ct < D/8) for N index n (0..7): the columns a
// lane loads contiguously.
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

template <int D, bool kF8>
__global__ void __launch_bounds__(kDecThreads, 3)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const DecParams p) {
  using Cfg = DecCfg<D, kF8>;
  constexpr int G = Cfg::kGroups, KW = Cfg::kKWords, VW = Cfg::kVWords;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float2 sml[4][16];
  __shared__ long long scratch[16];
  __shared__ uint64_t full[kDecStages], empty[kDecStages];
  __shared__ uint32_t abort_word;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  auto so = reinterpret_cast<float(*)[16][Cfg::kRowStride]>(smem);
  volatile uint32_t* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int row_tiles = p.row_tiles;
  const int kg = warp / row_tiles, rt = warp - kg * row_tiles, ways = 4 / row_tiles;
  const int stages = kDecStages / ways;                 // of this way's ring
  const uint32_t ring = smem_u32(smem) + kg * stages * kDecStageBytes;
  uint64_t* ring_full = full + kg * stages;
  uint64_t* ring_empty = empty + kg * stages;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDecStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], row_tiles);
    }
    *abort_flag = 0u;
    fence_mbar_init();
    if (p.cap > 0 || p.prefix_len > 0) {   // (without any key there are no tensor maps)
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
    }
  }

  int seq;
  long long first;
  const DecLine ln = dec_locate(p, gridDim.x, blockIdx.x, -1, scratch, seq, first);   // (its barriers order the above)
  const long long begin = (long long)blockIdx.x * ln.share, end = min(ln.total, begin + ln.share);
  // ring positions: steps issued (the way's first warp) and left behind, over all units
  uint32_t issued = 0u, done = 0u;
  bool ok = true;

  for (long long x = begin; x < end;) {
    // ---- the unit at line position x, and the part of it in this CTA's range
    const bool prefix = seq < 0;
    const int len = prefix ? p.prefix_len : dec_len(p, seq);
    const int nblk = prefix ? (p.whole_units ? 1 : (len + kDecBlock - 1) / kDecBlock) : dec_blocks(p, len);
    const int row_blocks = prefix ? p.prefix_row_blocks : p.row_blocks;
    const int rows = prefix ? p.B * p.GT : p.GT;
    const int unit = (int)((x - first) / nblk);
    const int blk0 = (int)((x - first) - (long long)unit * nblk);
    const int blk1 = (int)min((long long)nblk, blk0 + (end - x));
    const int h = unit / row_blocks, rb = unit - h * row_blocks;
    const int* table = prefix ? p.prefix_table : (p.table ? p.table + (size_t)seq * p.max_pages : nullptr);
    const int i0 = rb * 16 * row_tiles + rt * 16;   // first row of this warp's tile
    const int key_begin = p.whole_units ? 0 : blk0 * kDecBlock;
    const int key_end = p.whole_units ? len : (int)min((long long)len, (long long)blk1 * kDecBlock);

    // row i of the unit -> its index in q, o, lse
    auto row_index = [&](int i) -> long long {
      if (!prefix) return ((long long)seq * p.Hkv + h) * p.GT + i;
      const uint32_t b = fast_div((uint32_t)i, p.div_gt);
      return ((long long)b * p.Hkv + h) * p.GT + (i - (int)b * p.GT);
    };
    // this way's steps: keys key_begin + (kg + ways * n) * kStep
    const int stride = ways * Cfg::kStep;
    const int k_first = key_begin + kg * Cfg::kStep;
    const int steps = k_first < key_end ? (key_end - k_first + stride - 1) / stride : 0;
    // key position k -> (page's plane in the tensor maps, row in the page); no page: plane past the end
    auto place = [&](int k, int& plane, int& row) {
      const uint32_t pg = fast_div((uint32_t)k, p.div_page);
      const int id = table ? __ldg(table + pg) : seq;
      row = k - (int)(pg * (uint32_t)p.page);
      plane = (unsigned)id < (unsigned)p.num_pages ? id * p.Hkv + h : p.num_pages * p.Hkv;
    };
    // Loads of step n (one lane): boxes with a key only.
    auto issue = [&](int n) {
      const uint32_t st = issued % (uint32_t)stages;
      const int k = k_first + n * stride;
      const int boxes = min(Cfg::kStep / p.box, (key_end - k + p.box - 1) / p.box);
      mbar_arrive_expect_tx(&ring_full[st], (uint32_t)(2 * Cfg::kChunks * boxes * p.box * 128));
      for (int i = 0; i < boxes; ++i) {
        int plane, row;
        place(k + i * p.box, plane, row);
#pragma unroll
        for (int c = 0; c < Cfg::kChunks; ++c) {
          uint8_t* dst = smem + (kg * stages + st) * kDecStageBytes + c * Cfg::kChunkBytes + i * p.box * 128;
          tma_load_3d(dst, &tmap_k, &ring_full[st], c * (128 / Cfg::kElem), row, plane, l2_policy_evict_first());
          tma_load_3d(dst + Cfg::kVOff, &tmap_v, &ring_full[st], c * (128 / Cfg::kElem), row, plane,
                      l2_policy_evict_first());
        }
      }
    };
    const bool issuer = rt == 0 && lane == 0;
    if (issuer && ok)
      for (int n = 0; n < min(stages - 1, steps) && ok; ++n) {
        if (issued >= (uint32_t)stages)
          ok = wait_phase(&ring_empty[issued % (uint32_t)stages], (issued / (uint32_t)stages - 1u) & 1u, abort_flag,
                          kSiteDecodeEmpty);
        if (!ok) break;
        issue(n);
        ++issued;
      }
    ok = __all_sync(0xffffffffu, ok);

    float o[D / 8][4];
#pragma unroll
    for (int ct = 0; ct < D / 8; ++ct)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[ct][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    const bool active = i0 < rows;   // (a tile past the rows only keeps the ring going)

    // Q as the A operand of Q K^T: words 2s, 2s+1 of a row are K step s
    uint32_t q0[2 * (D / 16)], q1[2 * (D / 16)];
    {
      const bool r0 = i0 + g < rows, r1 = i0 + g + 8 < rows;
      const __nv_bfloat16* qa = p.q + (r0 ? row_index(i0 + g) : 0) * D;
      const __nv_bfloat16* qb = p.q + (r1 ? row_index(i0 + g + 8) : 0) * D;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const int off = dec_koff<D, kF8>(s, t4);
        const uint2 a = r0 ? __ldg(reinterpret_cast<const uint2*>(qa + off)) : make_uint2(0u, 0u);
        const uint2 b = r1 ? __ldg(reinterpret_cast<const uint2*>(qb + off)) : make_uint2(0u, 0u);
        q0[2 * s] = a.x, q0[2 * s + 1] = a.y;
        q1[2 * s] = b.x, q1[2 * s + 1] = b.y;
      }
    }
    // keys below the limits are seen by rows g and g + 8 of the tile
    int lim0 = len, lim1 = len, lim_min = len;
    if (p.causal && !prefix) {
      lim0 = len - p.T + 1 + (i0 + g) % p.T;
      lim1 = len - p.T + 1 + (i0 + g + 8) % p.T;
      lim_min = len - p.T + 1;
    }
    // E4M3: exponent bytes of keys 2t, 2t+1 of each half group of a step (1 for no page: zero rows)
    uint32_t sk[G][2], sv[G][2];
    auto load_scales = [&](int n) {
      if constexpr (kF8) {
        const int k = k_first + n * stride;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
#pragma unroll
          for (int j = 0; j < 2; ++j) sk[gr][j] = sv[gr][j] = 0x7f7fu;
          if (n >= steps || k + 16 * gr >= key_end) continue;
          int plane, row;
          place(k + 16 * gr, plane, row);
          if (plane >= p.num_pages * p.Hkv) continue;
          const long long e = (long long)plane * p.page + row + 2 * t4;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            sk[gr][j] = __ldg(reinterpret_cast<const uint16_t*>(p.ks + e + 8 * j));
            sv[gr][j] = __ldg(reinterpret_cast<const uint16_t*>(p.vs + e + 8 * j));
          }
        }
      }
    };
    load_scales(0);

    for (int n = 0; n < steps && ok; ++n, ++done) {
      const int k = k_first + n * stride;
      if (issuer && n + stages - 1 < steps) {
        // the stage of the step before last is free once the way's warps have left it
        if (issued >= (uint32_t)stages)
          ok = wait_phase(&ring_empty[issued % (uint32_t)stages], (issued / (uint32_t)stages - 1u) & 1u, abort_flag,
                          kSiteDecodeEmpty);
        if (ok) {
          issue(n + stages - 1);
          ++issued;
        }
      }
      const uint32_t st = done % (uint32_t)stages;
      ok = wait_phase(&ring_full[st], (done / (uint32_t)stages) & 1u, abort_flag, kSiteDecodeFull) && ok;
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (active) {
        const uint32_t tile_k = ring + st * kDecStageBytes, tile_v = tile_k + Cfg::kVOff;
        // S = Q K^T
        float s[G][2][4];
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t kw[KW];
            dec_load_k<D, kF8>(kw, tile_k, 16 * gr + 8 * j + g, t4);
            s[gr][j][0] = s[gr][j][1] = s[gr][j][2] = s[gr][j][3] = 0.f;
#pragma unroll
            for (int q = 0; q < D / 16; ++q) {
              const uint32_t a[4] = {q0[2 * q], q1[2 * q], q0[2 * q + 1], q1[2 * q + 1]};
              if constexpr (kF8) {
                mma_16816(s[gr][j], a, e4m3_hi2_to_bf16(__byte_perm(kw[q], 0u, 0x1000)),
                          e4m3_hi2_to_bf16(__byte_perm(kw[q], 0u, 0x3020)));
              } else {
                mma_16816(s[gr][j], a, kw[2 * q], kw[2 * q + 1]);
              }
            }
          }
        }
        float f[G][4];   // E4M3: factor of P for keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if constexpr (kF8) {
              const float c0 = p.c * e8_scale((int)(sk[gr][j] & 255u)), c1 = p.c * e8_scale((int)(sk[gr][j] >> 8));
              s[gr][j][0] *= c0;
              s[gr][j][1] *= c1;
              s[gr][j][2] *= c0;
              s[gr][j][3] *= c1;
              f[gr][2 * j] = e8_scale((int)(sv[gr][j] & 255u));
              f[gr][2 * j + 1] = e8_scale((int)(sv[gr][j] >> 8));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) s[gr][j][e] *= p.c;
            }
          }
        }
        load_scales(n + 1);
        const bool tail = k + Cfg::kStep > key_end;
        if (tail || k + Cfg::kStep > lim_min) {
#pragma unroll
          for (int gr = 0; gr < G; ++gr)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = k + 16 * gr + 8 * j + 2 * t4 + e;
                if (key >= min(lim0, key_end)) s[gr][j][e] = -INFINITY;
                if (key >= min(lim1, key_end)) s[gr][j][2 + e] = -INFINITY;
                if (kF8 && key >= key_end) f[gr][2 * j + e] = 0.f;
              }
        }
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mx0 = fmaxf(mx0, fmaxf(s[gr][j][0], s[gr][j][1]));
            mx1 = fmaxf(mx1, fmaxf(s[gr][j][2], s[gr][j][3]));
          }
        if (__any_sync(0xffffffffu, mx0 > m0 + kRescaleLog2 || mx1 > m1 + kRescaleLog2)) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
          mx0 = fmaxf(m0, fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2)));
          mx1 = fmaxf(m1, fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2)));
          const float a0 = mx0 == m0 ? 1.f : ex2_approx(m0 - mx0), a1 = mx1 == m1 ? 1.f : ex2_approx(m1 - mx1);
          m0 = mx0;
          m1 = mx1;
          l0 *= a0;
          l1 *= a1;
#pragma unroll
          for (int ct = 0; ct < D / 8; ++ct) {
            o[ct][0] *= a0;
            o[ct][1] *= a0;
            o[ct][2] *= a1;
            o[ct][3] *= a1;
          }
        }
        const float n0 = m0 == -INFINITY ? 0.f : m0, n1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
          uint32_t a[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float p0 = ex2_approx(s[gr][j][0] - n0), p1 = ex2_approx(s[gr][j][1] - n0);
            const float p2 = ex2_approx(s[gr][j][2] - n1), p3 = ex2_approx(s[gr][j][3] - n1);
            l0 += p0 + p1;
            l1 += p2 + p3;
            if constexpr (kF8) {
              a[2 * j] = pack_bf16x2(p0 * f[gr][2 * j], p1 * f[gr][2 * j + 1]);
              a[2 * j + 1] = pack_bf16x2(p2 * f[gr][2 * j], p3 * f[gr][2 * j + 1]);
            } else {
              a[2 * j] = pack_bf16x2(p0, p1);
              a[2 * j + 1] = pack_bf16x2(p2, p3);
            }
          }
          // O += P V
          uint32_t vr[4][VW];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 16 * gr + 2 * t4 + (e & 1) + 8 * (e >> 1);
            dec_load_v<D, kF8>(vr[e], tile_v, j, g);
            if (tail && k + j >= key_end) {   // not a key: its row may hold anything, and 0 * NaN would stay
#pragma unroll
              for (int w = 0; w < VW; ++w) vr[e][w] = 0u;
            }
          }
#pragma unroll
          for (int ct = 0; ct < D / 8; ++ct) {
            uint32_t b0, b1;
            if constexpr (kF8) {
              const int w = ct / 4;
              const uint32_t sel = ((uint32_t)(4 + ct % 4) << 12) | ((uint32_t)(ct % 4) << 4);
              b0 = e4m3_hi2_to_bf16(__byte_perm(vr[0][w], vr[1][w], sel));
              b1 = e4m3_hi2_to_bf16(__byte_perm(vr[2][w], vr[3][w], sel));
            } else {
              const uint32_t sel = (ct & 1) ? 0x7632u : 0x5410u;
              b0 = __byte_perm(vr[0][ct / 2], vr[1][ct / 2], sel);
              b1 = __byte_perm(vr[2][ct / 2], vr[3][ct / 2], sel);
            }
            mma_16816(o[ct], a, b0, b1);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring_empty[st]);   // this warp has left the stage
    }
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    // all rings are empty: the join may take their place, unless a wait gave up
    if (__syncthreads_or(!ok)) {
      ok = false;
      break;
    }

    // ---- join the warps' results, and write the unit out or its part to a slot
    if (t4 == 0) {
      sml[warp][g] = make_float2(m0, l0);
      sml[warp][g + 8] = make_float2(m1, l1);
    }
#pragma unroll
    for (int ct = 0; ct < D / 8; ++ct) {
      so[warp][g][dec_col<D, kF8>(ct, 2 * t4)] = o[ct][0];
      so[warp][g][dec_col<D, kF8>(ct, 2 * t4 + 1)] = o[ct][1];
      so[warp][g + 8][dec_col<D, kF8>(ct, 2 * t4)] = o[ct][2];
      so[warp][g + 8][dec_col<D, kF8>(ct, 2 * t4 + 1)] = o[ct][3];
    }
    __syncthreads();
    const bool whole = blk0 == 0 && blk1 == nblk;
    const long long slot = 2LL * blockIdx.x + (x == begin ? 0 : 1);
    const int tile_rows = min(16 * row_tiles, rows - rb * 16 * row_tiles);
    for (int idx = threadIdx.x; idx < tile_rows * (D / 4); idx += kDecThreads) {
      const int r = idx / (D / 4), d = (idx - r * (D / 4)) * 4;
      const int tile = r >> 4, rr = r & 15;
      float mt = -INFINITY;
      for (int w = 0; w < ways; ++w) mt = fmaxf(mt, sml[tile + w * row_tiles][rr].x);
      float lt = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < ways; ++w) {
        const float2 ml = sml[tile + w * row_tiles][rr];
        const float a = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2_approx(ml.x - mt);
        const float4 ov = *reinterpret_cast<const float4*>(&so[tile + w * row_tiles][rr][d]);
        lt = fmaf(ml.y, a, lt);
        acc.x = fmaf(ov.x, a, acc.x);
        acc.y = fmaf(ov.y, a, acc.y);
        acc.z = fmaf(ov.z, a, acc.z);
        acc.w = fmaf(ov.w, a, acc.w);
      }
      if (whole && p.area_o[0] == nullptr) {
        const long long row = row_index(rb * 16 * row_tiles + r);
        const float inv = lt == 0.f ? 0.f : 1.f / lt;
        *reinterpret_cast<uint2*>(p.o + row * D + d) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (d == 0)
          p.lse[row] = lt == 0.f ? -INFINITY : ((mt == -INFINITY ? 0.f : mt) + log2f(lt)) * 0.69314718055994530942f;
      } else {
        const long long at = whole ? row_index(rb * 16 * row_tiles + r) : slot * p.slot_rows + r;
        float* dst = whole ? p.area_o[prefix] : p.slot_o;
        *reinterpret_cast<float4*>(dst + at * D + d) = acc;
        if (d == 0) (whole ? p.area_ml[prefix] : p.slot_ml)[at] = make_float2(mt, lt);
      }
    }
    fence_proxy_async_smem();   // the next unit's copies follow these accesses
    __syncthreads();

    // ---- the next unit
    x += blk1 - blk0;
    const long long seq_blocks = (long long)p.Hkv * row_blocks * nblk;
    if (x >= first + seq_blocks) {
      first += seq_blocks;
      ++seq;
    }
  }
  // Drain after a wait gave up: every issued copy lands before the CTA exits.
  if (!ok && rt == 0 && lane == 0)
    for (uint32_t i = issued > (uint32_t)stages ? issued - (uint32_t)stages : 0u; i < issued; ++i)
      drain_phase(&ring_full[i % (uint32_t)stages], (i / (uint32_t)stages) & 1u, abort_flag);
}

// Joins the parts of every split unit in key order, and, behind a shared prefix (area_o set), the
// prefix's result with each row's own.  One block per (sequence, KV head, row block).  Bound by
// launch and a few dependent reads; the parts are still in L2.
template <int D>
__global__ void __launch_bounds__(kDecThreads) attn_decode_join_kernel(const DecParams p, unsigned ctas) {
  __shared__ long long scratch[16];
  const unsigned unit = blockIdx.x;
  const unsigned per_seq = (unsigned)p.Hkv * (unsigned)p.row_blocks;
  const int b = (int)(unit / per_seq);
  const int hr = (int)(unit - (unsigned)b * per_seq);
  const int h = hr / p.row_blocks, rb = hr - h * p.row_blocks;
  int seq;
  long long first;
  const DecLine ln = dec_locate(p, ctas, 0, b, scratch, seq, first);
  const int nblk = dec_blocks(p, dec_len(p, b));
  const long long u0 = first + (long long)hr * nblk, u1 = u0 + nblk;
  const long long c0 = u0 / ln.share, c1 = (u1 - 1) / ln.share;
  const bool shared = p.area_o[0] != nullptr;
  if (!shared && c0 == c1) return;   // written by the one CTA that had it

  const int tile_rows = min(16 * p.row_tiles, p.GT - rb * 16 * p.row_tiles);
  // prefix unit of a row (few rows: computed by the same kernel): its parts, if it was split
  const int pre_nblk = p.whole_units ? 1 : (p.prefix_len + kDecBlock - 1) / kDecBlock;
  for (int idx = threadIdx.x; idx < tile_rows * (D / 4); idx += kDecThreads) {
    const int r = idx / (D / 4), d = (idx - r * (D / 4)) * 4;
    const int i = rb * 16 * p.row_tiles + r;
    const long long row = ((long long)b * p.Hkv + h) * p.GT + i;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float* po, const float2* pml, long long at) {
      const float2 ml = pml[at];
      if (ml.x == -INFINITY && ml.y == 0.f) return;   // no keys: nothing to add
      const float4 v = *reinterpret_cast<const float4*>(po + at * D + d);
      const float mn = fmaxf(m, ml.x);
      const float a = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2_approx(m - mn);
      const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2_approx(ml.x - mn);
      m = mn;
      l = fmaf(ml.y, w, l * a);
      acc.x = fmaf(v.x, w, acc.x * a);
      acc.y = fmaf(v.y, w, acc.y * a);
      acc.z = fmaf(v.z, w, acc.z * a);
      acc.w = fmaf(v.w, w, acc.w * a);
    };
    // the parts of the unit [a0, a1) of the line; its rows start at `r` of a slot
    auto add_unit = [&](long long a0, long long a1, int part, int slot_row) {
      const long long f = a0 / ln.share, e = (a1 - 1) / ln.share;
      if (f == e) {
        add(p.area_o[part], p.area_ml[part], row);
        return;
      }
      for (long long c = f; c <= e; ++c)
        add(p.slot_o, p.slot_ml, (2 * c + ((c == f && a0 != c * ln.share) ? 1 : 0)) * p.slot_rows + slot_row);
    };
    if (p.prefix_len > 0) {
      const int pr = b * p.GT + i, per = 16 * p.row_tiles;
      const long long a0 = ((long long)h * p.prefix_row_blocks + pr / per) * pre_nblk;
      add_unit(a0, a0 + pre_nblk, 1, pr % per);
    }
    for (int s = 0; s < p.prefix_splits; ++s) add(p.split_o, p.split_ml, (long long)s * p.B * p.Hkv * p.GT + row);
    add_unit(u0, u1, 0, r);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(p.o + row * D + d) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (d == 0) p.lse[row] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * 0.69314718055994530942f;
  }
}

}  // namespace attn
