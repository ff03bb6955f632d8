// attn_fwd_rows_kernel.cuh -- attention of many query rows to keys of another length on B200
// (sm_100a): cross attention, and the prefix that a decoding batch shares.
//
// The computation is attn_fwd_colsplit_kernel.cuh's -- one 128-row tile per unit, two score buffers,
// each 128-key block's columns split between two softmax warpgroups with maxima, sums and
// accumulators of their own, joined exactly at the end of the unit -- without a causal mask, and with
// rows, keys and work that come from elsewhere:
//
//  * Rows.  All query rows that see the same keys may share a tile: the group * Nq rows of a KV head
//    (contiguous in q), or for a shared prefix those of several sequences, which a four-dimensional
//    TMA box (columns, rows of a sequence, head, sequences) lays one after the other.
//  * Keys, bf16: contiguous, or in pages, by TMA boxes of the largest of 128, 64, 32, 16 rows that
//    divides a page.  Each batch row has its own count of them; the MMA warp overwrites the last
//    value tile's rows behind it with zeros (its probabilities are 0, and 0 * NaN would not be).
//  * Keys, E4M3 (kF8): codes and exponents go by TMA to a raw ring; two more warpgroups convert them,
//    every other tile each, to bf16, exactly (a power-of-two scale rounds nothing), and store them as
//    TMA would, 128-byte swizzled.  One conversion serves 128 rows and is hidden behind their
//    exponentials (with one warpgroup it was not: 4100 clocks a block instead of 2100).
//  * Work: as in the decode kernel, the units' 128-key blocks stand in one line and each CTA
//    takes an equal, contiguous range of it, whatever the lengths; a range holds whole units and at
//    most two parts of units, which go unnormalised, in fp32, to the CTA's two slots of the workspace
//    and are joined by a second kernel.  (Dealing whole units out left the GPU a third idle for the
//    uneven lengths of B8 H16 Nq500 Nk<=1500.)  One warp finds the range and hands the units to the
//    other roles through a ring in shared memory: their code is then small enough for the
//    instruction cache (each role computing its own schedule took 130 KB of code, and 20 to 30 % of
//    the time).
//
// Bound by the tensor pipe's feeding: a 128-key block takes about 1650 clocks at D = 128 (the products
// alone 1024), the exponentials and the issue of products in turn.  Measured (B200): B4 Hq32 Hkv8 Nq2048
// Nk<=4096 D128 284 us, 1090 TFLOP/s; B8 H16 Nq500 Nk<=1500 D64 37 us and 8 us for the joining.
//
//   warps 0-3, 4-7  softmax warpgroups     warp 8   TMA producer     warp 9  MMA issuer
//   warp 10  output store (cross)          warp 11  scheduler        warps 12-19 (kF8) converters
//
// Every mbarrier wait is bounded; named barriers are only reached by all their participants.
#pragma once

#include <cuda_bf16.h>

#include "attn_decode_kernel.cuh"

namespace attn {

enum : unsigned {
  kSiteRowsProducer = 41,
  kSiteRowsMma = 42,
  kSiteRowsSoftmax = 43,
  kSiteRowsEpilogue = 44,
  kSiteRowsStore = 45,
  kSiteRowsConvert = 46,
  kSiteRowsSchedule = 47,
};

// Register split.  bf16: the forward kernel's (384 threads at 168).  kF8: 640 threads at 96;
// 2 * 128 * 152 + 128 * 48 + 2 * 128 * 64 == 640 * 96.
template <bool kF8>
struct RowsCfg {
  static constexpr int kThreads = kF8 ? 640 : 384;
  static constexpr int kRegsLaunch = kF8 ? 96 : kRegsAtLaunch;
  static constexpr int kSoftmax = kF8 ? 152 : kRegsSoftmax;
  static constexpr int kControl = kF8 ? 48 : kRegsControl;
  static constexpr int kConvert = 64;
  static_assert(2 * 128 * kSoftmax + 128 * kControl + (kF8 ? 256 * kConvert : 0) <= kThreads * kRegsLaunch,
                "register split exceeds the launch allocation");
};

constexpr int kRowsQueue = 4;   // units in the scheduler's ring

template <int D, bool kF8>
struct RowsSmem {
  static_assert(D == 32 || D == 64 || D == 96 || D == 128, "head dim must be 32, 64, 96 or 128");
  static constexpr int kChunks = (D + 63) / 64;          // 64-column (128-byte) swizzle chunks of a bf16 row
  static constexpr int kChunkBytes = kBlockM * 128;
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kStages = kF8 ? (kChunks == 2 ? 3 : 6) : (kChunks == 2 ? 4 : 8);   // K/V ring (bf16 tiles)
  // raw ring (E4M3 tiles and their exponents): with three a block took 3500 clocks, the tiles' latency
  static constexpr int kRaw = kF8 ? 5 : 0;
  static constexpr int kRawBytes = kBlockN * D;
  static constexpr int kOChunks = D / 32;                 // 32-column output chunks (64-byte rows)
  static constexpr int kStageBytes = kBlockM * 64;        // one staged output chunk: 8 KB
  static_assert(kOChunks * kStageBytes <= kTileBytes, "staged O must fit in a Q buffer");
  // Q buffers: two (O staging after their last use); one for kF8, whose units are long
  static constexpr int kQBufs = kF8 ? 1 : 2;
  static constexpr int kQOff = 0;
  static constexpr int kKVOff = kQBufs * kTileBytes;
  static constexpr int kRawOff = kKVOff + kStages * kTileBytes;
  static constexpr int kExpOff = kRawOff + kRaw * kRawBytes;
  static constexpr int kXOff = kExpOff + kRaw * kBlockN;  // (m, l) exchange [unit parity][warpgroup][row]
  static constexpr int kUnitOff = kXOff + 2 * 2 * kBlockM * 8;
  static constexpr int kBarOff = kUnitOff + kRowsQueue * 32;
  // q_full[2] q_empty[2] o_staged[2] kv_full[S] kv_empty[S] s_full[2] p_full[2 buffers][2 halves]
  // pv_done o_full o_free drain u_full[Q] u_empty[Q] raw_full[R] raw_empty[R]
  static constexpr int kNumBars = 6 + 2 * kStages + 2 + 4 + 4 + 2 * kRowsQueue + 2 * kRaw;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;  // tmem base, abort flag
  static constexpr int kAlloc = kMiscOff + 16 + 1024;      // slack for 1024-byte alignment
  static_assert(kAlloc <= 232448, "many-row kernel shared memory plan exceeds 227 KB");
};

struct RowsParams {
  float* lse;                // [B][Hkv][GT]
  __nv_bfloat16* o;          // [B][Hkv][GT][D]
  // unnormalised results [slot][128 rows][D] and (max, sum) [slot][128]: two slots a CTA for parts of
  // units; prefix: whole units' after them, by unit
  float* slot_o;
  float2* slot_ml;
  int B, Hkv, GT;
  int tiles;                 // of a key group: (b, h), or for a prefix h
  int prefix;                // 1: a tile has rows of all sequences
  int behind;                // 1: the keys are written by the kernel before
  int seqs;                  // sequences in a tile (prefix; else 1)
  int seq_tiles;             // tiles of a sequence (prefix with GT > 128; else 1)
  int q_box_rows;            // rows a Q tile load fills
  int min_share;             // places a CTA takes at least
  const int* k_lens;         // [B] or null
  int len_all;               // keys where k_lens is null; no batch row has more
  // paged keys
  const int* table;          // or null: page b
  int page, num_pages;
  int box;                   // key rows of a TMA box
  const uint8_t* ks;         // kF8: exponents
  const uint8_t* vs;
  float c;                   // |scale| * log2(e)
  uint32_t idesc_s;          // S = Q K^T: 128 x 128 x D (negates A when scale < 0)
  uint32_t idesc_pv;         // O_h += P_h V_h: 128 x D x 64
};

// A unit as the scheduler hands it out: the tile's first sequence, first row and head, the sequence
// of its keys, the 128-key blocks [jb, je) and the keys; where the result goes: -1 to O and LSE, else
// the slot.  je < 0 ends the CTA's work.
struct RowsUnit {
  int b0, i0, h, b;
  int jb, je, len, slot;
};
static_assert(sizeof(RowsUnit) == 32, "queue entry");

__device__ __forceinline__ int rows_len(const RowsParams& p, int b) {
  return p.k_lens != nullptr ? max(0, min(__ldg(p.k_lens + b), p.len_all)) : p.len_all;
}
__device__ __forceinline__ int rows_blocks(int len) { return (int)(((long long)len + kBlockN - 1) / kBlockN); }

// The line of work: key group by key group (sequences and heads; heads for a prefix), tile by tile; a
// unit takes kRowsOver places for its start and end (2000 clocks, a block 1700 to 2000), then one for
// each of its blocks.  Batch rows without keys have no place.
constexpr int kRowsOver = 1;
__host__ __device__ __forceinline__ int rows_places(int blocks) { return blocks > 0 ? blocks + kRowsOver : 0; }
// Blocks of a unit before place `p` of it.
__host__ __device__ __forceinline__ int rows_block_at(int p) { return p > kRowsOver ? p - kRowsOver : 0; }

struct RowsLine {
  long long total, share;
};

// One warp: the line, and the sequence that holds position x with the position of its first block
// (find >= 0: those of sequence `find`).
__device__ __forceinline__ RowsLine rows_locate(const RowsParams& p, unsigned ctas, long long x_cta, int find, int& b,
                                                long long& first) {
  const int lane = threadIdx.x & 31;
  const long long per_seq = (long long)p.Hkv * p.tiles;
  RowsLine ln;
  const int n = p.prefix ? 1 : p.B;
  long long total = 0;
  for (int c = 0; c < n; c += 32) total += c + lane < n ? rows_places(rows_blocks(rows_len(p, c + lane))) : 0;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  ln.total = total * per_seq;
  ln.share = max((long long)p.min_share, (ln.total + ctas - 1) / ctas);
  const long long x = x_cta * ln.share;
  b = n;
  first = ln.total;
  long long at = 0;
  for (int c = 0; c < n; c += 32) {
    const long long mine = c + lane < n ? per_seq * rows_places(rows_blocks(rows_len(p, c + lane))) : 0;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const long long begin = at + incl - mine;
    const unsigned hit =
        __ballot_sync(0xffffffffu, find >= 0 ? c + lane == find : (mine > 0 && x >= begin && x < begin + mine));
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = c + src;
      first = __shfl_sync(0xffffffffu, begin, src);
      break;
    }
    at += __shfl_sync(0xffffffffu, incl, 31);
  }
  return ln;
}

// First sequence, row and head of tile `tile` of key group (b, h).
__device__ __forceinline__ void rows_tile(const RowsParams& p, int b, int h, int tile, RowsUnit& w) {
  w.b = b;
  w.h = h;
  w.b0 = !p.prefix ? b : p.seq_tiles > 1 ? tile / p.seq_tiles : tile * p.seqs;
  w.i0 = (p.prefix ? (p.seq_tiles > 1 ? tile - w.b0 * p.seq_tiles : 0) : tile) * kBlockM;
}

// Row r of the tile: its index in q, o, lse, or -1 where the tile has no such row.
__device__ __forceinline__ long long rows_index(const RowsParams& p, int b0, int i0, int h, int r) {
  int b = b0, i = i0 + r;
  if (p.prefix && p.seq_tiles == 1) {
    const int s = r / p.GT;
    if (s >= p.seqs) return -1;
    b += s;
    i -= s * p.GT;
  }
  if (b >= p.B || i >= p.GT) return -1;
  return ((long long)b * p.Hkv + h) * p.GT + i;
}

// 4-D tiled bulk tensor load global -> shared, as tma_load_3d.
ATTN_DEV void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2, int c3,
                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

template <int D, bool kF8>
__global__ void __launch_bounds__(RowsCfg<kF8>::kThreads, 1)
    attn_fwd_rows_sm100(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_o,
                        const RowsParams p) {
  using Plan = RowsSmem<D, kF8>;
  using Cfg = RowsCfg<kF8>;
  constexpr int S = Plan::kStages, R = Plan::kRaw;
  constexpr int kSSteps = D / 16;  // K = 16 steps of S = Q K^T
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);

  uint8_t* sQ = smem + Plan::kQOff;
  uint8_t* sKV = smem + Plan::kKVOff;
  uint8_t* sRaw = smem + Plan::kRawOff;
  uint8_t* sExp = smem + Plan::kExpOff;
  float2* xml = reinterpret_cast<float2*>(smem + Plan::kXOff);
  int4* units = reinterpret_cast<int4*>(smem + Plan::kUnitOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Plan::kBarOff);
  uint64_t* q_full = bars;                 // [2]
  uint64_t* q_empty = bars + 2;            // [2]: by the store warp, or (results to a slot) after the unit's last S
  uint64_t* o_staged = bars + 4;           // [2]: the unit's O is staged in Q buffer [qb]
  uint64_t* kv_full = bars + 6;            // [S]
  uint64_t* kv_empty = kv_full + S;        // [S]
  uint64_t* s_full = kv_empty + S;         // [2]
  uint64_t* p_full = s_full + 2;           // [2 buffers][2 halves]
  uint64_t* pv_done = p_full + 4;
  uint64_t* o_full = pv_done + 1;
  uint64_t* o_free = pv_done + 2;
  uint64_t* drain = pv_done + 3;
  uint64_t* u_full = pv_done + 4;          // [kRowsQueue]
  uint64_t* u_empty = u_full + kRowsQueue; // [kRowsQueue]
  uint64_t* raw_full = u_empty + kRowsQueue;  // [R]
  uint64_t* raw_empty = raw_full + R;         // [R]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Plan::kMiscOff);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Plan::kMiscOff + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&o_staged[i], 8);
      mbar_init(&s_full[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], 4);
    for (int i = 0; i < S; ++i) {
      mbar_init(&kv_full[i], kF8 ? 4 : 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(pv_done, 1);
    mbar_init(o_full, 1);
    mbar_init(o_free, 8);
    mbar_init(drain, 1);
    for (int i = 0; i < kRowsQueue; ++i) {
      mbar_init(&u_full[i], 1);
      // softmax warps, producer, MMA warp, store warp, converter warps
      mbar_init(&u_empty[i], 8 + 1 + 1 + (p.prefix ? 0 : 1) + (kF8 ? 8 : 0));
    }
    for (int i = 0; i < R; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmap_q);
    tma_prefetch_desc(&tmap_k);
    tma_prefetch_desc(&tmap_v);
    if (!p.prefix) tma_prefetch_desc(&tmap_o);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  launch_dependents();

  // Unit `ord` of the ring, once the scheduler has written it (false: a wait gave up).
  auto take = [&](uint32_t ord, RowsUnit& w, unsigned site) -> bool {
    const uint32_t q = ord % kRowsQueue;
    if (!wait_phase(&u_full[q], (ord / kRowsQueue) & 1u, abort_flag, site)) return false;
    const int4 a = units[2 * q], b = units[2 * q + 1];
    w = RowsUnit{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    return true;
  };
  auto release = [&](uint32_t ord) { mbar_arrive(&u_empty[ord % kRowsQueue]); };
  // A position in the CTA's sequence of (unit, key block) pairs.
  struct Cursor {
    uint32_t ord = 0u;   // units taken
    int j = 0;
    bool valid = false;
    RowsUnit w;
  };
  // The next unit (valid = false: none, or a wait gave up); with `give` the one left behind is given
  // back.  `wide`: a whole warp calls (every lane has read a unit before one gives it back), else one
  // lane.  (A role's first cursor keeps nothing back: it is never more than two units ahead of its
  // second, and the ring holds four.)
  auto next_unit = [&](Cursor& c, bool give, bool wide, unsigned site) {
    if (c.valid && give) {
      if (wide) __syncwarp();
      if (!wide || lane == 0) release(c.ord - 1u);
    }
    c.valid = take(c.ord, c.w, site) && c.w.je >= 0;   // (the end marker is given back by no one)
    c.j = c.w.jb;
    ++c.ord;
  };

  if (warp == 11) {
    // ------------------------------------------------------------ scheduler
    regs_decrease<Cfg::kControl>();
    int b;
    long long first;
    const RowsLine ln = rows_locate(p, gridDim.x, blockIdx.x, -1, b, first);
    const long long begin = (long long)blockIdx.x * ln.share, end = min(ln.total, begin + ln.share);
    const long long per_seq = (long long)p.Hkv * p.tiles;
    uint32_t ord = 0u;
    bool ok = true;
    auto put = [&](const RowsUnit& w) {
      const uint32_t q = ord % kRowsQueue;
      if (ord >= kRowsQueue)
        ok = wait_phase(&u_empty[q], (ord / kRowsQueue - 1u) & 1u, abort_flag, kSiteRowsSchedule);
      if (!ok) return;
      units[2 * q] = make_int4(w.b0, w.i0, w.h, w.b);
      units[2 * q + 1] = make_int4(w.jb, w.je, w.len, w.slot);
      mbar_arrive(&u_full[q]);
      ++ord;
    };
    // The units of the range to the ring (one lane).
    if (lane == 0) {
      for (long long x = begin; x < end && ok;) {
        RowsUnit w;
        w.len = rows_len(p, b);
        const int nblk = rows_blocks(w.len), n = rows_places(nblk);
        if (n == 0) {
          ++b;
          continue;
        }
        const int unit = (int)((x - first) / n);
        const int p0 = (int)((x - first) - (long long)unit * n);
        const int p1 = (int)min((long long)n, p0 + (end - x));
        const int h = unit / p.tiles;
        rows_tile(p, b, h, unit - h * p.tiles, w);
        w.jb = rows_block_at(p0);
        w.je = rows_block_at(p1);
        const bool whole = w.jb == 0 && w.je == nblk;
        w.slot = !whole ? 2 * (int)blockIdx.x + (x == begin ? 0 : 1) : p.prefix ? 2 * (int)gridDim.x + unit : -1;
        if (w.jb < w.je) put(w);
        x += p1 - p0;
        if (x >= first + per_seq * n) {
          first += per_seq * n;
          ++b;
        }
      }
      if (ok) {
        RowsUnit w{};
        w.je = -1;
        put(w);
      }
    }
    __syncwarp();
    // Zeros for the tiles of batch rows without keys (the whole warp, while the last units are
    // computed), dealt out to all CTAs.
    if (!p.prefix) {
      for (int c = 0; c < p.B; c += 32) {
        unsigned none = __ballot_sync(0xffffffffu, c + lane < p.B && rows_len(p, c + lane) == 0);
        for (; none != 0u; none &= none - 1u) {
          const int seq = c + __ffs(none) - 1;
          for (long long u = blockIdx.x; u < per_seq; u += gridDim.x) {
            const int h = (int)(u / p.tiles), i0 = (int)(u - (long long)h * p.tiles) * kBlockM;
            const int n = min(kBlockM, p.GT - i0);
            const long long row = ((long long)seq * p.Hkv + h) * p.GT + i0;
            for (int i = lane; i < n * (D / 8); i += 32)
              reinterpret_cast<uint4*>(p.o + row * D)[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int i = lane; i < n; i += 32) p.lse[row + i] = -INFINITY;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    // The whole warp: lane i loads box i of a tile (at most eight), whose page it has looked up before
    // the wait for the stage.
    regs_decrease<Cfg::kControl>();
    {
      const uint64_t pol_kv = l2_policy_evict_last();
      const uint64_t pol_q = l2_policy_evict_first();
      constexpr int kLoadStages = kF8 ? R : S;
      uint64_t* full = kF8 ? raw_full : kv_full;
      uint64_t* empty = kF8 ? raw_empty : kv_empty;
      Ring ring;
      uint32_t filled = 0u, fill_par = 0u;      // per stage: ever filled / parity of its last fill
      uint32_t q_par = 3u, q_filled = 0u, q_fill_par = 0u;   // per Q buffer, as in the column-split kernel
      auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool mine = wait_phase(bar, parity, abort_flag, kSiteRowsProducer);
        return __all_sync(0xffffffffu, mine);
      };
      // Block j of the unit's keys: one box, or several that lie one after the other in the tile.
      // Boxes behind the last key are not loaded (their rows are masked, and V's overwritten).
      auto load_kv = [&](bool is_k, const RowsUnit& w, int j) -> bool {
        const int rows = min(kBlockN, w.len - j * kBlockN);
        const bool mine = lane * p.box < rows;
        int id = w.b, row = j * kBlockN + lane * p.box;
        if (p.table != nullptr && mine) {
          const int pg = row / p.page;
          id = __ldg(p.table + pg);
          row -= pg * p.page;
        }
        if (!wait_all(&empty[ring.stage], ring.phase ^ 1u)) return false;
        const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
        uint64_t* bar = &full[ring.stage];
        // a page that is none lies outside the tensor: zeros, and (kF8) exponents of 1
        const bool is_page = (unsigned)id < (unsigned)p.num_pages;
        const int plane = is_page ? id * p.Hkv + w.h : p.num_pages * p.Hkv;
        const unsigned boxes = __popc(__ballot_sync(0xffffffffu, mine));
        uint32_t bytes = boxes * (uint32_t)p.box * (kF8 ? (uint32_t)D : 128u * Plan::kChunks);
        if constexpr (kF8) {
          bytes += __popc(__ballot_sync(0xffffffffu, mine && is_page)) * (uint32_t)p.box;
          if (mine && !is_page) {
            for (int q = 0; q < p.box; q += 16)
              *reinterpret_cast<uint4*>(sExp + ring.stage * kBlockN + lane * p.box + q) =
                  make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
            fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (mine) {
          if constexpr (kF8) {
            tma_load_3d(sRaw + ring.stage * Plan::kRawBytes + lane * p.box * D, map, bar, 0, row, plane, pol_kv);
            if (is_page)
              bulk_load_1d(sExp + ring.stage * kBlockN + lane * p.box,
                           (is_k ? p.ks : p.vs) + ((long long)plane * p.page + row), (uint32_t)p.box, bar);
          } else {
            uint8_t* dst = sKV + ring.stage * Plan::kTileBytes + lane * p.box * 128;
#pragma unroll
            for (int ch = 0; ch < Plan::kChunks; ++ch)
              tma_load_3d(dst + ch * Plan::kChunkBytes, map, bar, ch * 64, row, plane, pol_kv);
          }
        }
        filled |= 1u << ring.stage;
        fill_par = (fill_par & ~(1u << ring.stage)) | (ring.phase << ring.stage);
        ring.advance<kLoadStages>();
        return true;
      };
      // Tiles in the order the MMA warp reads them: K(0), K(1), then V(g), K(g+2) for g = 0, 1, ...
      if (p.behind) wait_for_previous();
      Cursor sc, pc;
      next_unit(sc, false, true, kSiteRowsProducer);
      next_unit(pc, true, true, kSiteRowsProducer);
      bool ok = true;
      for (int i = 0; ok && __all_sync(0xffffffffu, sc.valid || pc.valid); ++i) {
#pragma unroll 1
        for (int half = 0; half < 2 && ok; ++half) {   // V(i-2), then K(i)
          if ((half == 0 && i < 2) || !__all_sync(0xffffffffu, half ? sc.valid : pc.valid)) continue;
          if (half && sc.j == sc.w.jb) {   // the unit's Q tile
            const int qb = (int)(sc.ord - 1u) % Plan::kQBufs;
            if (!(ok = wait_all(&q_empty[qb], (q_par >> qb) & 1u))) break;
            q_par ^= 1u << qb;
            if (lane == 0) {
              mbar_arrive_expect_tx(&q_full[qb], (uint32_t)(p.q_box_rows * 128 * Plan::kChunks));
#pragma unroll
              for (int ch = 0; ch < Plan::kChunks; ++ch)
                tma_load_4d(sQ + qb * Plan::kTileBytes + ch * Plan::kChunkBytes, &tmap_q, &q_full[qb], ch * 64,
                            sc.w.i0, sc.w.h, sc.w.b0, pol_q);
            }
            __syncwarp();
            if (q_filled & (1u << qb)) q_fill_par ^= 1u << qb;
            q_filled |= 1u << qb;
          }
          if (!(ok = load_kv(half != 0, half ? sc.w : pc.w, half ? sc.j : pc.j))) break;
          if (half) {
            if (++sc.j >= sc.w.je) next_unit(sc, false, true, kSiteRowsProducer);
          } else {
            if (++pc.j >= pc.w.je) next_unit(pc, true, true, kSiteRowsProducer);
          }
        }
      }
      // Drain: every issued copy must have landed before the CTA may exit.
      for (int s = 0; s < kLoadStages; ++s)
        if (filled & (1u << s)) drain_phase(&full[s], (fill_par >> s) & 1u, abort_flag);
      for (int t = 0; t < 2; ++t)
        if (q_filled & (1u << t)) drain_phase(&q_full[t], (q_fill_par >> t) & 1u, abort_flag);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the units (warp-uniform control flow); one elected lane issues.
    regs_decrease<Cfg::kControl>();
    {
      Ring ring;
      uint32_t q_par = 0u, of_par = 1u;  // q_par bit qb: parity of the next wait on q_full[qb]
      const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
      const uint64_t desc_q = smem_desc_kmajor_sw128(smem_u32(sQ));
      const uint64_t desc_k = smem_desc_kmajor_sw128(smem_u32(sKV));
      const uint64_t desc_v = smem_desc_mnmajor_sw128(smem_u32(sKV), Plan::kChunkBytes);
      const uint32_t idesc_s = p.idesc_s, idesc_pv = p.idesc_pv;
      auto adv = [](uint64_t d, uint32_t bytes) -> uint64_t { return d + (uint64_t)(bytes >> 4); };
      auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool mine = wait_phase(bar, parity, abort_flag, kSiteRowsMma);
        return __all_sync(0xffffffffu, mine);
      };
      // Rows of the unit's last V tile behind its keys become zeros (the converters do it for kF8;
      // TMA does where the keys end with the tensor).
      auto clear_padding = [&](int first, uint32_t st) {
#pragma unroll 1
        for (int i = first * 8 + lane; i < kBlockN * 8; i += 32)
#pragma unroll
          for (int ch = 0; ch < Plan::kChunks; ++ch)
            st_shared_v4(smem_u32(sKV) + st * Plan::kTileBytes + ch * Plan::kChunkBytes + i * 16, 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      };
      Cursor sc, pc;
      next_unit(sc, false, true, kSiteRowsMma);
      next_unit(pc, true, true, kSiteRowsMma);
      bool ok = true;
      // S(i) goes to score buffer i & 1 after P(i-2) V(i-2) has been issued (issue order).
      for (uint32_t i = 0; ok && __all_sync(0xffffffffu, sc.valid || pc.valid); ++i) {
        if (i >= 2u) {
          const uint32_t g = i - 2u, b = g & 1u, ph = (g >> 1) & 1u;
          if (!__all_sync(0xffffffffu, pc.valid)) break;
          const bool first = pc.j == pc.w.jb, last = pc.j == pc.w.je - 1;
          const uint32_t vst = ring.stage;
          if (!(ok = wait_all(&kv_full[vst], ring.phase))) break;
          ring.advance<S>();
          const int live = pc.w.len - pc.j * kBlockN;
          if (!kF8 && live < kBlockN && !(p.table == nullptr && pc.w.len == p.page)) clear_padding(live, vst);
          if (first) {
            if (!(ok = wait_all(o_free, of_par))) break;
            of_par ^= 1u;
          }
          const uint64_t dv = adv(desc_v, vst * Plan::kTileBytes);
          // O_h += P_h(g) V(g)[64h : 64h+64]: four K = 16 steps, P_h from TMEM (8 columns per step),
          // V as an MN-major operand (16 key rows of 128 bytes per step)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!(ok = wait_all(&p_full[2 * b + h], ph))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_ts(tmem + 256 + 128 * h, tmem + b * 128 + 64 * h + kk * 8, adv(dv, (4 * h + kk) * 2048), idesc_pv,
                       (!first || kk > 0) ? 1u : 0u);
              if (h == 1) {
                tc_commit(pv_done);
                tc_commit(&kv_empty[vst]);
                if (last) tc_commit(o_full);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (++pc.j >= pc.w.je) next_unit(pc, true, true, kSiteRowsMma);
        }
        if (__all_sync(0xffffffffu, sc.valid)) {
          const int qb = (int)(sc.ord - 1u) % Plan::kQBufs;
          const bool last = sc.j == sc.w.je - 1;
          if (sc.j == sc.w.jb) {
            if (!(ok = wait_all(&q_full[qb], (q_par >> qb) & 1u))) break;
            q_par ^= 1u << qb;
          }
          const uint32_t st = ring.stage;
          if (!(ok = wait_all(&kv_full[st], ring.phase))) break;
          ring.advance<S>();
          tc_fence_after();
          const uint64_t da = adv(desc_q, qb * Plan::kTileBytes);
          const uint64_t db = adv(desc_k, st * Plan::kTileBytes);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kSSteps; ++kk) {
              const uint32_t off = (kk >> 2) * Plan::kChunkBytes + (kk & 3) * 32;
              mma_ss(tmem + (i & 1u) * 128, adv(da, off), adv(db, off), idesc_s, kk > 0 ? 1u : 0u);
            }
            tc_commit(&s_full[i & 1u]);
            tc_commit(&kv_empty[st]);
            if (last && sc.w.slot >= 0) tc_commit(&q_empty[qb]);
          }
          __syncwarp();
          if (++sc.j >= sc.w.je) next_unit(sc, false, true, kSiteRowsMma);
        }
      }
      // Drain: all MMAs issued by this warp complete before TMEM is released.
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      drain_phase(drain, 0u, abort_flag);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax warpgroups
    regs_increase<Cfg::kSoftmax>();
    const int h = warp >> 2;                        // score columns 64h .. 64h+63
    const int r = threadIdx.x & 127;                // query row within the tile == TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_o0 = tmem_base + lane_off + 256;  // O_0; O_1 at +128
    const uint32_t t_oh = t_o0 + 128 * h;
    const float c = p.c;
    uint32_t g = 0, o_par = 0;
    bool ok = true;
    int u = 0;
    for (uint32_t ord = 0; ok; ++ord) {
      RowsUnit w;
      if (!__all_sync(0xffffffffu, take(ord, w, kSiteRowsSoftmax)) || w.je < 0) {
        // the end, or a wait that gave up: each warp leaves through one more agreement, which those
        // still in a unit join with its own
        bar_and(7, 2 * kBlockM, false);
        break;
      }
      __syncwarp();
      if (lane == 0) release(ord);
      const long long row = rows_index(p, w.b0, w.i0, w.h, r);
      const int key_lim = w.len - 1;
      float m = -INFINITY, l = 0.f;

#pragma unroll 1
      for (int j = w.jb; j < w.je; ++j, ++g) {
        if (!ok) continue;  // after a failed wait: reach the end-of-unit agreement without further waits
        const uint32_t b = g & 1u;
        if (!(ok = wait_phase(&s_full[b], (g >> 1) & 1u, abort_flag, kSiteRowsSoftmax))) continue;
        tc_fence_after();
        const uint32_t t_s = tmem_base + lane_off + b * 128 + 64 * h;
        float s[64];
        {
          uint32_t a0[32], a1[32];
          tmem_ld32(t_s + 0, a0);
          tmem_ld32(t_s + 32, a1);
          tmem_ld_wait();
          reg_fence32(a0);
          reg_fence32(a1);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            s[i] = __uint_as_float(a0[i]);
            s[32 + i] = __uint_as_float(a1[i]);
          }
        }
        const int k0 = j * kBlockN + 64 * h;
        if (k0 + 63 > key_lim) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (k0 + i > key_lim) s[i] = -INFINITY;
        }
        float mx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max3f(s[e], s[4 + e], s[8 + e]);
#pragma unroll
        for (int i = 12; i < 60; i += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3f(mx[e], s[i + e], s[i + 4 + e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[60 + e]);
        const float m_new = fmaxf(m, fmaxf(max3f(mx[0], mx[1], mx[2]), mx[3]) * c);
        // Lazy correction, as in the column-split kernel.
        bool any_rescale = false;
        float alpha = 1.f;
        if (j == w.jb) {
          m = m_new;
        } else {
          const bool need = m_new > m + kRescaleLog2;
          any_rescale = __any_sync(0xffffffffu, need);
          if (need) {
            alpha = ex2_approx(m - m_new);  // 0 while m is still -inf (no key of this half seen yet)
            l *= alpha;
            m = m_new;
          }
        }
        if (any_rescale) {
          // S(g) completing implies P(g-2) V has; P(g-1) V may still be running.
          if (!(ok = wait_phase(pv_done, (g - 1u) & 1u, abort_flag, kSiteRowsSoftmax))) continue;
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t ov[32];
            tmem_ld32(t_oh + ch * 32, ov);
            tmem_ld_wait();
            reg_fence32(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(t_oh + ch * 32, ov);
          }
        }
        // All exponentials on the special-function unit (the maximum drops a NaN score, its exponential does not).
        // A quarter of the columns on the FMA pipe's polynomial, as the column-split kernel has it, lost: B4 Hq32 Nq2048
        // Nk<=4096 D128 372 us against 359, D96 105 / 101, B8 H32 Nq500 Nk<=1500 D32 66 / 63, D64 41.6 / 41.8.
        const float m_use = (m == -INFINITY) ? 0.f : m;
        {
          const float2 c2 = make_float2(c, c);
          const float2 nm2 = make_float2(-m_use, -m_use);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                           make_float2(0.f, 0.f)};
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            const float2 x = fma2(make_float2(s[i], s[i + 1]), c2, nm2);
            const float2 pr = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            acc[(i >> 1) & 3] = add2(acc[(i >> 1) & 3], pr);
            pk[i >> 1] = pack_bf16x2(pr.x, pr.y);
          }
          tmem_st32(t_s, pk);
          const float2 a = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
          l += a.x + a.y;
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * b + h]);
      }

      // ---- end of the unit: agree on success, exchange (m_h, l_h), join and write O and LSE.
      if (ok) ok = wait_phase(o_full, o_par, abort_flag, kSiteRowsEpilogue);
      o_par ^= 1u;
      xml[((u & 1) * 2 + h) * kBlockM + r] = make_float2(m, l);
      ok = bar_and(7, 2 * kBlockM, ok);
      if (!ok) break;
      const float2 ml0 = xml[((u & 1) * 2 + 0) * kBlockM + r];
      const float2 ml1 = xml[((u & 1) * 2 + 1) * kBlockM + r];
      const float mt = fmaxf(ml0.x, ml1.x);
      const float a0 = (ml0.x == -INFINITY) ? 0.f : ex2_approx(ml0.x - mt);
      const float a1 = (ml1.x == -INFINITY) ? 0.f : ex2_approx(ml1.x - mt);
      const float lt = fmaf(ml1.y, a1, ml0.y * a0);
      const float inv_l = w.slot >= 0 ? 1.f : 1.f / lt;
      const float w0 = a0 * inv_l, w1 = a1 * inv_l;
      tc_fence_after();
      if (h >= Plan::kOChunks) {
        // no output chunk for this warpgroup (D = 32): its O columns are not read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
      const uint32_t stage_row = smem_u32(sQ + (u & 1) * Plan::kTileBytes) + r * 64;
#pragma unroll 1
      for (int ch = h; ch < Plan::kOChunks; ch += 2) {
        uint32_t x0[32], x1[32];
        tmem_ld32(t_o0 + ch * 32, x0);
        tmem_ld32(t_o0 + 128 + ch * 32, x1);
        tmem_ld_wait();
        reg_fence32(x0);
        reg_fence32(x1);
        if (ch + 2 >= Plan::kOChunks) {
          // this warpgroup's last reads of O: the next unit's P V may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = fmaf(__uint_as_float(x1[i]), w1, __uint_as_float(x0[i]) * w0);
        if (w.slot >= 0) {
          float4* dst = reinterpret_cast<float4*>(p.slot_o + ((long long)w.slot * kBlockM + r) * D + ch * 32);
          if (row >= 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        } else {
          // staged in this unit's Q buffer (its last S has completed), 64-byte swizzle, as in the
          // column-split kernel
          const uint32_t row_addr = stage_row + ch * Plan::kStageBytes;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            st_shared_v4(row_addr + ((q ^ ((r >> 1) & 3)) << 4), pack_bf16x2(x[8 * q], x[8 * q + 1]),
                         pack_bf16x2(x[8 * q + 2], x[8 * q + 3]), pack_bf16x2(x[8 * q + 4], x[8 * q + 5]),
                         pack_bf16x2(x[8 * q + 6], x[8 * q + 7]));
        }
      }
      if (w.slot >= 0) {
        if (h == 0) p.slot_ml[(long long)w.slot * kBlockM + r] = make_float2(mt, lt);
      } else {
        // make the staged rows visible to the TMA (async proxy), then hand them to the store warp
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_staged[u & 1]);
        if (h == 0 && row >= 0) p.lse[row] = (mt + log2f(lt)) * 0.69314718055994530942f;
      }
      ++u;
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ output store warp (cross attention)
    // Per whole unit: wait until both softmax warpgroups have staged O in the unit's Q buffer, store
    // it with TMA tensor stores (rows past the tensor are not written), wait until the stores have
    // read the buffer and give it back to the producer.
    regs_decrease<Cfg::kControl>();
    if (lane == 0 && !p.prefix) {
      uint32_t st_par = 0u;  // bit qb: parity of the next wait on o_staged[qb]
      Cursor c;
      for (next_unit(c, true, false, kSiteRowsStore); c.valid; next_unit(c, true, false, kSiteRowsStore)) {
        if (c.w.slot >= 0) continue;
        const int qb = (int)(c.ord - 1u) & 1;
        if (!wait_phase(&o_staged[qb], (st_par >> qb) & 1u, abort_flag, kSiteRowsStore)) break;
        st_par ^= 1u << qb;
        const uint8_t* stage = sQ + qb * Plan::kTileBytes;
#pragma unroll
        for (int ch = 0; ch < Plan::kOChunks; ++ch)
          tma_store_3d(&tmap_o, stage + ch * Plan::kStageBytes, ch * 32, c.w.i0, c.w.b * p.Hkv + c.w.h);
        bulk_commit_group();
        bulk_wait_group_read0();
        mbar_arrive(&q_empty[qb]);
      }
      // every TMA store has completed before the CTA exits
      bulk_wait_group0();
    }
    __syncwarp();
  } else if constexpr (kF8) {
    // ------------------------------------------------------------ converters: E4M3 -> bf16 tiles
    // Warpgroup c (0, 1) takes the tiles of its parity in the order of the ring.  A 128-row tile takes
    // kPasses passes; in each, kLanes lanes share a row (16 codes each).
    regs_decrease<Cfg::kConvert>();
    constexpr int kLanes = D / 16;                    // 2, 4, 6, 8
    constexpr int kRows = 128 / kLanes / 16 * 16;     // 64, 32, 16 (96 of the 128 threads), 16
    constexpr int kPasses = kBlockN / kRows;
    constexpr int kBatch = kPasses < 4 ? kPasses : 4;   // passes at a time (registers)
    const uint32_t group = (uint32_t)(warp - 12) >> 2;
    const int tid = (threadIdx.x - 384) & 127;
    // This thread's row of a pass and its columns.  D = 128, where shared memory's bandwidth bounds the
    // block (S reads 64 KB, P V 32, the conversion 96, all at 128 bytes a clock): the raw rows are
    // 128-byte swizzled too, and the eight lanes of a 128-byte access take one 64-column chunk of rows r
    // and r ^ 5, whose swizzles send their pieces to different banks in both layouts.
    constexpr bool kPairs = D == 128;
    int pr = tid / kLanes, col = (tid - pr * kLanes) * 16;
    if constexpr (kPairs) {
      const int pair = tid >> 3;   // 16: eight row pairs, two chunks
      pr = ((pair >> 1 & 3) | (pair >> 1 & 4) << 1) ^ ((tid >> 2 & 1) ? 5 : 0);
      col = (pair & 1) * 64 + (tid & 3) * 16;
    }
    const bool mine = pr < kRows;
    const uint32_t at = (uint32_t)((col >> 6) * Plan::kChunkBytes), q = (uint32_t)(col & 63) >> 3;
    Ring ring, raw;
    uint32_t tile = 0u;
    bool ok = true;
    auto convert = [&](int len, int j) -> bool {
      if (!wait_phase(&raw_full[raw.stage], raw.phase, abort_flag, kSiteRowsConvert)) return false;
      if (!wait_phase(&kv_empty[ring.stage], ring.phase ^ 1u, abort_flag, kSiteRowsConvert)) return false;
      const uint8_t* codes = sRaw + raw.stage * Plan::kRawBytes;
      const uint8_t* exps = sExp + raw.stage * kBlockN;
      const uint32_t base = smem_u32(sKV) + ring.stage * Plan::kTileBytes + at;
#pragma unroll 1
      for (int p0 = 0; p0 < kPasses; p0 += kBatch) {
        uint4 x[kBatch];
        uint32_t e[kBatch], top = 0u;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = (p0 + i) * kRows + pr;
          const bool live = mine && j * kBlockN + r < len;
          x[i] = live ? *reinterpret_cast<const uint4*>(codes + r * D + (kPairs ? col ^ ((r & 7) << 4) : col))
                      : make_uint4(0u, 0u, 0u, 0u);
          e[i] = live ? exps[r] : 127u;
          top = max(top, e[i]);
        }
        // bits -> value * 2^-120, times 2^(e - 7) in one multiplication while that is a bf16 number,
        // else (exponents above 2^7, and rows marked NaN) times 2^120 and the scale
        const bool far = __any_sync(0xffffffffu, top > 134u);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = (p0 + i) * kRows + pr;
          const uint32_t f = far ? 0x7b807b80u : (e[i] + 120u) * 0x00800080u;
          uint2 y[4] = {e4m3x4_scaled(x[i].x, f), e4m3x4_scaled(x[i].y, f), e4m3x4_scaled(x[i].z, f),
                        e4m3x4_scaled(x[i].w, f)};
          if (far) {
            const uint32_t f2 = e8_bf16x2((int)e[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = make_uint2(mul_bf16x2(y[k].x, f2), mul_bf16x2(y[k].y, f2));
          }
          if (mine) {
            const uint32_t row = base + r * 128;
            st_shared_v4(row + ((q ^ (r & 7)) << 4), y[0].x, y[0].y, y[1].x, y[1].y);
            st_shared_v4(row + (((q + 1) ^ (r & 7)) << 4), y[2].x, y[2].y, y[3].x, y[3].y);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&raw_empty[raw.stage]);
        mbar_arrive(&kv_full[ring.stage]);
      }
      return true;
    };
    Cursor sc, pc;
    next_unit(sc, false, true, kSiteRowsConvert);
    next_unit(pc, true, true, kSiteRowsConvert);
    for (int i = 0; ok && __all_sync(0xffffffffu, sc.valid || pc.valid); ++i) {
      // V(i-2), then K(i): one copy of the code serves both
#pragma unroll 1
      for (int half = 0; half < 2 && ok; ++half) {
        if ((half == 0 && i < 2) || !__all_sync(0xffffffffu, half ? sc.valid : pc.valid)) continue;
        if ((tile & 1u) == group)
          ok = __all_sync(0xffffffffu, convert(half ? sc.w.len : pc.w.len, half ? sc.j : pc.j));
        ++tile;
        raw.advance<R == 0 ? 1 : R>();
        ring.advance<S>();
        if (!ok) break;
        if (half) {
          if (++sc.j >= sc.w.je) next_unit(sc, false, true, kSiteRowsConvert);
        } else {
          if (++pc.j >= pc.w.je) next_unit(pc, true, true, kSiteRowsConvert);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Cross attention: joins the parts of every unit that was split, in key order, into O and LSE.  Block
// (c, y): the unit at the end of CTA c's range, where its first part is in that range; 32 rows a block,
// four a warp, whose loads stand side by side (one row after another, most of the kernel's 13 us for
// 9 MB was the chain of their latencies).
template <int D>
__global__ void __launch_bounds__(256) attn_rows_join_kernel(const RowsParams p, unsigned ctas) {
  __shared__ int4 unit_s;
  __shared__ long long place_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    int b;
    long long first;
    const long long c = blockIdx.x;
    const RowsLine ln = rows_locate(p, ctas, c + 1, -1, b, first);
    const long long x = (c + 1) * ln.share;
    int n = 0;
    RowsUnit w{};
    long long u0 = 0;
    if (x < ln.total) {
      const int places = rows_places(rows_blocks(rows_len(p, b)));
      const int unit = (int)((x - first) / places);
      u0 = first + (long long)unit * places;
      // split here (the unit's first block is before x, in range c), and not before
      if (u0 + kRowsOver < x && (u0 + kRowsOver) / ln.share == c) {
        n = (int)((u0 + places - 1) / ln.share - c) + 1;
        const int h = unit / p.tiles;
        rows_tile(p, b, h, unit - h * p.tiles, w);
      }
    }
    if (lane == 0) {
      unit_s = make_int4(w.b0, w.i0, w.h, n);
      place_s = 2 * c + (u0 > c * ln.share ? 1 : 0);
    }
  }
  __syncthreads();
  const int4 unit = unit_s;
  const long long first_slot = place_s, c0 = blockIdx.x;
  const int n = unit.w;
  // what follows in the stream waits for this kernel alone, so some block always waits for the one before
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) wait_for_previous();
  if (n == 0) return;
  // rows r0 + 8 i of the unit (those that are none come last); lane (i, k): part k of row i
  const int r0 = blockIdx.y * 32 + warp, part = lane & 7;
  long long row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = rows_index(p, unit.x, unit.y, unit.z, r0 + 8 * i);
  if (row[0] < 0) return;
  wait_for_previous();
  float m = -INFINITY, l = 0.f;   // of row lane / 8
  float acc[4][D / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < D / 32; ++e) acc[i][e] = 0.f;
  auto slot_row = [&](int k) { return (k == 0 ? first_slot : 2 * (c0 + k)) * kBlockM + r0; };   // of row 0
  for (int k0 = 0; k0 < n; k0 += 8) {
    const float2 ml = k0 + part < n ? p.slot_ml[slot_row(k0 + part) + 8 * (lane >> 3)] : make_float2(-INFINITY, 0.f);
    float mn = ml.x;
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
    mn = fmaxf(m, mn);
    const float a = dec_weight(make_float2(m, l), mn), w = dec_weight(ml, mn);
    float sum = ml.y * w;
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    m = mn;
    l = fmaf(l, a, sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float ai = __shfl_sync(0xffffffffu, a, 8 * i);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[i][e] *= ai;
    }
    const int here = min(8, n - k0);
#pragma unroll 2
    for (int k = 0; k < here; ++k) {
      const float* o = p.slot_o + slot_row(k0 + k) * D + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float wk = __shfl_sync(0xffffffffu, w, 8 * i + k);
        if (row[i] >= 0)
#pragma unroll
          for (int e = 0; e < D / 32; ++e) acc[i][e] = fmaf(o[8 * i * D + 32 * e], wk, acc[i][e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float inv = 1.f / __shfl_sync(0xffffffffu, l, 8 * i);
    if (row[i] < 0) continue;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) p.o[row[i] * D + 32 * e + lane] = __float2bfloat16_rn(acc[i][e] * inv);
  }
  if (part == 0) {
    const long long mine = rows_index(p, unit.x, unit.y, unit.z, r0 + 8 * (lane >> 3));
    if (mine >= 0) p.lse[mine] = dec_lse(m, l);
  }
}

}  // namespace attn
