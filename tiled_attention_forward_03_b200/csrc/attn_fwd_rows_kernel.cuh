// attn_fwd_rows_kernel.cuh -- attention of many query rows to keys of another length on B200
// (sm_100a): cross attention, and the prefix that a decoding batch shares.
//
// The same computation as attn_fwd_colsplit_kernel.cuh -- one 128-row tile per unit, two score
// buffers, each 128-key block's columns split between two softmax warpgroups with maxima, sums and
// accumulators of their own, joined exactly at the end of the unit -- without a causal mask, and
// with rows and keys that come from elsewhere:
//
//  * Rows.  All query rows that see the same keys may share a tile: the group * Nq rows of a KV head
//    (contiguous in q), or for a shared prefix those of several sequences, which a four-dimensional
//    TMA box (columns, rows of a sequence, head, sequences) lays one after the other.
//  * Keys, bf16: contiguous, or in pages, by TMA boxes of the largest of 128, 64, 32, 16 rows that
//    divides a page.  Each batch row has its own count of them; the MMA warp overwrites the last
//    value tile's rows behind it with zeros (its probabilities are 0, and 0 * NaN would not be).
//  * Keys, E4M3 (kF8): a fourth warpgroup loads codes and exponents, converts them to bf16 exactly
//    (a power-of-two scale rounds nothing) and stores them as TMA would, 128-byte swizzled; the next
//    tile's loads are in flight meanwhile.  Converting once per 128 rows costs less than the
//    exponentials of the same block, which bound the kernel, so it is hidden.
//  * Results: O (bf16) and LSE; or (kPart) unnormalised fp32 O, maximum and sum of the unit's part
//    of the keys, which a second kernel joins: used when the units alone would not fill the GPU and
//    for prefixes.
//
//   warps 0-3, 4-7  softmax warpgroups     warp 8  TMA producer (kF8: Q only)     warp 9  MMA issuer
//   warp 10  output store (not kPart)      warp 11 idle      warps 12-15 (kF8) converters
//
// Every mbarrier wait is bounded; named barriers are only reached by all their participants.
#pragma once

#include <cuda_bf16.h>

#include "attn_cache_kernel.cuh"
#include "attn_fwd_colsplit_kernel.cuh"

namespace attn {

enum : unsigned {
  kSiteRowsProducer = 41,
  kSiteRowsMma = 42,
  kSiteRowsSoftmax = 43,
  kSiteRowsEpilogue = 44,
  kSiteRowsStore = 45,
  kSiteRowsConvert = 46,
};

// Register split.  bf16: the forward kernel's (384 threads at 168).  kF8: 512 threads at 128;
// 2 * 128 * 168 + 128 * 56 + 128 * 120 == 512 * 128.
template <bool kF8>
struct RowsCfg {
  static constexpr int kThreads = kF8 ? 512 : 384;
  static constexpr int kRegsLaunch = kF8 ? 128 : kRegsAtLaunch;
  static constexpr int kSoftmax = kF8 ? 168 : kRegsSoftmax;
  static constexpr int kControl = kRegsControl;
  static constexpr int kConvert = 120;
  static_assert(2 * 128 * kSoftmax + 128 * kControl + (kF8 ? 128 * kConvert : 0) <= kThreads * kRegsLaunch,
                "register split exceeds the launch allocation");
};

struct RowsParams {
  float* lse;                // [B][Hkv][GT]
  __nv_bfloat16* o;          // rows without a key are zeroed directly
  float* part_o;             // kPart: [parts][B*Hkv*GT][D]
  float2* part_ml;           // kPart: [parts][B*Hkv*GT]
  int B, Hkv, GT;
  int num_units;             // key groups * parts * tiles
  int tiles, parts;
  int prefix;                // 0: a key group is (b, h); 1: it is h, with rows of all sequences
  int seqs;                  // sequences in a tile (prefix; else 1)
  int seq_tiles;             // tiles of a sequence (prefix with GT > 128; else 1)
  int q_box_rows;            // rows a Q tile load fills: min(GT, 128) * seqs (box 128 rows when seqs == 1)
  const int* k_lens;         // [B] or null
  int len_all;               // keys where k_lens is null
  int max_len;               // keys there is room for
  // paged keys
  const int* table;          // or null: page b
  int page, num_pages;
  int box;                   // key rows of a TMA box
  const void* k;             // kF8: codes and exponents
  const void* v;
  const uint8_t* ks;
  const uint8_t* vs;
  float c;                   // |scale| * log2(e)
  uint32_t idesc_s;          // S = Q K^T: 128 x 128 x D (negates A when scale < 0)
  uint32_t idesc_pv;         // O_h += P_h V_h: 128 x D x 64
};

struct RowsUnit {
  int b0, i0, h;  // first sequence, first row and head of the tile
  int b;          // sequence of the keys (cross)
  int part;
  int jb, je;     // 128-key blocks
  int len;        // keys
};

__device__ __forceinline__ void rows_unit(const RowsParams& p, int u, RowsUnit& w) {
  const int per_group = p.tiles * p.parts;
  const int group = u / per_group;
  int r = u - group * per_group;
  w.part = r / p.tiles;
  const int tile = r - w.part * p.tiles;
  if (p.prefix) {
    w.h = group;
    w.b = 0;
    w.b0 = p.seq_tiles > 1 ? tile / p.seq_tiles : tile * p.seqs;
    w.i0 = p.seq_tiles > 1 ? (tile - w.b0 * p.seq_tiles) * kBlockM : 0;
  } else {
    w.b = w.b0 = group / p.Hkv;
    w.h = group - w.b * p.Hkv;
    w.i0 = tile * kBlockM;
  }
  w.len = p.k_lens != nullptr ? __ldg(p.k_lens + w.b) : p.len_all;
  w.len = max(0, min(w.len, p.max_len));
  const long long nb = ((long long)w.len + kBlockN - 1) / kBlockN;
  w.jb = (int)(nb * w.part / p.parts);
  w.je = (int)(nb * (w.part + 1) / p.parts);
}

// Row r of the tile: its index in q, o, lse, or -1 where the tile has no such row.
__device__ __forceinline__ long long rows_index(const RowsParams& p, const RowsUnit& w, int r) {
  int b = w.b0, i = w.i0 + r;
  if (p.prefix && p.seq_tiles == 1) {
    const int s = r / p.GT;
    if (s >= p.seqs) return -1;
    b += s;
    i -= s * p.GT;
  }
  if (b >= p.B || i >= p.GT) return -1;
  return ((long long)b * p.Hkv + w.h) * p.GT + i;
}

// Position in the CTA's sequence of (unit, key block) pairs; units without a block are skipped.
struct RowsCursor {
  int next;       // next unit index
  RowsUnit w;
  int j = 0;
  int u = -1;     // ordinal of the current unit among this CTA's units with blocks
  bool valid = false;
};

__device__ __forceinline__ void rows_next_unit(const RowsParams& p, RowsCursor& c) {
  for (; c.next < p.num_units;) {
    rows_unit(p, c.next, c.w);
    c.next += (int)gridDim.x;
    if (c.w.jb < c.w.je) {
      c.valid = true;
      c.j = c.w.jb;
      ++c.u;
      return;
    }
  }
  c.valid = false;
}

__device__ __forceinline__ void rows_advance(const RowsParams& p, RowsCursor& c) {
  if (++c.j >= c.w.je) rows_next_unit(p, c);
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

template <int D, bool kPart, bool kF8>
__global__ void __launch_bounds__(RowsCfg<kF8>::kThreads, 1)
    attn_fwd_rows_sm100(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                        const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_o,
                        const RowsParams p) {
  using Plan = CsPlan<D>;
  using Cfg = RowsCfg<kF8>;
  constexpr int S = Plan::kStages;
  constexpr int kSSteps = D / 16;  // K = 16 steps of S = Q K^T
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);

  uint8_t* sQ = smem + Plan::kQOff;
  uint8_t* sKV = smem + Plan::kKVOff;
  float2* xml = reinterpret_cast<float2*>(smem + Plan::kXOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Plan::kBarOff);
  uint64_t* q_full = bars;                 // [2]
  uint64_t* q_empty = bars + 2;            // [2]: released by the store warp, or (kPart) after the unit's last S
  uint64_t* o_staged = bars + 4;           // [2]: the unit's O is staged in Q buffer [qb]
  uint64_t* kv_full = bars + 6;            // [S]
  uint64_t* kv_empty = kv_full + S;        // [S]
  uint64_t* s_full = kv_empty + S;         // [2]
  uint64_t* p_full = s_full + 2;           // [2 buffers][2 halves]
  uint64_t* pv_done = p_full + 4;
  uint64_t* o_full = pv_done + 1;
  uint64_t* o_free = pv_done + 2;
  uint64_t* drain = pv_done + 3;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Plan::kMiscOff);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Plan::kMiscOff + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&o_staged[i], 2 * kBlockM);
      mbar_init(&s_full[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], kBlockM);
    for (int i = 0; i < S; ++i) {
      mbar_init(&kv_full[i], kF8 ? 128 : 1);
      mbar_init(&kv_empty[i], 1);
    }
    mbar_init(pv_done, 1);
    mbar_init(o_full, 1);
    mbar_init(o_free, 2 * kBlockM);
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmap_q);
    if (!kF8) {
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
    }
    if (!kPart) tma_prefetch_desc(&tmap_o);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    regs_decrease<Cfg::kControl>();
    if (lane == 0) {
      const uint64_t pol_kv = l2_policy_evict_last();
      const uint64_t pol_q = l2_policy_evict_first();
      Ring ring;
      uint32_t filled = 0u, fill_par = 0u;      // per stage: ever filled / parity of its last fill
      uint32_t q_par = 3u, q_filled = 0u, q_fill_par = 0u;   // per Q buffer, as in the column-split kernel
      // Block j of the unit's keys: one box, or several that lie one after the other in the tile.
      // Boxes behind the last key are not loaded (their rows are masked, and V's overwritten).
      auto load_kv = [&](const CUtensorMap* map, const RowsUnit& w, int j) -> bool {
        if (!wait_phase(&kv_empty[ring.stage], ring.phase ^ 1u, abort_flag, kSiteRowsProducer)) return false;
        const int rows = min(kBlockN, w.len - j * kBlockN);
        const int boxes = (rows + p.box - 1) / p.box;
        mbar_arrive_expect_tx(&kv_full[ring.stage], (uint32_t)(boxes * p.box * 128 * Plan::kChunks));
        uint8_t* dst = sKV + ring.stage * Plan::kTileBytes;
        for (int i = 0; i < boxes; ++i) {
          const int pos = j * kBlockN + i * p.box;
          int id = w.b, row = pos;
          if (p.table != nullptr) {
            const int pg = pos / p.page;
            id = __ldg(p.table + pg);
            row = pos - pg * p.page;
          }
          // a page that is none lies outside the tensor: zeros
          const int plane = (unsigned)id < (unsigned)p.num_pages ? id * p.Hkv + w.h : p.num_pages * p.Hkv;
#pragma unroll
          for (int ch = 0; ch < Plan::kChunks; ++ch)
            tma_load_3d(dst + ch * Plan::kChunkBytes + i * p.box * 128, map, &kv_full[ring.stage], ch * 64, row, plane,
                        pol_kv);
        }
        filled |= 1u << ring.stage;
        fill_par = (fill_par & ~(1u << ring.stage)) | (ring.phase << ring.stage);
        ring.advance<S>();
        return true;
      };
      // The unit's Q tile when the block is its first, then (bf16) the block's K.
      auto load_k = [&](const RowsCursor& c) -> bool {
        if (c.j == c.w.jb) {
          const int qb = c.u & 1;
          if (!wait_phase(&q_empty[qb], (q_par >> qb) & 1u, abort_flag, kSiteRowsProducer)) return false;
          q_par ^= 1u << qb;
          mbar_arrive_expect_tx(&q_full[qb], (uint32_t)(p.q_box_rows * 128 * Plan::kChunks));
#pragma unroll
          for (int ch = 0; ch < Plan::kChunks; ++ch)
            tma_load_4d(sQ + qb * Plan::kTileBytes + ch * Plan::kChunkBytes, &tmap_q, &q_full[qb], ch * 64, c.w.i0,
                        c.w.h, c.w.b0, pol_q);
          if (q_filled & (1u << qb)) q_fill_par ^= 1u << qb;
          q_filled |= 1u << qb;
        }
        return kF8 ? true : load_kv(&tmap_k, c.w, c.j);
      };
      RowsCursor sc, pc;
      sc.next = pc.next = (int)blockIdx.x;
      rows_next_unit(p, sc);
      bool ok = true;
      if constexpr (kF8) {
        while (ok && sc.valid) {
          ok = load_k(sc);
          rows_next_unit(p, sc);
        }
      } else {
        rows_next_unit(p, pc);
        // The order the MMA warp reads the ring in: K(0), K(1), then V(g), K(g+2) for g = 0, 1, ...
        for (int i = 0; i < 2 && ok && sc.valid; ++i) {
          ok = load_k(sc);
          rows_advance(p, sc);
        }
        while (ok && pc.valid) {
          ok = load_kv(&tmap_v, pc.w, pc.j);
          if (ok && sc.valid) {
            ok = load_k(sc);
            rows_advance(p, sc);
          }
          rows_advance(p, pc);
        }
      }
      // Drain: every issued copy must have landed before the CTA may exit.
      for (int s = 0; s < S; ++s)
        if (filled & (1u << s)) drain_phase(&kv_full[s], (fill_par >> s) & 1u, abort_flag);
      for (int t = 0; t < 2; ++t)
        if (q_filled & (1u << t)) drain_phase(&q_full[t], (q_fill_par >> t) & 1u, abort_flag);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer (as the column-split kernel's)
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
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) tc_commit(bar);
        __syncwarp();
      };
      auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool mine = wait_phase(bar, parity, abort_flag, kSiteRowsMma);
        return __all_sync(0xffffffffu, mine);
      };
      auto next_stage = [&](bool& ok) -> uint32_t {
        const uint32_t st = ring.stage;
        ok = wait_all(&kv_full[st], ring.phase);
        ring.advance<S>();
        return st;
      };
      uint32_t gs = 0;  // blocks whose S has been issued
      auto issue_s = [&](const RowsCursor& c) -> bool {
        const int qb = c.u & 1;
        if (c.j == c.w.jb) {
          if (!wait_all(&q_full[qb], (q_par >> qb) & 1u)) return false;
          q_par ^= 1u << qb;
        }
        bool ok;
        const uint32_t st = next_stage(ok);
        if (!ok) return false;
        tc_fence_after();
        const uint64_t da = adv(desc_q, qb * Plan::kTileBytes);
        const uint64_t db = adv(desc_k, st * Plan::kTileBytes);
        const uint32_t d_tmem = tmem + (gs & 1u) * 128;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kSSteps; ++kk) {
            const uint32_t off = (kk >> 2) * Plan::kChunkBytes + (kk & 3) * 32;
            mma_ss(d_tmem, adv(da, off), adv(db, off), idesc_s, kk > 0 ? 1u : 0u);
          }
        }
        __syncwarp();
        commit(&s_full[gs & 1u]);
        commit(&kv_empty[st]);
        if (kPart && c.j == c.w.je - 1) commit(&q_empty[qb]);
        ++gs;
        return true;
      };
      auto issue_pv = [&](int h, uint32_t sbuf, uint32_t vst, bool accumulate) {
        const uint64_t dv = adv(desc_v, vst * Plan::kTileBytes);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(tmem + 256 + 128 * h, tmem + sbuf * 128 + 64 * h + kk * 8, adv(dv, (4 * h + kk) * 2048),
                   idesc_pv, (accumulate || kk > 0) ? 1u : 0u);
        }
        __syncwarp();
      };
      // Rows of the unit's last V tile behind its keys become zeros (the converters do it for kF8;
      // TMA does where the keys end with the tensor).
      auto clear_padding = [&](const RowsCursor& c, uint32_t st) {
        const int first = c.w.len - c.j * kBlockN;
        if (kF8 || first >= kBlockN || (p.table == nullptr && c.w.len == p.page)) return;
        for (int i = first * 8 + lane; i < kBlockN * 8; i += 32)
#pragma unroll
          for (int ch = 0; ch < Plan::kChunks; ++ch)
            st_shared_v4(smem_u32(sKV) + st * Plan::kTileBytes + ch * Plan::kChunkBytes + i * 16, 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      };

      RowsCursor sc, pc;
      sc.next = pc.next = (int)blockIdx.x;
      rows_next_unit(p, sc);
      rows_next_unit(p, pc);
      bool ok = true;
      for (int i = 0; i < 2 && ok && sc.valid; ++i) {
        ok = issue_s(sc);
        rows_advance(p, sc);
      }
      uint32_t gp = 0;  // blocks whose P V has been issued
      while (ok && pc.valid) {
        const uint32_t b = gp & 1u, ph = (gp >> 1) & 1u;
        const bool first = pc.j == pc.w.jb;
        if (!(ok = wait_all(&p_full[2 * b], ph))) break;
        if (first) {
          if (!(ok = wait_all(o_free, of_par))) break;
          of_par ^= 1u;
        }
        const uint32_t vst = next_stage(ok);
        if (!ok) break;
        clear_padding(pc, vst);
        tc_fence_after();
        issue_pv(0, b, vst, !first);
        if (!(ok = wait_all(&p_full[2 * b + 1], ph))) break;
        tc_fence_after();
        issue_pv(1, b, vst, !first);
        commit(pv_done);
        commit(&kv_empty[vst]);
        if (pc.j == pc.w.je - 1) commit(o_full);
        if (sc.valid) {
          if (!(ok = issue_s(sc))) break;
          rows_advance(p, sc);
        }
        ++gp;
        rows_advance(p, pc);
      }
      // Drain: all MMAs issued by this warp complete before TMEM is released.
      commit(drain);
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
    for (int unit = blockIdx.x; ok && unit < p.num_units; unit += (int)gridDim.x) {
      RowsUnit w;
      rows_unit(p, unit, w);
      const long long row = rows_index(p, w, r);
      if (w.jb == w.je) {
        // no keys (in this part): nothing is computed, the row's result is empty
        if (row >= 0) {
          if constexpr (kPart) {
            if (h == 0) p.part_ml[(long long)w.part * p.B * p.Hkv * p.GT + row] = make_float2(-INFINITY, 0.f);
          } else {
            for (int ch = h; ch < Plan::kOChunks; ch += 2)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                reinterpret_cast<uint4*>(p.o + row * D + ch * 32)[q] = make_uint4(0u, 0u, 0u, 0u);
            if (h == 0) p.lse[row] = -INFINITY;
          }
        }
        continue;
      }
      const int key_lim = w.len - 1;
      float m = -INFINITY, l = 0.f;

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
#pragma unroll
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
            float2 pr;
            if (((i >> 1) & 7) < poly_pairs_per8<D>()) {
              pr = exp2_poly2(x);
            } else {
              pr.x = ex2_approx(x.x);
              pr.y = ex2_approx(x.y);
            }
            acc[(i >> 1) & 3] = add2(acc[(i >> 1) & 3], pr);
            pk[i >> 1] = pack_bf16x2(pr.x, pr.y);
          }
          tmem_st32(t_s, pk);
          const float2 a = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
          l += a.x + a.y;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[2 * b + h]);
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
      const float inv_l = kPart ? 1.f : 1.f / lt;
      const float w0 = a0 * inv_l, w1 = a1 * inv_l;
      tc_fence_after();
      if (h >= Plan::kOChunks) {
        // no output chunk for this warpgroup (D = 32): its O columns are not read
        tc_fence_before();
        mbar_arrive(o_free);
      }
      const uint32_t stage_row = smem_u32(sQ + (u & 1) * Plan::kTileBytes) + r * 64;
#pragma unroll
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
          mbar_arrive(o_free);
        }
        auto joined = [&](int i) { return fmaf(__uint_as_float(x1[i]), w1, __uint_as_float(x0[i]) * w0); };
        if constexpr (kPart) {
          if (row >= 0) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + ((long long)w.part * p.B * p.Hkv * p.GT + row) * D + ch * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(joined(4 * i), joined(4 * i + 1), joined(4 * i + 2), joined(4 * i + 3));
          }
        } else {
          // staged in this unit's Q buffer, 64-byte swizzle, as in the column-split kernel
          uint32_t packed[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) packed[i] = pack_bf16x2(joined(2 * i), joined(2 * i + 1));
          const uint32_t row_addr = stage_row + ch * Plan::kStageBytes;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            st_shared_v4(row_addr + ((q ^ ((r >> 1) & 3)) << 4), packed[4 * q], packed[4 * q + 1], packed[4 * q + 2],
                         packed[4 * q + 3]);
        }
      }
      if constexpr (kPart) {
        if (h == 0 && row >= 0) p.part_ml[(long long)w.part * p.B * p.Hkv * p.GT + row] = make_float2(mt, lt);
      } else {
        // make the staged rows visible to the TMA (async proxy), then hand them to the store warp
        fence_proxy_async_smem();
        mbar_arrive(&o_staged[u & 1]);
        if (h == 0 && row >= 0) p.lse[row] = (mt + log2f(lt)) * 0.69314718055994530942f;
      }
      ++u;
    }
  } else if (warp == 10 && !kPart) {
    // ------------------------------------------------------------ output store warp (as the column-split kernel's)
    regs_decrease<Cfg::kControl>();
    if (lane == 0) {
      uint32_t st_par = 0u;  // bit qb: parity of the next wait on o_staged[qb]
      RowsCursor c;
      c.next = (int)blockIdx.x;
      for (rows_next_unit(p, c); c.valid; rows_next_unit(p, c)) {
        const int qb = c.u & 1;
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
  } else if (warp < 12) {
    regs_decrease<Cfg::kControl>();
  } else if constexpr (kF8) {
    // ------------------------------------------------------------ converters: E4M3 pages -> bf16 tiles
    // A 128-row tile takes kPasses passes; in each, kLanes lanes share a row (16 codes each) and the
    // warpgroup covers kRows rows, a whole number of 16-row groups or a whole fraction of one.
    regs_decrease<Cfg::kConvert>();
    constexpr int kLanes = D / 16;                    // 2, 4, 6, 8
    constexpr int kRows = kLanes == 6 ? 16 : 128 / kLanes;   // D = 96: 96 of the 128 threads have a piece
    constexpr int kPasses = kBlockN / kRows;
    const int tid = threadIdx.x - 384;
    const int pr = tid / kLanes, piece = tid - pr * kLanes;
    const bool mine = pr < kRows;
    Ring ring;
    bool ok = true;
    auto load_tile = [&](const RowsCursor& c, bool is_k, uint4 (&w)[kPasses], uint32_t (&e)[kPasses]) {
      const uint8_t* codes = static_cast<const uint8_t*>(is_k ? p.k : p.v);
      const uint8_t* exps = is_k ? p.ks : p.vs;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int pos = c.j * kBlockN + i * kRows + pr;
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        e[i] = 127u;
        if (!mine || pos >= c.w.len) continue;
        const int pg = pos / p.page;
        const int id = __ldg(p.table + pg);
        if ((unsigned)id >= (unsigned)p.num_pages) continue;
        const long long row = ((long long)id * p.Hkv + c.w.h) * p.page + (pos - pg * p.page);
        w[i] = __ldg(reinterpret_cast<const uint4*>(codes + row * D) + piece);
        e[i] = __ldg(exps + row);
      }
    };
    auto store_tile = [&](const uint4 (&w)[kPasses], const uint32_t (&e)[kPasses]) {
      ok = ok && wait_phase(&kv_empty[ring.stage], ring.phase ^ 1u, abort_flag, kSiteRowsConvert);
      if (!ok) return;
      const uint32_t base = smem_u32(sKV) + ring.stage * Plan::kTileBytes;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        if (!mine) continue;
        const int r = i * kRows + pr, col = piece * 16;
        const uint32_t at = base + (col >> 6) * Plan::kChunkBytes + r * 128;
        const uint32_t q = (uint32_t)(col & 63) >> 3;
        const uint32_t f = e8_bf16x2((int)e[i]);
        const uint2 x0 = e4m3x4_times(w[i].x, f), x1 = e4m3x4_times(w[i].y, f);
        const uint2 x2 = e4m3x4_times(w[i].z, f), x3 = e4m3x4_times(w[i].w, f);
        st_shared_v4(at + ((q ^ (r & 7)) << 4), x0.x, x0.y, x1.x, x1.y);
        st_shared_v4(at + (((q + 1) ^ (r & 7)) << 4), x2.x, x2.y, x3.x, x3.y);
      }
      fence_proxy_async_smem();
      mbar_arrive(&kv_full[ring.stage]);
      ring.advance<S>();
    };
    // Tiles in the order the MMA warp reads them: K(0), K(1), then V(g), K(g+2); the loads of the
    // next one are issued before the current one is converted.
    RowsCursor sc, pc;
    sc.next = pc.next = (int)blockIdx.x;
    rows_next_unit(p, sc);
    rows_next_unit(p, pc);
    int nk = 0, nv = 0;   // K and V tiles handed out
    auto next_tile = [&](uint4 (&w)[kPasses], uint32_t (&e)[kPasses]) -> bool {
      if (sc.valid && nk < nv + 2) {
        load_tile(sc, true, w, e);
        rows_advance(p, sc);
        ++nk;
        return true;
      }
      if (!pc.valid) return false;
      load_tile(pc, false, w, e);
      rows_advance(p, pc);
      ++nv;
      return true;
    };
    uint4 wa[kPasses], wb[kPasses];
    uint32_t ea[kPasses], eb[kPasses];
    bool have = next_tile(wa, ea);
    while (have && ok) {
      have = next_tile(wb, eb);
      store_tile(wa, ea);
      if (!have || !ok) break;
      have = next_tile(wa, ea);
      store_tile(wb, eb);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Joins the parts of every row in key order: O (bf16) and LSE.  One thread per four columns.
template <int D>
__global__ void __launch_bounds__(256) attn_rows_join_kernel(const float* __restrict__ part_o,
                                                             const float2* __restrict__ part_ml, int parts,
                                                             long long rows, __nv_bfloat16* __restrict__ o,
                                                             float* __restrict__ lse) {
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long row = idx / (D / 4);
  const int d = (int)(idx - row * (D / 4)) * 4;
  if (row >= rows) return;
  float m = -INFINITY, l = 0.f;
  for (int s = 0; s < parts; ++s) m = fmaxf(m, part_ml[s * rows + row].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < parts; ++s) {
    const float2 ml = part_ml[s * rows + row];
    if (ml.x == -INFINITY && ml.y == 0.f) continue;   // a part without keys: nothing was written
    const float w = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - m);
    const float4 v = *reinterpret_cast<const float4*>(part_o + (s * rows + row) * D + d);
    l = fmaf(ml.y, w, l);
    acc.x = fmaf(v.x, w, acc.x);
    acc.y = fmaf(v.y, w, acc.y);
    acc.z = fmaf(v.z, w, acc.z);
    acc.w = fmaf(v.w, w, acc.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(o + row * D + d) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (d == 0) lse[row] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * 0.69314718055994530942f;
}

}  // namespace attn
