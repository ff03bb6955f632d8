// attn_serve_api.cuh -- host side of the key/value cache and of attention over keys of another
// length (include/attn.h): argument checks, schedules and launches.  Part of attn_api.cu's
// translation unit: it uses that file's device set-up, error records and tensor-map encoders.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attn_cache_kernel.cuh"
#include "attn_decode_kernel.cuh"
#include "attn_fwd_rows_kernel.cuh"

namespace {

// ---------------------------------------------------------------- paged cache: shared checks

struct CacheArgs {
  const void *k, *v, *ks, *vs;
  const int *table, *lens;
  int B, Hkv, D, num_pages, page, max_pages;
};

// Sizes of a cache and of the call on it (no CUDA call, no pointer looked at).
int cache_size_checks(const CacheArgs& a) {
  if (a.B < 0 || a.Hkv < 1 || a.num_pages < 1 || a.page < 1 || a.max_pages < 0) return ATTN_ERR_INVALID_ARG;
  if (!narrow_head_dim(a.D) || a.page % 16 != 0) return ATTN_ERR_UNSUPPORTED;
  if ((long long)a.num_pages * a.Hkv > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

int cache_pointer_checks(const CacheArgs& a) {
  if (!a.k || !a.v || !a.lens || (a.max_pages > 0 && !a.table)) return ATTN_ERR_INVALID_ARG;
  if ((a.ks == nullptr) != (a.vs == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.table, 4) || !aligned(a.lens, 4) || !aligned(a.ks, 16) ||
      !aligned(a.vs, 16))
    return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

attn::CacheView cache_view(const CacheArgs& a) {
  attn::CacheView c;
  c.k = const_cast<void*>(a.k);
  c.v = const_cast<void*>(a.v);
  c.ks = static_cast<uint8_t*>(const_cast<void*>(a.ks));
  c.vs = static_cast<uint8_t*>(const_cast<void*>(a.vs));
  c.table = a.table;
  c.lens = a.lens;
  c.len_all = 0;
  c.max_pages = a.max_pages;
  c.num_pages = a.num_pages;
  c.page = a.page;
  c.Hkv = a.Hkv;
  c.div_page = attn::make_fast_div((uint32_t)a.page);
  return c;
}

int launch_status(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return ATTN_OK;
  record_cuda_error(what, e);
  return ATTN_ERR_CUDA;
}

// A tensor of bf16 (elem_bytes 2) or E4M3 bytes (1) as TMA loads it: `rank` dimensions, D fastest,
// boxes of the given extents, with 128-byte swizzle (rows of 128 bytes) or without; elements outside
// read as zero.
int encode_rows_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint32_t* box,
                    int elem_bytes = 2, bool swizzle = true) {
  auto enc = tensor_map_encoder();
  if (!enc) {
    std::snprintf(g_last_cuda_error, sizeof(g_last_cuda_error), "cuTensorMapEncodeTiled entry point unavailable");
    return ATTN_ERR_CUDA;
  }
  cuuint64_t strides[3];
  cuuint64_t bytes = (cuuint64_t)elem_bytes;
  for (int i = 0; i + 1 < rank; ++i) strides[i] = bytes *= dims[i];
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = enc(map, elem_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r == CUDA_SUCCESS) return ATTN_OK;
  record_driver_error("cuTensorMapEncodeTiled", (int)r);
  return ATTN_ERR_CUDA;
}

// Positions [0, N) of B sequences into k, v [B][Hkv][N][D].
void launch_cache_read(const attn::CacheView& c, bool f8, void* k, void* v, int B, int N, int D, cudaStream_t s) {
  const unsigned long long items = (unsigned long long)B * c.Hkv * N * (D / 8);
  const unsigned grid = (unsigned)((items + 255) / 256);
  const auto kb = reinterpret_cast<__nv_bfloat16*>(k);
  const auto vb = reinterpret_cast<__nv_bfloat16*>(v);
  const attn::FastDiv dn = attn::make_fast_div((uint32_t)N), dh = attn::make_fast_div((uint32_t)c.Hkv);
  auto go = [&](auto kern) { kern<<<grid, 256, 0, s>>>(c, kb, vb, N, dn, dh, items); };
  auto pick = [&](auto dim) {
    constexpr int D_ = decltype(dim)::value;
    f8 ? go(attn::attn_cache_read_kernel<D_, true>) : go(attn::attn_cache_read_kernel<D_, false>);
  };
  switch (D) {
    case 32: pick(std::integral_constant<int, 32>()); break;
    case 64: pick(std::integral_constant<int, 64>()); break;
    case 96: pick(std::integral_constant<int, 96>()); break;
    default: pick(std::integral_constant<int, 128>()); break;
  }
}

// ---------------------------------------------------------------- decode schedule

// Launches a kernel that may start before the one before it in the stream has ended (it waits for that
// end itself, where it reads its results).
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

struct DecodeDeviceInfo {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};

// Few rows over long keys: how attn_decode_kernel is launched, and its workspace.
struct DecPlan {
  int tile_rows;             // rows of a warp: 8 or 16
  int row_tiles, unit_rows, row_blocks, prefix_row_blocks = 0;
  int whole_units;           // units are not split
  bool warps;                // and warps take them
  unsigned grid;
  bool join;                 // the second kernel is needed
  size_t slot_o, slot_ml;    // bytes
  size_t area_o, area_ml;    // bytes of one area (shared prefix: two areas)
  size_t bytes() const { return slot_o + slot_ml + 2 * (area_o + area_ml); }
};

constexpr int kDecMinShare = 4;     // places of the line: a unit's two, and 64-key blocks
constexpr int kDecCtasPerSm = 3, kDecWarpCtasPerSm = 2;   // resident CTAs (the kernel's launch bounds)
// A warp takes whole units where no sequence has more than kDecShortBlocks blocks and there are units for
// all CTAs, or, behind a shared prefix (where it saves the joining kernel), kDecTinyBlocks.  Measured with
// Hq32 Hkv8 D128 E4M3, in us, warps against the CTA form: B64 N<=250 18.4 / 20.5, B256 N<=250 35 / 47, B256
// N<=500 55 / 68, B64 N<=500 both 28.7, B64 N<=1000 49 / 33; behind a prefix of 16384, B128 N<=500 98 / 106, B32
// N<=120 47 / 55; without one, B4 N128 14 / 10.
constexpr int kDecShortBlocks = 8, kDecTinyBlocks = 2;
// Else a CTA takes whole units where no sequence has more than kDecWholeBlocks blocks, or, with a unit (of
// up to 8 rows) for each SM and no more than there are CTAs, kDecEvenBlocks (kDecEvenNarrow at D <= 64,
// where a step has more keys): a launch less, and nothing to join.  Whole units against split ones, in us on the
// GPU (Hq32, tables that just fit):
//   8 blocks: Hkv8 D128 bf16 B1 N384 9.8 / 10.9, N500 11.8 / 11.1, B4 N500 11.7 / 12.2, B12 12.8 / 14.8, E4M3 B1 11.4 /
//   12.7, B12 11.7 / 15.4, D64 bf16 B1 8.5 / 9.3; 16 rows (Hkv2) B1 N256 11.5 / 14.1, N500 16.4 / 14.5, B24 17.3 / 16.4, B40
//   17.6 / 19.3; behind the border, B4 N1000 25 / 16;
//   a unit for each SM: D64 Hkv16 B10 N<=1500 18.1 / 18.4, all 1500 18.4 / 21.0, N<=2000 22.6 / 20.0, all 2000 23.0 / 25.0,
//   N<=2500 26.4 / 22.1; D32 Hkv8 B30 N<=1500 16.5 / 17.8, N<=2000 19.9 / 19.7; D128 Hkv8 B20 N<=1000 E4M3 19.7 / 20.7, bf16
//   21.8 / 20.7, N<=1300 22.9 / 22.4 and 26.6 / 23.8, E4M3 B48 N<=1000 22.7 / 27.4;
//   16 rows, E4M3 B20 N<=2000 74 / 46; more units than CTAs, B64 N<=700 38.0 / 31.7.
// (The table's width stands for the lengths, which the host does not know: a table wider than the border splits.)
constexpr int kDecWholeBlocks = 8, kDecEvenBlocks = 16, kDecEvenNarrow = 24;

// `cap`: keys a sequence can have at most.  `shared`: a prefix of `prefix_len` keys comes first;
// `prefix_here`: this kernel computes it too.
DecPlan dec_plan(int B, int Hkv, long long GT, int D, long long cap, int num_sms, bool shared, bool prefix_here,
                 long long prefix_len) {
  DecPlan pl;
  const long long cap_blocks = cap > 0 ? (cap + attn::kDecBlock - 1) / attn::kDecBlock : 1;
  const long long pre_blocks = (prefix_len + attn::kDecBlock - 1) / attn::kDecBlock;
  const long long most_rows = prefix_here ? (long long)B * GT : GT;
  pl.tile_rows = most_rows <= 8 ? 8 : 16;
  pl.row_tiles = most_rows <= 16 ? 1 : most_rows <= 32 ? 2 : 4;
  pl.unit_rows = pl.tile_rows * pl.row_tiles;
  pl.row_blocks = (int)((GT + pl.unit_rows - 1) / pl.unit_rows);
  const long long ctas = (long long)kDecCtasPerSm * num_sms;
  const long long units = (long long)B * Hkv * pl.row_blocks;
  pl.warps = !prefix_here && pl.row_tiles == 1 &&
             ((shared && cap_blocks <= kDecTinyBlocks) || (cap_blocks <= kDecShortBlocks && units >= ctas));
  const bool even = pl.tile_rows == 8 && units >= num_sms && units <= ctas;
  const int whole_blocks = !even ? kDecWholeBlocks : D <= 64 ? kDecEvenNarrow : kDecEvenBlocks;
  pl.whole_units = pl.warps || (!shared && cap_blocks <= whole_blocks) ? 1 : 0;
  double blocks = (double)units * (double)(cap_blocks + 2);   // places of the line, at most
  if (prefix_here) {
    const long long rows = (long long)B * GT;
    pl.prefix_row_blocks = (int)((rows + pl.unit_rows - 1) / pl.unit_rows);
    blocks += (double)Hkv * pl.prefix_row_blocks * (double)(pre_blocks + 2);
  }
  const double most = pl.warps ? (double)((units + 3) / 4) : pl.whole_units ? (double)units : blocks / kDecMinShare + 1;
  const long long resident = pl.warps ? (long long)kDecWarpCtasPerSm * num_sms : ctas;
  pl.grid = (unsigned)(most < (double)resident ? (long long)most : resident);
  if (pl.grid < 1) pl.grid = 1;
  pl.join = !pl.whole_units;
  const size_t slots = pl.whole_units ? 0 : 2 * (size_t)pl.grid * pl.unit_rows;
  pl.slot_o = slots * D * sizeof(float);
  pl.slot_ml = (slots * sizeof(float2) + 255) / 256 * 256;
  const size_t rows = shared && !pl.whole_units ? ((size_t)B * Hkv * (size_t)GT + 63) / 64 * 64 : 0;
  pl.area_o = rows * D * sizeof(float);
  pl.area_ml = rows * sizeof(float2);
  return pl;
}

template <int D, bool kF8, int kN, bool kWarp>
int launch_decode_dim(attn::DecParams& p, const DecPlan& pl, const void* k, const void* v, cudaStream_t s) {
  using Cfg = attn::DecCfg<D, kF8>;
  static DecodeDeviceInfo info[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevices)) e = cudaErrorInvalidDevice;
  if (e == cudaSuccess) {
    std::call_once(info[dev].once, [&] {
      info[dev].err = cudaFuncSetAttribute(reinterpret_cast<const void*>(attn::attn_decode_kernel<D, kF8, kN, kWarp>),
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, attn::dec_smem(kWarp));
    });
    e = info[dev].err;
  }
  if (e != cudaSuccess) {
    record_cuda_error("decode device setup", e);
    return ATTN_ERR_CUDA;
  }
  // boxes of a whole step where pages hold whole steps (contiguous keys are one page), else of 16 keys; a call
  // may have a table for its prefix alone (max_pages == 0)
  const bool paged = p.table != nullptr || p.prefix_table != nullptr;
  p.box = (!paged || p.page % Cfg::kStep == 0) ? Cfg::kStep : 16;
  CUtensorMap mk, mv;
  int st;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)p.page, (cuuint64_t)p.num_pages * (cuuint64_t)p.Hkv};
  const cuuint32_t box[3] = {(cuuint32_t)(128 / Cfg::kElem), (cuuint32_t)p.box, 1};
  if (p.cap > 0 || p.prefix_len > 0) {
    if ((st = encode_rows_map(&mk, k, 3, dims, box, Cfg::kElem)) != ATTN_OK) return st;
    if ((st = encode_rows_map(&mv, v, 3, dims, box, Cfg::kElem)) != ATTN_OK) return st;
  } else {   // no keys at all: nothing is loaded
    std::memset(&mk, 0, sizeof(mk));
    std::memset(&mv, 0, sizeof(mv));
  }
  // behind the many-row kernel of a shared prefix it may start early
  auto kern = attn::attn_decode_kernel<D, kF8, kN, kWarp>;
  if (p.many.tiles > 0)
    e = launch_behind(kern, dim3(pl.grid), attn::kDecThreads, attn::dec_smem(kWarp), s, mk, mv, p);
  else
    kern<<<pl.grid, attn::kDecThreads, attn::dec_smem(kWarp), s>>>(mk, mv, p);
  if (e == cudaSuccess && pl.join)
    e = launch_behind(attn::attn_decode_join_kernel<D>,
                      dim3((unsigned)((long long)p.B * p.Hkv * p.row_blocks), (unsigned)((pl.unit_rows + 3) / 4)),
                      attn::kDecThreads, 0, s, p, pl.grid);
  if (e != cudaSuccess) {
    cudaGetLastError();
    record_cuda_error("decode kernel launch", e);
    return ATTN_ERR_CUDA;
  }
  return launch_status("decode kernel launch");
}

// Fills the schedule and workspace part of `p` and launches.
int launch_decode(attn::DecParams& p, const DecPlan& pl, const void* k, const void* v, int D, bool shared,
                  void* workspace, cudaStream_t s) {
  p.row_tiles = pl.row_tiles;
  p.row_blocks = pl.row_blocks;
  p.prefix_row_blocks = pl.prefix_row_blocks;
  p.whole_units = pl.whole_units;
  p.min_share = pl.whole_units ? 3 : kDecMinShare;
  p.unit_rows = pl.unit_rows;
  char* w = static_cast<char*>(workspace);
  p.slot_o = reinterpret_cast<float*>(w);
  p.slot_ml = reinterpret_cast<float2*>(w + pl.slot_o);
  w += pl.slot_o + pl.slot_ml;
  for (int i = 0; i < 2; ++i) {
    p.area_o[i] = shared && pl.join ? reinterpret_cast<float*>(w) : nullptr;
    p.area_ml[i] = shared && pl.join ? reinterpret_cast<float2*>(w + pl.area_o) : nullptr;
    w += pl.area_o + pl.area_ml;
  }
  auto pick = [&](auto dim, auto tiles, auto warps) {
    constexpr int D_ = decltype(dim)::value, N_ = decltype(tiles)::value;
    constexpr bool W_ = decltype(warps)::value;
    return p.ks ? launch_decode_dim<D_, true, N_, W_>(p, pl, k, v, s) : launch_decode_dim<D_, false, N_, W_>(p, pl, k, v, s);
  };
  auto go = [&](auto dim) {
    if (pl.tile_rows == 8)
      return pl.warps ? pick(dim, std::integral_constant<int, 1>(), std::true_type())
                            : pick(dim, std::integral_constant<int, 1>(), std::false_type());
    return pl.warps ? pick(dim, std::integral_constant<int, 2>(), std::true_type())
                          : pick(dim, std::integral_constant<int, 2>(), std::false_type());
  };
  switch (D) {
    case 32: return go(std::integral_constant<int, 32>());
    case 64: return go(std::integral_constant<int, 64>());
    case 96: return go(std::integral_constant<int, 96>());
    default: return go(std::integral_constant<int, 128>());
  }
}

// Sizes common to decode and shared prefix; rows of a KV head in `GT`.
int decode_size_checks(const CacheArgs& a, int Hq, int T, float scale, long long* GT) {
  const int st = cache_size_checks(a);
  if (st == ATTN_ERR_INVALID_ARG || Hq < 1 || T < 0 || Hq % a.Hkv != 0 || !std::isfinite(scale))
    return ATTN_ERR_INVALID_ARG;
  if (st != ATTN_OK) return st;
  *GT = (long long)(Hq / a.Hkv) * T;
  // rows and work units are indexed in 32 bits; a batch's rows of one KV head too (shared prefix)
  if ((long long)a.B * a.Hkv > 0x7fffffffLL || *GT > (1LL << 30) || (double)a.B * (double)*GT > 2147483647.0 ||
      (double)a.B * a.Hkv * ((double)*GT / 16 + 1) > 2147483647.0)
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

int sm_count(int* num_sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && *num_sms >= 1) return ATTN_OK;
  record_cuda_error("cudaDeviceGetAttribute", e);
  return ATTN_ERR_CUDA;
}

long long cache_cap(int page, int max_pages) {
  const long long n = (long long)page * max_pages;
  return n < 0x7fffffffLL ? n : 0x7fffffffLL;
}

void fill_decode(attn::DecParams& p, const CacheArgs& a, const void* q, void* o, float* lse, int T, long long GT,
                 float scale, int causal) {
  std::memset(&p, 0, sizeof(p));
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.ks = static_cast<const uint8_t*>(a.ks);
  p.vs = static_cast<const uint8_t*>(a.vs);
  p.v = static_cast<const __nv_bfloat16*>(a.v);
  p.table = a.table;
  p.lens = a.lens;
  p.cap = cache_cap(a.page, a.max_pages);
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.page = a.page;
  p.Hkv = a.Hkv;
  p.B = a.B;
  p.div_page = attn::make_fast_div((uint32_t)a.page);
  p.GT = (int)GT;
  p.T = T;
  p.causal = causal;
  p.div_gt = attn::make_fast_div((uint32_t)GT);
  p.c = scale * attn::kLog2e;
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  p.lse = lse;
}

// ---------------------------------------------------------------- many rows: the tensor-core kernel

struct RowsDeviceInfo {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
RowsDeviceInfo g_rows_dev[kMaxDevices];

template <int D>
cudaError_t rows_setup_dim() {
  cudaError_t e = cudaSuccess;
  auto setup = [&](const void* fn, int regs, int smem) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaFuncAttributes fa{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, fn);
    // the register split (setmaxnreg) needs exactly the launch allocation it was sized for
    if (e == cudaSuccess && fa.numRegs != regs) e = cudaErrorInvalidDeviceFunction;
  };
  setup(reinterpret_cast<const void*>(attn::attn_fwd_rows_sm100<D, false>), attn::RowsCfg<false>::kRegsLaunch,
        attn::RowsSmem<D, false>::kAlloc);
  setup(reinterpret_cast<const void*>(attn::attn_fwd_rows_sm100<D, true>), attn::RowsCfg<true>::kRegsLaunch,
        attn::RowsSmem<D, true>::kAlloc);
  return e;
}

bool rows_device_setup() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= kMaxDevices)) e = cudaErrorInvalidDevice;
  if (e != cudaSuccess) {
    record_cuda_error("cudaGetDevice", e);
    return false;
  }
  RowsDeviceInfo& d = g_rows_dev[dev];
  std::call_once(d.once, [&d] {
    cudaError_t x = rows_setup_dim<32>();
    if (x == cudaSuccess) x = rows_setup_dim<64>();
    if (x == cudaSuccess) x = rows_setup_dim<96>();
    if (x == cudaSuccess) x = rows_setup_dim<128>();
    d.err = x;
  });
  if (d.err == cudaSuccess) return true;
  record_cuda_error("many-row kernel device setup", d.err);
  return false;
}

template <int D>
void launch_rows_dim(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                     const attn::RowsParams& p, bool f8, bool join, unsigned grid, cudaStream_t s) {
  if (f8)
    attn::attn_fwd_rows_sm100<D, true>
        <<<grid, attn::RowsCfg<true>::kThreads, attn::RowsSmem<D, true>::kAlloc, s>>>(mq, mk, mv, mo, p);
  else if (p.behind)
    launch_behind(attn::attn_fwd_rows_sm100<D, false>, dim3(grid), attn::RowsCfg<false>::kThreads,
                  attn::RowsSmem<D, false>::kAlloc, s, mq, mk, mv, mo, p);
  else
    attn::attn_fwd_rows_sm100<D, false>
        <<<grid, attn::RowsCfg<false>::kThreads, attn::RowsSmem<D, false>::kAlloc, s>>>(mq, mk, mv, mo, p);
  if (join) launch_behind(attn::attn_rows_join_kernel<D>, dim3(grid - 1, attn::kBlockM / 32), 256, 0, s, p, grid);
}

constexpr int kRowsMinShare = 3;   // places of the line: a unit's one, and 128-key blocks

// The tiles of a problem, the grid and the workspace.
struct RowsPlan {
  int tiles = 0, seqs = 1, seq_tiles = 1;
  long long blocks = 0;            // of a unit, at most
  unsigned grid = 1;
  size_t slot_o = 0, slot_ml = 0;  // bytes
  size_t bytes() const { return slot_o + slot_ml; }
};

RowsPlan rows_plan(int B, int Hkv, long long GT, int D, long long max_len, int num_sms, bool prefix) {
  RowsPlan pl;
  const long long per_seq = (GT + attn::kBlockM - 1) / attn::kBlockM;
  pl.blocks = max_len > 0 ? (max_len + attn::kBlockN - 1) / attn::kBlockN : 1;
  if (!prefix) {
    pl.tiles = (int)per_seq;
  } else if (GT <= attn::kBlockM) {
    pl.seqs = (int)(attn::kBlockM / GT);
    pl.tiles = (B + pl.seqs - 1) / pl.seqs;
  } else {
    pl.seq_tiles = (int)per_seq;
    pl.tiles = (int)(B * per_seq);
  }
  const long long units = (long long)(prefix ? Hkv : (long long)B * Hkv) * pl.tiles;
  const double most = (double)units * (double)(pl.blocks + 1) / kRowsMinShare + 1;
  pl.grid = most < (double)num_sms ? (unsigned)most : (unsigned)num_sms;
  const size_t slots = 2 * (size_t)pl.grid + (prefix ? (size_t)units : 0);
  pl.slot_o = slots * attn::kBlockM * D * sizeof(float);
  pl.slot_ml = slots * attn::kBlockM * sizeof(float2);
  return pl;
}

// Fills the sizes and launches; p's key, output and length fields are the caller's.
int launch_rows(attn::RowsParams& p, const RowsPlan& pl, const void* q, const void* k, const void* v, void* o, int D,
                bool prefix, float scale, void* workspace, cudaStream_t s) {
  if (!rows_device_setup()) return ATTN_ERR_CUDA;
  const bool f8 = p.ks != nullptr;
  p.tiles = pl.tiles;
  p.seqs = pl.seqs;
  p.seq_tiles = pl.seq_tiles;
  p.prefix = prefix ? 1 : 0;
  p.min_share = kRowsMinShare;
  p.slot_o = reinterpret_cast<float*>(workspace);
  p.slot_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + pl.slot_o);
  p.o = reinterpret_cast<__nv_bfloat16*>(o);
  const bool many = prefix && pl.seq_tiles == 1;   // a tile holds whole sequences
  p.q_box_rows = many ? p.GT * pl.seqs : attn::kBlockM;
  // c > 0 always: masked scores are -inf and must stay so (scale == 0: every 2^(s c) is 1)
  p.c = std::fmax(std::fabs(scale) * 1.44269504088896340736f, 1e-30f);
  p.idesc_s = attn::idesc_bf16_f32(attn::kBlockM, attn::kBlockN, false, false, scale < 0.f);
  p.idesc_pv = attn::idesc_bf16_f32(attn::kBlockM, D, false, true, false);
  CUtensorMap mq, mk, mv, mo;
  std::memset(&mo, 0, sizeof(mo));
  int st;
  const cuuint64_t qd[4] = {(cuuint64_t)D, (cuuint64_t)p.GT, (cuuint64_t)p.Hkv, (cuuint64_t)p.B};
  const cuuint32_t qb[4] = {64, (cuuint32_t)(many ? p.GT : attn::kBlockM), 1, (cuuint32_t)pl.seqs};
  if ((st = encode_rows_map(&mq, q, 4, qd, qb)) != ATTN_OK) return st;
  p.box = attn::kBlockN;
  if (p.table != nullptr)
    while (p.page % p.box != 0) p.box /= 2;
  const cuuint64_t kd[3] = {(cuuint64_t)D, (cuuint64_t)p.page, (cuuint64_t)p.num_pages * (cuuint64_t)p.Hkv};
  const cuuint32_t kb[3] = {(cuuint32_t)(f8 ? D : 64), (cuuint32_t)p.box, 1};
  const bool swizzle = !f8 || D == 128;   // (raw E4M3 tiles: as the converters read them)
  if ((st = encode_rows_map(&mk, k, 3, kd, kb, f8 ? 1 : 2, swizzle)) != ATTN_OK) return st;
  if ((st = encode_rows_map(&mv, v, 3, kd, kb, f8 ? 1 : 2, swizzle)) != ATTN_OK) return st;
  if (!prefix && (st = encode_map_o(&mo, o, (long long)p.B * p.Hkv, p.GT, D)) != ATTN_OK) return st;
  const bool join = !prefix && pl.grid > 1;
  switch (D) {
    case 32: launch_rows_dim<32>(mq, mk, mv, mo, p, f8, join, pl.grid, s); break;
    case 64: launch_rows_dim<64>(mq, mk, mv, mo, p, f8, join, pl.grid, s); break;
    case 96: launch_rows_dim<96>(mq, mk, mv, mo, p, f8, join, pl.grid, s); break;
    default: launch_rows_dim<128>(mq, mk, mv, mo, p, f8, join, pl.grid, s); break;
  }
  return launch_status("many-row kernel launch");
}

// At most this many rows of a KV head go through the decode kernel; more, through the tensor-core
// kernel.  Measured, in us, decode kernel against the other: cross attention, B8 Hkv16 N<=1500 D64, 16 rows 20.5 /
// 23.6, 20 to 32 rows 24.6 / 22.5 (B2 N<=8000 32.8 / 26.6); a prefix of 8000 bf16 keys (Hkv16 D64), 32 rows
// 34 / 38 (the other is two more kernels there), 48 rows 50 / 38.
constexpr int kFewRows = 16, kFewPrefixRows = 32;

// Shared prefix: the plans of its two kernels, and the workspace's layout (decode's part first).
struct PrefixPlan {
  bool here;        // the decode kernel computes the prefix too
  size_t wide;      // bytes of the prefix's keys, and of its values, as bf16 (0: converted in the kernel)
  DecPlan dec;
  RowsPlan rows;
  size_t bytes() const { return dec.bytes() + rows.bytes() + 2 * wide; }
};

// An E4M3 prefix is converted to bf16 once, ahead, where at least this many 128-row tiles of each head
// would convert it themselves and the copy is no larger than this (a bound on the workspace).  Prefix of 16384, Hq32 Hkv8 D128, in us,
// converted ahead against in the kernel: one tile (B32) 80 / 65, two (B64) 81 / 75, three (B96) 89 / 89, four (B128)
// 101 / 108, eight (B256) 153 / 187.
constexpr int kWideTiles = 4;
constexpr size_t kWideBytes = (size_t)256 << 20;

PrefixPlan prefix_plan(int B, int Hkv, long long GT, int D, int page, int max_pages, long long prefix_len,
                       int num_sms, bool f8) {
  PrefixPlan pl;
  pl.here = prefix_len > 0 && (long long)B * GT <= kFewPrefixRows;
  pl.dec = dec_plan(B, Hkv, GT, D, cache_cap(page, max_pages), num_sms, true, pl.here, prefix_len);
  if (prefix_len > 0 && !pl.here) pl.rows = rows_plan(B, Hkv, GT, D, prefix_len, num_sms, true);
  const size_t wide = ((size_t)Hkv * (size_t)prefix_len * D * 2 + 255) / 256 * 256;
  pl.wide = f8 && !pl.here && pl.rows.tiles >= kWideTiles && 2 * wide <= kWideBytes ? wide : 0;
  return pl;
}

// Sizes of a cross-attention problem; query rows of a KV head in `GT`.
int cross_size_checks(int B, int Hq, int Hkv, int Nq, int Nk, int D, float scale, long long* GT) {
  if (B < 0 || Nq < 0 || Nk < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !std::isfinite(scale))
    return ATTN_ERR_INVALID_ARG;
  if (!narrow_head_dim(D)) return ATTN_ERR_UNSUPPORTED;
  *GT = (long long)(Hq / Hkv) * Nq;
  if ((long long)B * Hkv > 0x7fffffffLL || *GT > (1LL << 30) ||
      (double)B * Hkv * ((double)*GT / 16 + 1) > 2147483647.0 ||
      (double)B * Hkv * ((double)Nk / 128 + 1) > 1073741824.0)
    return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

}  // namespace

extern "C" {

int attn_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                      const int* block_table, const int* lens, const int* new_lens, int B, int Hkv, int T, int D,
                      int num_pages, int page_size, int max_pages, void* stream) {
  const CacheArgs a{k_cache, v_cache, k_scale, v_scale, block_table, lens, B, Hkv, D, num_pages, page_size, max_pages};
  int st = cache_size_checks(a);
  if (st != ATTN_OK) return st;
  if (T < 0) return ATTN_ERR_INVALID_ARG;
  // rows are indexed in 32 bits, 2^31 blocks of 8 rows
  if ((double)B * Hkv * (double)T >= 4294967296.0) return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return ATTN_OK;
  if (!k || !v) return ATTN_ERR_INVALID_ARG;
  if ((st = cache_pointer_checks(a)) != ATTN_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(new_lens, 4)) return ATTN_ERR_MISALIGNED;
  const uint32_t rows = (uint32_t)((long long)B * Hkv * T);
  const int lanes = D / 8 <= 4 ? 4 : D / 8 <= 8 ? 8 : 16;
  // four rows a group where that still leaves blocks for every SM several times over
  const bool many = (unsigned long long)rows * lanes >= (1u << 20);
  const unsigned long long groups = many ? ((unsigned long long)rows + 3) / 4 : rows;
  const unsigned grid = (unsigned)((groups * lanes + 255) / 256);
  const attn::CacheView c = cache_view(a);
  const auto kb = reinterpret_cast<const __nv_bfloat16*>(k);
  const auto vb = reinterpret_cast<const __nv_bfloat16*>(v);
  const attn::FastDiv dt = attn::make_fast_div((uint32_t)T), dh = attn::make_fast_div((uint32_t)Hkv);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto kern) { kern<<<grid, 256, 0, s>>>(kb, vb, c, new_lens, T, dt, dh, rows); };
  auto pick = [&](auto dim) {
    constexpr int D_ = decltype(dim)::value;
    if (k_scale != nullptr)
      many ? go(attn::attn_cache_append_kernel<D_, true, 4>) : go(attn::attn_cache_append_kernel<D_, true, 1>);
    else
      many ? go(attn::attn_cache_append_kernel<D_, false, 4>) : go(attn::attn_cache_append_kernel<D_, false, 1>);
  };
  switch (D) {
    case 32: pick(std::integral_constant<int, 32>()); break;
    case 64: pick(std::integral_constant<int, 64>()); break;
    case 96: pick(std::integral_constant<int, 96>()); break;
    default: pick(std::integral_constant<int, 128>()); break;
  }
  return launch_status("cache append kernel launch");
}

int attn_cache_read(const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale,
                    const int* block_table, const int* lens, void* k, void* v, int B, int Hkv, int N, int D,
                    int num_pages, int page_size, int max_pages, void* stream) {
  const CacheArgs a{k_cache, v_cache, k_scale, v_scale, block_table, lens, B, Hkv, D, num_pages, page_size, max_pages};
  int st = cache_size_checks(a);
  if (st != ATTN_OK) return st;
  if (N < 0) return ATTN_ERR_INVALID_ARG;
  if ((double)B * Hkv * (double)N >= 4294967296.0) return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || N == 0) return ATTN_OK;
  if (!k || !v) return ATTN_ERR_INVALID_ARG;
  if ((st = cache_pointer_checks(a)) != ATTN_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16)) return ATTN_ERR_MISALIGNED;
  launch_cache_read(cache_view(a), k_scale != nullptr, k, v, B, N, D, reinterpret_cast<cudaStream_t>(stream));
  return launch_status("cache read kernel launch");
}

long long attn_fwd_decode_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int page_size, int max_pages) {
  const CacheArgs a{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, B, Hkv, D, 1, page_size, max_pages};
  long long GT = 0;
  if (decode_size_checks(a, Hq, T, 1.f, &GT) != ATTN_OK) return -1;
  if (B == 0 || T == 0) return 0;
  int num_sms = 0;
  if (sm_count(&num_sms) != ATTN_OK) return -1;
  return (long long)dec_plan(B, Hkv, GT, D, cache_cap(page_size, max_pages), num_sms, false, false, 0).bytes();
}

int attn_fwd_decode(const void* q, const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale,
                    const int* block_table, const int* lens, void* o, float* lse, int B, int Hq, int Hkv, int T,
                    int D, int num_pages, int page_size, int max_pages, float scale, void* workspace,
                    size_t workspace_bytes, void* stream) {
  const CacheArgs a{k_cache, v_cache, k_scale, v_scale, block_table, lens, B, Hkv, D, num_pages, page_size, max_pages};
  long long GT = 0;
  int st = decode_size_checks(a, Hq, T, scale, &GT);
  if (st != ATTN_OK) return st;
  if (B == 0 || T == 0) return ATTN_OK;
  if (!q || !o || !lse) return ATTN_ERR_INVALID_ARG;
  if ((st = cache_pointer_checks(a)) != ATTN_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256)) return ATTN_ERR_MISALIGNED;
  int num_sms = 0;
  if ((st = sm_count(&num_sms)) != ATTN_OK) return st;
  const DecPlan pl = dec_plan(B, Hkv, GT, D, cache_cap(page_size, max_pages), num_sms, false, false, 0);
  if (pl.bytes() > workspace_bytes || (pl.bytes() > 0 && !workspace)) return ATTN_ERR_INVALID_ARG;
  attn::DecParams p;
  fill_decode(p, a, q, o, lse, T, GT, scale, 1);
  return launch_decode(p, pl, k_cache, v_cache, D, false, workspace, reinterpret_cast<cudaStream_t>(stream));
}

long long attn_fwd_shared_prefix_workspace_bytes(int B, int Hq, int Hkv, int T, int D, int page_size, int max_pages,
                                                 int prefix_len, int e4m3) {
  const CacheArgs a{nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, B, Hkv, D, 1, page_size, max_pages};
  long long GT = 0;
  if (prefix_len < 0 || decode_size_checks(a, Hq, T, 1.f, &GT) != ATTN_OK) return -1;
  if (B == 0 || T == 0) return 0;
  int num_sms = 0;
  if (sm_count(&num_sms) != ATTN_OK) return -1;
  return (long long)prefix_plan(B, Hkv, GT, D, page_size, max_pages, prefix_len, num_sms, e4m3 != 0).bytes();
}

int attn_fwd_shared_prefix(const void* q, const void* k_cache, const void* v_cache, const void* k_scale,
                           const void* v_scale, const int* prefix_table, int prefix_len, const int* block_table,
                           const int* lens, void* o, float* lse, int B, int Hq, int Hkv, int T, int D, int num_pages,
                           int page_size, int max_pages, float scale, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const CacheArgs a{k_cache, v_cache, k_scale, v_scale, block_table, lens, B, Hkv, D, num_pages, page_size, max_pages};
  long long GT = 0;
  int st = decode_size_checks(a, Hq, T, scale, &GT);
  if (st != ATTN_OK) return st;
  if (prefix_len < 0) return ATTN_ERR_INVALID_ARG;
  if (B == 0 || T == 0) return ATTN_OK;
  if (!q || !o || !lse || (prefix_len > 0 && !prefix_table)) return ATTN_ERR_INVALID_ARG;
  if ((st = cache_pointer_checks(a)) != ATTN_OK) return st;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(workspace, 256) || !aligned(prefix_table, 4))
    return ATTN_ERR_MISALIGNED;
  int num_sms = 0;
  if ((st = sm_count(&num_sms)) != ATTN_OK) return st;
  const PrefixPlan pl = prefix_plan(B, Hkv, GT, D, page_size, max_pages, prefix_len, num_sms, k_scale != nullptr);
  if (pl.bytes() > workspace_bytes || (pl.bytes() > 0 && !workspace)) return ATTN_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  attn::DecParams p;
  fill_decode(p, a, q, o, lse, T, GT, scale, 1);
  if (pl.here) {
    p.prefix_table = prefix_table;
    p.prefix_len = prefix_len;
  } else if (prefix_len > 0) {
    // many rows: the prefix on the tensor-core kernel, its parts joined by the decode's second kernel
    attn::RowsParams r;
    std::memset(&r, 0, sizeof(r));
    r.B = B;
    r.Hkv = Hkv;
    r.GT = (int)GT;
    r.len_all = prefix_len;
    r.table = prefix_table;
    r.page = page_size;
    r.num_pages = num_pages;
    r.ks = p.ks;
    r.vs = p.vs;
    // (every part of the workspace is a multiple of 256 bytes)
    char* w = static_cast<char*>(workspace) + pl.dec.bytes();
    const void *kp = k_cache, *vp = v_cache;
    if (pl.wide) {
      char* wide = w + pl.rows.bytes();
      attn::CacheView c = cache_view(a);
      c.table = prefix_table;
      c.lens = nullptr;
      c.len_all = prefix_len;
      c.max_pages = (prefix_len + page_size - 1) / page_size;
      launch_cache_read(c, true, wide, wide + pl.wide, 1, prefix_len, D, s);
      if ((st = launch_status("prefix conversion launch")) != ATTN_OK) return st;
      kp = wide;
      vp = wide + pl.wide;
      r.behind = 1;
      r.table = nullptr;
      r.page = prefix_len;
      r.num_pages = 1;
      r.ks = r.vs = nullptr;
    }
    if ((st = launch_rows(r, pl.rows, q, kp, vp, o, D, true, scale, w, s)) != ATTN_OK) return st;
    p.many.o = r.slot_o;
    p.many.ml = r.slot_ml;
    p.many.tiles = r.tiles;
    p.many.seqs = r.seqs;
    p.many.seq_tiles = r.seq_tiles;
    p.many.places = attn::rows_places((int)pl.rows.blocks);
    p.many.over = attn::kRowsOver;
    p.many.ctas = pl.rows.grid;
    const long long total = (long long)Hkv * r.tiles * p.many.places;
    p.many.share = (total + p.many.ctas - 1) / p.many.ctas;
    if (p.many.share < kRowsMinShare) p.many.share = kRowsMinShare;
  }
  return launch_decode(p, pl.dec, k_cache, v_cache, D, true, workspace, s);
}

// ---------------------------------------------------------------- cross attention

long long attn_fwd_cross_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int D) {
  long long GT = 0;
  if (cross_size_checks(B, Hq, Hkv, Nq, Nk, D, 1.f, &GT) != ATTN_OK) return -1;
  if (B == 0 || Nq == 0) return 0;
  int num_sms = 0;
  if (sm_count(&num_sms) != ATTN_OK) return -1;
  return (long long)(GT <= kFewRows || Nk == 0 ? dec_plan(B, Hkv, GT, D, Nk, num_sms, false, false, 0).bytes()
                                               : rows_plan(B, Hkv, GT, D, Nk, num_sms, false).bytes());
}

int attn_fwd_cross(const void* q, const void* k, const void* v, const int* k_lens, void* o, float* lse, int B, int Hq,
                   int Hkv, int Nq, int Nk, int D, float scale, void* workspace, size_t workspace_bytes,
                   void* stream) {
  long long GT = 0;
  int st = cross_size_checks(B, Hq, Hkv, Nq, Nk, D, scale, &GT);
  if (st != ATTN_OK) return st;
  if (B == 0 || Nq == 0) return ATTN_OK;
  if (!q || !o || !lse || (Nk > 0 && (!k || !v))) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(k_lens, 4) || !aligned(workspace, 256))
    return ATTN_ERR_MISALIGNED;
  int num_sms = 0;
  if ((st = sm_count(&num_sms)) != ATTN_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (GT <= kFewRows || Nk == 0) {
    const DecPlan pl = dec_plan(B, Hkv, GT, D, Nk, num_sms, false, false, 0);
    if (pl.bytes() > workspace_bytes || (pl.bytes() > 0 && !workspace)) return ATTN_ERR_INVALID_ARG;
    // contiguous keys: sequence b is page b of Nk rows
    const CacheArgs a{k, v, nullptr, nullptr, nullptr, k_lens, B, Hkv, D, B, Nk > 0 ? Nk : 1, 1};
    attn::DecParams p;
    fill_decode(p, a, q, o, lse, Nq, GT, scale, 0);
    p.cap = p.len_all = Nk;
    return launch_decode(p, pl, k, v, D, false, workspace, s);
  }
  const RowsPlan pl = rows_plan(B, Hkv, GT, D, Nk, num_sms, false);
  if (pl.bytes() > workspace_bytes || (pl.bytes() > 0 && !workspace)) return ATTN_ERR_INVALID_ARG;
  attn::RowsParams r;
  std::memset(&r, 0, sizeof(r));
  r.lse = lse;
  r.B = B;
  r.Hkv = Hkv;
  r.GT = (int)GT;
  r.k_lens = k_lens;
  r.len_all = Nk;
  r.page = Nk;
  r.num_pages = B;
  return launch_rows(r, pl, q, k, v, o, D, false, scale, workspace, s);
}

}  // extern "C"

// ---------------------------------------------------------------- cross attention, backward

namespace {

struct CrossBwdDeviceInfo {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
CrossBwdDeviceInfo g_cross_bwd_dev[kMaxDevices];

template <int D>
cudaError_t cross_bwd_setup_dim() {
  cudaError_t e = cudaSuccess;
  auto setup = [&](const void* fn, int smem) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaFuncAttributes fa{};
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, fn);
    // the register split (setmaxnreg) needs exactly the launch allocation it was sized for
    if (e == cudaSuccess && attn::BwdCfg<D>::kSplit && fa.numRegs != attn::kRegsAtLaunch)
      e = cudaErrorInvalidDeviceFunction;
  };
  setup(reinterpret_cast<const void*>(attn::attn_bwd_sm100<D, true, true>), attn::BwdPlan<D, true>::kAlloc);
  setup(reinterpret_cast<const void*>(attn::attn_bwd_sm100<D, false, true>), attn::BwdPlan<D, false>::kAlloc);
  return e;
}

bool cross_bwd_device_setup(int dev) {
  if (dev < 0 || dev >= kMaxDevices) return false;
  CrossBwdDeviceInfo& d = g_cross_bwd_dev[dev];
  std::call_once(d.once, [&d] {
    cudaError_t e = cross_bwd_setup_dim<32>();
    if (e == cudaSuccess) e = cross_bwd_setup_dim<64>();
    if (e == cudaSuccess) e = cross_bwd_setup_dim<96>();
    if (e == cudaSuccess) e = cross_bwd_setup_dim<128>();
    d.err = e;
  });
  if (d.err == cudaSuccess) return true;
  record_cuda_error("cross-attention backward device setup", d.err);
  return false;
}

// The Q pass starts as the KV pass's CTAs end: its work is what fills the SMs that the KV pass leaves early (units of
// batch rows without keys at their block are empty), so it is cut into up to kCrossCtas CTAs an SM, of kCrossTiles
// column tiles at least, which the hardware deals out.  B4 Hq32 Hkv8 Nq2048 Nk<=4096 D128: one CTA an SM 1158 us for
// both passes, two 1088, four 1062, eight 1029; one after the other's end, 1187.  With four tiles an item
// (Nk 512) eight CTAs an SM took 147 us instead of 138.  The KV pass gains nothing from more CTAs than SMs.
constexpr int kCrossTiles = 8, kCrossCtas = 8;
template <int D>
void launch_cross_bwd_dim(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo,
                          const attn::BwdParams& pkv, const attn::BwdParams& pq, int num_sms, cudaStream_t s) {
  launch_behind(attn::attn_bwd_sm100<D, true, true>, dim3((unsigned)std::min(pkv.num_items, num_sms)),
                attn::BwdCfg<D>::kThreads, attn::BwdPlan<D, true>::kAlloc, s, mk, mv, mq, mdo, pkv);
  const int each = (kCrossTiles + pkv.num_blocks - 1) / pkv.num_blocks;
  const int ctas = std::max(num_sms, std::min((pq.num_items + each - 1) / each, kCrossCtas * num_sms));
  launch_behind(attn::attn_bwd_sm100<D, false, true>, dim3((unsigned)std::min(pq.num_items, ctas)),
                attn::BwdCfg<D>::kThreads, attn::BwdPlan<D, false>::kAlloc, s, mq, mdo, mk, mv, pq);
}

}  // namespace

extern "C" {

long long attn_bwd_cross_workspace_bytes(int B, int Hq, int Hkv, int Nq) {
  long long GT = 0;
  if (cross_size_checks(B, Hq, Hkv, Nq, 0, 32, 1.f, &GT) != ATTN_OK) return -1;
  return attn_bwd_workspace_bytes(B, Hkv, (int)GT);
}

int attn_bwd_cross(const void* q, const void* k, const void* v, const int* k_lens, const void* o, const float* lse,
                   const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Nq, int Nk, int D,
                   float scale, void* workspace, size_t workspace_bytes, void* stream) {
  // ---- host-side validation (no CUDA call before this block passes)
  long long GT = 0;
  int st = cross_size_checks(B, Hq, Hkv, Nq, Nk, D, scale, &GT);
  if (st != ATTN_OK) return st;
  if (B == 0 || (Nq == 0 && Nk == 0)) return ATTN_OK;
  if (Nq > 0 && (!q || !o || !lse || !dout || !dq || !workspace)) return ATTN_ERR_INVALID_ARG;
  if (Nk > 0 && (!k || !v || !dk || !dv)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16) || !aligned(lse, 4) || !aligned(k_lens, 4) ||
      !aligned(workspace, 256))
    return ATTN_ERR_MISALIGNED;
  const size_t part = bwd_part_bytes(B, Hkv, (int)GT);
  if (workspace_bytes < 2 * part) return ATTN_ERR_INVALID_ARG;
  int dev = 0, num_sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    record_cuda_error("cudaGetDevice", e);
    return ATTN_ERR_CUDA;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // one side empty: the other's gradients are zero
  const size_t q_bytes = (size_t)B * Hkv * (size_t)GT * D * 2, k_bytes = (size_t)B * Hkv * (size_t)Nk * D * 2;
  if (Nq == 0 || Nk == 0) {
    if (q_bytes) e = cudaMemsetAsync(dq, 0, q_bytes, s);
    if (k_bytes) e = cudaMemsetAsync(dk, 0, k_bytes, s);
    if (k_bytes && e == cudaSuccess) e = cudaMemsetAsync(dv, 0, k_bytes, s);
    if (e == cudaSuccess) return ATTN_OK;
    record_cuda_error("cudaMemsetAsync", e);
    return ATTN_ERR_CUDA;
  }
  if ((st = sm_count(&num_sms)) != ATTN_OK) return st;
  if (!cross_bwd_device_setup(dev)) return ATTN_ERR_CUDA;

  CUtensorMap mq, mk, mv, mdo;
  const long long heads = (long long)B * Hkv;
  if ((st = encode_map(&mq, q, heads, (int)GT, D)) != ATTN_OK) return st;
  if ((st = encode_map(&mk, k, heads, Nk, D)) != ATTN_OK) return st;
  if ((st = encode_map(&mv, v, heads, Nk, D)) != ATTN_OK) return st;
  if ((st = encode_map(&mdo, dout, heads, (int)GT, D)) != ATTN_OK) return st;

  const int nq = (int)((GT + attn::kBlockM - 1) / attn::kBlockM);
  const int nk = (int)(((long long)Nk + attn::kBlockN - 1) / attn::kBlockN);
  attn::BwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.dq = reinterpret_cast<__nv_bfloat16*>(dq);
  p.dk = reinterpret_cast<__nv_bfloat16*>(dk);
  p.dv = reinterpret_cast<__nv_bfloat16*>(dv);
  float* nlse2 = reinterpret_cast<float*>(workspace);
  float* ndelta = reinterpret_cast<float*>(static_cast<char*>(workspace) + part);
  p.nlse2 = nlse2;
  p.ndelta = ndelta;
  p.Hq = Hkv;
  p.Hkv = Hkv;
  p.Npad = nq * attn::kBlockN;
  p.group = 1;
  p.c = scale * attn::kLog2e;
  p.scale = scale;
  p.idesc_s = attn::idesc_bf16_f32(attn::kBlockM, attn::kBlockN, false, false, false);
  p.idesc_acc = attn::idesc_bf16_f32(attn::kBlockM, D, false, true, false);
  p.k_lens = k_lens;
  p.Nk = Nk;
  p.col_blocks = nq;
  attn::BwdParams pkv = p, pq = p;
  pkv.N = Nk;
  pkv.num_blocks = nk;
  pkv.num_items = (int)(heads * nk);
  pq.N = (int)GT;
  pq.num_blocks = nq;
  pq.num_items = (int)(heads * nq);

  const long long rows = heads * p.Npad;
  const long long rows_per_block = 256 / 16 * attn::kPrepRows;
  attn::attn_bwd_prep<<<(unsigned)((rows + rows_per_block - 1) / rows_per_block), 256, 0, s>>>(
      reinterpret_cast<const __nv_bfloat16*>(o), reinterpret_cast<const __nv_bfloat16*>(dout), lse, nlse2, ndelta,
      rows, (int)GT, p.Npad, D);
  switch (D) {
    case 32: launch_cross_bwd_dim<32>(mq, mk, mv, mdo, pkv, pq, num_sms, s); break;
    case 64: launch_cross_bwd_dim<64>(mq, mk, mv, mdo, pkv, pq, num_sms, s); break;
    case 96: launch_cross_bwd_dim<96>(mq, mk, mv, mdo, pkv, pq, num_sms, s); break;
    default: launch_cross_bwd_dim<128>(mq, mk, mv, mdo, pkv, pq, num_sms, s); break;
  }
  return launch_status("cross-attention backward kernel launch");
}

}  // extern "C"
