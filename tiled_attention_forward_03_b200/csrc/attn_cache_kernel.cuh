// attn_cache_kernel.cuh -- writing key/value rows into a paged cache and reading them back, for
// B200 (sm_100a).
//
// A cache is [num_pages][Hkv][page][D], bf16 or E4M3; position p of sequence b is row p % page of
// page table[b][p / page].  An E4M3 cache has one exponent e for each token and head, stored as an
// E8M0 byte e + 127 in [num_pages][Hkv][page]: a value is code * 2^e.  With amax the largest
// magnitude of the row,
//
//   e = the least integer >= -120 with amax <= 448 * 2^e,   code = E4M3(x * 2^-e)  (nearest even).
//
// A power of two moves the binade of the codes and rounds nothing, so every code * 2^e is a bf16
// number exactly (4 significant bits; 2^-9 * 2^-120 is above bf16's least subnormal) and the only
// rounding of the round trip is the one to E4M3, at most 2^-4 of the value (2^-10 * 2^e below the
// codes' least normal number).  The exponent comes from the largest magnitude's own bits: for
// amax = (1 + M/128) 2^(E-127), 448 = 1.75 * 2^8 gives e = E - 135, plus 1 when M > 96.  At e = 120
// codes stop at 240, because 256 * 2^120 is infinite.  A row with an infinity or a NaN is marked:
// e byte 255 (E8M0's NaN) and codes 0; it reads back as NaN.
//
// Both kernels move each byte once and are bound by HBM (short calls by launch and the
// dependent look-ups lens -> table -> row).  Measured: reading 340 MB of a batch back (B16 Hkv8 N<=4096
// D128 E4M3 to bf16) 57 us, 5.9 TB/s; appending 57 MB (B4 Hkv8 T<=4096) 18 us (20.5 with L2 flushed
// before), with the quantising's integer work as large as the copy's time.
#pragma once

#include <cuda_bf16.h>

#include "attn_fwd_kernel.cuh"  // FastDiv, and the PTX wrappers

namespace attn {

constexpr int kE8Nan = 255;

// The factor an E8M0 byte stands for: 2^(e8 - 127), NaN for 255.
__device__ __forceinline__ float e8_scale(int e8) {
  return __uint_as_float(e8 == kE8Nan ? 0x7fffffffu : e8 == 0 ? 0x00400000u : (uint32_t)e8 << 23);
}

// Where the cache lives and how long its sequences are.
struct CacheView {
  void* k;
  void* v;
  uint8_t* ks;        // E8M0 bytes, null for a bf16 cache
  uint8_t* vs;
  const int* table;   // [B][max_pages]
  const int* lens;    // [B], or null (reading): len_all
  int len_all;
  int max_pages, num_pages, page, Hkv;
  FastDiv div_page;
};

// Row (p of sequence b, head h) of the cache, or -1: the position is outside the table, or the
// table's entry is not a page.
__device__ __forceinline__ long long cache_row(const CacheView& c, int b, int h, long long pos) {
  if (pos < 0 || pos > 0x7fffffffLL) return -1;
  const uint32_t pg = fast_div((uint32_t)pos, c.div_page);
  if (pg >= (uint32_t)c.max_pages) return -1;
  const int id = __ldg(c.table + (size_t)b * c.max_pages + pg);
  if ((unsigned)id >= (unsigned)c.num_pages) return -1;
  return ((long long)id * c.Hkv + h) * c.page + ((uint32_t)pos - pg * (uint32_t)c.page);
}

// Larger of each pair of unsigned 16-bit halves.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// E8M0 byte of a row from the largest magnitude bits (bf16 without the sign) of its elements.
__device__ __forceinline__ int e8_of_amax(uint32_t bits) {
  if (bits >= 0x7f80u) return kE8Nan;
  const int e = (int)(bits >> 7) - 135 + ((bits & 127u) > 96u ? 1 : 0);
  return max(e, -120) + 127;
}

// Appends rows t < new_lens[b] of k, v [B][Hkv][T][D] at positions lens[b] + t.  A group of G lanes
// takes kRows rows of K and of V (16 bytes a lane and row, all loads issued before any use); a row's
// largest magnitude is a shuffle over the group.  kRows = 4 where the rows fill the GPU several times
// over: 57 MB of a quantised prompt batch (B4 Hkv8 T<=4096 D128) take 20.5 us (L2 flushed), with one row 22.5;
// T512 10.4 and 8.2.
template <int D, bool kF8, int kRows>
__global__ void __launch_bounds__(256) attn_cache_append_kernel(const __nv_bfloat16* __restrict__ k,
                                                                const __nv_bfloat16* __restrict__ v, CacheView c,
                                                                const int* __restrict__ new_lens, int T,
                                                                FastDiv div_t, FastDiv div_h, uint32_t rows) {
  constexpr int kLanes = D / 8;                                       // lanes with data
  constexpr int G = kLanes <= 4 ? 4 : kLanes <= 8 ? 8 : 16;
  const unsigned long long first = ((unsigned long long)blockIdx.x * blockDim.x + threadIdx.x) / G * kRows;
  const int lane = threadIdx.x & (G - 1);
  if (first >= rows) return;   // whole groups leave together
  // each step's loads of all rows before the next step's: counts and lengths, data and pages
  uint32_t bs[kRows], hs[kRows];
  int ts[kRows], have[kRows], news[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t row = (uint32_t)min(first + i, (unsigned long long)rows - 1);
    const uint32_t bh = fast_div(row, div_t);
    ts[i] = (int)(row - bh * (uint32_t)T);
    bs[i] = fast_div(bh, div_h);
    hs[i] = bh - bs[i] * (uint32_t)c.Hkv;
    news[i] = first + i < rows ? (new_lens != nullptr ? __ldg(new_lens + bs[i]) : T) : 0;
    have[i] = __ldg(c.lens + bs[i]);
  }
  uint4 x[kRows][2];
  int ids[kRows];
  uint32_t in_page[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const long long pos = (long long)have[i] + ts[i];
    const bool live = ts[i] < news[i] && pos >= 0 && pos <= 0x7fffffffLL;
    const uint32_t pg = fast_div((uint32_t)pos, c.div_page);
    in_page[i] = (uint32_t)pos - pg * (uint32_t)c.page;
    const bool placed = live && pg < (uint32_t)c.max_pages;
    ids[i] = placed ? __ldg(c.table + (size_t)bs[i] * c.max_pages + pg) : -1;
    const bool load = placed && lane < kLanes;
    x[i][0] = load ? __ldcs(reinterpret_cast<const uint4*>(k + (size_t)(first + i) * D) + lane) : make_uint4(0u, 0u, 0u, 0u);
    x[i][1] = load ? __ldcs(reinterpret_cast<const uint4*>(v + (size_t)(first + i) * D) + lane) : make_uint4(0u, 0u, 0u, 0u);
  }
  long long dst[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    dst[i] = (unsigned)ids[i] < (unsigned)c.num_pages ? ((long long)ids[i] * c.Hkv + hs[i]) * c.page + in_page[i] : -1;
  const unsigned mask = ((G == 16 ? 0xffffu : G == 8 ? 0xffu : 0xfu)) << (threadIdx.x & 31 & ~(G - 1));
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (dst[i] < 0) continue;   // (the whole group)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (!kF8) {
        if (lane < kLanes) reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(j ? c.v : c.k) + dst[i] * D)[lane] = x[i][j];
      } else {
        const uint32_t w[4] = {x[i][j].x, x[i][j].y, x[i][j].z, x[i][j].w};
        // largest magnitude bits, two columns at a time (integer order is the order of magnitudes)
        uint32_t top = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                 max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
#pragma unroll
        for (int d = G / 2; d > 0; d >>= 1) top = max_u16x2(top, __shfl_xor_sync(mask, top, d, G));
        const int e8 = e8_of_amax(max(top & 0xffffu, top >> 16));
        uint2 out = make_uint2(0u, 0u);
        if (e8 != kE8Nan) {
          const float inv = __uint_as_float((uint32_t)(254 - e8) << 23);   // 2^-e
          float y[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[2 * e] = __uint_as_float(w[e] << 16) * inv;
            y[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * inv;
          }
          if (e8 >= 247) {   // (the conversion itself stops at 448)
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fminf(fmaxf(y[e], -240.f), 240.f);
          }
          out.x = pack_e4m3x4(y[0], y[1], y[2], y[3]);
          out.y = pack_e4m3x4(y[4], y[5], y[6], y[7]);
        }
        if (lane < kLanes) reinterpret_cast<uint2*>(static_cast<uint8_t*>(j ? c.v : c.k) + dst[i] * D)[lane] = out;
        if (lane == 0) (j ? c.vs : c.ks)[dst[i]] = (uint8_t)e8;
      }
    }
  }
}

// Four E4M3 codes -> two bf16 pairs times 2^(e8 - 127), exactly; all NaN for e8 = 255.  The halves
// of each 16-bit float the hardware converts to are exact, and so is the fp32 product.
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t w, int e8) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  const float s = e8_scale(e8);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_uint2(pack_bf16x2(a.x * s, a.y * s), pack_bf16x2(b.x * s, b.y * s));
}

// Positions [0, N) of every sequence into k_out, v_out [B][Hkv][N][D] (bf16): zeros at and past
// lens[b] and where the table names no page.  A thread takes 8 columns (16 bytes of output, so that a
// warp's stores are contiguous) of one row of K and of V; two rows a thread took as long at 340 MB, and
// 9 us instead of 8 at 4 MB.
template <int D, bool kF8>
__global__ void __launch_bounds__(256) attn_cache_read_kernel(CacheView c, __nv_bfloat16* __restrict__ k_out,
                                                              __nv_bfloat16* __restrict__ v_out, int N, FastDiv div_n,
                                                              FastDiv div_h, unsigned long long items) {
  constexpr int kPieces = D / 8;
  const unsigned long long item = (unsigned long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= items) return;
  const uint32_t row = (uint32_t)(item / kPieces);
  const int d = (int)(item - (unsigned long long)row * kPieces) * 8;
  const uint32_t bh = fast_div(row, div_n);
  const int pos = (int)(row - bh * (uint32_t)N);
  const uint32_t b = fast_div(bh, div_h);
  const bool live = pos < (c.lens != nullptr ? __ldg(c.lens + b) : c.len_all);
  const long long src = live ? cache_row(c, (int)b, (int)(bh - b * (uint32_t)c.Hkv), pos) : -1;
  uint4 o[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  int e[2] = {127, 127};
  if (src >= 0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (kF8) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(j ? c.v : c.k) + src * D + d));
        o[j].x = w.x;
        o[j].y = w.y;
        e[j] = (j ? c.vs : c.ks)[src];
      } else {
        o[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(j ? c.v : c.k) + src * D + d));
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if constexpr (kF8) {
      const uint2 x = e4m3x4_to_bf16(o[j].x, e[j]), y = e4m3x4_to_bf16(o[j].y, e[j]);
      o[j] = make_uint4(x.x, x.y, y.x, y.y);
    }
    __stcs(reinterpret_cast<uint4*>(j ? v_out : k_out) + item, o[j]);
  }
}

// Products of bf16 pairs (nearest even; subnormal operands and results count).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two E4M3 codes in the high bytes of r's halves (the low bytes are ignored) as a bf16 pair times
// 2^-120, exactly: the sign stays, exponent and mantissa move four bits down.
__device__ __forceinline__ uint32_t e4m3_hi2_bits(uint32_t r) { return ((r >> 4) & 0x07f007f0u) | (r & 0x80008000u); }

// Four E4M3 codes times 2^-120 f -> two bf16 pairs, exactly where the products are bf16 numbers.
__device__ __forceinline__ uint2 e4m3x4_scaled(uint32_t w, uint32_t f) {
  return make_uint2(mul_bf16x2(e4m3_hi2_bits(__byte_perm(w, 0u, 0x1000)), f),
                    mul_bf16x2(e4m3_hi2_bits(__byte_perm(w, 0u, 0x3020)), f));
}

// An E8M0 factor as a bf16 pair.
__device__ __forceinline__ uint32_t e8_bf16x2(int e8) {
  const uint32_t b = e8 == kE8Nan ? 0x7fc0u : e8 == 0 ? 0x0040u : (uint32_t)e8 << 7;
  return b | (b << 16);
}

}  // namespace attn
