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
// dependent look-ups lens -> table -> row).
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
  const int* lens;    // [B]
  int max_pages, num_pages, page, Hkv;
  FastDiv div_page;
};

// Row (p of sequence b, head h) of the cache, or -1: the position is outside the table, or the
// table's entry is not a page.
__device__ __forceinline__ long long cache_row(const CacheView& c, int b, int h, long long pos) {
  if (pos < 0 || pos > 0x7fffffffLL) return -1;
  const uint32_t pg = fast_div((uint32_t)pos, c.div_page);
  if (pg >= (uint32_t)c.max_pages) return -1;
  const int id = c.table[(size_t)b * c.max_pages + pg];
  if ((unsigned)id >= (unsigned)c.num_pages) return -1;
  return ((long long)id * c.Hkv + h) * c.page + ((uint32_t)pos - pg * (uint32_t)c.page);
}

// E8M0 byte of a row from the largest magnitude bits (bf16 without the sign) of its elements.
__device__ __forceinline__ int e8_of_amax(uint32_t bits) {
  if (bits >= 0x7f80u) return kE8Nan;
  const int e = (int)(bits >> 7) - 135 + ((bits & 127u) > 96u ? 1 : 0);
  return max(e, -120) + 127;
}

// Appends rows t < new_lens[b] of k, v [B][Hkv][T][D] at positions lens[b] + t.  A group of G lanes
// takes one row of K and the same row of V (16 bytes a lane, both loads issued before any use); the
// row's largest magnitude is a shuffle over the group.  Measured on B200: the 57 MB of a quantised
// prompt batch (B4 H8 T4096 ragged, D128) at the rate given in the table of the design notes; a
// single token a sequence is launch-bound.
template <int D, bool kF8>
__global__ void __launch_bounds__(256) attn_cache_append_kernel(const __nv_bfloat16* __restrict__ k,
                                                                const __nv_bfloat16* __restrict__ v, CacheView c,
                                                                const int* __restrict__ new_lens, int T,
                                                                FastDiv div_t, FastDiv div_h, uint32_t rows) {
  constexpr int kLanes = D / 8;                                       // lanes with data
  constexpr int G = kLanes <= 4 ? 4 : kLanes <= 8 ? 8 : kLanes <= 16 ? 16 : 32;
  const uint32_t row = (uint32_t)(((unsigned long long)blockIdx.x * blockDim.x + threadIdx.x) / G);
  const int lane = threadIdx.x & (G - 1);
  if (row >= rows) return;   // whole groups leave together
  const bool live = lane < kLanes;
  uint4 x[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (live) {
    x[0] = __ldcs(reinterpret_cast<const uint4*>(k + (size_t)row * D) + lane);
    x[1] = __ldcs(reinterpret_cast<const uint4*>(v + (size_t)row * D) + lane);
  }
  const uint32_t bh = fast_div(row, div_t);
  const int t = (int)(row - bh * (uint32_t)T);
  const uint32_t b = fast_div(bh, div_h);
  const int h = (int)(bh - b * (uint32_t)c.Hkv);
  if (new_lens != nullptr && t >= new_lens[b]) return;
  const long long dst = cache_row(c, (int)b, h, (long long)c.lens[b] + t);
  if (dst < 0) return;
  if constexpr (!kF8) {
    if (live) {
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.k) + dst * D)[lane] = x[0];
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.v) + dst * D)[lane] = x[1];
    }
  } else {
    const unsigned mask = (G == 32 ? 0xffffffffu : ((1u << G) - 1u) << (threadIdx.x & 31 & ~(G - 1)));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t top = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
      for (int d = G / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(mask, top, d, G));
      const int e8 = e8_of_amax(top);
      uint2 out = make_uint2(0u, 0u);
      if (e8 != kE8Nan) {
        const float inv = __uint_as_float((uint32_t)(254 - e8) << 23);   // 2^-e
        const float lim = e8 >= 247 ? 240.f : 448.f;
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = __uint_as_float(w[e] << 16) * inv;
          y[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * inv;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fminf(fmaxf(y[e], -lim), lim);
        out.x = pack_e4m3x4(y[0], y[1], y[2], y[3]);
        out.y = pack_e4m3x4(y[4], y[5], y[6], y[7]);
      }
      if (live) reinterpret_cast<uint2*>(static_cast<uint8_t*>(i ? c.v : c.k) + dst * D)[lane] = out;
      if (lane == 0) (i ? c.vs : c.ks)[dst] = (uint8_t)e8;
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
// lens[b] and where the table names no page.  A thread takes 16 columns of one row of K and of V.
template <int D, bool kF8>
__global__ void __launch_bounds__(256) attn_cache_read_kernel(CacheView c, __nv_bfloat16* __restrict__ k_out,
                                                              __nv_bfloat16* __restrict__ v_out, int N, FastDiv div_n,
                                                              FastDiv div_h, unsigned long long items) {
  constexpr int kPieces = D / 16;
  const unsigned long long item = (unsigned long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (item >= items) return;
  const uint32_t row = (uint32_t)(item / kPieces);
  const int d = (int)(item - (unsigned long long)row * kPieces) * 16;
  const uint32_t bh = fast_div(row, div_n);
  const int pos = (int)(row - bh * (uint32_t)N);
  const uint32_t b = fast_div(bh, div_h);
  const int h = (int)(bh - b * (uint32_t)c.Hkv);
  const long long src = pos < c.lens[b] ? cache_row(c, (int)b, h, pos) : -1;
  uint4 o[2][2] = {};
  if (src >= 0) {
    if constexpr (kF8) {
      const uint4 kw = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.k) + src * D + d));
      const uint4 vw = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.v) + src * D + d));
      const int ek = c.ks[src], ev = c.vs[src];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 w = i ? vw : kw;
        const int e = i ? ev : ek;
        const uint2 a0 = e4m3x4_to_bf16(w.x, e), a1 = e4m3x4_to_bf16(w.y, e);
        const uint2 a2 = e4m3x4_to_bf16(w.z, e), a3 = e4m3x4_to_bf16(w.w, e);
        o[i][0] = make_uint4(a0.x, a0.y, a1.x, a1.y);
        o[i][1] = make_uint4(a2.x, a2.y, a3.x, a3.y);
      }
    } else {
      const uint4* kp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.k) + src * D + d);
      const uint4* vp = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.v) + src * D + d);
      o[0][0] = __ldcs(kp);
      o[0][1] = __ldcs(kp + 1);
      o[1][0] = __ldcs(vp);
      o[1][1] = __ldcs(vp + 1);
    }
  }
  uint4* ko = reinterpret_cast<uint4*>(k_out + (size_t)row * D + d);
  uint4* vo = reinterpret_cast<uint4*>(v_out + (size_t)row * D + d);
  ko[0] = o[0][0];
  ko[1] = o[0][1];
  vo[0] = o[1][0];
  vo[1] = o[1][1];
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
