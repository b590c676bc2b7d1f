// Warp-level pieces of the single-token kernels over the 8-bit cache: codes
// to fp16 MMA fragments, query fragments, exponentials.
//
// Tokens are the MMA's rows and query rows its columns (m16n8k16, fp16 in,
// fp32 sums): S^T[16 tokens][8 rows] = K q^T, then O^T[dims][8 rows] = V^T p^T.
// A group of eight query rows on one key head fills a column tile exactly,
// where rows of 16 would be half empty, and every code is read and converted
// once for all of them.  Codes become fp16 exactly: byte u under the
// pattern 0x6400 is 1024 + u, minus 1152 gives u - 128 (one byte permute and
// one packed subtraction for two codes).
#pragma once

#include <cuda_fp16.h>

#include "kv8.cuh"

namespace w4 {
namespace kv8 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t sub1152(uint32_t v) {
  const __half2 k = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&v), k);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Codes 0, 1 (lo) and 2, 3 (hi) of a word as fp16 pairs u - 128.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  return sub1152(__byte_perm(w, 0x64646464u, 0x4140));
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  return sub1152(__byte_perm(w, 0x64646464u, 0x4342));
}

__device__ __forceinline__ void mma16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Power of two that brings a row whose largest |value| is m to [2^14, 2^15)
// (fp16's upper end, so that only values 2^-28 below it lose bits), and its
// inverse.  m = 0 or not finite: 1.
__device__ __forceinline__ void row_scale(float m, float* up, float* down) {
  const int e = (int)(__float_as_uint(m) >> 23) - 127;
  const int s = (m == 0.0f || e == 128) ? 0 : max(-113, min(126, 14 - e));
  *up = __uint_as_float((uint32_t)(s + 127) << 23);
  *down = __uint_as_float((uint32_t)(127 - s) << 23);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Query fragments of one tile of 8 rows for the column operand.  Lane (i, j)
// = (lane / 4, lane % 4) holds row i; its D / 4 channels are, for each
// 128-channel half of the head (or all 64), the 16-byte chunks of codes that
// the same j reads from a key row: 2j and 2j + 1 of eight, or j of four.
// Step s of 16 channels multiplies word s of those.  `row` null: zeros.  The
// loads are apart from their use, so that other chains run in between.
template <int D>
__device__ __forceinline__ void load_query(const __nv_bfloat16* row, int j, uint2 (&raw)[D / 16]) {
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    const int ch = D == 64 ? 16 * j + 4 * s : 128 * (s / 8) + 32 * j + 4 * (s % 8);
    raw[s] = row == nullptr ? make_uint2(0, 0) : load_in(reinterpret_cast<const uint2*>(row + ch));
  }
}

// The loaded row as fragments; returns the row's down factor.
template <int D>
__device__ __forceinline__ float scale_query(const uint2 (&raw)[D / 16], uint32_t (&b)[D / 16][2]) {
  float m = 0.0f;
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
    m = fmaxf(m, fmaxf(fmaxf(fabsf(bf16_lo(raw[s].x)), fabsf(bf16_hi(raw[s].x))),
                       fmaxf(fabsf(bf16_lo(raw[s].y)), fabsf(bf16_hi(raw[s].y)))));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
  float up, down;
  row_scale(m, &up, &down);
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    b[s][0] = pack_half2(bf16_lo(raw[s].x) * up, bf16_hi(raw[s].x) * up);
    b[s][1] = pack_half2(bf16_lo(raw[s].y) * up, bf16_hi(raw[s].y) * up);
  }
  return down;
}

// 16-byte chunk `chunk` of row `row` of a 16-token slice in shared memory, as
// the tiled copy swizzles it: rows of 128 bytes, chunk ^ (row % 8); rows of
// 64 bytes, chunk ^ (row / 2 % 4).
template <int D>
__device__ __forceinline__ uint32_t slice_offset(int row, int chunk) {
  if (D == 64) return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
  return (uint32_t)((chunk >> 3) * 2048 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// S^T of one slice: keys at shared address `ks` (16 rows), NQ column tiles.
// acc[n][0..3]: tokens i, i, i + 8, i + 8 by rows 2j, 2j + 1, 2j, 2j + 1 of tile n.
template <int D, int NQ>
__device__ __forceinline__ void key_scores(uint32_t ks, int i, int j,
                                           const uint32_t (&q)[NQ][D / 16][2], float (&acc)[NQ][4]) {
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {   // this lane's chunks
    const int chunk = D == 64 ? j : 8 * (c / 2) + 2 * j + (c & 1);
    const uint4 x = lds128(ks + slice_offset<D>(i, chunk));
    const uint4 y = lds128(ks + slice_offset<D>(i + 8, chunk));
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t a0 = codes_lo(xw[w]), a1 = codes_lo(yw[w]);
      const uint32_t a2 = codes_hi(xw[w]), a3 = codes_hi(yw[w]);
#pragma unroll
      for (int n = 0; n < NQ; ++n)
        mma16816(acc[n], a0, a1, a2, a3, q[n][4 * c + w][0], q[n][4 * c + w][1]);
    }
  }
}

// O^T += V^T p^T of one slice: values at shared address `vs`; p[n][0..1] the
// column operand (tokens 2j, 2j + 1 and 2j + 8, 2j + 9 of row i of tile n).
// o[n][t][0..3]: channels c, c, c + 1, c + 1 by rows 2j, 2j + 1, 2j, 2j + 1, where
// c = value_channel<D>(i, t).
template <int D>
__device__ __forceinline__ int value_channel(int i, int t) {
  return D == 64 ? 8 * i + 2 * t : 128 * (t / 8) + 16 * i + 2 * (t % 8);
}

// kScaled: the products are added times `factor` (an exact power of two).
template <bool kScaled, int NQ, int T>
__device__ __forceinline__ void value_mma(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          const uint32_t (&p)[NQ][2], float (&o)[NQ][T][4], int t,
                                          float factor) {
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    if (kScaled) {
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      mma16816(x, a0, a1, a2, a3, p[n][0], p[n][1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][t][e] = fmaf(x[e], factor, o[n][t][e]);
    } else {
      mma16816(o[n][t], a0, a1, a2, a3, p[n][0], p[n][1]);
    }
  }
}

template <bool kScaled, int NQ, int T>
__device__ __forceinline__ void value_word(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3,
                                           const uint32_t (&p)[NQ][2], float (&o)[NQ][T][4],
                                           int t, float factor) {
  // bytes of tokens 2j and 2j + 1 (and 2j + 8, 2j + 9) side by side
  const uint32_t x0 = __byte_perm(r0, r1, 0x5140), x1 = __byte_perm(r0, r1, 0x7362);
  const uint32_t y0 = __byte_perm(r2, r3, 0x5140), y1 = __byte_perm(r2, r3, 0x7362);
  value_mma<kScaled, NQ>(codes_lo(x0), codes_hi(x0), codes_lo(y0), codes_hi(y0), p, o, t, factor);
  value_mma<kScaled, NQ>(codes_lo(x1), codes_hi(x1), codes_lo(y1), codes_hi(y1), p, o, t + 1, factor);
}

template <bool kScaled, int D, int NQ>
__device__ __forceinline__ void value_sums(uint32_t vs, int i, int j, const uint32_t (&p)[NQ][2],
                                           float (&o)[NQ][D / 16][4], float factor = 1.0f) {
  if (D == 64) {
    const uint32_t off = (i & 1) * 8;
    const uint2 a = lds64(vs + slice_offset<D>(2 * j, i >> 1) + off);
    const uint2 b = lds64(vs + slice_offset<D>(2 * j + 1, i >> 1) + off);
    const uint2 c = lds64(vs + slice_offset<D>(2 * j + 8, i >> 1) + off);
    const uint2 d = lds64(vs + slice_offset<D>(2 * j + 9, i >> 1) + off);
    value_word<kScaled, NQ>(a.x, b.x, c.x, d.x, p, o, 0, factor);
    value_word<kScaled, NQ>(a.y, b.y, c.y, d.y, p, o, 2, factor);
  } else {
#pragma unroll
    for (int half = 0; half < D / 128; ++half) {
      const uint4 a = lds128(vs + slice_offset<D>(2 * j, 8 * half + i));
      const uint4 b = lds128(vs + slice_offset<D>(2 * j + 1, 8 * half + i));
      const uint4 c = lds128(vs + slice_offset<D>(2 * j + 8, 8 * half + i));
      const uint4 d = lds128(vs + slice_offset<D>(2 * j + 9, 8 * half + i));
      value_word<kScaled, NQ>(a.x, b.x, c.x, d.x, p, o, 8 * half, factor);
      value_word<kScaled, NQ>(a.y, b.y, c.y, d.y, p, o, 8 * half + 2, factor);
      value_word<kScaled, NQ>(a.z, b.z, c.z, d.z, p, o, 8 * half + 4, factor);
      value_word<kScaled, NQ>(a.w, b.w, c.w, d.w, p, o, 8 * half + 6, factor);
    }
  }
}

}  // namespace kv8
}  // namespace w4
