// dsa_int4.cuh - packed latent rows (mla_dtype = DSA_INT4): layout, the 8-bit
// group scale and the conversions in both directions.  The format is defined in
// include/dsa.h.
//
// Decoding costs three instructions per pair of dims, by a method in common use: a
// small integer placed under the bits of a floating-point number converts itself.  A
// 4-bit two's complement code q XOR 8 is q + 8, so (nibble ^ 8) placed under the bf16
// pattern of 128 reads as 136 + q; times the scale S minus 136 S gives q S.  All of it
// is exact in bf16: S has at most 4 significant bits, 136 S = 17 * 8 * S at most 8
// (17 * 15 < 256), and q S at most 8.
#pragma once

#include <cuda_bf16.h>

#include "dsa_common.cuh"

namespace dsa {

constexpr int kInt4Group = 16;             // latent dims per scale
constexpr uint32_t kScaleMax = 0xF7;       // 61440, the largest scale the writers use

// Byte offsets within a packed row.
struct Int4Row {
  int rope, scale, bytes;
};
__host__ __device__ constexpr Int4Row int4_row(int d_c, int d_r) {
  return Int4Row{d_c / 2, d_c / 2 + 2 * d_r, (d_c / 2 + 2 * d_r + d_c / kInt4Group + 15) / 16 * 16};
}

// Value of scale byte b: 5 exponent bits (bias 15), 3 mantissa bits, subnormals.
__device__ __forceinline__ float scale_value(uint32_t b) {
  const uint32_t e = b >> 3, m = b & 7u;
  return e ? __uint_as_float(((e + 112u) << 23) | (m << 20)) : (float)m * 7.62939453125e-6f;   // 2^-17
}
// Nearest scale byte to r >= 0 (ties to even), at most kScaleMax.
__device__ __forceinline__ uint32_t scale_code(float r) {
  uint32_t c;
  if (r < 6.103515625e-5f) {                                     // 2^-14: steps of 2^-17
    c = (uint32_t)__float2int_rn(r * 131072.f);
  } else {
    const uint32_t u = __float_as_uint(r);
    c = ((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - (112u << 3);  // round to 3 mantissa bits
  }
  return c < kScaleMax ? c : kScaleMax;
}

// The bf16x2 constants (S, S) and (-136 S, -136 S) of scale byte `b`.  Shifted
// left by 4 the byte is the bf16 pattern of S * 2^-112 (subnormals included).
struct ScalePair {
  __nv_bfloat162 s, off;
};
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t u) {
  return *reinterpret_cast<__nv_bfloat162*>(&u);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ ScalePair scale_pair(uint32_t b) {
  ScalePair p;
  // 0x7780 = 2^112, 0xFB08 = -136 * 2^112
  const __nv_bfloat162 x = as_bf162((b << 4) * 0x00010001u);
  p.s = __hmul2(x, as_bf162(0x77807780u));
  p.off = __hmul2(x, as_bf162(0xFB08FB08u));
  return p;
}
// Eight dims of one word as four bf16x2, in order.  (The and-xor is written as one
// lop3 with both constants in registers: with literals it became two.)
__device__ __forceinline__ uint4 decode_word(uint32_t w, const ScalePair& p) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(x) : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(0x43084308u));   // (a & b) ^ c
    r[i] = as_u32(__hfma2(as_bf162(x), p.s, p.off));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Latent dim d of a packed row as fp32 (exact).
__device__ __forceinline__ float int4_dim(const uint8_t* row, int d, const Int4Row& ly) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(row)[d >> 3];
  const int nib = ((d & 1) << 2) + ((d & 7) >> 1);
  const int q = (int)((w >> (4 * nib)) << 28) >> 28;
  return (float)q * scale_value(row[ly.scale + d / kInt4Group]);
}

}  // namespace dsa
