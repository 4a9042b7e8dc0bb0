// mla_common.cuh - what the tensor-core attention kernels (bf16 rows, packed
// 4-bit rows) share: softmax constants, roundings and profiling stamps.
#pragma once

#include <cuda_bf16.h>

#include "dsa_kernels.cuh"

namespace dsa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// 2^x with the hardware approximation (ex2.approx.ftz.f32; 2^-inf = +0).
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// f[0..8) * inv as eight bf16 (round to nearest even) in one 16-byte piece.
__device__ __forceinline__ uint4 pack8(const float* f, float inv) {
  return make_uint4(pack_bf16x2(f[0] * inv, f[1] * inv), pack_bf16x2(f[2] * inv, f[3] * inv),
                    pack_bf16x2(f[4] * inv, f[5] * inv), pack_bf16x2(f[6] * inv, f[7] * inv));
}
// Profiling stamp: event `ev` of block j in the first cluster's first pair.
__device__ __forceinline__ void tstamp(long long* tr, uint32_t rank, int ev, int j) {
  if (tr != nullptr && blockIdx.x < 2 && j < kTraceBlocks)
    tr[((int)rank * kTraceEvents + ev) * kTraceBlocks + j] = clock64();
}

}  // namespace dsa
