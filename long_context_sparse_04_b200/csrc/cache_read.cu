// cache_read.cu - gather cached tokens by physical row and dequantise them: the
// first step of an un-absorbed prefill over a cached context ("DeepSeek Sparse
// Attention DSA Architecture Guide", section "The Classical Multi-Head Latent
// Attention (MLA) Mechanism": keys and values are up-projected from the latent),
// and of moving a sequence to another cache.
//
//   k_out[n]      = fl32(e4m3 code * scale)          (one rounding)
//   latent_out[n] = code * scale per 16 dims, bf16   (exact), RoPE key copied
//
// A stream: with 4-bit latents 548 bytes in and 1,664 out per token, so writes
// bound it.  One warp per token; a lane decodes one group of 16 dims (8 bytes of
// codes) into 32 bytes.
#include <cuda_fp8.h>

#include "dsa_int4.cuh"
#include "dsa_kernels.cuh"

namespace dsa {
namespace {

constexpr int kWarpsPerCta = 8;

__device__ __forceinline__ float4 e4m3x4_to_f32(uint32_t w, float s) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half_raw h =
        __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>((w >> (8 * i)) & 0xFFu), __NV_E4M3);
    f[i] = __half2float(__half(h)) * s;
  }
  return make_float4(f[0], f[1], f[2], f[3]);
}

template <bool kInt4>
__global__ void __launch_bounds__(kWarpsPerCta * 32) cache_read_kernel(const ReadArgs a) {
  pdl_launch_dependents();
  trace_kernel(a.status, DSA_KERNEL_CACHE_READ);
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  if (n >= a.n) return;
  const int64_t row = a.slot[n];
  if (row < 0) return;
  if (row >= a.num_tokens) {
    if (lane == 0) set_status(a.status, DSA_ERR_OUT_OF_RANGE, n);
    return;
  }
  if (a.k_out != nullptr) {
    float4* dst = reinterpret_cast<float4*>(a.k_out + (int64_t)n * a.d_idx);
    const int chunks = a.d_idx >> 2;
    if (a.idx_dtype == DSA_FP8_E4M3) {
      const float s = a.idx_k_scale[row];
      const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.idx_k) + row * a.d_idx);
      for (int c = lane; c < chunks; c += 32) dst[c] = e4m3x4_to_f32(src[c], s);
    } else {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.idx_k) + row * a.d_idx);
      for (int c = lane; c < chunks; c += 32) dst[c] = src[c];
    }
  }
  if (a.latent_out == nullptr) return;
  const uint8_t* src = static_cast<const uint8_t*>(a.latent) + row * a.latent_row_bytes;
  if constexpr (kInt4) {
    const Int4Row ly = int4_row(a.d_c, a.d_r);
    const int groups = a.d_c / kInt4Group, pieces = a.d_r >> 3;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.latent_out) + (int64_t)n * (a.d_c + a.d_r));
    for (int g = lane; g < groups; g += 32) {
      const uint2 w = reinterpret_cast<const uint2*>(src)[g];
      const ScalePair s = scale_pair(src[ly.scale + g]);
      dst[2 * g] = decode_word(w.x, s);
      dst[2 * g + 1] = decode_word(w.y, s);
    }
    for (int c = lane; c < pieces; c += 32)
      dst[2 * groups + c] = reinterpret_cast<const uint4*>(src + ly.rope)[c];
  } else {
    const int pieces = a.latent_row_bytes >> 4;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.latent_out) + (int64_t)n * a.latent_row_bytes);
    for (int c = lane; c < pieces; c += 32) dst[c] = reinterpret_cast<const uint4*>(src)[c];
  }
}

}  // namespace

dsa_status launch_cache_read(const ReadArgs& a, cudaStream_t stream) {
  if (a.n == 0) return DSA_OK;
  const unsigned grid = (unsigned)(((int64_t)a.n + kWarpsPerCta - 1) / kWarpsPerCta);
  (a.int4 ? cache_read_kernel<true> : cache_read_kernel<false>)<<<grid, kWarpsPerCta * 32, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("cache read launch failed: %s", cudaGetErrorString(e));
    return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

}  // namespace dsa
