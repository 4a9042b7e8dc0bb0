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
// bound it.  131,072 tokens take 55.4 us, 5.3 TB/s (a kernel that copies 218 MB of
// such output alone ran at 5.9); bf16 rows (387 MB) 79.6 us against a floor of 59.2, fp32
// (739 MB) 122 against 113.  One warp per token, CTAs of four, fourteen an SM, for whose 32
// registers a thread the compiler spills 28 bytes and reloads 60: ten CTAs, without a spill,
// took 57.4, twelve 65.5, sixteen the same as fourteen.  Eight warps a CTA took 57.6 us,
// sixteen 61.7, two 71; two tokens a warp, persistent warps and a ring filled by cp.async
// 70-89; 32-byte stores 66.7.
#include <cuda_fp8.h>

#include "dsa_int4.cuh"
#include "dsa_kernels.cuh"

namespace dsa {
namespace {

constexpr int kWarpsPerCta = 4;

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

// Streaming stores: the output is not read again here.
__device__ __forceinline__ void st_stream(uint4* p, const uint4& v) { __stcs(p, v); }

__device__ __forceinline__ int64_t slot_of(const ReadArgs& a, int64_t n) {
  if (n >= a.n) return -1;
  const int64_t row = __ldg(reinterpret_cast<const long long*>(a.slot) + n);
  if (row < a.num_tokens) return row;
  if ((threadIdx.x & 31) == 0) set_status(a.status, DSA_ERR_OUT_OF_RANGE, (int)n);
  return -1;
}

// Packed rows, one warp per token.  A lane decodes words of eight dims, 32 apart, so
// that a warp's stores are whole lines, and all of a token's loads are issued before
// its first store (d_c <= 512: two words a lane).
__global__ void __launch_bounds__(kWarpsPerCta * 32, 14) cache_read_int4_kernel(const __grid_constant__ ReadArgs a) {
  pdl_launch_dependents();
  trace_kernel(a.status, DSA_KERNEL_CACHE_READ);
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5), row = slot_of(a, n);
  if (row < 0) return;
  const Int4Row ly = int4_row(a.d_c, a.d_r);
  const uint8_t* src = static_cast<const uint8_t*>(a.latent) + row * ly.bytes;
  const bool lat = a.latent_out != nullptr, fp8 = a.idx_dtype == DSA_FP8_E4M3;
  const int words = lat ? a.d_c >> 3 : 0, pieces = lat ? a.d_r >> 3 : 0, keys = a.k_out != nullptr ? a.d_idx >> 2 : 0;
  uint32_t code[2], scale[2], key = 0;
  float ks = 0.f;
  uint4 rope;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int w = lane + 32 * i;
    if (w < words) {
      code[i] = __ldg(reinterpret_cast<const uint32_t*>(src) + w);
      scale[i] = __ldg(src + ly.scale + (w >> 1));
    }
  }
  if (lane < pieces) rope = __ldg(reinterpret_cast<const uint4*>(src + ly.rope) + lane);
  const uint32_t* kw = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.idx_k) + row * a.d_idx);
  if (fp8 && lane < keys) {
    key = __ldg(kw + lane);
    ks = __ldg(a.idx_k_scale + row);
  }
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.latent_out) + n * (a.d_c + a.d_r));
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 32 * i < words) st_stream(dst + lane + 32 * i, decode_word(code[i], scale_pair(scale[i])));
  if (lane < pieces) st_stream(dst + words + lane, rope);
  for (int c = lane + 32; c < pieces; c += 32) st_stream(dst + words + c, __ldg(reinterpret_cast<const uint4*>(src + ly.rope) + c));
  float4* kdst = reinterpret_cast<float4*>(a.k_out + n * a.d_idx);
  if (fp8) {
    if (lane < keys) __stcs(kdst + lane, e4m3x4_to_f32(key, ks));
    for (int c = lane + 32; c < keys; c += 32) __stcs(kdst + c, e4m3x4_to_f32(__ldg(kw + c), ks));
  } else {
    const float4* kf = reinterpret_cast<const float4*>(static_cast<const float*>(a.idx_k) + row * a.d_idx);
    for (int c = lane; c < keys; c += 32) __stcs(kdst + c, __ldg(kf + c));
  }
}

// Caches of the values' own type: a copy of the latent row, the key as above.
__global__ void __launch_bounds__(kWarpsPerCta * 32) cache_read_kernel(const __grid_constant__ ReadArgs a) {
  pdl_launch_dependents();
  trace_kernel(a.status, DSA_KERNEL_CACHE_READ);
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5), row = slot_of(a, n);
  if (row < 0) return;
  const int words = a.k_out != nullptr ? a.d_idx >> 2 : 0;
  const int pieces = a.latent_out != nullptr ? a.latent_row_bytes >> 4 : 0;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.latent) + row * a.latent_row_bytes);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.latent_out) + n * a.latent_row_bytes);
#pragma unroll 4
  for (int c = lane; c < pieces; c += 32) st_stream(dst + c, __ldg(src + c));
  if (a.idx_dtype == DSA_FP8_E4M3) {
    const uint32_t* key = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.idx_k) + row * a.d_idx);
    const float s = words > 0 ? __ldg(a.idx_k_scale + row) : 0.f;
    for (int c = lane; c < words; c += 32)
      __stcs(reinterpret_cast<float4*>(a.k_out + n * a.d_idx) + c, e4m3x4_to_f32(__ldg(key + c), s));
  } else {
    const float4* key = reinterpret_cast<const float4*>(static_cast<const float*>(a.idx_k) + row * a.d_idx);
    for (int c = lane; c < words; c += 32) __stcs(reinterpret_cast<float4*>(a.k_out + n * a.d_idx) + c, __ldg(key + c));
  }
}

}  // namespace

dsa_status launch_cache_read(const ReadArgs& a, cudaStream_t stream) {
  if (a.n == 0) return DSA_OK;
  const unsigned grid = (unsigned)(((int64_t)a.n + kWarpsPerCta - 1) / kWarpsPerCta);
  (a.int4 ? cache_read_int4_kernel : cache_read_kernel)<<<grid, kWarpsPerCta * 32, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("cache read launch failed: %s", cudaGetErrorString(e));
    return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

}  // namespace dsa
