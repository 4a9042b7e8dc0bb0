// cache_append.cu - fused FP8 quantise + paged cache write of new tokens.
//
// Each decoding step writes its new tokens into the layer's caches before the
// indexer reads them ("Sparse Attention Architectures for Long-Context
// Inference: Evolution and Engineering Practices", section 6, item
// "Incremental inference adaptation").  The indexer key cache is FP8
// ("DeepSeek Sparse Attention DSA Architecture Guide", section "Stage 1: The
// Lightning Indexer", item "Native FP8 Precision") with one fp32 scale per
// token, and both caches are paged ("Sparse Attention in Large Language
// Models: Architecture Evolution and Engineering Practice", section 4, item
// "Memory Management and KV Cache Optimization").
//
// One warp per token, eight tokens per CTA.  The work is a stream: per token
// 4*d_I bytes of key and (d_c+d_r)*elt bytes of latent in, d_I codes, a scale
// and the latent row out, so the kernel is HBM-bound and its design is about
// bytes in flight: every lane issues its key float4s and its first latent
// 16-byte chunks before the destination lookup (two dependent loads through
// the block table), so the table walk overlaps the payload.  No shared
// memory, no tensor cores: nothing here is a contraction.
//
//   amax  = max |k|            (lane max, then a butterfly over the warp)
//   s     = fl32(amax / 448)   (div.rn.f32; 1 when the quotient is 0)
//   code  = E4M3(fl32(k / s))  (div.rn.f32, then cvt.rn.satfinite.e4m3x2)
//
// The divisions are IEEE round-to-nearest and take no flush-to-zero, so the
// codes are exactly those of the rule as written; the hardware conversion
// rounds to nearest even and saturates finite overflow at +-448.
#include <cfloat>

#include "dsa_int4.cuh"
#include "dsa_kernels.cuh"

namespace dsa {
namespace {

constexpr int kWarpsPerCta = 8;     // tokens per CTA
constexpr int kPackedWarps = 4;     // the same for packed rows
constexpr int kMaxKeyChunks = 4;    // float4 per lane: d_I <= 4 * 32 * 4 = 512
constexpr int kLatGroup = 3;        // 16-byte latent chunks per lane in flight (1152 B rows: one group)

__device__ __forceinline__ float div_rn(float a, float b) {
  float r;
  asm("div.rn.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Four floats -> four e4m3 bytes, x0 in the lowest byte (the lowest address).
// cvt packs its first source into the upper byte of the pair.
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ float4 ld_stream_f4(const float4* p) {
  float4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint4 ld_stream_u4(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ bool finite4(const float4& v) {
  return fabsf(v.x) <= FLT_MAX && fabsf(v.y) <= FLT_MAX && fabsf(v.z) <= FLT_MAX &&
         fabsf(v.w) <= FLT_MAX;
}

// The largest magnitude of eight bf16 pairs as a bf16 pattern (infinities and NaN are
// the patterns from 0x7F80 on).
__device__ __forceinline__ uint32_t amax_bf16(const uint4& x, const uint4& y) {
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 8; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

__device__ __forceinline__ float amax4(const float4& v) {
  return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// The warp's key scale: fl32(amax / 448), 1 when that is 0.
__device__ __forceinline__ float key_scale(float amax) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = div_rn(amax, 448.f);
  return s > 0.f ? s : 1.f;
}
__device__ __forceinline__ uint32_t key_codes(const float4& v, float s) {
  return e4m3x4(div_rn(v.x, s), div_rn(v.y, s), div_rn(v.z, s), div_rn(v.w, s));
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The same codes, mostly without divisions.  k * rcp(s) is within 4 units in the last
// place of fl32(k / s); E4M3 keeps 4 significant bits from 2^-6 on, so both round alike
// unless the product's 20 dropped bits lie within 8 of half: those, and smaller values
// (fewer bits kept), are divided.
__device__ __forceinline__ float key_quotient(float k, float s, float r) {
  const float y = k * r;
  const uint32_t u = __float_as_uint(y);
  if ((u & 0xFFFFFu) - 0x7FFF8u <= 16u || (u & 0x7FFFFFFFu) < 0x3C800000u) return div_rn(k, s);
  return y;
}
__device__ __forceinline__ uint32_t key_codes_fast(const float4& v, float s) {
  const float r = rcp_approx(s);
  if (!(r < 3e38f)) return key_codes(v, s);       // the reciprocal of a subnormal scale
  return e4m3x4(key_quotient(v.x, s, r), key_quotient(v.y, s, r), key_quotient(v.z, s, r), key_quotient(v.w, s, r));
}

// Cache row of position `pos` of sequence `seq`; false when out of range.
__device__ __forceinline__ bool position_row(const AppendArgs& a, int seq, int pos, int64_t& row) {
  bool ok = seq >= 0 && seq < a.num_seqs && pos >= 0;
  if (ok) row = a.map.row(seq, pos, nullptr, &ok);
  return ok;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The code words of a group whose scale's reciprocal is r.
__device__ __forceinline__ void int4_codes(const uint32_t (&v)[8], float r, uint32_t (&w)[2]) {
  const uint64_t r2 = pair_f32(r, r), to_grid = pair_f32(6144.f, 6144.f), to_int = pair_f32(12576768.f, 12576768.f);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t x = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t p = v[4 * h + i];
      uint64_t c = mul_f32x2(pair_f32(bf16_lo(p), bf16_hi(p)), r2);
      // (c + 6144) - 6144 + 1.5 * 2^23: the low bits are the code in two's complement,
      // rounded to even (the last two constants are one, exactly)
      c = add_f32x2(add_f32x2(c, to_grid), to_int);
      // nibble i of each half
      const uint32_t q = __byte_perm((uint32_t)c, (uint32_t)(c >> 32), 0x5410), keep = 0x00010001u * ((1u << (4 * i)) - 1u);
      x = (x & keep) | ((q << (4 * i)) & ~keep);
    }
    w[h] = x;
  }
}

// One group of 16 latent dims (eight bf16 pairs) as its scale byte and two code
// words: the scale is fl32(amax / 7) rounded to 8 bits, the code the nearest integer
// to c / scale, ties to even, within +-7.
//
// Neither needs a division.  The largest |c| is A 2^i with A <= 255, so A 2^i / 7 either
// is a tie of the scale's rounding (a number of at most 5 significant bits) or differs
// from one by 2^-11 of itself at least; the product with fl32(1 / 7) is within two units
// in the last place, so rounding its last four bits away restores ties and moves nothing
// else across one.  With c = a 2^i (a <= 255) and scale = m 2^j (m <= 15), a quotient
// of at least 1/4 in magnitude is a / (m 2^w) with m 2^w <= 4 a, so it either is a tie
// k + 1/2 or is at least 1 / (2 m 2^w) >= 1 / 2040 from one; a smaller one rounds to 0.
// c * rcp(scale) is within 2e-6 of it below 8, so rounding that product to a multiple of
// 2^-11 (adding 6144) restores ties exactly and moves nothing else across one.
// `amax`: the largest |c| as a bf16 pattern.
__device__ __forceinline__ uint32_t int4_group(uint32_t (&v)[8], uint32_t amax, uint32_t (&w)[2]) {
  const float a7 = bf16_lo(amax) * (1.f / 7.f);
  const uint32_t code = scale_code(__uint_as_float((__float_as_uint(a7) + 8u) & ~15u));
  w[0] = w[1] = 0u;
  if (code == 0u) return 0u;
  const float scale = scale_value(code), r = rcp_approx(scale);
  // a normal, unsaturated scale is at least 16/17 of amax / 7, so quotients stay below
  // 7.5; with other scales the dims are clamped to 7 of them first (exact: a bf16)
  if (code < 8u || code == kScaleMax) {
    const uint32_t top = __float_as_uint(7.f * scale) >> 16, hi = __byte_perm(top, top, 0x1010), lo = hi | 0x80008000u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      asm("min.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(hi));
      asm("max.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(lo));
    }
  }
  int4_codes(v, r, w);
  return code;
}

// Rows of the caches' own element types; by position or by slot.
template <bool kSlots>
__global__ void __launch_bounds__(kWarpsPerCta * 32)
cache_append_kernel(const AppendArgs a) {
  pdl_launch_dependents();
  trace_kernel(a.status, DSA_KERNEL_CACHE_APPEND);
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  if (n >= a.n_new) return;

  // 1. the payload: key chunks and the first latent group, all in flight
  // (by slot, a NULL source has no chunks)
  const int kc = kSlots && a.k_new == nullptr ? 0 : a.d_idx >> 2;
  const float4* ksrc = reinterpret_cast<const float4*>(a.k_new) + (int64_t)n * kc;
  float4 v[kMaxKeyChunks];
#pragma unroll
  for (int i = 0; i < kMaxKeyChunks; ++i) {
    const int c = lane + 32 * i;
    v[i] = c < kc ? ld_stream_f4(ksrc + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int lc = kSlots && a.latent_new == nullptr ? 0 : a.latent_row_bytes >> 4;
  const uint4* lsrc = reinterpret_cast<const uint4*>(a.latent_new) + (int64_t)n * lc;
  uint4 t[kLatGroup];
#pragma unroll
  for (int i = 0; i < kLatGroup; ++i) {
    const int c = lane + 32 * i;
    if (c < lc) t[i] = ld_stream_u4(lsrc + c);
  }

  // 2. the destination row (the same map the attention stage reads)
  bool ok;
  int64_t row = 0;
  if constexpr (kSlots) {
    row = __ldg(reinterpret_cast<const long long*>(a.slot) + n);
    if (row < 0) return;                   // padding
    ok = row < a.map.num_tokens;
  } else {
    ok = position_row(a, __ldg(a.tok_seq + n), __ldg(a.tok_pos + n), row);
  }
  if (!ok) {
    if (lane == 0) set_status(a.status, DSA_ERR_OUT_OF_RANGE, n);
    return;
  }

  // 3. the key: reject non-finite, then quantise (or copy) and store
  bool fin = true;
#pragma unroll
  for (int i = 0; i < kMaxKeyChunks; ++i) fin = fin && finite4(v[i]);
  if (!__all_sync(0xffffffffu, fin)) {
    if (lane == 0) set_status(a.status, DSA_ERR_INVALID_ARG, n);
    return;
  }
  if (a.idx_dtype == DSA_FP8_E4M3) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxKeyChunks; ++i) amax = fmaxf(amax, amax4(v[i]));
    const float s = key_scale(amax);
    uint32_t* kdst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.idx_k) + row * a.d_idx);
#pragma unroll
    for (int i = 0; i < kMaxKeyChunks; ++i) {
      const int c = lane + 32 * i;
      if (c < kc) kdst[c] = key_codes(v[i], s);
    }
    if (lane == 0 && kc > 0) a.idx_k_scale[row] = s;
  } else {
    float4* kdst = reinterpret_cast<float4*>(static_cast<float*>(a.idx_k) + row * a.d_idx);
#pragma unroll
    for (int i = 0; i < kMaxKeyChunks; ++i) {
      const int c = lane + 32 * i;
      if (c < kc) kdst[c] = v[i];
    }
  }

  // 4. the latent row: store the group in flight, load the next (rows wider
  //    than 32 * kLatGroup chunks only)
  uint4* ldst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.latent) + row * a.latent_row_bytes);
  for (int base = 0;;) {
#pragma unroll
    for (int i = 0; i < kLatGroup; ++i) {
      const int c = base + lane + 32 * i;
      if (c < lc) ldst[c] = t[i];
    }
    base += 32 * kLatGroup;
    if (base >= lc) break;
#pragma unroll
    for (int i = 0; i < kLatGroup; ++i) {
      const int c = base + lane + 32 * i;
      if (c < lc) t[i] = ld_stream_u4(lsrc + c);
    }
  }
}

// Packed rows.  A lane quantises whole groups of 16 latent dims (d_c = 512: one each),
// so a group's maximum needs no exchange.  65,536 tokens take 37 us against a floor of
// 22 us for their 146 MB: what bounds it is the integer pipe (unpacking, packing and
// comparing; a warp instruction takes it two cycles).  fp32 pairs and bf16 pair maxima
// took it from 42.4 to 39.2, CTAs of four warps instead of eight to 37.2.  Persistent
// warps with the next token's loads in flight measured the same.  Ten CTAs an SM leave a
// thread 48 registers, for which it spills 100 bytes and reloads 96; eight CTAs, without
// a spill (60 registers), took 2 us more, twelve (40 registers) 1 us.
struct Token {
  float4 key;              // this lane's first key chunk (d_I > 128: the others are loaded late)
  uint4 lat[2], rope;      // its group of 16 dims, its piece of the RoPE key
  int64_t row;             // by slot
  int seq, pos;            // by position
};

template <bool kSlots>
__device__ __forceinline__ void load_token(const AppendArgs& a, int64_t n, Token& x) {
  const int lane = threadIdx.x & 31;
  if constexpr (kSlots) {
    x.row = __ldg(reinterpret_cast<const long long*>(a.slot) + n);
  } else {
    x.seq = __ldg(a.tok_seq + n);
    x.pos = __ldg(a.tok_pos + n);
  }
  const int kc = a.k_new == nullptr ? 0 : a.d_idx >> 2;
  x.key = lane < kc ? ld_stream_f4(reinterpret_cast<const float4*>(a.k_new) + n * kc + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
  x.lat[0] = x.lat[1] = make_uint4(0u, 0u, 0u, 0u);
  if (a.latent_new != nullptr) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.latent_new) + n * a.latent_new_row_bytes);
    const int groups = a.d_c / kInt4Group;
    if (lane < groups) {
      x.lat[0] = ld_stream_u4(src + 2 * lane);
      x.lat[1] = ld_stream_u4(src + 2 * lane + 1);
    }
    if (lane < (a.d_r >> 3)) x.rope = ld_stream_u4(src + 2 * groups + lane);
  }
}

template <bool kSlots>
__device__ __forceinline__ void store_token(const AppendArgs& a, int64_t n, const Token& x) {
  const int lane = threadIdx.x & 31;
  int64_t row = 0;
  bool ok;
  if constexpr (kSlots) {
    row = x.row;
    if (row < 0) return;                   // padding
    ok = row < a.map.num_tokens;
  } else {
    ok = position_row(a, x.seq, x.pos, row);
  }
  if (!ok) {
    if (lane == 0) set_status(a.status, DSA_ERR_OUT_OF_RANGE, (int)n);
    return;
  }
  const int kc = a.k_new == nullptr ? 0 : a.d_idx >> 2;
  const float4* ksrc = reinterpret_cast<const float4*>(a.k_new) + n * kc;
  const uint32_t lat_max = amax_bf16(x.lat[0], x.lat[1]);
  float amax = amax4(x.key);
  bool fin = finite4(x.key) && lat_max < 0x7F80u;
  for (int c = lane + 32; c < kc; c += 32) {
    const float4 v = ld_stream_f4(ksrc + c);
    fin = fin && finite4(v);
    amax = fmaxf(amax, amax4(v));
  }
  if (!__all_sync(0xffffffffu, fin)) {
    if (lane == 0) set_status(a.status, DSA_ERR_INVALID_ARG, (int)n);
    return;
  }
  const Int4Row ly = int4_row(a.d_c, a.d_r);
  const int groups = a.d_c / kInt4Group, pieces = a.d_r >> 3;
  uint8_t* dst = static_cast<uint8_t*>(a.latent) + row * a.latent_row_bytes;
  if (a.latent_new != nullptr && lane < pieces) reinterpret_cast<uint4*>(dst + ly.rope)[lane] = x.rope;
  if (kc > 0) {
    if (a.idx_dtype == DSA_FP8_E4M3) {
      const float s = key_scale(amax);
      uint32_t* kdst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.idx_k) + row * a.d_idx);
      if (lane < kc) kdst[lane] = key_codes_fast(x.key, s);
      for (int c = lane + 32; c < kc; c += 32) kdst[c] = key_codes_fast(ld_stream_f4(ksrc + c), s);
      if (lane == 0) a.idx_k_scale[row] = s;
    } else {
      float4* kdst = reinterpret_cast<float4*>(static_cast<float*>(a.idx_k) + row * a.d_idx);
      if (lane < kc) kdst[lane] = x.key;
      for (int c = lane + 32; c < kc; c += 32) kdst[c] = ld_stream_f4(ksrc + c);
    }
  }
  if (a.latent_new == nullptr) return;
  if (lane < groups) {
    uint32_t v[8] = {x.lat[0].x, x.lat[0].y, x.lat[0].z, x.lat[0].w, x.lat[1].x, x.lat[1].y, x.lat[1].z, x.lat[1].w};
    uint32_t w[2];
    const uint32_t code = int4_group(v, lat_max, w);
    reinterpret_cast<uint2*>(dst)[lane] = make_uint2(w[0], w[1]);
    dst[ly.scale + lane] = (uint8_t)code;
  }
  const uint4* rsrc = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.latent_new) + n * a.latent_new_row_bytes) + 2 * groups;
  for (int c = lane + 32; c < pieces; c += 32) reinterpret_cast<uint4*>(dst + ly.rope)[c] = ld_stream_u4(rsrc + c);
  const int pad = ly.scale + groups + lane;
  if (pad < ly.bytes) dst[pad] = 0u;
}

template <bool kSlots>
__global__ void __launch_bounds__(kPackedWarps * 32, 10)
cache_append_int4_kernel(const __grid_constant__ AppendArgs a) {
  pdl_launch_dependents();
  trace_kernel(a.status, DSA_KERNEL_CACHE_APPEND);
  const int64_t n = (int64_t)blockIdx.x * kPackedWarps + (threadIdx.x >> 5);
  if (n >= a.n_new) return;
  Token x;
  load_token<kSlots>(a, n, x);
  store_token<kSlots>(a, n, x);
}

}  // namespace

dsa_status launch_cache_append(const AppendArgs& a, cudaStream_t stream) {
  if (a.n_new == 0) return DSA_OK;
  const int warps = a.int4 ? kPackedWarps : kWarpsPerCta;
  const unsigned grid = (unsigned)(((int64_t)a.n_new + warps - 1) / warps);
  void (*kernel)(AppendArgs) = a.slot ? cache_append_kernel<true> : cache_append_kernel<false>;
  if (a.int4) kernel = a.slot ? cache_append_int4_kernel<true> : cache_append_int4_kernel<false>;
  kernel<<<grid, warps * 32, 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("cache append launch failed: %s", cudaGetErrorString(e));
    return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

int cache_append_max_d_idx() { return kMaxKeyChunks * 32 * 4; }

}  // namespace dsa
