// mla_int4_tc.cu - sparse absorbed MLA over packed 4-bit latent rows on the
// 5th-generation tensor cores.
//
// The mathematics is that of mla_tc.cu ("DeepSeek Sparse Attention DSA
// Architecture Guide", section "Stage 2: Fine-Grained Token Selection and Output
// Computation"), over rows whose latent dims are 4-bit codes with a scale per 16
// (include/dsa.h).  A decoded value is exact in bf16 (dsa_int4.cuh), so decoding
// adds no rounding: what is rounded is each softmax weight, to bf16 once for the
// second product (relative 2^-8 at most, its sum is kept in fp32), and the output.
//
// Work unit: (row t, key split), one cluster of two CTAs.  The pair runs every
// product as one two-CTA tcgen05.mma (M = 128 heads, 64 of them in each CTA), so
// each CTA has its own heads' logits, softmax state and output rows, and nothing
// of the softmax crosses between them:
//   S = Q K^T   M=128, N=64 keys, K=576.  CTA r holds the 64 heads' Q and keys
//               [32r, 32r+32) of the block, all 576 dims.
//   O += P V    M=128, N=2x256 dims, K=64 keys.  CTA r holds its heads' P and
//               dims [256r, 256r+256) of all 64 keys.
// In tensor memory lane l < 64 of a CTA is head l with the first half of N, lane
// l + 64 the same head with the second half.
// The two operands overlap in a quarter of the block only, and each CTA decodes
// both for itself straight from the packed rows: at three instructions a pair of
// values that is cheaper than an exchange through distributed shared memory.
//
// Roles per CTA (672 threads):
//   warps 0-3    softmax and output: thread (l) = TMEM lane; 32 keys of a head per
//                block, the two halves of a head share the maximum through shared
//                memory.  Lazy rescale as in mla_tc.cu.
//   warps 4-11   decode the keys' tile: packed pieces from global memory to
//                registers one block ahead, then 16-byte stores, swizzled.
//   warps 12-19  decode the values' tile, the same way
//   warp 20      tensor memory; in the pair's first CTA one thread issues the MMAs
// The tiles have two stages each; S of block j+1 is issued before P V of block j,
// so that the tensor cores work while the softmax of block j runs.
#include "dsa_int4.cuh"
#include "dsa_kernels.cuh"
#include "mla_common.cuh"

namespace dsa {
namespace {

constexpr int kHc = 64;                         // heads per CTA
constexpr int kDC = 512, kDR = 64, kD = kDC + kDR;
constexpr Int4Row kRow = int4_row(kDC, kDR);
constexpr int kBlk = 64, kHalfBlk = 32;
constexpr int kMaxKeys = 2048;
constexpr int kKWarp0 = 4, kVWarp0 = 12, kDecWarps = 8, kMmaWarp = 20;
constexpr int kThreads = 32 * 21;
constexpr int kDecThreads = 2 * kDecWarps * 32;
constexpr int kQChunks = kD / 64;               // 64-dim SW128 chunks: 8 latent, 1 RoPE
constexpr uint32_t kColS = 0, kColO = 64, kTmemCols = 512;
// polls of a bounded wait (20 ms at least; real waits take microseconds)
constexpr uint32_t kWaitPolls = 1u << 20;

struct __align__(1024) Smem {
  uint8_t q[kQChunks][kHc * 128];               // this CTA's heads
  uint8_t k[2][kQChunks][kHalfBlk * 128];       // its 32 keys, 576 dims
  uint8_t v[2][4][kBlk * 128];                  // 64 keys, its 256 dims
  uint8_t p[kHc * 128];                         // its heads' weights of 64 keys
  int32_t rows[kMaxKeys];                       // physical cache row per selected key, -1 = none
  uint32_t valid[kMaxKeys / 32];                // per 32 keys: bit i set = key i has a row
  float red[2][2 * kHc];                        // block maxima by lane; the final sums
  // waited for by the issuing thread, in the first CTA's shared memory
  uint64_t q_full, k_full[2], v_full[2], p_full, s_free[2];
  // arrivals of finished products, in both CTAs
  uint64_t s_full[2], pv_done[2];
  uint64_t drained;
  uint32_t tmem_base;
  int last_flag;
};
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "shared memory of the attention kernel");

// ---------------------------------------------------------------- two-CTA tcgen05
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)),
               "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// D (+)= A B over the pair: each CTA's shared memory holds half of A's rows and
// half of B's, at the same offsets.
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// Arrive on `bar` of both CTAs when the products issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ bool wait_local(uint64_t* bar, uint32_t parity, DeviceStatus* st, int site) {
  return mbar_wait(bar, parity, st, site, kWaitPolls);
}
// Waits for arrivals of the other CTA too (acquire at cluster scope).
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, DeviceStatus* st, int site) {
  for (uint32_t i = 0; i < kWaitPolls; ++i)
    if (mbar_try_wait_cluster(bar, parity)) return true;
  set_status(st, DSA_ERR_TIMEOUT, site);
  return false;
}
// One arrival per warp on a barrier of the pair's first CTA.
__device__ __forceinline__ void warp_arrive_first(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive_cluster(bar, 0);
}

// ---------------------------------------------------------------- MMA issue (first CTA, one thread)
__device__ __forceinline__ void issue_products(Smem& S, DeviceStatus* status, uint32_t tmem, int nblk) {
  constexpr uint32_t idesc_s = idesc_bf16(kBlk, false);
  constexpr uint32_t idesc_pv = idesc_bf16(256, true);
  bool ok = wait_pair(&S.q_full, 0, status, 41);
  const uint32_t qa = smem_u32(S.q), pa = smem_u32(S.p);
  for (int j = 0; ok && j <= nblk; ++j) {
    if (j < nblk) {
      const int b = j & 1;
      ok = wait_pair(&S.k_full[b], (j >> 1) & 1, status, 42) && wait_pair(&S.s_free[b], ((j >> 1) & 1) ^ 1, status, 43);
      if (!ok) break;
      fence_proxy_async_smem();
      tc_fence_after();
      const uint32_t ka = smem_u32(S.k[b]);
#pragma unroll
      for (int ch = 0; ch < kQChunks; ++ch)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_bf16_pair(tmem + kColS + b * 32, sdesc_sw128(qa + ch * kHc * 128 + 32 * kk, 16, 1024),
                        sdesc_sw128(ka + ch * kHalfBlk * 128 + 32 * kk, 16, 1024), idesc_s, (ch | kk) != 0);
      mma_commit_pair(&S.s_full[b]);
    }
    if (j >= 1) {
      const int jj = j - 1, b = jj & 1;
      ok = wait_pair(&S.v_full[b], (jj >> 1) & 1, status, 44) && wait_pair(&S.p_full, jj & 1, status, 45);
      if (!ok) break;
      fence_proxy_async_smem();
      tc_fence_after();
      const uint32_t va = smem_u32(S.v[b]);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          mma_bf16_pair(tmem + kColO + n * 128, sdesc_sw128(pa + 32 * kk, 16, 1024),
                        sdesc_sw128(va + n * 2 * kBlk * 128 + kk * 16 * 128, kBlk * 128, 1024), idesc_pv,
                        (jj | kk) != 0);
      mma_commit_pair(&S.pv_done[b]);
    }
  }
  // every product issued is done before the pair's shared and tensor memory go
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&S.drained))
               : "memory");
  wait_local(&S.drained, 0, status, 46);
}

// ---------------------------------------------------------------- decoding
// A warp's share of one block: two pieces of 32 dims of a key per lane.  Eight
// neighbouring lanes take eight keys (their 16-byte stores fall into distinct
// banks of the swizzled tile), the four lane groups four neighbouring pieces (64
// bytes of codes of one key: two whole sectors).
template <bool kV>
struct Decoder {
  uint4 codes[2];
  uint32_t scales[2];
  uint4 rope;

  static __device__ __forceinline__ void place(int wt, int i, int& key, int& piece) {
    const int lane = threadIdx.x & 31, task = wt + kDecWarps * i;
    key = (kV ? task & 7 : task & 3) * 8 + (lane & 7);
    piece = (kV ? task >> 3 : task >> 2) * 4 + (lane >> 3);
  }
  // Loads block j's packed pieces (zeros for a key without a row).
  __device__ __forceinline__ void load(const Smem& S, const uint8_t* latent, int j, int wt, uint32_t rank) {
    const int32_t* rows = S.rows + j * kBlk + (kV ? 0 : kHalfBlk * (int)rank);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int key, piece;
      place(wt, i, key, piece);
      if (kV) piece += 8 * (int)rank;
      const int row = rows[key];
      const uint8_t* src = latent + (int64_t)row * kRow.bytes;
      codes[i] = make_uint4(0u, 0u, 0u, 0u);
      scales[i] = 0u;
      if (row >= 0) {
        codes[i] = __ldg(reinterpret_cast<const uint4*>(src) + piece);
        scales[i] = __ldg(reinterpret_cast<const unsigned short*>(src + kRow.scale) + piece);
      }
    }
    if (!kV) {
      const int kt = wt * 32 + (threadIdx.x & 31), row = rows[kt >> 3];
      rope = make_uint4(0u, 0u, 0u, 0u);
      if (row >= 0)
        rope = __ldg(reinterpret_cast<const uint4*>(latent + (int64_t)row * kRow.bytes + kRow.rope) + (kt & 7));
    }
  }
  __device__ __forceinline__ void store(uint8_t* tile, int wt) const {
    constexpr int kChunk = (kV ? kBlk : kHalfBlk) * 128;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int key, piece;
      place(wt, i, key, piece);
      uint8_t* dst = tile + (piece >> 1) * kChunk;
      const int p0 = (piece & 1) * 4;
      const ScalePair s0 = scale_pair(scales[i] & 0xFFu), s1 = scale_pair(scales[i] >> 8);
      *reinterpret_cast<uint4*>(dst + sw128_off(key, p0)) = decode_word(codes[i].x, s0);
      *reinterpret_cast<uint4*>(dst + sw128_off(key, p0 + 1)) = decode_word(codes[i].y, s0);
      *reinterpret_cast<uint4*>(dst + sw128_off(key, p0 + 2)) = decode_word(codes[i].z, s1);
      *reinterpret_cast<uint4*>(dst + sw128_off(key, p0 + 3)) = decode_word(codes[i].w, s1);
    }
    if (!kV) {
      const int kt = wt * 32 + (threadIdx.x & 31);
      *reinterpret_cast<uint4*>(tile + 8 * kChunk + sw128_off(kt >> 3, kt & 7)) = rope;
    }
  }
};

template <bool kV>
__device__ __forceinline__ void decode_blocks(Smem& S, const MlaArgs& a, int nblk, uint32_t rank, int wt) {
  const uint8_t* latent = static_cast<const uint8_t*>(a.latent);
  Decoder<kV> cur, nxt;
  cur.load(S, latent, 0, wt, rank);
  cp_async_wait_all();                            // this thread's pieces of Q
  fence_proxy_async_smem();
  warp_arrive_first(&S.q_full);
  for (int j = 0; j < nblk; ++j) {
    const int b = j & 1;
    if (j + 1 < nblk) nxt.load(S, latent, j + 1, wt, rank);
    // the stage is free once the products of block j-2 have read it
    if (!wait_local(kV ? &S.pv_done[b] : &S.s_full[b], ((j >> 1) & 1) ^ 1, a.status, kV ? 48 : 47)) break;
    cur.store(kV ? S.v[b][0] : S.k[b][0], wt);
    fence_proxy_async_smem();                     // generic stores -> tensor cores
    warp_arrive_first(kV ? &S.v_full[b] : &S.k_full[b]);
    cur = nxt;
  }
}

// 32 columns of this thread's lane of O (zeros when no product was issued).
__device__ __forceinline__ void load_o32(uint32_t taddr, bool empty, float (&o)[32]) {
  if (empty) {
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.f;
    return;
  }
  tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(&o[0]));
  tmem_wait_ld();
}

__global__ void __launch_bounds__(kThreads, 1) mla_int4_tc_kernel(MlaArgs a, int keys_per_split) {
  extern __shared__ __align__(1024) uint8_t smraw[];
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit = blockIdx.x >> 1;
  const int t = unit / a.splits, sp = unit % a.splits;
  pdl_launch_dependents();

  // setup that reads no input memory overlaps the predecessor's tail
  if (threadIdx.x == 0) {
    mbar_init(&S.q_full, 2 * 2 * kDecWarps);
    mbar_init(&S.p_full, 2 * 4);
    mbar_init(&S.drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], 2 * kDecWarps);
      mbar_init(&S.v_full[i], 2 * kDecWarps);
      mbar_init(&S.s_free[i], 2 * 4);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.pv_done[i], 1);
    }
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == kMmaWarp) tmem_alloc_pair(&S.tmem_base, kTmemCols);
  pdl_wait();
  trace_kernel(a.status, DSA_KERNEL_MLA_INT4_TC);
  const int klen = a.row_klen[t];
  const int seq = a.row_seq[t];
  const bool known = (seq >= 0 && seq < a.num_seqs) || !a.map.uses_seq();
  if (!known && klen > 0 && threadIdx.x == 0) set_status(a.status, DSA_ERR_OUT_OF_RANGE, t);
  const int nsel = known ? min(klen, a.topk) : 0;
  const int k0 = sp * keys_per_split;
  const int nvalid = max(0, min(nsel - k0, keys_per_split));
  const int nblk = (nvalid + kBlk - 1) / kBlk;
  {
    constexpr int kPer = (kMaxKeys + kThreads - 1) / kThreads;
    const int32_t* idx = a.idx + (int64_t)t * a.topk + k0;
    int sv[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = threadIdx.x + u * kThreads;
      sv[u] = i < nvalid ? __ldg(idx + i) : -1;
    }
    // Q lands while the selection is resolved; heads beyond H are zeros
    const int g = threadIdx.x - 32 * kKWarp0;
    if (nblk > 0 && g >= 0 && g < kDecThreads) {
      const int h0 = kHc * (int)rank;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)t * a.n_heads * kD;
#pragma unroll
      for (int i = 0; i < kHc * kD / 8 / kDecThreads; ++i) {
        const int qi = g + i * kDecThreads, h = qi / (kD / 8), c = qi - h * (kD / 8);
        const bool in = h0 + h < a.n_heads;
        cp_async_16_zfill(S.q[c >> 3] + sw128_off(h, c & 7), q + (int64_t)(in ? h0 + h : 0) * kD + 8 * c, in);
      }
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = threadIdx.x + u * kThreads;
      int row = -1;
      if (i < nblk * kBlk) {
        const int sk = sv[u];
        if (sk >= 0 && sk < klen) {
          bool ok = true;
          const int64_t r = a.map.row(seq, sk, a.status, &ok);
          row = ok ? (int32_t)r : -1;
        }
        S.rows[i] = row;
      }
      const uint32_t bits = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0 && i < nblk * kBlk) S.valid[i >> 5] = bits;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();                       // the pair's barriers are initialised
  const uint32_t tmem = S.tmem_base;

  if (warp == kMmaWarp) {
    if (rank == 0 && lane == 0 && nblk > 0) issue_products(S, a.status, tmem, nblk);
    __syncwarp();
  } else if (warp >= kVWarp0) {
    if (nblk > 0) decode_blocks<true>(S, a, nblk, rank, warp - kVWarp0);
  } else if (warp >= kKWarp0) {
    if (nblk > 0) decode_blocks<false>(S, a, nblk, rank, warp - kKWarp0);
  } else {
    // -------------------------------------------------- softmax and output (128 threads)
    const int l = threadIdx.x, half = l >> 6, hl = l & 63;
    const int head = kHc * (int)rank + hl;
    const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
    const float c = a.sm_scale * kLog2e;
    float m_used = -INFINITY, sum = 0.f;
    // a wait that runs out marks the thread dead; the loop is left together
    bool dead = false;
    for (int j = 0; j < nblk; ++j) {
      const int b = j & 1;
      dead = dead || !wait_local(&S.s_full[b], (j >> 1) & 1, a.status, 49);
      tc_fence_after();
      float s[32];
      tmem_ld32(tmem + lane_off + kColS + b * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
      tmem_wait_ld();
      tc_fence_before();
      warp_arrive_first(&S.s_free[b]);
      // logits in the log2 domain; masked keys are -inf
      const uint32_t mask = S.valid[2 * j + half];
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] *= c;
      if (mask != 0xFFFFFFFFu) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!((mask >> i) & 1u)) s[i] = -INFINITY;
      }
      float pm[8];
#pragma unroll
      for (int i = 0; i < 32; ++i) pm[i & 7] = (i < 8) ? s[i] : fmaxf(pm[i & 7], s[i]);
      const float mh = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])),
                             fmaxf(fmaxf(pm[4], pm[5]), fmaxf(pm[6], pm[7])));
      S.red[b][l] = mh;
      if (named_bar_or(1, 128, dead)) { dead = true; break; }
      const float mb = fmaxf(mh, S.red[b][l ^ 64]);
      // lazy rescale: P stays <= 2^8.  Warp-uniform; a head's two lanes decide alike
      const bool need = mb > m_used + kRescale;
      if (__any_sync(0xffffffffu, need)) {
        const float m_new = need ? mb : m_used;
        const float alpha = need ? (m_used == -INFINITY ? 0.f : exp2f(m_used - m_new)) : 1.f;
        if (j > 0) {
          dead = dead || !wait_local(&S.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, a.status, 50);
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            uint32_t o[32];
            const uint32_t col = tmem + lane_off + kColO + 32 * cc;
            tmem_ld32(col, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(col, o);
          }
          tmem_wait_st();
        }
        sum *= alpha;
        m_used = m_new;
      }
      // p = 2^(z - m); while no key of the head has been visible m counts as 0
      const float mu = (m_used == -INFINITY) ? 0.f : m_used;
      uint32_t p2[16];
      float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p0 = ex2_approx(s[2 * i] - mu);
        const float p1 = ex2_approx(s[2 * i + 1] - mu);
        ls[i & 3] += p0 + p1;
        p2[i] = pack_bf16x2(p0, p1);
      }
      sum += (ls[0] + ls[1]) + (ls[2] + ls[3]);
      // the weights' tile is free once P V of the block before is done
      if (j > 0) dead = dead || !wait_local(&S.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, a.status, 51);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(S.p + sw128_off(hl, 4 * half + i)) =
            make_uint4(p2[4 * i], p2[4 * i + 1], p2[4 * i + 2], p2[4 * i + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      warp_arrive_first(&S.p_full);
    }
    if (!dead && nblk > 0) {
      dead = !wait_local(&S.pv_done[(nblk - 1) & 1], ((nblk - 1) >> 1) & 1, a.status, 52);
      tc_fence_after();
    }
    // the head's sum over its two lanes; a wait that ran out anywhere fails the CTA
    named_bar_sync(1, 128);
    S.red[0][l] = sum;
    const bool fail = named_bar_or(1, 128, dead);
    const float lt = S.red[0][hl] + S.red[0][hl + 64];
    const bool empty = nblk == 0;
    const int heads_here = max(0, min(kHc, a.n_heads - kHc * (int)rank));
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)t * a.n_heads + kHc * (int)rank) * kDC;
    if (fail) {
      // recorded in the status word: zeros
      for (int i = l; i < heads_here * (kDC / 8); i += 128) reinterpret_cast<uint4*>(out)[i] = make_uint4(0u, 0u, 0u, 0u);
    } else {
      // the finished rows go through shared memory (the values' tiles, idle now) so
      // that global writes are whole rows: 64 heads x 64 pieces of 16 bytes, piece
      // c of head h at c ^ (h % 32)
      uint8_t* stg = S.v[0][0];
      const auto stage = [&](const float (&o)[32], int cc, float inv) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(stg + hl * 1024 + (((32 * half + 4 * cc + q) ^ (hl & 31)) << 4)) = pack8(&o[8 * q], inv);
      };
      bool write_out = true;
      if (a.splits == 1) {
        const float inv = lt > 0.f ? 1.f / lt : 0.f;
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {
          float o[32];
          load_o32(tmem + lane_off + kColO + 32 * cc, empty, o);
          stage(o, cc, inv);
        }
        if (a.lse && half == 0 && head < a.n_heads)
          a.lse[(int64_t)t * a.n_heads + head] = lt > 0.f ? (m_used + log2f(lt)) * kLn2 : -INFINITY;
      } else {
        // key splits: publish O and (max, sum); the row's last split to arrive (per
        // CTA rank) merges them in split order:
        //   out = sum_s w_s O_s / sum_s w_s l_s,  w_s = 2^(m_s - max m)
        float4* po = reinterpret_cast<float4*>(a.part_o);
        float2* pml = reinterpret_cast<float2*>(a.part_ml);
        constexpr int64_t kUnit = (kDC / 4) * kHc;
        const auto unit_of = [&](int s2) { return ((int64_t)t * a.splits + s2) * 2 + rank; };
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {
          float o[32];
          load_o32(tmem + lane_off + kColO + 32 * cc, empty, o);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            po[unit_of(sp) * kUnit + (64 * half + 8 * cc + i) * kHc + hl] =
                make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        if (half == 0) pml[unit_of(sp) * kHc + hl] = make_float2(m_used, lt);
        named_bar_sync(1, 128);
        if (l == 0) {
          __threadfence();
          unsigned long long* slot = &a.part_cnt[(int64_t)t * 2 + rank];
          const bool last = take_ticket(slot, a.launch_id, a.status) == (uint32_t)a.splits;
          if (last) *slot = (unsigned long long)a.launch_id << 32;   // a replay counts from zero again
          S.last_flag = last;
          __threadfence();
        }
        named_bar_sync(1, 128);
        write_out = S.last_flag != 0;
        if (write_out) {
          if (l == 0 && a.status != nullptr) atomicOr(&a.status->ran, DSA_KERNEL_MLA_COMBINE);
          float w[kMaxSplits];
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int s2 = 0; s2 < kMaxSplits; ++s2) {
            w[s2] = s2 < a.splits ? __ldcg(&pml[unit_of(s2) * kHc + hl]).x : -INFINITY;
            M = fmaxf(M, w[s2]);
          }
#pragma unroll
          for (int s2 = 0; s2 < kMaxSplits; ++s2) {
            w[s2] = w[s2] == -INFINITY ? 0.f : exp2f(w[s2] - M);
            if (s2 < a.splits) L += w[s2] * __ldcg(&pml[unit_of(s2) * kHc + hl]).y;
          }
          const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll 1
          for (int cc = 0; cc < 8; ++cc) {
            float acc[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0.f;
#pragma unroll
            for (int s2 = 0; s2 < kMaxSplits; ++s2) {
              if (s2 >= a.splits) continue;
              const float4* src = po + unit_of(s2) * kUnit + (64 * half + 8 * cc) * kHc + hl;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 v = __ldcg(src + i * kHc);
                acc[4 * i] = fmaf(w[s2], v.x, acc[4 * i]);
                acc[4 * i + 1] = fmaf(w[s2], v.y, acc[4 * i + 1]);
                acc[4 * i + 2] = fmaf(w[s2], v.z, acc[4 * i + 2]);
                acc[4 * i + 3] = fmaf(w[s2], v.w, acc[4 * i + 3]);
              }
            }
            stage(acc, cc, inv);
          }
          if (a.lse && half == 0 && head < a.n_heads)
            a.lse[(int64_t)t * a.n_heads + head] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
        }
      }
      if (write_out) {
        named_bar_sync(1, 128);
#pragma unroll 4
        for (int i = l; i < heads_here * 64; i += 128) {
          const int h = i >> 6, ch = i & 63;
          reinterpret_cast<uint4*>(out)[i] = *reinterpret_cast<const uint4*>(stg + h * 1024 + ((ch ^ (h & 31)) << 4));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                       // no access to the pair's memory is still pending
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

}  // namespace

bool mla_int4_tc_supported(const MlaArgs& a) {
  return a.mla_dtype == DSA_INT4 && a.n_heads <= 2 * kHc && a.d_c == kDC && a.d_r == kDR && a.topk <= kMaxKeys;
}

dsa_status launch_mla_int4_tc(const MlaArgs& a, cudaStream_t stream) {
  if (a.num_rows == 0) return DSA_OK;
  const size_t smem = sizeof(Smem) + 1024;
  static std::atomic<bool> attr[kMaxDevices] = {};
  if (dsa_status st = set_smem_limit_once(reinterpret_cast<const void*>(mla_int4_tc_kernel), smem, attr)) return st;
  const int keys_per_split = (int)(ceil_div64(ceil_div64(a.topk, a.splits), kBlk) * kBlk);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.num_rows * a.splits * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  MlaArgs la = a;
  la.launch_id = next_launch_id();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, mla_int4_tc_kernel, la, keys_per_split);
  if (e != cudaSuccess) {
    set_error("mla_int4_tc launch: %s", cudaGetErrorString(e));
    return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

}  // namespace dsa
