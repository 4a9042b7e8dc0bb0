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
// Work unit: (row t, key split), one pair of CTAs.  The pair runs every product as
// two-CTA tcgen05.mma (M = 128 heads, 64 of them in each CTA), so each CTA has its
// own heads' logits, softmax state and output rows, and nothing of the softmax
// crosses between them:
//   S = Q K^T   M=128, N=64 keys, K=576.  CTA r holds the 64 heads' Q and keys
//               [32r, 32r+32) of the block, all 576 dims.
//   O += P V    M=128, N=2x256 dims, K=64 keys.  CTA r holds its heads' P and
//               dims [256r, 256r+256) of all 64 keys.
// In tensor memory lane l < 64 of a CTA is head l with the first half of N, lane
// l + 64 the same head with the second half.  A block of 64 keys takes the tensor
// cores 1,428 cycles (36 MMAs of 25 cycles, bound by the operands' shared-memory
// reads, and 8 of 65) against 1,088 at their peak; 128 keys would run the first
// product at the peak, but two stages of them do not fit beside Q.
// The two operands overlap in a quarter of the block only, and each CTA decodes
// both for itself straight from the packed rows: at three instructions a pair of
// values that is cheaper than an exchange through distributed shared memory.
//
// Roles per CTA (832 threads):
//   warps 0-7    softmax and output, two groups of four warps that take the blocks in
//                turn: a block's chain (wait, tensor-memory load, maximum, weights,
//                store) is longer than its products take, so one group would set the
//                pace.  Thread = TMEM lane, 32 keys of a head; the head's other 32 are
//                lane + 64.  The running maximum passes from group to group through
//                shared memory (a few hundred cycles a block); each thread keeps its
//                own sum.  Lazy rescale as in mla_tc.cu.
//   warps 8-23   decode, two groups of eight warps that take the blocks in turn, each
//                with its own stage: packed pieces from global memory to registers, two
//                blocks' time ahead of their use (one block's was too little: the loads
//                set the pace), then 16-byte stores, swizzled, of the keys' and the
//                values' tile
//   warp 24      tensor memory; in the pair's first CTA one thread issues the MMAs
//   warp 25      resolves the selection to cache rows, two blocks at a time
// Tiles, weights and logits have two stages each; S of block j+1 is issued before
// P V of block j, so that the tensor cores work while the softmax of block j runs.
//
// Decode batches split a row's keys over 2 or 4 pairs of one cluster, which merge
// through distributed shared memory: no scratch in global memory, no arrival order.
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
constexpr int kMaxPairs = 4;                    // key splits of a row: 1, 2 or 4 (a cluster of 8 CTAs)
constexpr int kSmWarps = 8, kDecWarps = 8;
constexpr int kDecWarp0 = 8, kMmaWarp = 24, kRowWarp = 25;
constexpr int kThreads = 32 * 26;
constexpr int kSmThreads = 32 * kSmWarps;
constexpr int kDecThreads = 2 * kDecWarps * 32;
constexpr int kQChunks = kD / 64;               // 64-dim SW128 chunks: 8 latent, 1 RoPE
constexpr uint32_t kColS = 0, kColO = 64, kTmemCols = 512;
// polls of a bounded wait (20 ms at least; real waits take microseconds)
constexpr uint32_t kWaitPolls = 1u << 20;

struct Smem {                                   // 1024-byte aligned
  uint8_t q[kQChunks][kHc * 128];               // this CTA's heads
  uint8_t k[2][kQChunks][kHalfBlk * 128];       // its 32 keys, 576 dims
  uint8_t v[2][4][kBlk * 128];                  // 64 keys, its 256 dims
  uint8_t p[2][kHc * 128];                      // its heads' weights of 64 keys
  float red[2][2 * kHc];                        // by softmax group and lane: block maxima; the final sums
  float m_run[2][kHc];                          // running maximum of a head after a group's block
  int32_t rows[2][2 * kBlk];                    // cache row per key of two blocks, -1 = none
  uint32_t valid[kMaxKeys / 32];                // per 32 keys: bit i set = key i has a row
  // waited for by the issuing thread, in the pair's first CTA
  uint64_t q_full, k_full[2], v_full[2], p_full[2];
  // arrivals of finished products, in both CTAs
  uint64_t s_full[2], pv_done[2];
  uint64_t rows_full[2], rows_free[2];
  uint64_t merged;                              // the other splits' parts have arrived
  uint64_t drained;
  uint32_t tmem_base;
};
static_assert(sizeof(Smem) <= 227 * 1024, "shared memory of the attention kernel");
static_assert(offsetof(Smem, k) % 1024 == 0 && offsetof(Smem, v) % 1024 == 0 && offsetof(Smem, p) % 1024 == 0, "swizzle");
// The merge of a row's key splits S: pair s finishes columns [256 s / S, 256 (s + 1) / S)
// of every lane and gets them from the other pairs, [source][column / 4][lane] float4,
// where Q lay, with (max, sum) per source and head; it sends its other columns from
// behind that.  Rows of the finished output are staged behind those.
constexpr size_t kRecvMl = 3 * 32768, kSendMl = kRecvMl + kMaxPairs * kHc * 8, kSend = kRecvMl + 4096;
template <int kSplits>
struct Merge {
  static constexpr int kCols = 256 / kSplits;                   // columns of a lane that a pair finishes
  static constexpr uint32_t kPart = kCols * 512, kMl = kHc * 8; // bytes of one source's part
  static constexpr size_t kOut = kSplits == 1 ? offsetof(Smem, v) : kSend + (kSplits - 1) * (size_t)kPart;
  static constexpr int kOutRow = 4 * kCols + 16;                // bytes of a staged head: odd in 16-byte pieces
  static_assert((kSplits - 1) * (size_t)kPart <= kRecvMl, "receive area");
  static_assert(kOut % 128 == 0 && kOut + kHc * (size_t)kOutRow <= offsetof(Smem, red), "send and output areas");
};

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
// True in one lane of a converged warp.  The compiler knows that what follows is
// run by one thread and keeps the descriptors in uniform registers; under
// `lane == 0` it moved every operand of every MMA there first, and issuing a
// block's 44 MMAs took 4,800 cycles.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Arrive on `bar` of the pair's two CTAs (cluster ranks `mask`) when the products
// issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)), "h"(mask) : "memory");
}
// Bounded wait; on time-out records DSA_ERR_TIMEOUT (detail = site) and returns
// false.  Written out so that a barrier already complete costs two instructions:
// every warp passes two to four of them a block.
__device__ __forceinline__ bool wait_local(uint64_t* bar, uint32_t parity, DeviceStatus* st, int site) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, %3;\n"
      "WAIT_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE_%=;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra WAIT_%=;\n"
      "DONE_%=:\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "n"(kWaitPolls) : "memory");
  if (!ok) set_status(st, DSA_ERR_TIMEOUT, site);
  return ok != 0;
}
// The same, agreed on by the warp (its lanes go on or leave together).
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, DeviceStatus* st, int site) {
  return __all_sync(0xffffffffu, wait_local(bar, parity, st, site));
}
// One arrival per warp on a barrier of the pair's first CTA.  What it announces
// lies in the arriving CTA's own shared or tensor memory and is read by the tensor
// cores only: fence.proxy.async (stores) or tcgen05.fence (tensor-memory reads),
// executed before it by every lane, makes that visible to them, so the arrive
// itself is ordered at CTA scope.  A release at cluster scope would also wait for
// this thread's global loads in flight: it cost 1,000 cycles an arrive, and a
// block 5,800 cycles instead of 2,700.
// `first`: this CTA's shared-memory window mapped to the pair's first CTA, minus the
// local window (mapa of the base, taken once).
__device__ __forceinline__ void warp_arrive_first(uint64_t* bar, uint32_t first) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .u32 l;\n\t"
      "mov.u32 l, %%laneid;\n\t"
      "setp.eq.u32 p, l, 0;\n\t"
      "@p mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar) + first) : "memory");
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---------------------------------------------------------------- MMA issue (first CTA, one thread)
__device__ __forceinline__ void issue_products(Smem& S, const MlaArgs& a, uint32_t tmem, int nblk, uint16_t mask) {
  DeviceStatus* status = a.status;
  constexpr uint32_t idesc_s = idesc_bf16(kBlk, false);
  constexpr uint32_t idesc_pv = idesc_bf16(256, true);
  bool ok = wait_local(&S.q_full, 0, status, 41);
  // descriptors: a byte offset within the tile adds offset >> 4 to the address field
  const uint64_t qd = sdesc_sw128(smem_u32(S.q), 16, 1024), pd = sdesc_sw128(smem_u32(S.p), 16, 1024);
  const uint64_t kd0 = sdesc_sw128(smem_u32(S.k[0]), 16, 1024);
  const uint64_t vd0 = sdesc_sw128(smem_u32(S.v[0]), kBlk * 128, 1024);
  for (int j = 0; ok && j <= nblk; ++j) {
    if (j < nblk) {
      const int b = j & 1;
      // (S of block j-2 has been read: P V of that block waited for its weights)
      if (!(ok = wait_local(&S.k_full[b], (j >> 1) & 1, status, 42))) break;
      tc_fence_after();
      const uint64_t kd = kd0 + (uint64_t)(b * (sizeof(S.k[0]) >> 4));
      const uint32_t d = tmem + kColS + b * 32;
#pragma unroll
      for (int ch = 0; ch < kQChunks; ++ch)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_bf16_pair(d, qd + (ch * kHc * 128 + 32 * kk >> 4), kd + (ch * kHalfBlk * 128 + 32 * kk >> 4), idesc_s,
                        (ch | kk) != 0);
      mma_commit_pair(&S.s_full[b], mask);
      tstamp(a.trace, 0, 2, j);
    }
    if (j >= 1) {
      const int jj = j - 1, b = jj & 1;
      ok = wait_local(&S.v_full[b], (jj >> 1) & 1, status, 44) && wait_local(&S.p_full[b], (jj >> 1) & 1, status, 45);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vd = vd0 + (uint64_t)(b * (sizeof(S.v[0]) >> 4));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          mma_bf16_pair(tmem + kColO + n * 128, pd + b * (sizeof(S.p[0]) >> 4) + (32 * kk >> 4),
                        vd + (n * 2 * kBlk * 128 + kk * 16 * 128 >> 4), idesc_pv, (jj | kk) != 0);
      mma_commit_pair(&S.pv_done[b], mask);
      tstamp(a.trace, 0, 3, jj);
    }
  }
  // every product issued is done before the pair's shared and tensor memory go
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&S.drained))
               : "memory");
  wait_local(&S.drained, 0, status, 46);
}

// ---------------------------------------------------------------- the selection
// One warp turns the selection into cache rows, two blocks (four keys a lane) at a
// time: their block-table entries and the next positions are in flight while the
// two before are handed over.
__device__ __forceinline__ void resolve_rows(Smem& S, const MlaArgs& a, int t, int seq, int klen, int k0, int nvalid,
                                             int nblk) {
  constexpr int kKeys = 2 * kBlk / 32;
  const int lane = threadIdx.x & 31;
  const int32_t* idx = a.idx + (int64_t)t * a.topk + k0;
  const CacheMap& m = a.map;
  const int32_t* table = m.block_table ? m.block_table + (int64_t)seq * m.max_pages_per_seq : nullptr;
  const int64_t start = !m.block_table && m.seq_start ? (int64_t)__ldg(m.seq_start + seq) : 0;
  const auto positions = [&](int p, int (&s)[kKeys]) {
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      const int i = p * 2 * kBlk + 32 * u + lane;
      s[u] = i < nvalid ? __ldg(idx + i) : -1;
      if (s[u] >= klen) s[u] = -1;
    }
  };
  const auto page_of = [&](int s) { return m.page_shift >= 0 ? s >> m.page_shift : s / m.page_size; };
  const auto entries = [&](const int (&s)[kKeys], int (&e)[kKeys]) {
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      e[u] = -1;
      if (s[u] < 0 || table == nullptr) continue;
      const int pg = page_of(s[u]);
      if (pg < m.max_pages_per_seq) e[u] = __ldg(table + pg);
      else set_status(a.status, DSA_ERR_OUT_OF_RANGE, s[u]);
    }
  };
  const auto row_of = [&](int s, int e) {
    if (s < 0) return -1;
    if (table != nullptr) {
      const int pg = page_of(s);
      if (pg >= m.max_pages_per_seq) return -1;
      if (e < 0 || e >= m.num_pages) {
        set_status(a.status, DSA_ERR_OUT_OF_RANGE, e);
        return -1;
      }
      return (int)((int64_t)e * m.page_size + (s - pg * m.page_size));
    }
    const int64_t r = start + s;
    if (r < 0 || r >= m.num_tokens) {
      set_status(a.status, DSA_ERR_OUT_OF_RANGE, s);
      return -1;
    }
    return (int)r;
  };
  int s0[kKeys], s1[kKeys], s2[kKeys], e0[kKeys], e1[kKeys];
  positions(0, s0);
  positions(1, s1);
  entries(s0, e0);
  cluster_wait();
  for (int p = 0; 2 * p < nblk; ++p) {
    positions(p + 2, s2);
    entries(s1, e1);
    if (!wait_warp(&S.rows_free[p & 1], ((p >> 1) & 1) ^ 1, a.status, 53)) break;
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      const int row = row_of(s0[u], e0[u]);
      S.rows[p & 1][32 * u + lane] = row;
      const uint32_t bits = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0) S.valid[kKeys * p + u] = bits;
      s0[u] = s1[u];
      s1[u] = s2[u];
      e0[u] = e1[u];
    }
    warp_arrive(&S.rows_full[p & 1]);
  }
}

// ---------------------------------------------------------------- decoding
// The packed codes of 64 dims of one key (32 bytes) and their four scales, first and
// second half swapped in odd units.
struct Unit {
  uint4 codes[2];
  uint32_t scales;

  // Unit `u` of the row (zeros for a key without a row).
  __device__ __forceinline__ void load(const uint8_t* latent, int row, int u) {
    codes[0] = codes[1] = make_uint4(0u, 0u, 0u, 0u);
    scales = 0u;
    if (row >= 0) {
      const uint8_t* src = latent + (int64_t)row * kRow.bytes;
      const int odd = (u & 1) * 16;
      codes[0] = __ldg(reinterpret_cast<const uint4*>(src + 32 * u + odd));
      codes[1] = __ldg(reinterpret_cast<const uint4*>(src + 32 * u + (odd ^ 16)));
      scales = __ldg(reinterpret_cast<const uint32_t*>(src + kRow.scale) + u);
    }
  }
  // Decoded to a tile's 128-byte row; `at`: its address with the swizzle of the first
  // piece in bits 4-6, from which piece e's differs by e (the tile's rows and bits are
  // aligned, so that an exclusive or does).
  __device__ __forceinline__ void store(uint32_t at, int odd) const {
    const uint32_t sc = odd ? __funnelshift_r(scales, scales, 16) : scales;
    const uint32_t w[8] = {codes[0].x, codes[0].y, codes[0].z, codes[0].w, codes[1].x, codes[1].y, codes[1].z, codes[1].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const ScalePair s = scale_pair((sc >> (8 * q)) & 0xFFu);
      st_smem_v4(at ^ (32u * q), decode_word(w[2 * q], s));
      st_smem_v4(at ^ (32u * q + 16u), decode_word(w[2 * q + 1], s));
    }
  }
};

// The blocks of one parity g: warp w of its eight.  Per block a lane decodes one unit
// of the keys' tile and one of the values'.  Eight neighbouring lanes take four keys
// and two neighbouring units of each: a load then touches four lines for every eight
// lanes (eight keys touched eight, and the L1's data stage set the pace), and with
// odd units' halves swapped the eight 16-byte stores still fall into distinct banks.
//   keys' tile:   keys 4 w.. of the CTA's 32, all 8 units
//   values' tile: keys 8 w.., the CTA's 4 units
__device__ __forceinline__ void decode_blocks(Smem& S, const MlaArgs& a, int nblk, uint32_t rank, uint32_t first, int w, int g) {
  const uint8_t* latent = static_cast<const uint8_t*>(a.latent);
  const int lane = threadIdx.x & 31, odd = lane & 1, quad = lane >> 3;
  const bool stamp = a.trace != nullptr && w == 0 && lane == 0;
  const int k_key = 4 * w + ((lane & 7) >> 1), k_unit = 2 * quad + odd;
  const int v_key = 8 * w + 4 * (quad & 1) + ((lane & 7) >> 1), v_unit = 2 * (quad >> 1) + odd;
  const uint32_t k_dst = smem_u32(S.k[g][k_unit]) + k_key * 128 + (((4 * odd) ^ (k_key & 7)) << 4);
  const uint32_t v_dst = smem_u32(S.v[g][v_unit]) + v_key * 128 + (((4 * odd) ^ (v_key & 7)) << 4);
  const int kt = w * 32 + lane;                                   // RoPE: 32 keys x 8 pieces, one per thread
  uint8_t* r_dst = S.k[g][8] + sw128_off(kt >> 3, kt & 7);
  const int own = g * kBlk + kHalfBlk * (int)rank;                // the CTA's keys in the two blocks' rows
  Unit ku, vu;
  uint4 rope;
  int k_row = -1, v_row = -1;
  const auto load_keys = [&](int j) {
    const int p = j >> 1;
    if (!wait_warp(&S.rows_full[p & 1], (p >> 1) & 1, a.status, 54)) return false;
    const int32_t* rows = S.rows[p & 1];
    k_row = rows[own + k_key];
    v_row = rows[g * kBlk + v_key];
    const int r_row = rows[own + (kt >> 3)];
    warp_arrive(&S.rows_free[p & 1]);
    ku.load(latent, k_row, k_unit);
    rope = make_uint4(0u, 0u, 0u, 0u);
    if (r_row >= 0) rope = __ldg(reinterpret_cast<const uint4*>(latent + (int64_t)r_row * kRow.bytes + kRow.rope + 16 * (kt & 7)));
    return true;
  };
  const auto load_values = [&] { vu.load(latent, v_row, 4 * (int)rank + v_unit); };
  bool ok = true;
  if (g < nblk) {
    ok = load_keys(g);
    load_values();
  }
  cp_async_wait_all();                            // this thread's pieces of Q
  fence_proxy_async_smem();
  cluster_wait();                                 // the first CTA's barriers are initialised
  warp_arrive_first(&S.q_full, first);
  for (int j = g; ok && j < nblk; j += 2) {
    const uint32_t free = ((j >> 1) & 1) ^ 1;
    // the keys' stage is free once S of block j-2 has read it
    if (!wait_warp(&S.s_full[g], free, a.status, 47)) break;
    if (stamp) tstamp(a.trace, rank, 5, j);
    ku.store(k_dst, odd);
    *reinterpret_cast<uint4*>(r_dst) = rope;
    fence_proxy_async_smem();                     // generic stores -> tensor cores
    warp_arrive_first(&S.k_full[g], first);
    if (stamp) tstamp(a.trace, rank, 0, j);
    if (j + 2 < nblk) ok = load_keys(j + 2);
    // the values' once P V of block j-2 has
    if (!ok || !wait_warp(&S.pv_done[g], free, a.status, 48)) break;
    if (stamp) tstamp(a.trace, rank, 7, j);
    vu.store(v_dst, odd);
    fence_proxy_async_smem();
    warp_arrive_first(&S.v_full[g], first);
    if (stamp) tstamp(a.trace, rank, 1, j);
    if (j + 2 < nblk) load_values();
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

// Two fp32 in one 64-bit register pair: one instruction for both.
__device__ __forceinline__ uint64_t pair_f32(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split_f32(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Softmax state of a thread: lane l of tensor memory (head l % 64, keys 32 (l / 64)..
// of a block), blocks of its group's parity.
struct Softmax {
  float m = -INFINITY, sum = 0.f;                 // maximum (log2 domain) that the sum refers to, sum
  bool dead = false;                              // a wait ran out

  // One block of group g = j % 2.  A thread whose wait ran out (dead) skips its waits
  // and goes on, so that every arrival and collective access stays uniform.
  __device__ __forceinline__ void block(Smem& S, const MlaArgs& a, uint32_t tmem_lane, int j, int nblk, int g, float c,
                                        uint32_t rank, uint32_t first) {
    const int l = threadIdx.x & 127, half = l >> 6, hl = l & 63;
    const uint32_t phase = (j >> 1) & 1;
    dead = dead || !wait_local(&S.s_full[g], phase, a.status, 49);
    tc_fence_after();
    if (l == 0 && a.trace != nullptr) tstamp(a.trace, rank, 4, j);
    float s[32];
    tmem_ld32(tmem_lane + kColS + g * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
    tmem_wait_ld();
    // masked keys are -inf (a full block needs no test)
    const uint32_t mask = S.valid[2 * j + half];
    if (mask != 0xFFFFFFFFu) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!((mask >> i) & 1u)) s[i] = -INFINITY;
    }
    float pm[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pm[i] = max3(s[2 * i], s[2 * i + 1], s[8 + i]);
#pragma unroll
    for (int i = 12; i < 32; i += 8)
#pragma unroll
      for (int k = 0; k < 4; ++k) pm[k] = i + 4 + k < 32 ? max3(pm[k], s[i + k], s[i + 4 + k]) : fmaxf(pm[k], s[i + k]);
    const float mh = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
    S.red[g][l] = mh;
    // named barriers, not mbarriers: even a wait that is already met costs ~200 cycles
    // on an mbarrier, and this chain sets the pace.  First the running maximum after
    // the other group's block j-1, then this block's from the group's other warps.
    if (j > 0) named_bar_sync(4 + (g ^ 1), kSmThreads);
    float m_now = j > 0 ? S.m_run[g ^ 1][hl] : -INFINITY;
    named_bar_sync(2 + g, kSmThreads / 2);
    const float mb = c * fmaxf(mh, S.red[g][l ^ 64]);
    // lazy rescale: P stays <= 2^8.  Warp-uniform (tensor-memory access is collective);
    // the two lanes of a head decide alike
    const bool need = mb > m_now + kRescale;
    if (__any_sync(0xffffffffu, need)) {
      const float m_new = need ? mb : m_now;
      const float alpha = need ? (m_now == -INFINITY ? 0.f : exp2f(m_now - m_new)) : 1.f;
      if (j > 0) {
        // no product is in flight: block j-1's is done, block j's waits for P below
        dead = dead || !wait_local(&S.pv_done[g ^ 1], ((j - 1) >> 1) & 1, a.status, 50);
        tc_fence_after();
#pragma unroll 1
        for (int cc = 0; cc < 16; ++cc) {
          uint32_t o[16];
          const uint32_t col = tmem_lane + kColO + 16 * cc;
          tmem_ld16(col, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
          tmem_st16(col, o);
        }
        tmem_wait_st();
      }
      m_now = m_new;
    }
    if (half == 0) S.m_run[g][hl] = m_now;
    if (j + 1 < nblk) named_bar_arrive(4 + g, kSmThreads);
    if (__any_sync(0xffffffffu, m != m_now)) {
      sum *= m == -INFINITY ? 0.f : exp2f(m - m_now);
      m = m_now;
    }
    // (the weights' tile is free: P V of block j-2 was issued before S of this block,
    // and a commit covers all that was issued before it)
    // p = 2^(c s - m); while no key of the head has been visible m counts as 0
    const float mu = (m == -INFINITY) ? 0.f : -m;
    const uint64_t c2 = pair_f32(c, c), mu2 = pair_f32(mu, mu);
    uint64_t ls = 0;                              // two running sums
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t p2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float z0, z1;
        split_f32(fma_f32x2(pair_f32(s[8 * q + 2 * i], s[8 * q + 2 * i + 1]), c2, mu2), z0, z1);
        const float p0 = ex2_approx(z0), p1 = ex2_approx(z1);
        ls = add_f32x2(ls, pair_f32(p0, p1));
        p2[i] = pack_bf16x2(p0, p1);
      }
      *reinterpret_cast<uint4*>(S.p[g] + sw128_off(hl, 4 * half + q)) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    warp_arrive_first(&S.p_full[g], first);
    float l0, l1;
    split_f32(ls, l0, l1);
    sum += l0 + l1;
    if (l == 0 && a.trace != nullptr) tstamp(a.trace, rank, 6, j);
  }
};

// S: key splits of a row = pairs of a cluster.
template <int kSplits>
__global__ void __launch_bounds__(kThreads, 1) mla_int4_tc_kernel(MlaArgs a) {
  extern __shared__ __align__(1024) uint8_t smraw[];
  Smem& S = *reinterpret_cast<Smem*>(smraw);
  const int warp = threadIdx.x >> 5;
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, first = crank & ~1u;
  const int sp = (int)(crank >> 1);
  const uint32_t to_first = mapa(smraw, first) - smem_u32(smraw);
  const int t = blockIdx.x / (2 * kSplits);
  pdl_launch_dependents();

  // setup that reads no input memory overlaps the predecessor's tail
  if (threadIdx.x == 0) {
    mbar_init(&S.q_full, 2 * 2 * kDecWarps);
    mbar_init(&S.drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], 2 * kDecWarps);
      mbar_init(&S.v_full[i], 2 * kDecWarps);
      mbar_init(&S.p_full[i], kSmWarps);         // a group's four warps in each CTA
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.pv_done[i], 1);
      mbar_init(&S.rows_full[i], 1);
      mbar_init(&S.rows_free[i], 2 * kDecWarps);
    }
    mbar_init(&S.merged, 1);
    fence_mbar_init();
    if (kSplits > 1) mbar_expect_tx(&S.merged, (kSplits - 1) * (Merge<kSplits>::kPart + Merge<kSplits>::kMl));
  }
  __syncwarp();
  if (warp == kMmaWarp) tmem_alloc_pair(&S.tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();                     // waited for before anything touches another CTA
  const uint32_t tmem = S.tmem_base;
  pdl_wait();
  trace_kernel(a.status, DSA_KERNEL_MLA_INT4_TC);
  const int klen = a.row_klen[t];
  const int seq = a.row_seq[t];
  const bool known = (seq >= 0 && seq < a.num_seqs) || !a.map.uses_seq();
  if (!known && klen > 0 && threadIdx.x == 0) set_status(a.status, DSA_ERR_OUT_OF_RANGE, t);
  const int nsel = known ? min(klen, a.topk) : 0;
  // whole blocks per split, shared out over what the row really selects
  const int keys_per_split = (max(nsel, 0) + kSplits * kBlk - 1) / (kSplits * kBlk) * kBlk;
  const int k0 = sp * keys_per_split;
  const int nvalid = max(0, min(nsel - k0, keys_per_split));
  const int nblk = (nvalid + kBlk - 1) / kBlk;
  const bool empty = nblk == 0;
  Softmax sm;

  if (warp == kMmaWarp) {
    cluster_wait();
    if (rank == 0 && !empty && elect_one()) issue_products(S, a, tmem, nblk, (uint16_t)(3u << first));
    __syncwarp();
  } else if (warp == kRowWarp) {
    if (!empty) resolve_rows(S, a, t, seq, klen, k0, nvalid, nblk);
    else cluster_wait();
  } else if (warp >= kDecWarp0) {
    if (!empty) {
      // Q lands while the selection is resolved; heads beyond H are zeros
      const int th = threadIdx.x - 32 * kDecWarp0, h0 = kHc * (int)rank;
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)t * a.n_heads * kD;
#pragma unroll
      for (int i = 0; i < kHc * kD / 8 / kDecThreads; ++i) {
        const int qi = th + i * kDecThreads, h = qi / (kD / 8), c = qi - h * (kD / 8);
        const bool in = h0 + h < a.n_heads;
        cp_async_16_zfill(S.q[c >> 3] + sw128_off(h, c & 7), q + (int64_t)(in ? h0 + h : 0) * kD + 8 * c, in);
      }
      const int w = warp - kDecWarp0;
      decode_blocks(S, a, nblk, rank, to_first, w % kDecWarps, w / kDecWarps);
    } else {
      cluster_wait();
    }
  } else {
    cluster_wait();
    const float c = a.sm_scale * kLog2e;
    const uint32_t tmem_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int g = warp >> 2;
    for (int j = g; j < nblk; j += 2) sm.block(S, a, tmem_lane, j, nblk, g, c, rank, to_first);
    if (!sm.dead && !empty) {
      sm.dead = !wait_local(&S.pv_done[(nblk - 1) & 1], ((nblk - 1) >> 1) & 1, a.status, 52);
      tc_fence_after();
    }
  }

  // The row's output.  With key splits the pairs of the cluster first exchange what
  // they hold, once every pair's products are done and its tiles may be overwritten.
  using Mg = Merge<kSplits>;
  constexpr int kCols = Mg::kCols;
  if (kSplits > 1) {
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
  }
  if (warp < kSmWarps) {
    const int l = threadIdx.x & 127, cw = threadIdx.x >> 7, half = l >> 6, hl = l & 63;
    const uint32_t o_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kColO;
    // the head's maximum and its sum over four threads; a wait that ran out anywhere
    // fails the CTA
    const bool fail = named_bar_or(1, kSmThreads, sm.dead);
    float M = empty ? -INFINITY : S.m_run[(nblk - 1) & 1][hl];
    S.red[cw][l] = sm.m == -INFINITY ? 0.f : sm.sum * exp2f(sm.m - M);
    named_bar_sync(1, kSmThreads);
    float L = (S.red[0][hl] + S.red[1][hl]) + (S.red[0][hl + 64] + S.red[1][hl + 64]);
    if (fail) L = __int_as_float(0x7FC00000);     // marks the row for the other pairs too
    float w[kSplits];
    w[0] = 1.f;
    bool got = true;
    if (kSplits > 1) {
      // parts for the other pairs, 32 columns at a time: staged, then one bulk copy
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        const int col = 128 * cw + 32 * cc, to = col / kCols;
        if (to == sp) continue;
        float o[32];
        load_o32(o_lane + col, empty || fail, o);
        const int out_slot = to < sp ? to : to - 1, in_slot = sp < to ? sp : sp - 1;
        const size_t off = (size_t)(col - to * kCols) * 512;
        uint8_t* src = smraw + kSend + out_slot * (size_t)Mg::kPart + off;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(src + (i * 128 + l) * 16) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        fence_proxy_async_smem();
        named_bar_sync(2 + cw, 128);
        if (l == 0)
          bulk_copy_to_peer(smraw + in_slot * (size_t)Mg::kPart + off, src, 32 * 512, &S.merged, (uint32_t)(2 * to) + rank);
      }
      float2* ml = reinterpret_cast<float2*>(smraw + kSendMl);
      if (cw == 0 && half == 0) ml[hl] = make_float2(M, L);
      fence_proxy_async_smem();
      named_bar_sync(1, kSmThreads);
      if (threadIdx.x < kSplits && threadIdx.x != sp)
        bulk_copy_to_peer(smraw + kRecvMl + sp * (size_t)Mg::kMl, ml, Mg::kMl, &S.merged, 2 * threadIdx.x + rank);
      bulk_commit();
      got = wait_local(&S.merged, 0, a.status, 57);
      // out = sum_s w_s O_s / sum_s w_s l_s,  w_s = 2^(m_s - max m), splits in order
      const float2 mine = make_float2(M, L);
      M = -INFINITY;
      L = 0.f;
      float2 v[kSplits];
#pragma unroll
      for (int s2 = 0; s2 < kSplits; ++s2) {
        v[s2] = s2 == sp ? mine : reinterpret_cast<const float2*>(smraw + kRecvMl + s2 * (size_t)Mg::kMl)[hl];
        M = fmaxf(M, v[s2].x);
      }
#pragma unroll
      for (int s2 = 0; s2 < kSplits; ++s2) {
        w[s2] = v[s2].x == -INFINITY ? 0.f : exp2f(v[s2].x - M);
        L += w[s2] * v[s2].y;                     // NaN of a failed pair stays
      }
    }
    const bool bad = named_bar_or(1, kSmThreads, !got) || L != L;
    const float inv = L > 0.f ? 1.f / L : 0.f;
    // Finished rows go through shared memory, so that each head's columns leave as
    // two bulk copies (one from each half of the dims).
    uint8_t* stg = smraw + Mg::kOut + (size_t)hl * Mg::kOutRow + half * 2 * kCols;
    constexpr int kMine = kCols / 2;              // columns of this thread: 128, 64 or 32
#pragma unroll 1
    for (int cc = 0; cc < kMine / 32; ++cc) {
      const int col = kMine * cw + 32 * cc;       // within the pair's columns
      float o[32];
      load_o32(o_lane + sp * kCols + col, empty || bad, o);
      if (kSplits > 1) {
        float acc[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[i] = 0.f;
#pragma unroll
        for (int s2 = 0; s2 < kSplits; ++s2) {
          if (s2 == sp) {
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = fmaf(w[s2], o[i], acc[i]);
          } else {
            const uint8_t* src = smraw + (s2 < sp ? s2 : s2 - 1) * (size_t)Mg::kPart + (size_t)col * 512 + l * 16;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 x = *reinterpret_cast<const float4*>(src + i * 2048);
              acc[4 * i] = fmaf(w[s2], x.x, acc[4 * i]);
              acc[4 * i + 1] = fmaf(w[s2], x.y, acc[4 * i + 1]);
              acc[4 * i + 2] = fmaf(w[s2], x.z, acc[4 * i + 2]);
              acc[4 * i + 3] = fmaf(w[s2], x.w, acc[4 * i + 3]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = bad ? 0.f : acc[i];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4*>(stg + 2 * col + 16 * q) = pack8(&o[8 * q], inv);
    }
    fence_proxy_async_smem();
    named_bar_sync(1, kSmThreads);
    const int head = kHc * (int)rank + hl;
    if (cw == 0 && head < a.n_heads) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + ((int64_t)t * a.n_heads + head) * kDC + 256 * half + sp * kCols;
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(out), "r"(smem_u32(stg)), "n"(2 * kCols)
                   : "memory");
      bulk_commit();
      if (a.lse && sp == 0 && half == 0)
        a.lse[(int64_t)t * a.n_heads + head] = L > 0.f ? (M + log2f(L)) * kLn2 : -INFINITY;
    }
    // this thread's copies are done before shared memory goes
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                       // no access to the pair's memory is still pending
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

using Kernel = void (*)(MlaArgs);
template <int kSplits>
constexpr Kernel kernel_of = mla_int4_tc_kernel<kSplits>;

cudaLaunchConfig_t launch_config(cudaLaunchAttribute (&at)[2], int splits, int rows) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * splits * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Smem);
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)(splits * 2);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

// Clusters of `splits` pairs that can be resident at once on this device (0 if the
// query fails), looked up once per device.
int resident_clusters(Kernel kernel, int splits) {
  static std::atomic<int> cached[kMaxPairs + 1][kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  const int have = cached[splits][dev].load();
  if (have > 0) return have - 1;
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = launch_config(at, splits, 1);
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  cached[splits][dev].store(n + 1);
  return n;
}

}  // namespace

bool mla_int4_tc_supported(const MlaArgs& a) {
  return a.mla_dtype == DSA_INT4 && a.n_heads <= 2 * kHc && a.d_c == kDC && a.d_r == kDR && a.topk <= kMaxKeys;
}

dsa_status launch_mla_int4_tc(const MlaArgs& a, cudaStream_t stream) {
  if (a.num_rows == 0) return DSA_OK;
  static std::atomic<bool> attr1[kMaxDevices] = {}, attr2[kMaxDevices] = {}, attr4[kMaxDevices] = {};
  dsa_status st;
  if ((st = set_smem_limit_once(reinterpret_cast<const void*>(kernel_of<1>), sizeof(Smem), attr1)) ||
      (st = set_smem_limit_once(reinterpret_cast<const void*>(kernel_of<2>), sizeof(Smem), attr2)) ||
      (st = set_smem_limit_once(reinterpret_cast<const void*>(kernel_of<4>), sizeof(Smem), attr4)))
    return st;
  // key splits: the most whose clusters are all resident at once (a second wave costs
  // more than a split saves), where the selection has a block of keys for each
  int splits = 1;
  Kernel kernel = kernel_of<1>;
  if (a.topk > 2 * kBlk && a.num_rows <= resident_clusters(kernel_of<4>, 4)) {
    splits = 4;
    kernel = kernel_of<4>;
  } else if (a.topk > kBlk && a.num_rows <= resident_clusters(kernel_of<2>, 2)) {
    splits = 2;
    kernel = kernel_of<2>;
  }
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = launch_config(at, splits, a.num_rows);
  cfg.stream = stream;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) {
    set_error("mla_int4_tc launch: %s", cudaGetErrorString(e));
    return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

}  // namespace dsa
