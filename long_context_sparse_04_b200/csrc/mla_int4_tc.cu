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
// Roles per CTA (896 threads):
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
//   warp 24      tensor memory; in the pair's first CTA one thread issues Q K^T
//   warps 25-26  resolve the selection to cache rows, up to four blocks ahead
//   warp 27      in the first CTA one thread issues P V
// Tiles, weights and logits have two stages each; S of block j+1 runs before P V of
// block j, so that the tensor cores work while the softmax of block j does.
// Without key splits the kernel is persistent: a pair takes rows t, t + pairs, ...,
// its blocks one stream across rows (block counter n: stage and group n % 2), so that
// the next row's selection, rows, tiles and Q come in while this row is finished.
//
// Decode batches split a row's keys over 2 or 4 pairs of one cluster, which merge
// through distributed shared memory: no scratch in global memory, no arrival order.
//
// Measured with 128 heads and 2,048 selected keys: 32 rows 32 us (56,000 cycles: 8,000
// to the first tile, 16 blocks, 12,000 of merge and output) against a floor of 11.1 us
// of tensor time; 2,048 rows 1.11 ms (1.05 PFLOP/s) on a cool card and 1.28 under its
// power cap, floor 0.71.  A block takes about 2,000 cycles: what a decoding group needs
// for its two tiles of two blocks, waits and arrivals included, at 8 cycles an
// instruction (148 rows: issue slots 64 % used, tensor pipe 46 %).
#include <cudaTypedefs.h>

#include "dsa_int4.cuh"
#include "dsa_kernels.cuh"
#include "mla_common.cuh"
#include "mla_int4_shape.h"

namespace dsa {
namespace {

constexpr int kHc = 64;                         // heads per CTA
constexpr int kDC = 512, kDR = 64, kD = kDC + kDR;
constexpr Int4Row kRow = int4_row(kDC, kDR);
constexpr int kBlk = 64, kHalfBlk = 32;
constexpr int kMaxKeys = 2048;
constexpr int kMaxPairs = 4;                    // key splits of a row: 1, 2 or 4 (a cluster of 8 CTAs)
constexpr int kSmWarps = 8, kDecWarps = 8;
constexpr int kDecWarp0 = 8, kMmaWarp = 24, kRowWarp = 25, kRowWarps = 2, kMmaWarp2 = 27;
constexpr int kThreads = 32 * 28;
constexpr int kSmThreads = 32 * kSmWarps;
constexpr int kDecThreads = 2 * kDecWarps * 32;
constexpr int kQChunks = kD / 64;               // 64-dim SW128 chunks: 8 latent, 1 RoPE
constexpr uint32_t kColS = 0, kColO = 64, kTmemCols = 512;
// Blocks in the ring of resolved rows, and in that of their validity bits: block n's are
// read by the softmax before its weights are stored, and resolving block n + 10 waits for
// those (rows n + 6 loaded, keys n + 4 stored, S of block n + 2 done, weights n stored).
constexpr int kRowRing = 4, kValidRing = 16;
// polls of a bounded wait (a poll that finds nothing takes up to 4 us: 4 s in all; real
// waits take microseconds), unless a test sets fewer: read from the arguments, which costs
// under 1 % of any case
constexpr uint32_t kWaitPolls = 1u << 20;

struct Smem {                                   // 1024-byte aligned
  uint8_t q[kQChunks][kHc * 128];               // this CTA's heads
  uint8_t k[2][kQChunks][kHalfBlk * 128];       // its 32 keys, 576 dims
  uint8_t v[2][4][kBlk * 128];                  // 64 keys, its 256 dims
  uint8_t p[2][kHc * 128];                      // its heads' weights of 64 keys
  float red[2][2 * kHc];                        // by softmax group and lane: block maxima; the final sums
  float m_run[2][kHc];                          // running maximum of a head after a group's block
  int32_t rows[kRowRing][kBlk];                 // cache row per key of a block, -1 = none
  uint32_t valid[kValidRing][2];                // per 32 keys: bit i set = key i has a row
  // waited for by the issuing thread, in the pair's first CTA
  uint64_t q_full, k_full[2], v_full[2], p_full[2], o_free;
  // arrivals of finished products, in both CTAs
  uint64_t s_full[2], pv_done[2], q_idle;       // q_idle: every S of a row
  uint64_t rows_full[kRowRing], rows_free[kRowRing];
  uint64_t merged;                              // the other splits' parts have arrived
  uint64_t v_idle[2];                           // the row's output has left a stage of the values' tiles
  uint64_t drained;
  uint32_t tmem_base;
};
static_assert(sizeof(Smem) <= 227 * 1024, "shared memory of the attention kernel");
static_assert(offsetof(Smem, k) % 1024 == 0 && offsetof(Smem, v) % 1024 == 0 && offsetof(Smem, p) % 1024 == 0, "swizzle");
// The merge of a row's key splits S: pair s finishes columns [256 s / S, 256 (s + 1) / S)
// of every lane and gets them from the other pairs, [source][column / 4][lane] float4,
// where Q lay, with (max, sum) per source and head; it sends its other columns from
// behind that.  Copies between CTAs run at 16 bytes a cycle, 2 us of a row of two splits
// and 128 heads, so only the lanes of heads that exist travel.  Finished columns are staged as tiles of 64 heads x 64 dims (128-byte
// rows, swizzled), one bulk tensor store each: in the values' tiles, idle between a
// row's last product and the next row's first, or with splits behind what is sent.
constexpr size_t kRecvMl = 3 * 32768, kSendMl = kRecvMl + kMaxPairs * kHc * 8, kSend = kRecvMl + 4096;
template <int kSplits>
struct Merge {
  static constexpr int kCols = 256 / kSplits;                   // columns of a lane that a pair finishes
  static constexpr uint32_t kPart = kCols * 512, kMl = kHc * 8; // bytes of one source's part, at most
  static constexpr int kTiles = 8 / kSplits;                    // staged tiles: kTiles / 2 from each half of the dims
  static constexpr size_t kOut =
      kSplits == 1 ? offsetof(Smem, v) : (kSend + (kSplits - 1) * (size_t)kPart + 1023) / 1024 * 1024;
  static_assert((kSplits - 1) * (size_t)kPart <= kRecvMl, "receive area");
  static_assert(kOut + kTiles * 8192 <= offsetof(Smem, p) || (kSplits > 1 && kOut + kTiles * 8192 <= offsetof(Smem, red)),
                "output tiles");
  static_assert(kSend + (kSplits - 1) * (size_t)kPart <= offsetof(Smem, red), "send area");
};

// The selected keys of a row (of its split sp of kSplits).
struct Row {
  int klen, seq, nsel, k0, nvalid, nblk;
};
template <int kSplits>
__device__ __forceinline__ Row row_of(const MlaArgs& a, int klen, int seq, int sp) {
  Row r;
  const bool known = (seq >= 0 && seq < a.num_seqs) || !a.map.uses_seq();
  r.klen = klen;
  r.seq = seq;
  r.nsel = known ? max(min(klen, a.topk), 0) : 0;
  // whole blocks per split, shared out over what the row really selects
  const int per_split = (r.nsel + kSplits * kBlk - 1) / (kSplits * kBlk) * kBlk;
  r.k0 = sp * per_split;
  r.nvalid = max(0, min(r.nsel - r.k0, per_split));
  r.nblk = (r.nvalid + kBlk - 1) / kBlk;
  return r;
}
// The rows t0, t0 + step, ... of a pair, the next one's lengths in flight.
template <int kSplits>
struct RowStream {
  const MlaArgs& a;
  int t, step, sp, klen_next = 0, seq_next = 0;
  __device__ __forceinline__ RowStream(const MlaArgs& a_, int t0, int step_, int sp_) : a(a_), t(t0 - step_), step(step_), sp(sp_) {
    fetch();
  }
  __device__ __forceinline__ void fetch() {
    if (t + step < a.num_rows) {
      klen_next = __ldg(a.row_klen + t + step);
      seq_next = __ldg(a.row_seq + t + step);
    }
  }
  // The next row; false behind the last.
  __device__ __forceinline__ bool next(Row& r) {
    t += step;
    if (t >= a.num_rows) return false;
    r = row_of<kSplits>(a, klen_next, seq_next, sp);
    fetch();
    return true;
  }
  // The next row that selects anything (r.nblk = 0 behind the last).
  __device__ __forceinline__ bool next_busy(Row& r) {
    while (next(r))
      if (r.nblk > 0) return true;
    r.nblk = 0;
    return false;
  }
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
// cluster_arrive() that orders no memory accesses.
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
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
// The same on `bar` of this CTA alone.
__device__ __forceinline__ void mma_commit_own(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Bounded wait; on time-out records DSA_ERR_TIMEOUT (detail = site) and returns
// false.  Written out so that a barrier already complete costs few instructions: every
// warp passes two to four of them a block.  kShort: a first try apart from the loop,
// cheaper where barriers are mostly complete.  With key splits that is so (32 rows: 29.8
// against 30.3 us); in the persistent kernel, whose warps wait more, it was slower (16
// heads: 27.5 against 26.6 us).
template <bool kShort>
__device__ __forceinline__ bool wait_local(uint64_t* bar, uint32_t parity, const MlaArgs& a, int site) {
  uint32_t ok;
  if (kShort) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    if (ok) return true;
  }
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
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(a.spin_limit) : "memory");
  if (!ok) set_status(a.status, DSA_ERR_TIMEOUT, site);
  return ok != 0;
}
// The same, agreed on by the warp (its lanes go on or leave together).
template <bool kShort>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const MlaArgs& a, int site) {
  return __all_sync(0xffffffffu, wait_local<kShort>(bar, parity, a, site));
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
  if ((threadIdx.x & 31) == 0)
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(smem_u32(bar) + first) : "memory");
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---------------------------------------------------------------- MMA issue (first CTA)
// One thread for each product: the 36 MMAs of S take an issuing warp, which shares its
// scheduler with six others, about as long as the tensor cores, so a wait for weights
// must not stand before them (148 rows: 85.2 us with two threads, 86.2 with one; the
// issuing loop rolled up, which costs a few more instructions an MMA, took it to 114).
// A byte offset within a tile adds offset >> 4 to a descriptor's address field.
template <int kSplits>
__device__ __forceinline__ void issue_logits(Smem& S, RowStream<kSplits> rows, uint32_t tmem, uint16_t mask) {
  const MlaArgs& a = rows.a;
  constexpr uint32_t idesc = idesc_bf16(kBlk, false);
  const uint64_t qd = sdesc_sw128(smem_u32(S.q), 16, 1024), kd0 = sdesc_sw128(smem_u32(S.k[0]), 16, 1024);
  Row r;
  bool ok = true;
  uint32_t busy = 0;                              // rows with keys so far
  for (int n0 = 0; ok && rows.next_busy(r); n0 += r.nblk, ++busy) {
    ok = wait_local<(kSplits > 1)>(&S.q_full, busy & 1, a, 41);
    for (int j = 0; ok && j < r.nblk; ++j) {
      const int n = n0 + j, b = n & 1;
      // the keys are there, and S of block n-2 has been read: its weights are there
      ok = wait_local<(kSplits > 1)>(&S.p_full[b], ((n >> 1) & 1) ^ 1, a, 43) && wait_local<(kSplits > 1)>(&S.k_full[b], (n >> 1) & 1, a, 42);
      if (!ok) break;
      tc_fence_after();
      const uint64_t kd = kd0 + (uint64_t)(b * (sizeof(S.k[0]) >> 4));
      const uint32_t d = tmem + kColS + b * 32;
#pragma unroll
      for (int ch = 0; ch < kQChunks; ++ch)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_bf16_pair(d, qd + (ch * kHc * 128 + 32 * kk >> 4), kd + (ch * kHalfBlk * 128 + 32 * kk >> 4), idesc, (ch | kk) != 0);
      mma_commit_pair(&S.s_full[b], mask);
      if (kSplits == 1 && j + 1 == r.nblk) mma_commit_pair(&S.q_idle, mask);
      tstamp(a.trace, 0, 2, n);
    }
  }
  mma_commit_own(&S.drained);
}
template <int kSplits>
__device__ __forceinline__ void issue_outputs(Smem& S, RowStream<kSplits> rows, uint32_t tmem, uint16_t mask) {
  const MlaArgs& a = rows.a;
  constexpr uint32_t idesc = idesc_bf16(256, true);
  const uint64_t pd0 = sdesc_sw128(smem_u32(S.p), 16, 1024), vd0 = sdesc_sw128(smem_u32(S.v[0]), kBlk * 128, 1024);
  Row r;
  bool ok = true;
  uint32_t busy = 0;
  for (int n0 = 0; ok && rows.next_busy(r); n0 += r.nblk, ++busy) {
    for (int j = 0; ok && j < r.nblk; ++j) {
      const int n = n0 + j, b = n & 1;
      ok = wait_local<(kSplits > 1)>(&S.v_full[b], (n >> 1) & 1, a, 44) && wait_local<(kSplits > 1)>(&S.p_full[b], (n >> 1) & 1, a, 45);
      // the row before has been read out of the accumulator
      if (j == 0 && busy > 0) ok = ok && wait_local<(kSplits > 1)>(&S.o_free, (busy - 1) & 1, a, 58);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vd = vd0 + (uint64_t)(b * (sizeof(S.v[0]) >> 4)), pd = pd0 + (uint64_t)(b * (sizeof(S.p[0]) >> 4));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mma_bf16_pair(tmem + kColO + h * 128, pd + (32 * kk >> 4), vd + (h * 2 * kBlk * 128 + kk * 16 * 128 >> 4), idesc,
                        (j | kk) != 0);
      mma_commit_pair(&S.pv_done[b], mask);
      tstamp(a.trace, 0, 3, n);
    }
  }
  // the last row's arrivals from the other CTA are in
  if (kSplits == 1 && ok && busy > 0) wait_local<(kSplits > 1)>(&S.o_free, (busy - 1) & 1, a, 58);
  mma_commit_own(&S.drained);
}

// ---------------------------------------------------------------- the selection
// Two warps turn the selection into cache rows, the blocks of parity p each, two keys of
// a block per lane: the positions of a warp's next block are in flight with the
// block-table entries of this one.  (One warp took 2,000 cycles a block, longer where
// the selection came from HBM, and set the pace: a prefill of 2,048 rows 1.33 ms
// instead of 1.14.  What is being loaded is neither copied nor tested before it is
// used, for either would wait for it.)
template <int kSplits>
__device__ __forceinline__ void resolve_rows(Smem& S, RowStream<kSplits> rows, uint32_t rank, int p) {
  const MlaArgs& a = rows.a;
  const CacheMap& m = a.map;
  const int lane = threadIdx.x & 31;
  // The first block's positions, where a full selection has them, go to L1 while the
  // row's length is on its way.
  const int guess = (a.topk + kSplits * kBlk - 1) / (kSplits * kBlk) * kBlk * rows.sp + kBlk * p + lane;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    int32_t unused;
    if (guess + 32 * u < a.topk)
      asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(unused) : "l"(a.idx + (int64_t)(rows.t + rows.step) * a.topk + guess + 32 * u));
  }
  Row r;
  r.nblk = 0;
  int j = 0;
  bool more = rows.next_busy(r);
  const auto advance = [&] {
    if (more && ++j == r.nblk) {
      j = 0;
      more = rows.next_busy(r);
      // the next row's Q comes to L2 some blocks before its tile is free: every pair
      // changes rows at about the same time, and from HBM that took 11,000 cycles
      const int heads = min(kHc, a.n_heads - kHc * (int)rank);
      if (more && heads > 0 && p == 0 && lane == 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                         static_cast<const __nv_bfloat16*>(a.q) + ((int64_t)rows.t * a.n_heads + kHc * (int)rank) * kD),
                     "r"(heads * kD * 2) : "memory");
    }
  };
  int s[2], seq = 0, klen = 0;                    // the next block's positions and row
  bool any = false;
  const auto positions = [&] {
    any = more;
    if (!more) return;
    seq = r.seq;
    klen = r.klen;
    const int32_t* idx = a.idx + (int64_t)rows.t * a.topk + r.k0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = j * kBlk + 32 * u + lane;
      s[u] = -1;
      if (i < r.nvalid) s[u] = __ldg(idx + i);
    }
    advance();
    advance();                                    // the other warp's block
  };
  if (p == 1) advance();
  positions();
  for (int n = p; any; n += 2) {
    int e[2], off[2];
    bool has[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      has[u] = s[u] >= 0 && s[u] < klen;
      off[u] = s[u];
      e[u] = 0;
      if (m.block_table != nullptr) {
        const int pg = m.page_shift >= 0 ? s[u] >> m.page_shift : s[u] / m.page_size;
        off[u] -= pg * m.page_size;
        if (has[u] && pg >= m.max_pages_per_seq) {
          set_status(a.status, DSA_ERR_OUT_OF_RANGE, s[u]);
          has[u] = false;
        }
        if (has[u]) e[u] = __ldg(m.block_table + (int64_t)seq * m.max_pages_per_seq + pg);
      } else if (has[u] && m.seq_start != nullptr) {
        e[u] = __ldg(m.seq_start + seq);
      }
    }
    positions();
    const int slot = n % kRowRing;
    if (!wait_warp<(kSplits > 1)>(&S.rows_free[slot], (n / kRowRing & 1) ^ 1, a, 53)) break;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      int64_t row = (int64_t)e[u] + off[u];
      bool in = row >= 0 && row < m.num_tokens;
      if (m.block_table != nullptr) {
        in = e[u] >= 0 && e[u] < m.num_pages;
        row = (int64_t)e[u] * m.page_size + off[u];
      }
      if (has[u] && !in) set_status(a.status, DSA_ERR_OUT_OF_RANGE, m.block_table != nullptr ? e[u] : off[u]);
      const bool ok = has[u] && in;
      S.rows[slot][32 * u + lane] = ok ? (int)row : -1;
      const uint32_t bits = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) S.valid[n % kValidRing][u] = bits;
    }
    warp_arrive(&S.rows_full[slot]);
  }
}

// ---------------------------------------------------------------- decoding
// The tiles hold dims in an order that suits the decoding: a unit is 64 dims (32 bytes
// of codes, four scales, one chunk of a tile), and its piece e of 8 dims lies at
// position e ^ f(unit) of the chunk, f = unit for the keys' tile, 2 unit for the
// values'.  Q's pieces are placed alike, and the output's columns are put back when
// they are stored, so the permutation costs nothing; it lets lanes that hold different
// units of a key store their e-th pieces, in register order, to distinct banks.
__device__ __forceinline__ int key_piece(int unit, int e) { return e ^ (unit & 7); }
__device__ __forceinline__ int value_piece(int unit, int e) { return e ^ (2 * (unit & 3)); }

struct Unit {
  uint32_t codes[8], scales;

  // Unit `u` of the row (zeros for a key without a row).  One 32-byte load: lanes that
  // share a 128-byte line then take one pass of the L1's data stage (8 a warp; as two
  // 16-byte loads they took 23, and that stage set the pace).
  __device__ __forceinline__ void load(const uint8_t* latent, int row, int u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) codes[i] = 0u;
    scales = 0u;
    if (row >= 0) {
      const uint8_t* src = latent + (int64_t)row * kRow.bytes;
      asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(codes[0]), "=r"(codes[1]), "=r"(codes[2]), "=r"(codes[3]), "=r"(codes[4]), "=r"(codes[5]),
                     "=r"(codes[6]), "=r"(codes[7])
                   : "l"(src + 32 * u));
      scales = __ldg(reinterpret_cast<const uint32_t*>(src + kRow.scale) + u);
    }
  }
  // Decoded to a tile's 128-byte row; `at`: its address with the first piece's swizzled
  // position in bits 4-6, from which piece e's differs by e (the tile's rows and bits
  // are aligned, so that an exclusive or does).
  __device__ __forceinline__ void store(uint32_t at) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const ScalePair s = scale_pair((scales >> (8 * q)) & 0xFFu);
      st_smem_v4(at ^ (32u * q), decode_word(codes[2 * q], s));
      st_smem_v4(at ^ (32u * q + 16u), decode_word(codes[2 * q + 1], s));
    }
  }
};

// The blocks of one parity g: warp w of its eight.  Per block a lane decodes one unit
// of the keys' tile and one of the values'.
//   keys' tile:   keys 4 w.. of the CTA's 32, eight lanes the 8 units of a key
//   values' tile: keys 8 w.., four lanes the CTA's 4 units of a key
// All sixteen warps bring in Q, once S of the row before has read it; heads beyond H
// are zeros.
template <int kSplits>
__device__ __forceinline__ void decode_blocks(Smem& S, RowStream<kSplits> rows, uint32_t rank, uint32_t first, int w, int g) {
  const MlaArgs& a = rows.a;
  const uint8_t* latent = static_cast<const uint8_t*>(a.latent);
  const int lane = threadIdx.x & 31;
  const bool stamp = a.trace != nullptr && w == 0 && lane == 0;
  const int k_key = 4 * w + (lane >> 3), k_unit = lane & 7;
  const int v_key = 8 * w + (lane >> 2), v_unit = lane & 3;
  const uint32_t k_dst = smem_u32(S.k[g][k_unit]) + sw128_off(k_key, key_piece(k_unit, 0));
  const uint32_t v_dst = smem_u32(S.v[g][v_unit]) + sw128_off(v_key, value_piece(v_unit, 0));
  const int kt = w * 32 + lane;                                   // RoPE: 32 keys x 8 pieces, one per thread
  uint8_t* r_dst = S.k[g][8] + sw128_off(kt >> 3, kt & 7);
  const int own = kHalfBlk * (int)rank;                           // the CTA's keys in the block's rows
  Unit ku, vu;
  uint4 rope;
  int v_row = -1;
  const auto load_keys = [&](int n) {
    const int slot = n % kRowRing;
    if (!wait_warp<(kSplits > 1)>(&S.rows_full[slot], n / kRowRing & 1, a, 54)) return false;
    const int k_row = S.rows[slot][own + k_key], r_row = S.rows[slot][own + (kt >> 3)];
    v_row = S.rows[slot][v_key];
    warp_arrive(&S.rows_free[slot]);
    ku.load(latent, k_row, k_unit);
    rope = make_uint4(0u, 0u, 0u, 0u);
    if (r_row >= 0) rope = __ldg(reinterpret_cast<const uint4*>(latent + (int64_t)r_row * kRow.bytes + kRow.rope + 16 * (kt & 7)));
    return true;
  };
  const auto load_values = [&] { vu.load(latent, v_row, 4 * (int)rank + v_unit); };
  const auto load_q = [&](int t) {
    const int th = (g * kDecWarps + w) * 32 + lane, h0 = kHc * (int)rank;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)t * a.n_heads * kD;
#pragma unroll 3
    for (int i = 0; i < kHc * kD / 8 / kDecThreads; ++i) {
      const int qi = th + i * kDecThreads, h = qi / (kD / 8), c = qi - h * (kD / 8);
      const bool in = h0 + h < a.n_heads;
      const int piece = c < kDC / 8 ? key_piece(c >> 3, c & 7) : c & 7;
      cp_async_16_zfill(S.q[c >> 3] + sw128_off(h, piece), q + (int64_t)(in ? h0 + h : 0) * kD + 8 * c, in);
    }
  };
  // blocks known to come, looked up ahead of their use: a load has one place in the
  // loop, for where two would meet the compiler moves what was loaded, and waits
  RowStream<kSplits> ahead = rows;
  int known = 0;
  const auto comes = [&](int n) {
    Row x;
    while (known <= n && ahead.next_busy(x)) known += x.nblk;
    return n < known;
  };
  const auto q_landed = [&] {
    cp_async_wait_all();
    fence_proxy_async_smem();
    warp_arrive_first(&S.q_full, first);
  };
  bool ok = true;
  Row r;
  // the first row's Q, while its selection is resolved (and done with before the first
  // tile's loads, for which the fence would wait)
  if (comes(0)) load_q(ahead.t);
  cluster_wait();                                 // the first CTA's barriers are initialised
  if (known > 0) q_landed();
  if (comes(g)) {
    ok = load_keys(g);
    load_values();
  }
  uint32_t busy = 0;                              // rows with keys so far
  for (int n0 = 0; ok && rows.next_busy(r); n0 += r.nblk, ++busy) {
    bool q_pending = n0 > 0, first_in_row = true;
    int n = n0 + ((n0 ^ g) & 1);
    do {
      const bool mine = n < n0 + r.nblk;
      const uint32_t free = ((n >> 1) & 1) ^ 1;
      if (q_pending) {
        // Q's tile is free once S of the row before's last block has read it.  (A barrier
        // of its own: this group may not have seen the S before on that block's.)
        if (!(ok = wait_warp<(kSplits > 1)>(&S.q_idle, (busy - 1) & 1, a, 59))) break;
        load_q(rows.t);
      }
      if (mine) {
        // the keys' stage is free once S of block n-2 has read it
        if (!(ok = wait_warp<(kSplits > 1)>(&S.s_full[g], free, a, 47))) break;
        if (stamp) tstamp(a.trace, rank, 5, n);
        ku.store(k_dst);
        *reinterpret_cast<uint4*>(r_dst) = rope;
        fence_proxy_async_smem();                 // generic stores -> tensor cores
        warp_arrive_first(&S.k_full[g], first);
        if (stamp) tstamp(a.trace, rank, 0, n);
      }
      // The output of the row before has left the values' stage.  Waited for in every
      // row, and in one without a block of this parity before its Q is handed over: a
      // parity tells two phases apart, not three, and such a row could end without this
      // group.
      const bool idle_wait = first_in_row && busy > 0;
      if (idle_wait && !mine && !(ok = wait_warp<(kSplits > 1)>(&S.v_idle[g], (busy - 1) & 1, a, 60))) break;
      if (q_pending) {
        q_landed();
        q_pending = false;
      }
      const bool more = mine && comes(n + 2);
      if (more && !(ok = load_keys(n + 2))) break;
      if (idle_wait && mine && !(ok = wait_warp<(kSplits > 1)>(&S.v_idle[g], (busy - 1) & 1, a, 60))) break;
      first_in_row = false;
      if (mine) {
        // the values' stage is free once P V of block n-2 has read it
        if (!(ok = wait_warp<(kSplits > 1)>(&S.pv_done[g], free, a, 48))) break;
        if (stamp) tstamp(a.trace, rank, 7, n);
        vu.store(v_dst);
        fence_proxy_async_smem();
        if (!(a.inject & DSA_FAULT_MLA_INT4_VALUES)) warp_arrive_first(&S.v_full[g], first);
        if (stamp) tstamp(a.trace, rank, 1, n);
        if (more) load_values();
      }
      n += 2;
    } while (n < n0 + r.nblk);
  }
  cp_async_wait_all();                            // after a wait that ran out
}

// N columns of this thread's lane of O (zeros when no product was issued).
template <int N>
__device__ __forceinline__ void load_o(uint32_t taddr, bool empty, float (&o)[N]) {
  if (empty) {
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.f;
    return;
  }
  if constexpr (N == 32) tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(&o[0]));
  else tmem_ld16(taddr, *reinterpret_cast<uint32_t(*)[16]>(&o[0]));
  tmem_wait_ld();
}

// Of a row's sum of weights: 0 for no key at all, NaN for a NaN logit or a wait that ran
// out, and 1 or so otherwise (its largest term is 2^-8 at least).
__device__ __forceinline__ float inverse_sum(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ float log_sum(float m, float sum) { return sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2; }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Softmax state of a thread for one row: lane l of tensor memory (head l % 64, keys
// 32 (l / 64).. of a block), blocks of its group's parity.
struct Softmax {
  float m = -INFINITY, sum = 0.f;                 // maximum (log2 domain) that the sum refers to, sum
  bool dead = false;                              // a wait ran out

  // Block j of the row, n = n0 + j of the pair, n % 2 = g.  A thread whose wait ran out (dead) skips its waits
  // and goes on, so that every arrival and collective access stays uniform.
  template <int kSplits>
  __device__ __forceinline__ void block(Smem& S, const MlaArgs& a, uint32_t tmem_lane, int n, int j, int nblk, int g, float c,
                                        uint32_t rank, uint32_t first) {
    const int l = threadIdx.x & 127, half = l >> 6, hl = l & 63;
    const uint32_t phase = (n >> 1) & 1;
    // the weights' tile is free once P V of block n-2 has read it (waited for here, where
    // the group waits for its logits anyway)
    dead = dead || !wait_local<(kSplits > 1)>(&S.pv_done[g], phase ^ 1, a, 51);
    dead = dead || !wait_local<(kSplits > 1)>(&S.s_full[g], phase, a, 49);
    tc_fence_after();
    if (l == 0 && a.trace != nullptr) tstamp(a.trace, rank, 4, n);
    float s[32];
    tmem_ld32(tmem_lane + kColS + g * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
    tmem_wait_ld();
    // masked keys are -inf (a full block needs no test)
    const uint32_t mask = S.valid[n % kValidRing][half];
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
        dead = dead || !wait_local<(kSplits > 1)>(&S.pv_done[g ^ 1], ((n - 1) >> 1) & 1, a, 50);
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
    if (l == 0 && a.trace != nullptr) tstamp(a.trace, rank, 6, n);
  }
};

// N columns (from `col`, of a lane's 256) of head hl, scaled and rounded, into the
// 128-byte row of its staged tile, the values' permutation undone.
template <int N>
__device__ __forceinline__ void stage_bf16(uint8_t* tile, int hl, int col, const float (&o)[N], float scale) {
#pragma unroll
  for (int q = 0; q < N / 8; ++q)
    *reinterpret_cast<uint4*>(tile + sw128_off(hl, value_piece(col >> 6, (col >> 3 & 7) + q))) = pack8(&o[8 * q], scale);
}
// A staged tile to dims [x, x + 64) of heads [y, y + 64) of row t (heads beyond H are
// dropped by the tensor map's bounds).
__device__ __forceinline__ void store_tile(const CUtensorMap* map, const uint8_t* tile, int x, int y, int t) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)), "r"(smem_u32(tile)), "r"(x), "r"(y), "r"(t) : "memory");
}

// S: key splits of a row = pairs of a cluster.
template <int kSplits>
__global__ void __launch_bounds__(kThreads, 1) mla_int4_tc_kernel(const __grid_constant__ MlaArgs a,
                                                                 const __grid_constant__ CUtensorMap out_map) {
  extern __shared__ __align__(1024) uint8_t smraw[];
  Smem& S = *reinterpret_cast<Smem*>(smraw);
  const int warp = threadIdx.x >> 5;
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, first = crank & ~1u;
  const int sp = (int)(crank >> 1);
  const uint32_t to_first = mapa(smraw, first) - smem_u32(smraw);
  const int heads = max(0, min(kHc, a.n_heads - kHc * (int)rank));  // of this CTA
  pdl_launch_dependents();

  if (threadIdx.x == 0) {
    mbar_init(&S.q_full, 2 * 2 * kDecWarps);
    mbar_init(&S.o_free, 2 * kSmWarps);
    mbar_init(&S.drained, 2);
    mbar_init(&S.q_idle, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], 2 * kDecWarps);
      mbar_init(&S.v_full[i], 2 * kDecWarps);
      mbar_init(&S.p_full[i], kSmWarps);         // a group's four warps in each CTA
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.pv_done[i], 1);
      mbar_init(&S.v_idle[i], 1);
    }
    for (int i = 0; i < kRowRing; ++i) {
      mbar_init(&S.rows_full[i], 1);
      mbar_init(&S.rows_free[i], kDecWarps);
    }
    mbar_init(&S.merged, 1);
    fence_mbar_init();
    if (kSplits > 1) mbar_expect_tx(&S.merged, (kSplits - 1) * (Merge<kSplits>::kCols * 8 * heads + Merge<kSplits>::kMl));
  }
  __syncwarp();
  if (warp == kMmaWarp) tmem_alloc_pair(&S.tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();                     // waited for before anything touches another CTA
  const uint32_t tmem = S.tmem_base;
  pdl_wait();
  trace_kernel(a.status, kSplits > 1 ? DSA_KERNEL_MLA_INT4_TC | DSA_KERNEL_MLA_COMBINE : DSA_KERNEL_MLA_INT4_TC);
  // with splits one row per cluster, else the pair's share of the rows
  RowStream<kSplits> rows(a, blockIdx.x / (2 * kSplits), kSplits > 1 ? a.num_rows : (int)gridDim.x / 2, sp);
  using Mg = Merge<kSplits>;

  if (warp == kMmaWarp || warp == kMmaWarp2) {
    cluster_wait();
    if (rank == 0 && elect_one()) {
      if (warp == kMmaWarp) issue_logits<kSplits>(S, rows, tmem, (uint16_t)(3u << first));
      else issue_outputs<kSplits>(S, rows, tmem, (uint16_t)(3u << first));
    }
    __syncwarp();
    // Every product issued is done before the pair's shared and tensor memory go, even if
    // all others have left because waits ran out: waited for (with the built-in limit)
    // before the cluster's last barrier.  Without splits that is this one; with them the
    // merge may begin, and the last one follows it.
    if (kSplits > 1) cluster_arrive();
    if (rank == 0) mbar_wait(&S.drained, 0, a.status, 46);
    __syncwarp();
    if (kSplits == 1) cluster_arrive();
  } else if (warp >= kRowWarp) {
    resolve_rows<kSplits>(S, rows, rank, warp - kRowWarp);
    cluster_wait();
    cluster_arrive();
  } else if (warp >= kDecWarp0) {
    const int w = warp - kDecWarp0;
    decode_blocks<kSplits>(S, rows, rank, to_first, w % kDecWarps, w / kDecWarps);
    cluster_arrive();
  } else {
    cluster_wait();
    const float c = a.sm_scale * kLog2e;
    const uint32_t tmem_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int l = threadIdx.x & 127, g = warp >> 2, half = l >> 6, hl = l & 63, head = kHc * (int)rank + hl;
    Softmax sm;
    Row r;
    bool settled = true;                          // no wait ran out in either group
    for (int n0 = 0; rows.next(r); n0 += r.nblk) {
      const int t_out = rows.t, last = (n0 + r.nblk - 1) & 1;
      const bool empty = r.nblk == 0;
      if (r.nsel == 0 && r.klen > 0 && threadIdx.x == 0) set_status(a.status, DSA_ERR_OUT_OF_RANGE, t_out);
      sm.m = -INFINITY;
      sm.sum = 0.f;
      for (int j = (n0 ^ g) & 1; j < r.nblk; j += 2) sm.block<kSplits>(S, a, tmem_lane, n0 + j, j, r.nblk, g, c, rank, to_first);
      if (kSplits > 1) cluster_arrive();
      // the last block's group waits for its product (to the other group's threads the
      // barrier may still be two phases back); all meet at the barrier below
      if (!empty && last == g) sm.dead = sm.dead || !wait_local<(kSplits > 1)>(&S.pv_done[last], ((n0 + r.nblk - 1) >> 1) & 1, a, 52);
      // the row's output: the head's maximum, its sum over four threads, then this
      // thread's half of the lane's columns
      const bool bad = named_bar_or(1, kSmThreads, sm.dead);
      settled = settled && !bad;
      tc_fence_after();
      const float M = empty ? -INFINITY : S.m_run[last][hl];
      // (a maximum of -inf goes with a sum of 0, or NaN from a NaN logit, which stays; a row
      // without a key depends on no wait)
      S.red[g][l] = bad && !empty ? __int_as_float(0x7FC00000) : sm.m == -INFINITY ? sm.sum : sm.sum * exp2f(sm.m - M);
      if (kSplits > 1) break;
      named_bar_sync(1, kSmThreads);
      const float L = (S.red[0][hl] + S.red[1][hl]) + (S.red[0][hl + 64] + S.red[1][hl + 64]);
      named_bar_sync(1, kSmThreads);              // read before the next row's maxima go there
      const float inv = inverse_sum(L);
      if (empty) {
        // the values' tiles may hold a later row's already: zeros go out directly
        uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t)t_out * a.n_heads * kDC);
        const int from = kHc * (int)rank * (kDC / 8), to = min(a.n_heads, kHc * ((int)rank + 1)) * (kDC / 8);
        for (int i = from + (int)threadIdx.x; i < to; i += kSmThreads) out[i] = make_uint4(0u, 0u, 0u, 0u);
      } else {
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          const int col = 128 * g + 32 * cc;
          float o[32];
          load_o(tmem_lane + kColO + col, bad, o);
          stage_bf16(smraw + Mg::kOut + (4 * half + (col >> 6)) * 8192, hl, col, o, inv);
        }
        tc_fence_before();
        warp_arrive_first(&S.o_free, to_first);
        fence_proxy_async_smem();
        named_bar_sync(1, kSmThreads);
        // the group that does not begin the next row sends the tiles out, those in the
        // stage of the next block first
        const int next = (n0 + r.nblk) & 1;
        if (g != next && l == 0) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int tile = (4 * next) ^ i;
            if (kHc * (int)rank < a.n_heads)
              store_tile(&out_map, smraw + Mg::kOut + tile * 8192, 64 * tile, kHc * (int)rank, t_out);
            if ((i & 3) == 3) bulk_commit();
          }
          bulk_wait_read<1>();
          mbar_arrive(&S.v_idle[next]);
          bulk_wait_read0();
          mbar_arrive(&S.v_idle[next ^ 1]);
        }
        __syncwarp();
      }
      if (a.lse && half == 0 && g == 0 && head < a.n_heads)
        a.lse[(int64_t)t_out * a.n_heads + head] = log_sum(M, L);
    }
    if (kSplits == 1) {
      // A release would wait for the output's stores as well (1,500 cycles).  There is no
      // need of one when what this warp sent to the other CTA has led to the products and
      // the end of the issue, o_free, that were waited for.
      bulk_wait_read0();                          // what this thread's copies read may go
      tc_fence_before();
      __syncwarp();
      if (settled) cluster_arrive_relaxed();
      else cluster_arrive();
    }
  }

  // With key splits the pairs of the cluster exchange what they hold, all of a CTA's
  // warps taking part (four read a column of tensor memory, so in groups of four).
  if constexpr (kSplits > 1) {
    constexpr int kCols = Mg::kCols, kItems = (kSplits - 1) * kCols / 32;
    static_assert(kItems <= kDecWarp0 / 4 + 2 * kDecWarps / 4, "a group sends 32 columns at most");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // A CTA's threads arrived when its last S was done, or with its last weights: Q's and
    // the keys' tiles, where the parts arrive, are free then, and the barrier is complete
    // by the time that the last product is.  Parts are sent from where the values lay.
    cluster_wait();
    if (warp < kMmaWarp) {
      const int l = threadIdx.x & 127, grp = warp >> 2, half = l >> 6, hl = l & 63;
      const uint32_t o_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kColO;
      const Row r = row_of<kSplits>(a, rows.klen_next, rows.seq_next, sp);
      const int t = blockIdx.x / (2 * kSplits);
      const bool none = r.nblk == 0;
      float M = none ? -INFINITY : S.m_run[(r.nblk - 1) & 1][hl];
      float L = (S.red[0][hl] + S.red[1][hl]) + (S.red[0][hl + 64] + S.red[1][hl + 64]);
      // a column group's 16 bytes of every lane that travels; this lane's place there
      const uint32_t lanes16 = 32u * heads, lane16 = 16u * (half * heads + hl);
      if (grp < kItems) {
        const int dst = grp * 32 / kCols, to = dst < sp ? dst : dst + 1, in_slot = sp < to ? sp : sp - 1;
        const int col = grp * 32 % kCols;
        float o[32];
        load_o(o_lane + to * kCols + col, none, o);
        uint8_t* src = smraw + kSend + grp * (size_t)(32 * 512);
        if (hl < heads) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(src + i * lanes16 + lane16) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        if (grp == 0 && half == 0) reinterpret_cast<float2*>(smraw + kSendMl)[hl] = make_float2(M, L);
        fence_proxy_async_smem();
        named_bar_sync(2 + grp, 128);
        if (l == 0 && heads > 0)
          bulk_copy_to_peer(smraw + in_slot * (size_t)Mg::kPart + (col / 4) * lanes16, src, 8 * lanes16, &S.merged,
                            (uint32_t)(2 * to) + rank);
        if (grp == 0 && l < kSplits && l != sp)
          bulk_copy_to_peer(smraw + kRecvMl + sp * (size_t)Mg::kMl, smraw + kSendMl, Mg::kMl, &S.merged,
                            (uint32_t)(2 * l) + rank);
      }
      if (grp < 4) {
        constexpr int kMine = kCols / 4;            // columns of this thread: 32 or 16
        const int col = kMine * grp;                // within the pair's columns
        float own[kMine];
        load_o(o_lane + sp * kCols + col, none, own);
        const bool got = wait_local<(kSplits > 1)>(&S.merged, 0, a, 57);
        // out = sum_s w_s O_s / sum_s w_s l_s,  w_s = 2^(m_s - max m), splits in order
        float w[kSplits];
        float2 v[kSplits];
        const float2 mine = make_float2(M, L);
        M = -INFINITY;
        L = 0.f;
#pragma unroll
        for (int s2 = 0; s2 < kSplits; ++s2) {
          v[s2] = s2 == sp ? mine : reinterpret_cast<const float2*>(smraw + kRecvMl + s2 * (size_t)Mg::kMl)[hl];
          M = fmaxf(M, v[s2].x);
        }
#pragma unroll
        for (int s2 = 0; s2 < kSplits; ++s2) {
          w[s2] = v[s2].x == -INFINITY ? 0.f : exp2f(v[s2].x - M);
          L += w[s2] * v[s2].y;                     // NaN stays
        }
        if (named_bar_or(1, 4 * 128, !got)) L = __int_as_float(0x7FC00000);
        const float inv = inverse_sum(L);
        const int head = kHc * (int)rank + hl;
        float acc[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) acc[i] = 0.f;
#pragma unroll
        for (int s2 = 0; s2 < kSplits; ++s2) {
          float o[kMine];
          if (s2 == sp) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) o[i] = own[i];
          } else {
            const uint8_t* src = smraw + (s2 < sp ? s2 : s2 - 1) * (size_t)Mg::kPart + (col / 4) * lanes16 + (hl < heads ? lane16 : 0u);
#pragma unroll
            for (int i = 0; i < kMine / 4; ++i) {
              const float4 x = *reinterpret_cast<const float4*>(src + i * lanes16);
              o[4 * i] = x.x, o[4 * i + 1] = x.y, o[4 * i + 2] = x.z, o[4 * i + 3] = x.w;
            }
          }
#pragma unroll
          for (int i = 0; i < kMine; ++i) acc[i] = fmaf(w[s2], o[i], acc[i]);
        }
        stage_bf16(smraw + Mg::kOut + (Mg::kTiles / 2 * half + (col >> 6)) * 8192, hl, sp * kCols + col, acc, inv);
        fence_proxy_async_smem();
        named_bar_sync(1, 4 * 128);
        if (threadIdx.x < Mg::kTiles && kHc * (int)rank < a.n_heads) {
          const int i = threadIdx.x, in_half = i % (Mg::kTiles / 2), x = 256 * (i / (Mg::kTiles / 2)) + sp * kCols + 64 * in_half;
          store_tile(&out_map, smraw + Mg::kOut + i * 8192, x, kHc * (int)rank, t);
          bulk_commit();
        }
        if (a.lse && sp == 0 && grp == 0 && half == 0 && head < a.n_heads)
          a.lse[(int64_t)t * a.n_heads + head] = log_sum(M, L);
      }
    }
    // what the CTAs sent one another has been received, or was released at the barrier before
    bulk_wait_read0();
    tc_fence_before();
    __syncwarp();
    cluster_arrive_relaxed();
  }
  // nothing of the cluster is still to be accessed behind this barrier
  cluster_wait();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

using Kernel = void (*)(MlaArgs, CUtensorMap);
template <int kSplits>
constexpr Kernel kernel_of = mla_int4_tc_kernel<kSplits>;

// out [T, H, d_c] bf16, stored as tiles of 64 heads x 64 dims.
bool make_out_map(CUtensorMap* m, const MlaArgs& a) {
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!fn) return false;
  const cuuint64_t dim[3] = {(cuuint64_t)kDC, (cuuint64_t)a.n_heads, (cuuint64_t)a.num_rows};
  const cuuint64_t stride[2] = {kDC * 2, (cuuint64_t)a.n_heads * kDC * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)kHc, 1}, step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.out, dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaLaunchConfig_t launch_config(cudaLaunchAttribute (&at)[2], int splits, int clusters) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * splits * 2));
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

// Clusters of `splits` pairs that can be resident at once on this device, negative if the
// query fails.  Kept per device; a context with a part of the SMs then gets the number of
// the context that asked first, which is a matter of speed only.
int resident_clusters(Kernel kernel, int splits) {
  static OnceAsked kept[kMaxPairs + 1][kMaxDevices];
  const auto ask = [&] {
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = launch_config(at, splits, 1);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) return n;
    (void)cudaGetLastError();
    return -1;
  };
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  return dev < kMaxDevices ? kept[splits][dev].get(ask) : ask();
}

}  // namespace

bool mla_int4_tc_supported(const MlaArgs& a) {
  return a.mla_dtype == DSA_INT4 && a.n_heads <= 2 * kHc && a.d_c == kDC && a.d_r == kDR && a.topk <= kMaxKeys;
}

dsa_status launch_mla_int4_tc(const MlaArgs& a, cudaStream_t stream) {
  if (a.num_rows == 0) return DSA_OK;
  CUtensorMap out_map;
  if (!make_out_map(&out_map, a)) {
    set_error("mla_int4_tc: cuTensorMapEncodeTiled failed");
    return DSA_ERR_CUDA;
  }
  static std::atomic<bool> attr1[kMaxDevices] = {}, attr2[kMaxDevices] = {}, attr4[kMaxDevices] = {};
  dsa_status st;
  if ((st = set_smem_limit_once(reinterpret_cast<const void*>(kernel_of<1>), sizeof(Smem), attr1)) ||
      (st = set_smem_limit_once(reinterpret_cast<const void*>(kernel_of<2>), sizeof(Smem), attr2)) ||
      (st = set_smem_limit_once(reinterpret_cast<const void*>(kernel_of<4>), sizeof(Smem), attr4)))
    return st;
  const auto kernel_for = [](int splits) { return splits == 4 ? kernel_of<4> : splits == 2 ? kernel_of<2> : kernel_of<1>; };
  const Int4Shape shape = int4_shape(a.num_rows, a.topk, kBlk, device_sm_count(),
                                     [&](int splits) { return resident_clusters(kernel_for(splits), splits); });
  Kernel kernel = kernel_for(shape.splits);
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = launch_config(at, shape.splits, shape.clusters);
  cfg.stream = stream;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  MlaArgs la = a;
  la.spin_limit = fault_spin_limit(kWaitPolls);
  la.inject = fault_inject();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, la, out_map);
  if (e != cudaSuccess) {
    set_error("mla_int4_tc launch: %s", cudaGetErrorString(e));
    return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

}  // namespace dsa
