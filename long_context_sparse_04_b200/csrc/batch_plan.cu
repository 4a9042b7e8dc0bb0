// batch_plan.cu - the block table, slot map and row map of one step from the
// requests' lengths, with the pages popped from and pushed back on a free list
// ("Sparse Attention in Large Language Models: Architecture Evolution and
// Engineering Practice", section 4, item "Memory Management and KV Cache
// Optimization": paged caches).  The rule is stated at dsa_batch_plan in
// include/dsa.h.
//
// Everything follows from five prefix sums over the requests: pages handed back and
// pages and rows asked for (the admission) in one scan, pages and rows granted in
// another.  Every CTA computes them for itself, keeps the three that the rest needs in
// shared memory, and writes its share of the rows, table entries and pages; a binary
// search in shared memory gives a row's request.  CTAs are launched by what the host
// knows: for the rows (a chunked prefill of 131,072 takes 128), and for the pages that a
// step may hand back (redoing the sums costs them nothing: one CTA after another would
// wait for them all the same, and a cluster, which could share them, is 8 CTAs).  200
// requests of up to 128K tokens in pages of 16 that hand back 239,770 take 24 us with 16
// CTAs and runs of eight pages a thread, 150 with one CTA, 519 without the runs as well;
// where nothing is handed back the further CTAs cost 0.2 to 0.4 us.  What bounds a
// decoding batch is latency: the launch, two loads in a chain, the scans' barriers, the
// arrival of the CTAs; thousands of requests are bound by what every CTA does for them
// (half of the time of 4,096).
// Lengths and the free count, which may be updated in place, are written by the CTA
// that finishes last, when every CTA has read them; free-list entries read (below the
// old count) and written (at or above it) never meet, nor do table entries read (pages
// held) and written.
#include <climits>
#include <type_traits>

#include "dsa_kernels.cuh"

namespace dsa {
namespace {

// Threads per CTA: few for a decoding batch, whose two scans are a chain of barriers (256
// requests: 6.5 us a plan with 256 threads, 7.8 with 1,024 and three scans; 4,096
// requests and 131,072 rows: 18.0).
constexpr int kFew = 256, kMany = 1024;
constexpr int kFewCtas = 16;           // at most, for the pages that may be handed back
constexpr int kMaxSeqs = 16384;        // three int32 prefix arrays in shared memory

// One request as the rule sees it.
struct Request {
  int64_t len, add;       // tokens cached, tokens asked for
  int32_t held, need;     // pages held, pages asked for (0 when it cannot run)
  int32_t give;           // pages handed back
  int err;                // 0, DSA_ERR_INVALID_ARG or DSA_ERR_OUT_OF_RANGE
  bool rel;
  // tokens of the request's candidate rows (0 when it cannot run)
  __device__ int64_t rows() const { return err == 0 && !rel ? add : 0; }
};

// ceil(tokens / page) for 0 <= tokens < 2^31 (32-bit: a 64-bit division costs ~5x)
__device__ __forceinline__ int32_t pages_of(int64_t tokens, int32_t page) {
  return (int32_t)(((uint32_t)tokens + (uint32_t)page - 1u) / (uint32_t)page);
}

// What the caller says of a request.
struct Lengths {
  int32_t len, add, rel;
};
__device__ __forceinline__ Lengths load_lengths(const PlanArgs& a, int b) {
  return Lengths{a.p.seq_len[b], a.p.n_new[b], a.p.release != nullptr ? a.p.release[b] : 0};
}

// `end`: of a contiguous cache, the row behind the last that the request may use.
template <bool kPaged>
__device__ __forceinline__ Request request_of(const PlanArgs& a, int b, const Lengths& x, int64_t end) {
  Request r;
  r.len = x.len;
  r.add = x.add;
  r.rel = x.rel != 0;
  r.held = r.need = r.give = 0;
  r.err = 0;
  const int64_t width = kPaged ? (int64_t)a.max_pages_per_seq * a.page_size
                                      : end - (a.seq_start ? a.seq_start[b] : 0);
  if (r.len < 0 || r.add < 0 || (r.rel && r.add != 0) || (kPaged && r.len > width)) {
    r.err = DSA_ERR_INVALID_ARG;
  } else if (!r.rel && r.add > 0 &&
             (r.len + r.add > width || r.len + r.add > INT_MAX || (!kPaged && a.seq_start && a.seq_start[b] < 0))) {
    r.err = DSA_ERR_OUT_OF_RANGE;
  }
  if (r.err != DSA_ERR_INVALID_ARG && kPaged) {
    r.held = pages_of(r.len, a.page_size);
    if (r.rel) r.give = r.held;
    else if (r.err == 0) r.need = pages_of(r.len + r.add, a.page_size) - r.held;
  }
  return r;
}

// Rows of a contiguous cache: a request's end where the next larger start of any request
// begins.  keys: 2 * start + (1 if the request holds or asks for tokens), ascending, in
// the shared memory of the page sums, which such a cache has no use for.
template <int kThreads>
__device__ __forceinline__ void sort_starts(const PlanArgs& a, uint32_t* keys, int n) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    uint32_t key = UINT_MAX;                      // behind the last request
    if (i < a.num_seqs) {
      const int32_t start = a.seq_start ? a.seq_start[i] : 0;
      key = start < 0 ? 0u : 2u * (uint32_t)start + (a.p.seq_len[i] > 0 || a.p.n_new[i] > 0 ? 1u : 0u);
    }
    keys[i] = key;
  }
  __syncthreads();
  bool falls = false;
  for (int i = threadIdx.x; i + 1 < n; i += kThreads) falls = falls || keys[i] > keys[i + 1];
  if (!__syncthreads_or(falls)) return;           // laid out in order, as a rule
  for (int size = 2; size <= n; size <<= 1) {     // bitonic
    for (int d = size >> 1; d > 0; d >>= 1) {
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const int j = i ^ d;
        const uint32_t x = keys[i], y = keys[j];  // (only the thread of the lower one writes)
        if (j > i && (x > y) == ((i & size) == 0)) {
          keys[i] = y;
          keys[j] = x;
        }
      }
      __syncthreads();
    }
  }
}
// The row behind the last of a request that begins at `start` and asks for tokens; none
// where another request that holds or asks for tokens begins there too.
__device__ __forceinline__ int64_t rows_end(const PlanArgs& a, const uint32_t* keys, int n, int32_t start) {
  if (start < 0) return 0;
  const uint32_t key = 2u * (uint32_t)start + 1u;
  int lo = 0, hi = n;                             // the first key above it
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (keys[mid] <= key) lo = mid + 1; else hi = mid;
  }
  if (lo > 1 && keys[lo - 2] == key) return 0;
  const int64_t next = lo < n ? (int64_t)(keys[lo] >> 1) : a.num_tokens;
  return next < a.num_tokens ? next : a.num_tokens;
}

// Exclusive prefixes of N values over the block's threads, and their totals.
template <int kThreads, int N>
__device__ __forceinline__ void block_scan(int64_t (&x)[N], int64_t (&total)[N], int64_t (*part)[kThreads / 32]) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t own[N];
#pragma unroll
  for (int k = 0; k < N; ++k) own[k] = x[k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int64_t u = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] += u;
    }
  }
  if (lane == 31) {
#pragma unroll
    for (int k = 0; k < N; ++k) part[k][warp] = x[k];
  }
  __syncthreads();
  if (kWarps > 8) {                             // warp k scans the warps' sums of value k
    if (warp < N) {
      int64_t u = lane < kWarps ? part[warp][lane] : 0;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, u, o);
        if (lane >= o) u += v;
      }
      if (lane < kWarps) part[warp][lane] = u;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      x[k] += (warp > 0 ? part[k][warp - 1] : 0) - own[k];
      total[k] = part[k][kWarps - 1];
    }
  } else {                                      // every warp adds them up
#pragma unroll
    for (int k = 0; k < N; ++k) {
      int64_t before = 0, all = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const int64_t p = part[k][i];
        before += i < warp ? p : 0;
        all += p;
      }
      x[k] += before - own[k];
      total[k] = all;
    }
  }
}

// Largest b of [0, n) with start[b] <= i, for start[0] = 0 <= i < start[n]: the
// owner of item i (empty requests share their successor's start).
__device__ __forceinline__ int owner(const int32_t* start, int n, int32_t i) {
  int lo = 0, hi = n;                       // start[lo] <= i < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// What the CTAs share in the workspace's status block, zero between calls: CTAs that
// are done, and INT_MAX - (8 * request + error) of the lowest request in error.
struct PlanShared {
  unsigned int done;
  int worst;
};
static_assert(sizeof(PlanShared) <= sizeof(DeviceStatus::pad), "status block");

// kPaged: a block table, else a contiguous cache (apart, for what it needs in the loop over
// the requests took the plan of 4,096 paged ones from 19.1 to 20.5 us).
template <int kThreads, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1) batch_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t part[5][kThreads / 32];  // of the first scan, of the second
  __shared__ int s_worst, s_refused, s_last;
  const int B = a.num_seqs, tid = threadIdx.x;
  int32_t* tok_start = sm;                  // rows granted before request b, [B + 1]
  int32_t* pg_start = sm + (B + 1);         // pages granted
  int32_t* give_start = sm + 2 * (B + 1);   // pages handed back
  PlanShared* shared = reinterpret_cast<PlanShared*>(a.status->pad);
  pdl_launch_dependents();
  trace_kernel(a.status, DSA_KERNEL_BATCH_PLAN);
  if (tid == 0) { s_worst = 0; s_refused = 0; }

  int64_t F = 0;
  bool bad_count = false;
  if (kPaged) {
    F = *a.p.free_count;
    bad_count = F < 0 || F > a.p.free_capacity;
    if (bad_count) F = 0;
  }
  __syncthreads();

  // thread i owns the requests [i * per, i * per + per); the three arrays first hold
  // what each request asks for or hands back
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  int64_t asked[3] = {0, 0, 0}, asked_all[3];  // pages handed back, pages and rows asked for
  int refused = 0;
  uint32_t* keys = reinterpret_cast<uint32_t*>(pg_start);   // of a contiguous cache; n_keys < 2 (B + 1)
  const int n_keys = kPaged || B == 1 ? 1 : 1 << (32 - __clz(B - 1));
  if (!kPaged) sort_starts<kThreads>(a, keys, n_keys);
  constexpr int kBatch = 4;                 // loads of as many requests at a time
  for (int bb = b0; bb < b1; bb += kBatch) {
    Lengths x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (bb + i < b1) x[i] = load_lengths(a, bb + i);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int b = bb + i;
      if (b >= b1) break;
      const int64_t end = kPaged || x[i].add <= 0 ? a.num_tokens : rows_end(a, keys, n_keys, a.seq_start ? a.seq_start[b] : 0);
      const Request r = request_of<kPaged>(a, b, x[i], end);
      tok_start[b] = (int32_t)r.rows();
      if (kPaged) {
        pg_start[b] = r.need;
        give_start[b] = r.give;
      }
      asked[0] += r.give;
      asked[1] += r.need;
      asked[2] += r.rows();
      if (r.err) {
        atomicMax(&s_worst, INT_MAX - (b * 8 + r.err));
        ++refused;
      }
    }
  }
  block_scan<kThreads>(asked, asked_all, part);
  const int64_t gives = asked_all[0], have = F + gives;
  // the admission: inclusive sums of pages and rows over every request that could run
  int64_t give = asked[0], need = asked[1], rows = asked[2], granted[2] = {0, 0}, granted_all[2];
  for (int b = b0; b < b1; ++b) {
    const int32_t n = tok_start[b], p = kPaged ? pg_start[b] : 0, g = kPaged ? give_start[b] : 0;
    need += p;
    rows += n;
    const bool go = (p == 0 || need <= have) && (n == 0 || rows <= a.p.max_tokens);
    if (!go) {
      tok_start[b] = 0;
      ++refused;
    }
    if (!go || !kPaged) pg_start[b] = 0;
    granted[0] += go ? n : 0;
    granted[1] += go ? p : 0;
    give_start[b] = (int32_t)give;
    give += g;
  }
  if (refused) atomicAdd(&s_refused, refused);
  block_scan<kThreads>(granted, granted_all, part + 3);
  const int64_t total = granted_all[0], taken = granted_all[1];
  for (int b = b0; b < b1; ++b) {
    const int32_t n = tok_start[b], p = pg_start[b];
    tok_start[b] = (int32_t)granted[0];
    pg_start[b] = (int32_t)granted[1];
    granted[0] += n;
    granted[1] += p;
  }
  if (tid == 0) {
    tok_start[B] = (int32_t)total;
    pg_start[B] = (int32_t)taken;
    give_start[B] = (int32_t)gives;
  }
  __syncthreads();

  // The stack of free pages: the list, then the pages handed back.
  const int64_t W = a.max_pages_per_seq;
  const auto handed_back = [&](int32_t i) {
    const int b = owner(give_start, B, i);
    return a.block_table[(int64_t)b * W + (i - give_start[b])];
  };
  // The k-th page taken, -1 when its id lies outside the cache.
  const auto taken_page = [&](int32_t k) {
    const int64_t i = have - 1 - k;
    const int32_t pg = i < F ? a.p.free_pages[i] : handed_back((int32_t)(i - F));
    return pg >= 0 && pg < a.num_pages ? pg : -1;
  };
  const int gid = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
  const int32_t n_rows = (int32_t)total;
  const int last = n_rows > 0 ? owner(tok_start, B, n_rows - 1) : 0;
  for (int64_t t64 = gid; t64 < a.p.max_tokens; t64 += step) {
    const int32_t t = (int32_t)t64;
    int b = last;
    int32_t pos = -1;
    int64_t slot = -1;
    if (t < n_rows) {
      b = owner(tok_start, B, t);
      const int32_t len = a.p.seq_len[b];
      pos = len + (t - tok_start[b]);
      if (kPaged) {
        const int32_t pg = pos / a.page_size, held = pages_of(len, a.page_size);
        int32_t page = pg >= held ? taken_page(pg_start[b] + pg - held) : a.block_table[(int64_t)b * W + pg];
        if (page < 0 || page >= a.num_pages) {
          atomicMax(&s_worst, INT_MAX - (b * 8 + DSA_ERR_OUT_OF_RANGE));
          page = -1;
        }
        if (page >= 0) slot = (int64_t)page * a.page_size + (pos - pg * a.page_size);
      } else {
        slot = (int64_t)(a.seq_start ? a.seq_start[b] : 0) + pos;
      }
    }
    a.p.row_seq[t] = b;
    a.p.row_klen[t] = pos + 1;
    a.p.tok_pos[t] = pos;
    a.p.slot[t] = slot;
  }
  for (int64_t k64 = gid; k64 < taken; k64 += step) {
    const int32_t k = (int32_t)k64;
    const int b = owner(pg_start, B, k);
    const int32_t held = pages_of(a.p.seq_len[b], a.page_size);
    a.block_table[(int64_t)b * W + held + (k - pg_start[b])] = taken_page(k);
  }
  const int64_t left = min(have - taken, (int64_t)a.p.free_capacity);
  // Pages handed back, in runs of kRun * 32 a warp: one search where a run is one request's,
  // and all its loads in flight before its first store.
  const int64_t back = left - F;
  const auto hand_back = [&](auto run) {
    constexpr int kRun = decltype(run)::value;
    for (int64_t i0 = (int64_t)(gid >> 5) * (32 * kRun); i0 < back; i0 += (int64_t)step * kRun) {
      const int b0 = owner(give_start, B, (int32_t)i0), end = give_start[b0 + 1];
      int32_t page[kRun];
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        const int64_t i = i0 + 32 * u + (tid & 31);
        const int b = i < end ? b0 : owner(give_start, B, (int32_t)min(i, back - 1));
        if (i < back) page[u] = a.block_table[(int64_t)b * W + (i - give_start[b])];
      }
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        const int64_t i = i0 + 32 * u + (tid & 31);
        if (i < back) a.p.free_pages[F + i] = page[u];
      }
    }
  };
  if (back <= step) hand_back(std::integral_constant<int, 1>());
  else hand_back(std::integral_constant<int, 8>());
  for (int b = gid; b <= B; b += step) a.p.tok_start[b] = tok_start[b];

  // the CTA that is done last has the rest: every CTA has read the lengths and the free
  // count, and said what it found wrong
  __syncthreads();
  if (tid == 0) {
    if (s_worst) atomicMax(&shared->worst, s_worst);
    __threadfence();
    s_last = gridDim.x == 1 || atomicAdd(&shared->done, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  for (int b = tid; b < B; b += kThreads) {
    const Request r = request_of<kPaged>(a, b, load_lengths(a, b), a.num_tokens);   // (a refused one has no rows)
    const int32_t n = tok_start[b + 1] - tok_start[b];
    a.p.seq_len_out[b] = r.rel && r.err == 0 ? 0 : (int32_t)(r.len + n);
  }
  if (tid == 0) {
    const int worst = *reinterpret_cast<volatile int*>(&shared->worst);
    if (worst) set_status(a.status, (INT_MAX - worst) & 7, (INT_MAX - worst) >> 3);
    shared->worst = 0;
    shared->done = 0;
    if (bad_count || (kPaged && have - taken > left)) set_status(a.status, DSA_ERR_INVALID_ARG, -1);
    if (kPaged) *a.p.free_count_out = (int32_t)left;
    a.p.totals[0] = n_rows;
    a.p.totals[1] = (int32_t)taken;
    a.p.totals[2] = s_refused;
    a.p.totals[3] = (int32_t)gives;
  }
}

}  // namespace

int batch_plan_max_seqs() { return kMaxSeqs; }

// CTAs for n items, `each` a CTA: one at least, `most` at most.
static int ctas_for(int64_t n, int each, int most) {
  const int64_t want = (n + each - 1) / each;
  return want < 1 ? 1 : want < most ? (int)want : most;
}

template <bool kPaged>
static dsa_status launch(const PlanArgs& a, cudaStream_t stream) {
  const size_t smem_max = (size_t)3 * (kMaxSeqs + 1) * sizeof(int32_t);
  static std::atomic<bool> attr[kMaxDevices] = {};
  if (dsa_status st = set_smem_limit_once(reinterpret_cast<const void*>(batch_plan_kernel<kMany, kPaged>), smem_max, attr))
    return st;
  const size_t smem = (size_t)3 * (a.num_seqs + 1) * sizeof(int32_t);
  // The pages that a step may hand back are as many as the tables or the cache hold: known
  // here only as that bound, so CTAs are launched for them that mostly find nothing to do.
  const int64_t table = (int64_t)a.num_seqs * a.max_pages_per_seq;
  const int64_t back = !kPaged || a.p.release == nullptr ? 0 : table < a.num_pages ? table : a.num_pages;
  if (a.num_seqs <= 2 * kFew && a.p.max_tokens <= 8 * kFew) {
    batch_plan_kernel<kFew, kPaged><<<ctas_for(back, 16 * kFew, kFewCtas), kFew, smem, stream>>>(a);
  } else {
    const int most = device_sm_count(), rows = ctas_for(a.p.max_tokens, kMany, most), pages = ctas_for(back, 8 * kMany, most);
    batch_plan_kernel<kMany, kPaged><<<rows > pages ? rows : pages, kMany, smem, stream>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("batch plan launch failed: %s", cudaGetErrorString(e));
    return DSA_ERR_CUDA;
  }
  return DSA_OK;
}

dsa_status launch_batch_plan(const PlanArgs& a, cudaStream_t stream) {
  return a.block_table != nullptr ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace dsa
