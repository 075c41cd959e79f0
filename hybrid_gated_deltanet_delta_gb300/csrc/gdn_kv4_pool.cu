// The page pool of the 4-bit key/value cache: truncate or free rows, branch
// rows onto the same pages, and grow rows with copy-on-write of a shared last
// page (include/gdn.h).  The pool's only state is the number of holders of each
// page, so freeing is an atomic decrement and a row's new pages are the
// lowest-numbered ones with no holder: the result does not depend on the order
// in which threads run.
#include "gdn_common.cuh"
#include "gdn_kv4.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ bool row_ok(const gdn_kv4_pool& p, int row) {
  return row >= 0 && row < p.n_rows && p.kv_len[row] >= 0 &&
         (int64_t)p.kv_len[row] <= (int64_t)p.max_pages * p.page_tokens;
}

__device__ __forceinline__ int pages_of(const gdn_kv4_pool& p, int tokens) {
  return tokens / p.page_tokens + (tokens % p.page_tokens != 0);
}

__device__ __forceinline__ bool page_ok(const gdn_kv4_pool& p, int page) {
  return page >= 0 && page < p.n_pages;
}

// One block per row.
__global__ void __launch_bounds__(kThreads)
release_kernel(gdn_kv4_pool p, const int32_t* rows, const int32_t* keep_len) {
  pdl_enter();
  const int row = rows[blockIdx.x], keep = keep_len[blockIdx.x];
  if (!row_ok(p, row) || keep < 0) {
    if (threadIdx.x == 0) report(p.status, GDN_ERR_ROW_RANGE);
    return;
  }
  const int len = p.kv_len[row];
  if (keep >= len) return;
  int32_t* t = p.table + (int64_t)row * p.table_stride;
  // all of the pages that are given up are looked at before any is
  bool bad = false;
  for (int j = pages_of(p, keep) + threadIdx.x; j < pages_of(p, len); j += kThreads)
    bad |= !page_ok(p, t[j]);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) report(p.status, GDN_ERR_PAGE_RANGE);
    return;
  }
  for (int j = pages_of(p, keep) + threadIdx.x; j < pages_of(p, len); j += kThreads) {
    atomicSub(p.ref + t[j], 1);
    t[j] = -1;
  }
  __syncthreads();
  if (threadIdx.x == 0) p.kv_len[row] = keep;
}

// One block per branch.  Source rows are only read (a dst row is never one).
__global__ void __launch_bounds__(kThreads)
fork_kernel(gdn_kv4_pool p, const int32_t* src, const int32_t* dst) {
  pdl_enter();
  const int from = src[blockIdx.x], to = dst[blockIdx.x];
  // the first entries are read beside the lengths, not after them
  int ahead = -1;
  if (from >= 0 && from < p.n_rows && (int)threadIdx.x < p.max_pages)
    ahead = p.table[(int64_t)from * p.table_stride + threadIdx.x];
  if (!row_ok(p, from) || !row_ok(p, to) || p.kv_len[to] != 0) {
    if (threadIdx.x == 0) report(p.status, GDN_ERR_ROW_RANGE);
    return;
  }
  const int32_t* s = p.table + (int64_t)from * p.table_stride;
  int32_t* d = p.table + (int64_t)to * p.table_stride;
  const int len = p.kv_len[from], held = pages_of(p, len);
  // a row is branched whole or not at all: its pages are looked at before any is counted
  bool bad = false;
  for (int j = threadIdx.x; j < held; j += kThreads)
    bad |= !page_ok(p, j < kThreads ? ahead : s[j]);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) report(p.status, GDN_ERR_PAGE_RANGE);
    return;
  }
  for (int j = threadIdx.x; j < p.max_pages; j += kThreads) {
    const int page = j >= held ? -1 : j < kThreads ? ahead : s[j];
    if (j < held) atomicAdd(p.ref + page, 1);
    d[j] = page;
  }
  __syncthreads();
  if (threadIdx.x == 0) p.kv_len[to] = len;
}

// ---------------------------------------------------------------- reserve
constexpr int kPlan = 512;

// What the copy kernel does for a row: nothing when `records` is 0.  While the plan
// is made: -1 for a row that is not served, and the row's first rank among the free
// pages in `start`.
struct Copy {
  int from, to, records, start;
};

// Inclusive sums over the block (kPlan threads); `total` is the block's.
__device__ __forceinline__ int block_scan(int x, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sum[w] = x;
  __syncthreads();
  int s = lane < kPlan / 32 ? warp_sum[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
  return x + (w > 0 ? before : 0);
}

struct Need {
  bool ok, copy;
  int err;                                  // why not ok
  int row, old_len, new_len, lowest, want;  // entries lowest .. want-1 are new
  int from;                                 // the shared last page, to be copied
};

__device__ __forceinline__ Need need_of(const gdn_kv4_pool& p, const int32_t* rows,
                                        const int32_t* new_len, int f) {
  Need n = {};
  n.err = GDN_ERR_ROW_RANGE;
  n.row = rows[f];
  n.new_len = new_len[f];
  n.ok = row_ok(p, n.row) && (int64_t)n.new_len <= (int64_t)p.max_pages * p.page_tokens;
  if (!n.ok) return n;
  n.old_len = p.kv_len[n.row];
  n.ok = n.new_len >= n.old_len;
  if (!n.ok) return n;
  n.lowest = pages_of(p, n.old_len);
  n.want = pages_of(p, n.new_len);
  if (n.old_len % p.page_tokens != 0 && n.new_len > n.old_len) {
    const int tail = p.table[(int64_t)n.row * p.table_stride + n.lowest - 1];
    if (!page_ok(p, tail)) {
      n.ok = false;
      n.err = GDN_ERR_PAGE_RANGE;
    } else if (p.ref[tail] > 1) {
      n.copy = true;
      n.from = tail;
      --n.lowest;
    }
  }
  return n;
}

// Which of the kScan pages from `at` on have no holder, by bits.
constexpr int kScan = 8;

struct Counts {
  int4 x[2];
};

__device__ __forceinline__ Counts load_counts(const gdn_kv4_pool& p, int at) {
  Counts c;
  const bool vec = (reinterpret_cast<uintptr_t>(p.ref) & 15u) == 0;
#pragma unroll
  for (int i = 0; i < 2; ++i, at += 4) {
    c.x[i] = make_int4(1, 1, 1, 1);
    if (vec && at + 4 <= p.n_pages) {
      c.x[i] = *reinterpret_cast<const int4*>(p.ref + at);
    } else if (at < p.n_pages) {
      c.x[i].x = p.ref[at];
      if (at + 1 < p.n_pages) c.x[i].y = p.ref[at + 1];
      if (at + 2 < p.n_pages) c.x[i].z = p.ref[at + 2];
      if (at + 3 < p.n_pages) c.x[i].w = p.ref[at + 3];
    }
  }
  return c;
}

__device__ __forceinline__ unsigned free_bits(const Counts& c) {
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    m |= ((c.x[i].x == 0) | (c.x[i].y == 0) << 1 | (c.x[i].z == 0) << 2 | (c.x[i].w == 0) << 3)
         << (4 * i);
  return m;
}

struct PlanRow {
  int start, row, lowest, served;
};

// One block: the rows' needs in order, the number of free pages, which rows
// are served, and then the pages themselves.  Bound by latency: the rows' chain of
// dependent reads (row, length, tail page, its holders) runs under the read of the
// counts, 8 consecutive pages a thread, so that a pool of 4096 pages takes one read
// and one scan; the free pages then go to shared memory by rank and a thread serves
// one rank, with what it needs of the row in shared memory as well.  One sequence
// branched four ways (four kernels: release, fork, this one and the copy): 12.3 us with a
// page a thread and the rows' plan in global memory, 13.6 us with each thread handing
// out its own eight pages, 10.9 us this way; 32 sequences 37.2, 41.0 and 36.0 us.  (Now
// 11.3 to 12.1 us over boxes and 36.6 us: release and fork look at all pages first, 0.2 us.)
__global__ void __launch_bounds__(kPlan, 1)
plan_kernel(gdn_kv4_pool p, const int32_t* rows, const int32_t* new_len, int F, Copy* plan,
            int32_t* granted) {
  __shared__ int warp_sum[32];
  __shared__ PlanRow kept[kPlan];              // of the first kPlan rows
  __shared__ uint16_t by_rank[kPlan * kScan];  // free pages of a chunk
  pdl_enter();
  const int tid = threadIdx.x;
  constexpr int kChunk = kPlan * kScan;
  Counts counts = load_counts(p, tid * kScan);
  // needs, by the counts before the call; the first kPlan rows stay in registers and
  // shared memory (row tid: `own`), the others in the plan
  auto look = [&](int f) {
    const Need n = need_of(p, rows, new_len, f);
    if (!n.ok) report(p.status, n.err);
    return n;
  };
  auto records = [&](const Need& n) {
    return !n.ok ? -1 : n.copy ? (n.old_len % p.page_tokens + kv4::kRec - 1) / kv4::kRec : 0;
  };
  int asked = 0, have = 0, total;
  Need own = {};
  for (int f0 = 0; f0 < F; f0 += kPlan) {
    const int f = f0 + tid;
    Need n = {};
    if (f < F) n = look(f);
    const int mine = n.ok ? n.want - n.lowest : 0;
    const int at = asked + block_scan(mine, warp_sum, total) - mine;
    if (f0 == 0) {
      own = n;
      kept[tid] = {at, n.row, n.lowest, n.ok};
    } else if (f < F) {
      plan[f] = {n.from, -1, records(n), at};
    }
    asked += total;
  }
  auto start = [&](int f) { return f < kPlan ? kept[f].start : plan[f].start; };
  // this thread's free pages and their first rank, of the last chunk of pages
  unsigned mine = 0;
  int rank = 0;
  for (int i0 = 0; i0 < p.n_pages; i0 += kChunk) {
    if (i0 > 0) counts = load_counts(p, i0 + tid * kScan);
    mine = free_bits(counts);
    rank = block_scan(__popc(mine), warp_sum, total) - __popc(mine);
    have += total;
  }
  // rows that do not fit: they and all later ones that need pages
  __syncthreads();
  for (int f = tid; f < F; f += kPlan) {
    if (f < kPlan ? !own.ok : plan[f].records < 0) continue;
    const int end = f + 1 < F ? start(f + 1) : asked;
    if (end > start(f) && end > have) {
      if (f < kPlan) own.ok = false, kept[f].served = 0;
      else plan[f].records = -1;
      report(p.status, GDN_ERR_POOL_EMPTY);
    }
  }
  // hand out the free pages by rank
  int rank0 = 0;
  for (int i0 = 0; i0 < p.n_pages && rank0 < asked; i0 += kChunk) {
    total = have;
    if (p.n_pages > kChunk) {
      mine = free_bits(load_counts(p, i0 + tid * kScan));
      rank = block_scan(__popc(mine), warp_sum, total) - __popc(mine);
    }
    for (; mine != 0; mine &= mine - 1) by_rank[rank++] = (uint16_t)(tid * kScan + __ffs(mine) - 1);
    __syncthreads();
    for (int k = tid; k < total && rank0 + k < asked; k += kPlan) {
      int lo = 0, hi = F - 1;  // the last row whose first rank is <= this one
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start(mid) <= rank0 + k) lo = mid;
        else hi = mid - 1;
      }
      PlanRow r;
      if (lo < kPlan) {
        r = kept[lo];
      } else {
        const int row = rows[lo], recs = plan[lo].records;
        r = {plan[lo].start, row, pages_of(p, p.kv_len[row]) - (recs > 0), recs >= 0};
      }
      if (r.served) {
        const int i = i0 + by_rank[k];
        p.table[(int64_t)r.row * p.table_stride + r.lowest + rank0 + k - r.start] = i;
        if (rank0 + k == r.start) plan[lo].to = i;  // of use when there is a tail to copy
        p.ref[i] = 1;
      }
    }
    rank0 += total;
    __syncthreads();
  }
  // (a row that was not served gets a length that every later call skips)
  auto grant = [&](int f, int n) {
    if (granted != nullptr) granted[f] = n;
  };
  for (int f = tid; f < F; f += kPlan) {
    if (f < kPlan) {
      const int recs = records(own);
      plan[f].from = own.from;
      plan[f].records = recs < 0 ? 0 : recs;
      if (recs > 0) atomicSub(p.ref + own.from, 1);
      if (recs >= 0) p.kv_len[own.row] = own.new_len;
      grant(f, recs >= 0 ? own.new_len : -1);
      continue;
    }
    if (plan[f].records < 0) {
      plan[f].records = 0;
      grant(f, -1);
      continue;
    }
    if (plan[f].records > 0) atomicSub(p.ref + plan[f].from, 1);
    p.kv_len[rows[f]] = new_len[f];
    grant(f, new_len[f]);
  }
}

// Grid (pieces, F, layers): the records of a page that hold tokens, head by head.
// Bound by HBM: each thread has four 16-byte loads in flight (32 sequences branched
// four ways copy 73 MB to 73 MB, most of 36.6 us with the three kernels before it).
__global__ void __launch_bounds__(kThreads)
copy_kernel(const Copy* plan, uint8_t* pages, int64_t page_stride, int64_t layer_stride, int Hkv,
            int recs, int rec_bytes) {
  constexpr int U = 4;
  pdl_enter();
  const Copy c = plan[blockIdx.y];
  if (c.records == 0) return;
  const int per_head = c.records * rec_bytes / 16, skip = (recs - c.records) * rec_bytes / 16;
  uint8_t* layer = pages + blockIdx.z * layer_stride;
  const uint4* from = reinterpret_cast<const uint4*>(layer + c.from * page_stride);
  uint4* to = reinterpret_cast<uint4*>(layer + c.to * page_stride);
  const int total = per_head * Hkv;
  for (int i0 = blockIdx.x * kThreads * U + threadIdx.x; i0 < total;
       i0 += gridDim.x * kThreads * U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i < total) x[u] = __ldcs(from + i + (int64_t)(i / per_head) * skip);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads;
      if (i < total) to[i + (int64_t)(i / per_head) * skip] = x[u];
    }
  }
}

}  // namespace

int launch_kv4_release(const gdn_kv4_pool& p, const int32_t* rows, const int32_t* keep, int F,
                       cudaStream_t s) {
  return launch_pdl(release_kernel, dim3(F), dim3(kThreads), 0, s, p, rows, keep);
}

int launch_kv4_fork(const gdn_kv4_pool& p, const int32_t* src, const int32_t* dst, int F,
                    cudaStream_t s) {
  return launch_pdl(fork_kernel, dim3(F), dim3(kThreads), 0, s, p, src, dst);
}

size_t kv4_reserve_workspace_bytes(int F) { return (size_t)F * sizeof(Copy); }

int launch_kv4_reserve(const gdn_kv4_pool& p, void* pages, int64_t page_stride,
                       int64_t layer_stride, int n_layers, int Hkv, int D, const int32_t* rows,
                       const int32_t* new_len, int F, int32_t* granted, void* workspace,
                       cudaStream_t s) {
  Copy* plan = static_cast<Copy*>(workspace);
  const int rc =
      launch_pdl(plan_kernel, dim3(1), dim3(kPlan), 0, s, p, rows, new_len, F, plan, granted);
  if (rc != GDN_OK) return rc;
  return launch_pdl(copy_kernel, dim3(8, F, n_layers), dim3(kThreads), 0, s, (const Copy*)plan,
                    static_cast<uint8_t*>(pages), page_stride, layer_stride, Hkv,
                    p.page_tokens / kv4::kRec, kv4::rec_bytes(D));
}

}  // namespace gdn
