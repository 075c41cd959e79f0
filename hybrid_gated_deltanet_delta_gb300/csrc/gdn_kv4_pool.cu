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
  for (int j = pages_of(p, keep) + threadIdx.x; j < pages_of(p, len); j += kThreads) {
    const int page = t[j];
    if (page_ok(p, page)) atomicSub(p.ref + page, 1);
    else report(p.status, GDN_ERR_PAGE_RANGE);
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
  if (!row_ok(p, from) || !row_ok(p, to) || p.kv_len[to] != 0) {
    if (threadIdx.x == 0) report(p.status, GDN_ERR_ROW_RANGE);
    return;
  }
  const int32_t* s = p.table + (int64_t)from * p.table_stride;
  int32_t* d = p.table + (int64_t)to * p.table_stride;
  const int len = p.kv_len[from], held = pages_of(p, len);
  for (int j = threadIdx.x; j < p.max_pages; j += kThreads) {
    const int page = j < held ? s[j] : -1;
    if (j < held) {
      if (page_ok(p, page)) atomicAdd(p.ref + page, 1);
      else report(p.status, GDN_ERR_PAGE_RANGE);
    }
    d[j] = page;
  }
  __syncthreads();
  if (threadIdx.x == 0) p.kv_len[to] = len;
}

// ---------------------------------------------------------------- reserve
constexpr int kPlan = 1024;

// What the copy kernel does for a row: nothing when `records` is 0.
struct Copy {
  int from, to, records, start;  // start: the row's first rank among the free pages (plan only)
};

// Inclusive sums over the block (1024 threads); `total` is the block's.
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
  int s = warp_sum[lane];
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
  int row, old_len, new_len, lowest, want;  // entries lowest .. want-1 are new
};

__device__ __forceinline__ Need need_of(const gdn_kv4_pool& p, const int32_t* rows,
                                        const int32_t* new_len, int f) {
  Need n = {};
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
    } else if (p.ref[tail] > 1) {
      n.copy = true;
      --n.lowest;
    }
  }
  return n;
}

// One block: the rows' needs in order, the number of free pages, which rows
// are served, and then the pages themselves.
__global__ void __launch_bounds__(kPlan)
plan_kernel(gdn_kv4_pool p, const int32_t* rows, const int32_t* new_len, int F, Copy* plan) {
  __shared__ int warp_sum[32];
  pdl_enter();
  const int tid = threadIdx.x;
  int asked = 0, have = 0, total;
  // needs, by the counts before the call
  for (int f0 = 0; f0 < F; f0 += kPlan) {
    const int f = f0 + tid;
    Need n = {};
    if (f < F) {
      n = need_of(p, rows, new_len, f);
      if (!n.ok) report(p.status, GDN_ERR_ROW_RANGE);
    }
    const int mine = n.ok ? n.want - n.lowest : 0;
    const int upto = block_scan(mine, warp_sum, total);
    if (f < F) {
      Copy c = {-1, -1, 0, asked + upto - mine};
      if (n.copy) {
        c.from = p.table[(int64_t)n.row * p.table_stride + n.lowest];
        c.records = (n.old_len % p.page_tokens + kv4::kRec - 1) / kv4::kRec;
      }
      if (!n.ok) c.to = -2;  // not served
      plan[f] = c;
    }
    asked += total;
  }
  for (int i0 = 0; i0 < p.n_pages; i0 += kPlan) {
    const int i = i0 + tid;
    have += __syncthreads_count(i < p.n_pages && p.ref[i] == 0);
  }
  // rows that do not fit: they and all later ones that need pages
  for (int f = tid; f < F; f += kPlan) {
    if (plan[f].to == -2) continue;
    const int end = f + 1 < F ? plan[f + 1].start : asked;
    if (end > plan[f].start && end > have) {
      plan[f].to = -2;
      report(p.status, GDN_ERR_POOL_EMPTY);
    }
  }
  __syncthreads();
  // hand out the free pages by rank
  int rank0 = 0;
  for (int i0 = 0; i0 < p.n_pages && rank0 < asked; i0 += kPlan) {
    const int i = i0 + tid;
    const int is_free = i < p.n_pages && p.ref[i] == 0;
    const int rank = rank0 + block_scan(is_free, warp_sum, total) - 1;
    if (is_free && rank < asked) {
      int lo = 0, hi = F - 1;  // the last row whose first rank is <= rank
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (plan[mid].start <= rank) lo = mid;
        else hi = mid - 1;
      }
      const Copy c = plan[lo];
      if (c.to != -2) {
        const int row = rows[lo];
        const int lowest = pages_of(p, p.kv_len[row]) - (c.records > 0);
        p.table[(int64_t)row * p.table_stride + lowest + rank - c.start] = i;
        if (c.records > 0 && rank == c.start) plan[lo].to = i;
        p.ref[i] = 1;
      }
    }
    rank0 += total;
  }
  __syncthreads();
  for (int f = tid; f < F; f += kPlan) {
    if (plan[f].to == -2) {
      plan[f].records = 0;
      continue;
    }
    if (plan[f].records > 0) atomicSub(p.ref + plan[f].from, 1);
    p.kv_len[rows[f]] = new_len[f];
  }
}

// Grid (pieces, F, layers): the records of a page that hold tokens, head by head.
// Bound by HBM: each thread has four 16-byte loads in flight.
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
                       const int32_t* new_len, int F, void* workspace, cudaStream_t s) {
  Copy* plan = static_cast<Copy*>(workspace);
  const int rc = launch_pdl(plan_kernel, dim3(1), dim3(kPlan), 0, s, p, rows, new_len, F, plan);
  if (rc != GDN_OK || n_layers == 0) return rc;
  return launch_pdl(copy_kernel, dim3(8, F, n_layers), dim3(kThreads), 0, s, (const Copy*)plan,
                    static_cast<uint8_t*>(pages), page_stride, layer_stride, Hkv,
                    p.page_tokens / kv4::kRec, kv4::rec_bytes(D));
}

}  // namespace gdn
