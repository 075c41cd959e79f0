// Attention over the 4-bit cache for sequences that share pages: the plan before, and the join
// after, the pass of gdn_kv4_attn.cuh (kShared) over what groups share and sequences have alone.
//
//   o = (2^(m_p - m) O_p + 2^(m_o - m) O_o) / (2^(m_p - m) l_p + 2^(m_o - m) l_o)
//
// with O, l and the reference m of the shared and of the own part, each in turn the sum of the
// parts that blocks left of it; m is the largest of them.
#include "gdn_common.cuh"
#include "gdn_kv4.cuh"
#include "gdn_kv4_attn.h"
#include "gdn_launch.h"

namespace gdn {
namespace {

using namespace kv4;

constexpr int kTile = 128;
constexpr float kNone = -3.402823466e38f;

// ---------------------------------------------------------------- plan
// A cluster of blocks a group, a share of its sequences each.  The group's first sequence with a
// whole tile before its block is the one whose table row the shared pages are taken from; the
// others share with it what lies on the same pages of both, in whole tiles.  What all of those
// share that share a tile at all is the group's prefix.  Bound by the latency of the groups and
// of the rows' entries after them: the first lengths are read beside the groups, and the least
// prefix is put where each block of the cluster reads it, so that one barrier is waited for (32
// branches 62.0 us in all before, here 60.9).
constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32, kPlanBlocks = 8;
constexpr int kKept = 512;  // sequences of a share whose numbers stay in shared memory

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t x;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(x));
  return x;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t x;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(x));
  return x;
}

// Every thread of the cluster; what was written before the one is seen after the other.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// The lesser of x and a word of shared memory of block `rank` of the cluster, there.
__device__ __forceinline__ void cluster_min(int* p, uint32_t rank, int x) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(gdn_kv4_cache c, int N, const int32_t* __restrict__ parent,
            const int32_t* __restrict__ group, int n_groups, SharedPlan plan) {
  __shared__ int ref, shortest, least;
  __shared__ int differ[kPlanWarps];  // first entry of a sequence's row that is another page
  __shared__ int kept[kKept];
  __shared__ int lens[kPlanThreads];  // of the first sequences, read before the groups are known
  int32_t* start = plan.extra + n_groups;  // -1 for a sequence that is skipped
  const int blocks = cluster_size(), rank = cluster_rank(), g = blockIdx.x / blocks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) ref = c.B, shortest = least = 0x7fffffff;
  __syncwarp();  // the barrier is one instruction of whole warps
  if (blocks > 1) cluster_arrive();  // waited for before the first write to another block
  pdl_enter();
  const int early = tid < c.B ? c.kv_len[tid] : 0;
  bool ok = true;
  for (int i = tid; i <= n_groups; i += kPlanThreads) {
    const int x = group[i];
    ok = ok && x >= 0 && x <= c.B && (i == n_groups || x <= group[i + 1]);
  }
  const int lo = group[g], hi = group[g + 1];
  lens[tid] = early;
  ok = __syncthreads_and(ok);
  auto length = [&](int b, bool report_it) {  // as seq_len
    return check_len(c, b < kPlanThreads ? lens[b] : c.kv_len[b], report_it);
  };
  if (!ok && g == 0 && rank == 0 && tid == 0) report(c.status, GDN_ERR_ROW_RANGE);
  const int first = ok ? lo : 0, end = ok ? hi : 0;
  // tokens before a sequence's block, -1 for one that is skipped; by a warp, which writes down
  // the sequence's numbers
  auto before = [&](int b) {
    int len = length(b, lane == 0);
    if (len > 0 && parent != nullptr) {
      const int32_t* p = parent + (int64_t)b * N;
      bool good = true;
      for (int n = lane; n < N; n += 32) {
        const int up = p[n];
        good = good && (n == 0 ? up == -1 : up >= 0 && up < n);
      }
      if (!__all_sync(0xffffffffu, good)) {
        if (lane == 0) report(c.status, GDN_ERR_BAD_TREE);
        len = 0;
      }
    }
    if (lane == 0) plan.len[n_groups + b] = len, plan.first[n_groups + b] = b | (uint32_t)b << 16;
    return len > 0 ? max(len - N, 0) : -1;
  };
  if (g == 0) {  // sequences of no group
    const int from = ok ? group[0] : c.B, to = ok ? group[n_groups] : c.B;
    for (int i = rank * kPlanWarps + warp; i < from + c.B - to; i += blocks * kPlanWarps) {
      const int b = i < from ? i : to + i - from, x = before(b);
      if (lane == 0) start[b] = x < 0 ? -1 : 0;
    }
  }
  // the first sequence with a tile (whether or not its tree is one: its pages serve as well)
  for (int b = first + tid; b < end; b += kPlanThreads)
    if (length(b, false) - N >= kTile) atomicMin(&ref, b);
  // this block's sequences are first + rank, first + rank + blocks, ..
  const int mine = end - first > rank ? (end - first - rank + blocks - 1) / blocks : 0;
  auto seq = [&](int i) { return first + rank + i * blocks; };
  // of sequence seq(i): tokens before its block, then tiles shared (kept, or in its place)
  auto held = [&](int i) -> int& { return mine <= kKept ? kept[i] : start[seq(i)]; };
  for (int i = warp; i < mine; i += kPlanWarps) {
    const int x = before(seq(i));
    if (lane == 0) held(i) = x < kTile ? min(x, 0) : x;
  }
  __syncthreads();
  const int r = ref, most = r < end ? length(r, false) - N : 0;
  const int32_t* row = c.table + (int64_t)(r < end ? r : 0) * c.table_stride;
  // up to kPlanWarps sequences at once, the warps spread over them
  for (int i0 = 0; i0 < mine; i0 += kPlanWarps) {
    const int count = min(mine - i0, kPlanWarps), each = kPlanWarps / count;
    if (tid < kPlanWarps) differ[tid] = 0x7fffffff;
    __syncthreads();
    const int m = warp / each, turn = warp % each, b = seq(i0 + m);
    if (m < count && b != r) {
      const int common = min(held(i0 + m), most);
      const int pages = common <= 0 ? 0 : (common + c.page_tokens - 1) / c.page_tokens;
      const int32_t* other = c.table + (int64_t)b * c.table_stride;
      constexpr int U = 8;
      for (int j0 = turn * 32 * U; j0 < pages; j0 += each * 32 * U) {
        int x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * 32 + lane;
          x[u] = j < pages ? other[j] ^ row[j] : 0;
        }
        int at = 0x7fffffff;
#pragma unroll
        for (int u = U - 1; u >= 0; --u)
          if (x[u] != 0) at = j0 + u * 32 + lane;
        at = __reduce_min_sync(0xffffffffu, at);
        if (at != 0x7fffffff) {
          if (lane == 0) atomicMin(&differ[m], at);
          break;
        }
      }
    }
    __syncthreads();
    if (tid < count) {
      int& x = held(i0 + tid);
      const int64_t same = (int64_t)differ[tid] * c.page_tokens;
      if (x > 0) {
        x = (int)min((int64_t)min(x, most), same) / kTile;
        if (x > 0 && seq(i0 + tid) != r) atomicMin(&shortest, x);
      }
    }
    __syncthreads();
  }
  // over the group's blocks
  int all = shortest;
  if (blocks > 1) {
    cluster_wait();
    if (tid < blocks) cluster_min(&least, tid, shortest);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    all = least;
  }
  const int tiles = all == 0x7fffffff ? 0 : all;  // (nobody shares with the first)
  for (int i = tid; i < mine; i += kPlanThreads) {
    const int x = held(i);
    start[seq(i)] = x > 0 ? tiles : x;
  }
  if (tid == 0 && rank == 0) {
    plan.len[g] = tiles * kTile;
    plan.extra[g] = end - first;
    plan.first[g] = first | (uint32_t)(r < end ? r : first) << 16;
  }
}

// ---------------------------------------------------------------- join
// A thread has four channels of one row; with few rows (ONE_ROW) the block's threads share one
// row and take every NP-th part each, else each D/4 of them take a row.  The parts are the own
// ones, in block order, and then the shared ones.  Bound by latency: the numbers of the plan and of
// the row, then the parts; 6 us after the pass for 8,192 rows of 128 channels.  With eight parts
// in flight 9.5 us, with two 6; one row a block up to 8 rows an SM (32 branches: 62.0 us in all,
// up to 2 rows 66.6; 8 x 8 chains, always one row a block, 115.7 against 92.8; branches of 4,096
// tokens, 24/4 heads of 256, one row a block / several: 16 of them 27.6 / 32.2, 32 33.3 / 35.3, 44
// 38.4 / 39.2, 56 (past the bound of 1,216 rows) 44.1 / 44.1, 64 46.9 / 46.3, 96 59.0 / 56.6; 32/8 of
// 128: 38 42.4 / 43.0, 44 44.7 / 44.4).
constexpr int kJoinThreads = 256;

template <int D, bool ONE_ROW>
__global__ void __launch_bounds__(kJoinThreads)
shared_join_kernel(const __grid_constant__ AttnArgs a, int NT, int blocks) {
  constexpr int Q = D / 4, NP = kJoinThreads / Q, STEP = ONE_ROW ? NP : 1;
  __shared__ __align__(16) float acc[ONE_ROW ? NP : 1][D];
  __shared__ float2 sums[NP];
  pdl_enter();
  const int quad = threadIdx.x % Q, lot = threadIdx.x / Q;
  const int row = ONE_ROW ? blockIdx.x : blockIdx.x * NP + lot;  // (31 bits hold them)
  if (row >= a.c.B * a.N * a.Hq) return;  // ONE_ROW: none
  const RowPart part[2] = {a.row_part[0][row], a.row_part[1][row]};  // (of a pass before, maybe)
  const int node = a.by_Hq(row), b = a.by_N(node), n = node - b * a.N, head = row - node * a.Hq;
  const int from = a.plan_extra[a.n_groups + b];
  const bool there = from >= 0 && a.plan_len[a.n_groups + b] - a.N + n >= 0;
  // first block, parts and row of the own (0) and the shared side (1); (a pass whose waits ran
  // out may have left no numbers here, so they are kept in range)
  int first[2], at[2], count[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    first[i] = min(part[i].blocks & 0xffff, blocks - 1);
    at[i] = min(max(part[i].row, 0), NT - 1);
    count[i] = min(max((part[i].blocks >> 16 & 0xffff) - first[i], 0), blocks - 1 - first[i]) + 1;
    if (!there || (i == 1 && from == 0)) count[i] = 0;
  }
  const int parts = count[0] + count[1];
  float top = kNone, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto larger = [](float p, float q) { return q > p || q != q ? q : p; };  // NaN stays
  constexpr int U = ONE_ROW ? 4 : 2;
#pragma unroll 1
  for (int i0 = ONE_ROW ? lot : 0; i0 < parts; i0 += U * STEP) {
    float2 ml[U];
    float4 p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * STEP;
      ml[u] = make_float2(kNone, 0.f);
      p[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < parts) {
        const bool shared = i >= count[0];
        const int k = shared ? i - count[0] : i;
        if (k == 0) {
          ml[u] = shared ? make_float2(part[1].m, part[1].l) : make_float2(part[0].m, part[0].l);
          p[u] = __ldcg(reinterpret_cast<const float4*>(a.row_o[shared] + (int64_t)row * D) + quad);
        } else {
          const int64_t slot = (int64_t)((shared ? first[1] : first[0]) + k) * NT +
                               (shared ? at[1] : at[0]);
          ml[u] = __ldcg(a.part_ml + slot);
          p[u] = __ldcg(reinterpret_cast<const float4*>(a.part_o + slot * D) + quad);
        }
      }
    }
    float m = top;
#pragma unroll
    for (int u = 0; u < U; ++u) m = larger(m, ml[u].x);
    const float keep = exp2f(top - m);
    top = m;
    sum *= keep;
    o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = exp2f(ml[u].x - m);
      sum += w * ml[u].y;
      o.x += w * p[u].x, o.y += w * p[u].y, o.z += w * p[u].z, o.w += w * p[u].w;
    }
  }
  if constexpr (ONE_ROW) {
    *reinterpret_cast<float4*>(&acc[lot][quad * 4]) = o;
    if (quad == 0) sums[lot] = make_float2(top, sum);
    __syncthreads();
    if (lot != 0) return;
#pragma unroll
    for (int k = 0; k < NP; ++k) top = larger(top, sums[k].x);
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const float4 p = *reinterpret_cast<const float4*>(&acc[k][quad * 4]);
      const float w = exp2f(sums[k].x - top);
      o.x += w * p.x, o.y += w * p.y, o.z += w * p.z, o.w += w * p.w;
      sum += w * sums[k].y;
    }
  }
  const float inv =
      sum != 0.f ? (a.c.v_scale != nullptr ? a.c.v_scale[a.by_G(head)] : 1.f) / sum : 0.f;
  const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = a.bf16 ? Elem<GDN_BF16>::from(v[i]) : Elem<GDN_F16>::from(v[i]);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + (int64_t)row * D + quad * 4) =
      make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
  if (a.lse != nullptr && quad == 0)
    a.lse[row] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

template <int D>
int join_d(const AttnArgs& a, int NT, int blocks, cudaStream_t s) {
  const int64_t rows = (int64_t)a.c.B * a.N * a.Hq;
  constexpr int NP = kJoinThreads / (D / 4);
  if (rows <= 8 * blocks)
    return launch_pdl(shared_join_kernel<D, true>, dim3((unsigned)rows), dim3(kJoinThreads), 0, s,
                      a, NT, blocks);
  return launch_pdl(shared_join_kernel<D, false>, dim3((unsigned)((rows + NP - 1) / NP)),
                    dim3(kJoinThreads), 0, s, a, NT, blocks);
}

}  // namespace

int launch_kv4_shared_plan(const gdn_kv4_cache& c, int N, const int32_t* parent,
                           const int32_t* group, int n_groups, const SharedPlan& plan,
                           cudaStream_t s) {
  // Several blocks where the usual group has many sequences.  One block / eight, us of the whole
  // call, pages of 64 tokens (24/4 heads of 256):
  //   members    32 pages      128 pages     512 pages     2,048 pages
  //     8       21.8 / 22.1   25.9 / 26.7   37.1 / 36.7    73.0 / 65.6
  //     9       22.0 / 22.5   26.1 / 27.1   39.8 / 36.8    84.3 / 66.3
  //    16       25.7 / 26.0   31.8 / 32.2   47.0 / 43.9    98.6 / 80.9
  //    24       30.0 / 28.8   38.4 / 36.1   63.2 / 55.5
  //    48       41.3 / 38.4   53.3 / 48.0   92.8 / 76.6
  // (the host does not know the lengths: a bound of 8 members loses up to 1 us with few pages and
  // wins up to 18 with many).
  const int blocks = c.B > 8 * (int64_t)n_groups ? kPlanBlocks : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n_groups * blocks);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, plan_kernel, c, N, parent, group, n_groups, plan) != cudaSuccess) {
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
  }
  return launch_status();
}

int launch_kv4_shared_join(const kv4::AttnArgs& a, int rows, int blocks, cudaStream_t s) {
  switch (a.c.D) {
    case 64: return join_d<64>(a, rows, blocks, s);
    case 128: return join_d<128>(a, rows, blocks, s);
    default: return join_d<256>(a, rows, blocks, s);
  }
}

}  // namespace gdn
