// Attention over the 4-bit key/value cache (include/gdn.h).
//
//     o[b][n][h] = sum_j p_j v_j,  p = softmax_j(scale * q . k_j)
//
// One block per (node, query head, sequence): its warps take the positions
// round robin, each with a running maximum and sum, and are joined at the end.
#include <cuda_fp16.h>
#include <math.h>

#include "gdn_common.cuh"
#include "gdn_kv4.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

using namespace kv4;

constexpr int kWarps = 4;

template <int DT, int D>
__global__ void __launch_bounds__(kWarps * 32)
attn_kernel(gdn_kv4_cache c, const void* __restrict__ qin, int64_t qsb, int64_t qsn, int N, int Hq,
            float scale, const int32_t* parent, void* __restrict__ out, float* lse) {
  constexpr int C = D / 32;  // channels of a lane
  using T = typename Elem<DT>::T;
  __shared__ float part[kWarps][D + 2];
  __shared__ unsigned long long seen_s;
  pdl_enter();
  const int n = blockIdx.x / Hq, hq = blockIdx.x % Hq, b = blockIdx.y;
  const int h = hq / (Hq / c.Hkv), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int len = seq_len(c, b, blockIdx.x == 0 && threadIdx.x == 0);
  if (threadIdx.x == 0) {
    unsigned long long seen = 0;
    if (parent != nullptr) {
      const int32_t* p = parent + (int64_t)b * N;
      if (tree_ok(p, N))
        for (int m = n; m >= 0; m = p[m]) seen |= 1ull << m;
      else
        report(c.status, GDN_ERR_BAD_TREE);
    }
    seen_s = seen;
  }
  __syncthreads();
  const unsigned long long seen = seen_s;
  if (parent != nullptr && seen == 0) len = 0;
  const int base = len - N;
  float q[C], acc[C] = {};
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const T raw = static_cast<const T*>(qin)[b * qsb + n * qsn + (int64_t)hq * D + lane * C + i];
    q[i] = DT == GDN_BF16 ? bf16_to_f32(raw) : __half2float(__ushort_as_half(raw));
  }
  const float x_scale = scale * (c.k_scale != nullptr ? c.k_scale[h] : 1.0f);
  float top = -INFINITY, sum = 0.f;
  for (int j = warp; j < len; j += kWarps) {
    const int u = j - base;
    if (u >= 0 && (parent != nullptr ? !((seen >> u) & 1) : u > n)) continue;
    const uint8_t* rec = record(c, b, h, j);
    if (rec == nullptr) {
      if (lane == 0) report(c.status, GDN_ERR_PAGE_RANGE);
      continue;
    }
    const int slot = j % kRec;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int ch = lane * C + i;
      const uint32_t k8 = rec[(ch >> 5) * 512 + slot * 16 + ((ch & 31) >> 1)];
      x += q[i] * e2m1((k8 >> (4 * (ch & 1))) & 15u) * e4m3(rec[off_ks(D) + slot * (D / 16) + (ch >> 4)]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= x_scale;
    const float t = fmaxf(top, x);
    const float keep = top == -INFINITY ? 0.f : __expf(top - t);
    const float p = x == -INFINITY ? 0.f : __expf(x - t);  // NaN stays
    top = t;
    sum = sum * keep + p;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int ch = lane * C + i;
      const uint32_t v8 = rec[off_v(D) + ch * 16 + (slot >> 1)];
      const float v = e2m1((v8 >> (4 * (slot & 1))) & 15u) * e4m3(rec[off_vs(D) + (ch >> 4) * kRec + slot]);
      acc[i] = acc[i] * keep + p * v;
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) part[warp][lane * C + i] = acc[i];
  if (lane == 0) part[warp][D] = top, part[warp][D + 1] = sum;
  __syncthreads();
  float all = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) all = fmaxf(all, part[w][D]);
  for (int w = 0; w < kWarps; ++w)
    if (part[w][D + 1] != 0.f) total += part[w][D + 1] * __expf(part[w][D] - all);
  const int64_t at = ((int64_t)b * N + n) * Hq + hq;
  const float v_scale = c.v_scale != nullptr ? c.v_scale[h] : 1.0f;
  for (int ch = threadIdx.x; ch < D; ch += kWarps * 32) {
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w)
      if (part[w][D + 1] != 0.f) o += part[w][ch] * __expf(part[w][D] - all);
    static_cast<T*>(out)[at * D + ch] = Elem<DT>::from(total != 0.f ? o / total * v_scale : 0.f);
  }
  if (lse != nullptr && threadIdx.x == 0) lse[at] = total != 0.f ? all + logf(total) : -INFINITY;
}

template <int DT>
int attn_d(const gdn_kv4_cache& c, const void* q, int64_t qsb, int64_t qsn, int N, int Hq,
           float scale, const int32_t* parent, void* o, float* lse, cudaStream_t s) {
  const dim3 grid(N * Hq, c.B), block(kWarps * 32);
  switch (c.D) {
    case 64: return launch_pdl(attn_kernel<DT, 64>, grid, block, 0, s, c, q, qsb, qsn, N, Hq, scale, parent, o, lse);
    case 128: return launch_pdl(attn_kernel<DT, 128>, grid, block, 0, s, c, q, qsb, qsn, N, Hq, scale, parent, o, lse);
    default: return launch_pdl(attn_kernel<DT, 256>, grid, block, 0, s, c, q, qsb, qsn, N, Hq, scale, parent, o, lse);
  }
}

}  // namespace

size_t kv4_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D) { return 16; }

int launch_kv4_attention(const gdn_kv4_cache& c, const void* q, int dtype, int64_t qsb, int64_t qsn,
                         int N, int Hq, float scale, const int32_t* parent, void* o, float* lse,
                         void* workspace, cudaStream_t s) {
  return dtype == GDN_BF16 ? attn_d<GDN_BF16>(c, q, qsb, qsn, N, Hq, scale, parent, o, lse, s)
                           : attn_d<GDN_F16>(c, q, qsb, qsn, N, Hq, scale, parent, o, lse, s);
}

}  // namespace gdn
