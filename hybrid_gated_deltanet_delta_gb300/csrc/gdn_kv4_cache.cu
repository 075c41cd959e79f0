// The 4-bit key/value cache outside attention: append (quantise on write),
// read back, and the commit of an accepted path.  Layout and value definition
// are in include/gdn.h.
//
// The unit of all three is a record (32 tokens of one head), because a byte of
// the V codes holds two neighbouring tokens of one channel: one thread block
// owns every byte of the records it writes, so a token appended next to an
// older one is merged with it without atomics.
#include "gdn_common.cuh"
#include "gdn_kv4.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

using namespace kv4;

constexpr int kThreads = 256;

// ---------------------------------------------------------------- append
// Grid (records a block can touch, Hkv, B).  A thread quantises 16 channels of
// one token: K codes are 8 contiguous bytes and go straight to the record; V
// codes are staged one byte each in shared memory ([token][channel]) and then
// packed by the thread that owns the channel, 16 bytes of 32 tokens, merged
// with the record's old bytes where the block covers only part of it.
template <int DT, int D>
__global__ void __launch_bounds__(kThreads)
append_kernel(gdn_kv4_cache c, const void* __restrict__ kin, const void* __restrict__ vin,
              int64_t ksb, int64_t ksn, int64_t vsb, int64_t vsn, int N) {
  constexpr int G = D / 16;  // scale groups
  using T = typename Elem<DT>::T;
  __shared__ __align__(16) uint8_t code[kRec][D];
  pdl_enter();
  const int b = blockIdx.z, h = blockIdx.y;
  const int len = seq_len(c, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  const int base = len - N;
  const int t0 = ((base > 0 ? base : 0) / kRec + (int)blockIdx.x) * kRec;  // first token here
  if (t0 >= len) return;
  const int lo = base > t0 ? base - t0 : 0, hi = len - t0 < kRec ? len - t0 : kRec;
  uint8_t* rec = record(c, b, h, t0);
  if (rec == nullptr) {
    if (threadIdx.x == 0) report(c.status, GDN_ERR_PAGE_RANGE);
    return;
  }
  const float inv_k = c.k_scale != nullptr ? 1.0f / c.k_scale[h] : 1.0f;
  const float inv_v = c.v_scale != nullptr ? 1.0f / c.v_scale[h] : 1.0f;
  bool bad = false;
  for (int i = threadIdx.x; i < 2 * (hi - lo) * G; i += kThreads) {
    const bool is_v = i >= (hi - lo) * G;
    const int u = is_v ? i - (hi - lo) * G : i;
    const int slot = lo + u / G, g = u % G;
    const int64_t n = t0 + slot - base;
    const T* src = is_v ? static_cast<const T*>(vin) + b * vsb + n * vsn + (int64_t)h * D + g * 16
                        : static_cast<const T*>(kin) + b * ksb + n * ksn + (int64_t)h * D + g * 16;
    float x[2][8];
    load8<DT>(src, x[0]);
    load8<DT>(src + 8, x[1]);
    const float inv = is_v ? inv_v : inv_k;
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float y = x[j >> 3][j & 7];
      bad |= !(fabsf(y) <= 3.4028235e38f);
      y *= inv;
      y = y == y ? fminf(fmaxf(y, -2688.f), 2688.f) : 0.f;
      a = fmaxf(a, fabsf(y));
      x[j >> 3][j & 7] = y;
    }
    const uint32_t s8 = to_e4m3(a * (1.0f / 6.0f));
    const float s = e4m3((uint8_t)s8);
    const float r = s > 0.f ? 1.0f / s : 0.f;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 16; j += 2)
      w[j >> 3] |= to_e2m1x2(x[j >> 3][j & 7] * r, x[j >> 3][(j & 7) + 1] * r) << (4 * (j & 7));
    if (is_v) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // 4 codes -> 4 bytes
        const uint32_t n4 = w[j >> 1] >> (16 * (j & 1));
        o[j] = (n4 & 0xfu) | ((n4 & 0xf0u) << 4) | ((n4 & 0xf00u) << 8) | ((n4 & 0xf000u) << 12);
      }
      *reinterpret_cast<uint4*>(&code[slot][g * 16]) = make_uint4(o[0], o[1], o[2], o[3]);
      rec[off_vs(D) + g * kRec + slot] = (uint8_t)s8;
    } else {
      *reinterpret_cast<uint2*>(rec + (g >> 1) * 512 + slot * 16 + (g & 1) * 8) =
          make_uint2(w[0], w[1]);
      rec[off_ks(D) + slot * G + g] = (uint8_t)s8;
    }
  }
  if (bad) report(c.status, GDN_ERR_NONFINITE);
  __syncthreads();
  for (int ch = threadIdx.x; ch < D; ch += kThreads) {
    uint4* at = reinterpret_cast<uint4*>(rec + off_v(D) + ch * 16);
    uint32_t w[4] = {0, 0, 0, 0}, m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < kRec; ++t)
      if (t >= lo && t < hi) {
        w[t >> 3] |= (uint32_t)code[t][ch] << (4 * (t & 7));
        m[t >> 3] |= 0xfu << (4 * (t & 7));
      }
    if (lo != 0 || hi != kRec) {
      const uint4 old = *at;
      w[0] |= old.x & ~m[0], w[1] |= old.y & ~m[1], w[2] |= old.z & ~m[2], w[3] |= old.w & ~m[3];
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------- read back
// Grid as append.  K: a thread takes 8 channels of a token (4 bytes); V: a
// thread takes a channel (16 bytes, 32 tokens), so that a warp's stores of one
// token are consecutive channels.
template <int DT, int D>
__global__ void __launch_bounds__(kThreads)
read_kernel(gdn_kv4_cache c, void* __restrict__ kout, void* __restrict__ vout, int N) {
  using E = Elem<DT>;
  using T = typename E::T;
  pdl_enter();
  const int b = blockIdx.z, h = blockIdx.y;
  const int len = seq_len(c, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  const int base = len - N;
  T* ko = static_cast<T*>(kout) + ((int64_t)b * N * c.Hkv + h) * D;
  T* vo = static_cast<T*>(vout) + ((int64_t)b * N * c.Hkv + h) * D;
  const int64_t step = (int64_t)c.Hkv * D;
  // nodes that do not exist: the blocks of this head share them
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
       i < (int64_t)(base < 0 ? -base : 0) * D; i += (int64_t)gridDim.x * kThreads) {
    ko[i / D * step + i % D] = E::from(0.f);
    vo[i / D * step + i % D] = E::from(0.f);
  }
  const int t0 = ((base > 0 ? base : 0) / kRec + (int)blockIdx.x) * kRec;
  if (t0 >= len) return;
  const int lo = base > t0 ? base - t0 : 0, hi = len - t0 < kRec ? len - t0 : kRec;
  const uint8_t* rec = record(c, b, h, t0);
  if (rec == nullptr && threadIdx.x == 0) report(c.status, GDN_ERR_PAGE_RANGE);
  const float gk = c.k_scale != nullptr ? c.k_scale[h] : 1.0f;
  const float gv = c.v_scale != nullptr ? c.v_scale[h] : 1.0f;
  for (int i = threadIdx.x; i < (hi - lo) * (D / 8); i += kThreads) {
    const int slot = lo + i / (D / 8), p = i % (D / 8);
    T* out = ko + (int64_t)(t0 + slot - base) * step + p * 8;
    uint32_t w = 0;
    float s = 0.f;
    if (rec != nullptr) {
      w = *reinterpret_cast<const uint32_t*>(rec + (p >> 2) * 512 + slot * 16 + (p & 3) * 4);
      s = e4m3(rec[off_ks(D) + slot * (D / 16) + (p >> 1)]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) out[j] = E::from(e2m1((w >> (4 * j)) & 15u) * s * gk);
  }
  for (int i = threadIdx.x; i < 4 * D; i += kThreads) {
    const int ch = i % D, quarter = i / D;  // 8 tokens
    uint32_t w = 0;
    uint2 s8 = make_uint2(0, 0);
    if (rec != nullptr) {
      w = *reinterpret_cast<const uint32_t*>(rec + off_v(D) + ch * 16 + quarter * 4);
      s8 = *reinterpret_cast<const uint2*>(rec + off_vs(D) + (ch >> 4) * kRec + quarter * 8);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int slot = quarter * 8 + j;
      if (slot < lo || slot >= hi) continue;
      const float s = e4m3((uint8_t)((j < 4 ? s8.x : s8.y) >> (8 * (j & 3))));
      vo[(int64_t)(t0 + slot - base) * step + ch] = E::from(e2m1((w >> (4 * j)) & 15u) * s * gv);
    }
  }
}

// ---------------------------------------------------------------- commit
// Grid (Hkv, B, layers).  A block of up to 64 nodes lies in at most three
// records.  K codes and scales are moved by word, each word position by one
// thread along the path in order (a node's source is never an earlier node's
// destination, since the i-th node of a path has index >= i); a V channel's
// nibbles are moved by the thread that owns the channel, in a shared-memory copy
// of its rows.
constexpr int kMaxNodes = 64;
constexpr int kWindow = 3;

template <int D>
__global__ void __launch_bounds__(kThreads)
commit_kernel(gdn_kv4_cache c, int64_t layer_stride, int N, const int32_t* parent,
              const int32_t* accept, int32_t* len_out) {
  __shared__ int path[kMaxNodes];
  __shared__ int count;
  __shared__ uint8_t* recs[kWindow];
  __shared__ __align__(16) uint8_t vrow[D][kWindow * 16];
  pdl_enter();
  const int h = blockIdx.x, b = blockIdx.y;
  if (threadIdx.x == 0) {
    const bool lead = h == 0 && blockIdx.z == 0;
    const int len = seq_len(c, b, lead), a = accept[b];
    int err = GDN_OK, m = 0;
    if (a < 0 || a >= N) err = GDN_ERR_ACCEPT_RANGE;
    else if (len < N) err = GDN_ERR_ROW_RANGE;
    else if (parent == nullptr) m = a + 1;
    else if (!tree_ok(parent + (int64_t)b * N, N)) err = GDN_ERR_BAD_TREE;
    if (err == GDN_OK && parent != nullptr) {
      for (int n = a; n >= 0; n = parent[(int64_t)b * N + n]) ++m;
      int i = m;
      for (int n = a; n >= 0; n = parent[(int64_t)b * N + n]) path[--i] = n;
    }
    if (lead) {
      if (err != GDN_OK) report(c.status, err);
      len_out[b] = err == GDN_OK ? len - N + m : c.kv_len[b];
    }
    if (parent == nullptr) m = 0;  // a chain's path is where it is
    while (m > 0 && path[m - 1] == m - 1) --m;  // only a prefix moves nothing: then m = 0
    count = err == GDN_OK ? m : 0;
    for (int w = 0; w < kWindow; ++w) {
      const int pos = ((len - N) / kRec + w) * kRec;
      recs[w] = nullptr;
      if (count > 0 && pos < len) {
        recs[w] = record(c, b, h, pos);
        if (recs[w] == nullptr) {
          if (lead) report(c.status, GDN_ERR_PAGE_RANGE);
          count = 0;
        } else {
          recs[w] += blockIdx.z * layer_stride;
        }
      }
    }
  }
  __syncthreads();
  const int m = count;
  if (m == 0) return;
  const int off = (c.kv_len[b] - N) % kRec;
  constexpr int kw = D / 8, sw = D / 64;  // words of a token's K codes, K scales
  for (int i = threadIdx.x; i < kw + sw + D / 16; i += kThreads) {
    for (int e = 0; e < m; ++e) {
      if (path[e] == e) continue;
      const int from = off + path[e], to = off + e;
      const uint8_t* s = recs[from / kRec];
      uint8_t* d = recs[to / kRec];
      const int fs = from % kRec, ts = to % kRec;
      if (i < kw) {
        *reinterpret_cast<uint32_t*>(d + (i >> 2) * 512 + ts * 16 + (i & 3) * 4) =
            *reinterpret_cast<const uint32_t*>(s + (i >> 2) * 512 + fs * 16 + (i & 3) * 4);
      } else if (i < kw + sw) {
        const int j = (i - kw) * 4;
        *reinterpret_cast<uint32_t*>(d + off_ks(D) + ts * (D / 16) + j) =
            *reinterpret_cast<const uint32_t*>(s + off_ks(D) + fs * (D / 16) + j);
      } else {
        const int g = (i - kw - sw) * kRec;
        d[off_vs(D) + g + ts] = s[off_vs(D) + g + fs];
      }
    }
  }
  for (int ch = threadIdx.x; ch < D; ch += kThreads) {
    uint8_t* row = vrow[ch];
    const int last = (off + path[m - 1]) / kRec;
#pragma unroll
    for (int w = 0; w < kWindow; ++w)
      if (w <= last)
        *reinterpret_cast<uint4*>(row + w * 16) =
            *reinterpret_cast<const uint4*>(recs[w] + off_v(D) + ch * 16);
    for (int e = 0; e < m; ++e) {
      const int from = off + path[e], to = off + e;
      const uint32_t x = (row[from >> 1] >> (4 * (from & 1))) & 15u;
      const uint32_t keep = row[to >> 1] & (to & 1 ? 0x0fu : 0xf0u);
      row[to >> 1] = (uint8_t)(keep | (x << (4 * (to & 1))));
    }
#pragma unroll
    for (int w = 0; w < kWindow; ++w)
      if (w <= (off + m - 1) / kRec)
        *reinterpret_cast<uint4*>(recs[w] + off_v(D) + ch * 16) =
            *reinterpret_cast<const uint4*>(row + w * 16);
  }
}

template <int DT>
int append_d(const gdn_kv4_cache& c, const void* k, const void* v, int64_t ksb, int64_t ksn,
             int64_t vsb, int64_t vsn, int N, dim3 grid, cudaStream_t s) {
  switch (c.D) {
    case 64: return launch_pdl(append_kernel<DT, 64>, grid, dim3(kThreads), 0, s, c, k, v, ksb, ksn, vsb, vsn, N);
    case 128: return launch_pdl(append_kernel<DT, 128>, grid, dim3(kThreads), 0, s, c, k, v, ksb, ksn, vsb, vsn, N);
    default: return launch_pdl(append_kernel<DT, 256>, grid, dim3(kThreads), 0, s, c, k, v, ksb, ksn, vsb, vsn, N);
  }
}

template <int DT>
int read_d(const gdn_kv4_cache& c, void* k, void* v, int N, dim3 grid, cudaStream_t s) {
  switch (c.D) {
    case 64: return launch_pdl(read_kernel<DT, 64>, grid, dim3(kThreads), 0, s, c, k, v, N);
    case 128: return launch_pdl(read_kernel<DT, 128>, grid, dim3(kThreads), 0, s, c, k, v, N);
    default: return launch_pdl(read_kernel<DT, 256>, grid, dim3(kThreads), 0, s, c, k, v, N);
  }
}

// Records that N tokens can touch, whatever the offset of the first.
int touched(int N) { return (int)(((int64_t)N + kRec - 2) / kRec + 1); }

}  // namespace

int launch_kv4_append(const gdn_kv4_cache& c, const void* k, const void* v, int dtype,
                      int64_t ksb, int64_t ksn, int64_t vsb, int64_t vsn, int N, cudaStream_t s) {
  const dim3 grid(touched(N), c.Hkv, c.B);
  switch (dtype) {
    case GDN_F32: return append_d<GDN_F32>(c, k, v, ksb, ksn, vsb, vsn, N, grid, s);
    case GDN_BF16: return append_d<GDN_BF16>(c, k, v, ksb, ksn, vsb, vsn, N, grid, s);
    default: return append_d<GDN_F16>(c, k, v, ksb, ksn, vsb, vsn, N, grid, s);
  }
}

int launch_kv4_read(const gdn_kv4_cache& c, void* k, void* v, int dtype, int N, cudaStream_t s) {
  const dim3 grid(touched(N), c.Hkv, c.B);
  switch (dtype) {
    case GDN_F32: return read_d<GDN_F32>(c, k, v, N, grid, s);
    case GDN_BF16: return read_d<GDN_BF16>(c, k, v, N, grid, s);
    default: return read_d<GDN_F16>(c, k, v, N, grid, s);
  }
}

int launch_kv4_commit(const gdn_kv4_cache& c, int64_t layer_stride, int n_layers, int N,
                      const int32_t* parent, const int32_t* accept, int32_t* len_out,
                      cudaStream_t s) {
  // a chain moves nothing: one block per sequence writes its length
  const dim3 grid(parent != nullptr ? c.Hkv : 1, c.B, parent != nullptr ? n_layers : 1);
  switch (c.D) {
    case 64: return launch_pdl(commit_kernel<64>, grid, dim3(kThreads), 0, s, c, layer_stride, N, parent, accept, len_out);
    case 128: return launch_pdl(commit_kernel<128>, grid, dim3(kThreads), 0, s, c, layer_stride, N, parent, accept, len_out);
    default: return launch_pdl(commit_kernel<256>, grid, dim3(kThreads), 0, s, c, layer_stride, N, parent, accept, len_out);
  }
}

}  // namespace gdn
