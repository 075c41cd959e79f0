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
#include "gdn_kv4_append.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

using namespace kv4;

// ---------------------------------------------------------------- append
// Grid (records a block can touch, Hkv, B).  A thread quantises 16 channels of
// two neighbouring tokens, the two that share the bytes of V codes.  K codes are 8
// contiguous bytes a token and go straight to the record; V codes are staged as
// bytes ([token pair][channel]) in shared memory and gathered by the thread that
// owns the channel, 16 bytes of 32 tokens, merged with the record's old bytes where
// the block covers only part of it.  Bound by the instructions on each value and
// the latency of a block's length, page and values: 8,192 tokens of 4 heads of 256
// channels (43 MB) were 30 us with a token a thread and a byte a code in shared
// memory, 17.7 us with every value clamped and checked by itself, and are 14.8 us
// this way.  Four blocks an SM (64 registers): with three 18.0 us, with five 16.9.
// Whole 32-byte sectors a store, by exchanges between lanes, gave 14.7 us and were
// left out.
template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 4)
append_kernel(gdn_kv4_cache c, const void* __restrict__ kin, const void* __restrict__ vin,
              int64_t ksb, int64_t ksn, int64_t vsb, int64_t vsn, int N) {
  constexpr int G = D / 16;  // scale groups
  using T = typename Elem<DT>::T;
  __shared__ __align__(16) uint8_t code[kRec / 2][D];
  pdl_enter();
  const int b = blockIdx.z, h = blockIdx.y;
  // (The place, and V's codes at the end, stand here although gdn_kv4_rotary.cu has functions for
  // them: with calls of those, inlined, eight chains of 16 take 3.32 us, here 3.20, one token 2.94
  // and 2.85, 512 tokens 4.22 and 4.10; 48 sequences 3.42 and 3.50.)
  const int len = seq_len(c, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
  Place at;
  at.base = len - N;
  at.t0 = ((at.base > 0 ? at.base : 0) / kRec + (int)blockIdx.x) * kRec;
  if (at.t0 >= len) return;
  at.lo = at.base > at.t0 ? at.base - at.t0 : 0, at.hi = len - at.t0 < kRec ? len - at.t0 : kRec;
  at.rec = record(c, b, h, at.t0);
  if (at.rec == nullptr) {
    if (threadIdx.x == 0) report(c.status, GDN_ERR_PAGE_RANGE);
    return;
  }
  const float inv_k = c.k_scale != nullptr ? 1.0f / c.k_scale[h] : 1.0f;
  const float inv_v = c.v_scale != nullptr ? 1.0f / c.v_scale[h] : 1.0f;
  const int pair0 = at.lo >> 1, pairs = ((at.hi + 1) >> 1) - pair0;
  bool bad = false;
  for (int i = threadIdx.x; i < 2 * pairs * G; i += kThreads) {
    const bool is_v = i >= pairs * G;
    const int u = is_v ? i - pairs * G : i, g = u % G;
    const T* src = is_v ? static_cast<const T*>(vin) + b * vsb : static_cast<const T*>(kin) + b * ksb;
    const int64_t step = is_v ? vsn : ksn;
    quantise_pair<D>(at, is_v, is_v ? inv_v : inv_k, pair0 + u / G, g, code, bad,
                     [&](int slot, float (&x)[2][8]) {
                       const T* p = src + (int64_t)(at.t0 + slot - at.base) * step +
                                    (int64_t)h * D + g * 16;
                       load8<DT>(p, x[0]);
                       load8<DT>(p + 8, x[1]);
                     });
  }
  if (bad) report(c.status, GDN_ERR_NONFINITE);
  __syncthreads();
  // nibbles of the block in each word of 8 tokens
  uint32_t mine[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int from = min(max(at.lo - 8 * w, 0), 8), to = min(max(at.hi - 8 * w, 0), 8);
    mine[w] = (uint32_t)(((1ull << (4 * to)) - 1) & ~((1ull << (4 * from)) - 1));
  }
  for (int ch = threadIdx.x; ch < D; ch += kThreads) {
    uint4* to = reinterpret_cast<uint4*>(at.rec + off_v(D) + ch * 16);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (code[4 * k][ch] | (uint32_t)code[4 * k + 1][ch] << 8 |
              (uint32_t)code[4 * k + 2][ch] << 16 | (uint32_t)code[4 * k + 3][ch] << 24) & mine[k];
    if (at.lo != 0 || at.hi != kRec) {
      const uint4 old = *to;
      w[0] |= old.x & ~mine[0], w[1] |= old.y & ~mine[1];
      w[2] |= old.z & ~mine[2], w[3] |= old.w & ~mine[3];
    }
    *to = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------- read back
// Grid as append.  K: a thread takes 16 bytes of output of a token, four tokens'
// codes in flight; V: 4 channels of 8 tokens (a word of each), four lanes beside
// each other the same channels, so that a warp's reads and stores are whole sectors.
// Bound by the stores: 67 MB of fp32 for 8,192 tokens of 4 heads of 256 channels,
// 35 us with a value a store, 16.4 us so; 16 tokens of 8 sequences 3.6 us with one
// token's codes in flight, 3.0 us with four.
template <int DT>
__device__ __forceinline__ void store4(void* p, const float (&x)[4]) {
  if constexpr (DT == GDN_F32) {
    st_f4(static_cast<float*>(p), x[0], x[1], x[2], x[3]);
  } else {
    using E = Elem<DT>;
    *reinterpret_cast<uint2*>(p) =
        make_uint2(E::from(x[0]) | (uint32_t)E::from(x[1]) << 16,
                   E::from(x[2]) | (uint32_t)E::from(x[3]) << 16);
  }
}

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
  constexpr int CH = 16 / (int)sizeof(T), PER = D / CH;  // channels of a K thread
  constexpr int U = 4;  // loads in flight before their stores
  for (int i0 = threadIdx.x; i0 < (hi - lo) * PER; i0 += U * kThreads) {
    uint32_t w[U];
    uint8_t s8[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads, slot = lo + i / PER, ch = i % PER * CH;
      w[u] = 0, s8[u] = 0;
      if (rec != nullptr && i < (hi - lo) * PER) {
        const uint8_t* at = rec + (ch >> 5) * 512 + slot * 16 + ((ch & 31) >> 1);
        w[u] = CH == 4 ? *reinterpret_cast<const uint16_t*>(at)
                       : *reinterpret_cast<const uint32_t*>(at);
        s8[u] = rec[off_ks(D) + slot * (D / 16) + (ch >> 4)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads, slot = lo + i / PER, ch = i % PER * CH;
      if (i >= (hi - lo) * PER) break;
      const float s = e4m3(s8[u]);
      T* out = ko + (int64_t)(t0 + slot - base) * step + ch;
#pragma unroll
      for (int half = 0; half < CH / 4; ++half) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = e2m1((w[u] >> (16 * half + 4 * j)) & 15u) * s * gk;
        store4<DT>(out + 4 * half, x);
      }
    }
  }
  for (int i = threadIdx.x; i < D; i += kThreads) {
    const int ch = i / 4 * 4, quarter = i % 4;  // 8 tokens
    uint32_t w[4] = {0, 0, 0, 0};
    uint2 s8 = make_uint2(0, 0);
    if (rec != nullptr) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = *reinterpret_cast<const uint32_t*>(rec + off_v(D) + (ch + k) * 16 + quarter * 4);
      s8 = *reinterpret_cast<const uint2*>(rec + off_vs(D) + (ch >> 4) * kRec + quarter * 8);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int slot = quarter * 8 + j;
      if (slot < lo || slot >= hi) continue;
      const float s = e4m3((uint8_t)((j < 4 ? s8.x : s8.y) >> (8 * (j & 3))));
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = e2m1((w[k] >> (4 * j)) & 15u) * s * gv;
      store4<DT>(vo + (int64_t)(t0 + slot - base) * step + ch, x);
    }
  }
}

// ---------------------------------------------------------------- commit
// Grid (pieces of the (layer, head) pairs, B).  A block of up to 64 nodes lies in at
// most three records.  The path is found once a block of threads, in shared memory;
// then each warp moves K and the scales, or 64 channels of V, of one (layer, head)
// pair at a time.  K codes and scales are moved by word, each word position by one
// lane, eight path nodes read before they are written (a node's source is never an
// earlier node's destination, since the i-th node of a path has index >= i).  A V
// channel's codes are gathered nibble by nibble by the lane that owns the channel,
// from its words in shared memory, two channels a lane: a nibble's place and turn are
// worked out once, and cost each channel a rotation and a select.  Bound by latency
// and those instructions: few bytes have to move, but the rows of V that hold them
// are read and written whole.  64 trees of 22 nodes, 8 heads of 128 channels, 16
// layers: 38 us with a block a (layer, head) pair that walks the path in global
// memory, 31 us with four layers to a block and the path in shared memory, 26 us with
// blocks that do not all fit at once, 23.5 us with one wave and a channel's nibbles
// moved one by one, 15.7 us this way (one tree: 6.2, 9.0, 4.9, 4.6 and 3.9 us).  Of
// waves of 456, 608, 760 and 912 blocks 608 (four on each of 152 SMs) took least: 16.9,
// 15.7, 18.0 and 17.2 us.
constexpr int kMaxNodes = 64;
constexpr int kWindow = 3;
constexpr int kCommitWarps = kThreads / 32;

template <int D>
__global__ void __launch_bounds__(kThreads)
commit_kernel(gdn_kv4_cache c, int64_t layer_stride, int n_layers, int N, const int32_t* parent,
              const int32_t* accept, int32_t* len_out) {
  __shared__ int up[kMaxNodes], back[kMaxNodes];  // parents; the path from its end
  __shared__ int count, bad_tree;
  __shared__ uint8_t* recs[kWindow];  // of head 0, layer 0
  __shared__ int src[kMaxNodes];  // where the i-th node of the path is, from the first record
  __shared__ uint2 rows[kCommitWarps][kWindow * 4][32];
  pdl_enter();
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool lead = blockIdx.x == 0;
  // what the path needs is read at once: length, node, parents, pages
  const int len = seq_len(c, b, lead && threadIdx.x == 0), a = accept[b];
  if (parent != nullptr) {
    if (threadIdx.x == 0) bad_tree = 0;
    __syncthreads();
    for (int n = threadIdx.x; n < N; n += kThreads) {
      const int p = parent[(int64_t)b * N + n];
      up[n] = p;
      if (n == 0 ? p != -1 : p < 0 || p >= n) bad_tree = 1;
    }
    if (threadIdx.x >= kMaxNodes && threadIdx.x < kMaxNodes + kWindow && len >= N) {
      const int w = threadIdx.x - kMaxNodes, pos = ((len - N) / kRec + w) * kRec;
      recs[w] = pos < len ? record(c, b, 0, pos) : nullptr;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    int err = GDN_OK, m = 0;
    if (a < 0 || a >= N) err = GDN_ERR_ACCEPT_RANGE;
    else if (len < N) err = GDN_ERR_ROW_RANGE;
    else if (parent == nullptr) m = a + 1;
    else if (bad_tree) err = GDN_ERR_BAD_TREE;
    if (err == GDN_OK && parent != nullptr)
      for (int n = a; n >= 0; n = up[n]) back[m++] = n;
    // a chain's path is where it is, and so is one of the nodes 0 .. m - 1
    const bool moves = err == GDN_OK && parent != nullptr && a != m - 1;
    if (moves)  // all of the block's pages, before anything is written
      for (int w = 0; w < kWindow; ++w)
        if (((len - N) / kRec + w) * kRec < len && recs[w] == nullptr) err = GDN_ERR_PAGE_RANGE;
    if (lead) {
      if (err != GDN_OK) report(c.status, err);
      len_out[b] = err == GDN_OK ? len - N + m : c.kv_len[b];
    }
    if (err != GDN_OK || !moves) m = 0;
    count = m;
  }
  __syncthreads();
  const int m = count;
  if (m == 0) return;
  const int off = (len - N) % kRec;
  for (int i = threadIdx.x; i < m; i += kThreads) src[i] = off + back[m - 1 - i];
  __syncthreads();
  int first = 0;  // nodes before it stay
  while (src[first] == off + first) ++first;
  constexpr int kw = D / 8, sw = D / 64;  // words of a token's K codes, K scales
  const int rec0 = (off + first) / kRec, rec1 = (off + m - 1) / kRec;  // written
  const int last = src[m - 1] / kRec;                                  // read
  const int64_t head_stride = (int64_t)(c.page_tokens / kRec) * rec_bytes(D);
  // a warp's work: a (layer, head) pair's K and scales, or 64 channels of its V
  constexpr int PARTS = 1 + D / 64;
  for (int i = blockIdx.x * kCommitWarps + warp; i < n_layers * c.Hkv * PARTS;
       i += gridDim.x * kCommitWarps) {
    const int part = i % PARTS, pair = i / PARTS;
    const int64_t at0 = pair / c.Hkv * layer_stride + pair % c.Hkv * head_stride;
    for (int j = part == 0 ? lane : D; j < kw + sw + D / 16; j += 32) {
      // where this lane's word (or V scale) of a token is
      const bool byte = j >= kw + sw;
      const int64_t at = at0 + (j < kw ? (j >> 2) * 512 + (j & 3) * 4
                                       : !byte ? off_ks(D) + (j - kw) * 4
                                               : off_vs(D) + (j - kw - sw) * kRec);
      const int step = j < kw ? 16 : !byte ? D / 16 : 1;
      for (int e0 = first; e0 < m; e0 += 8) {
        uint32_t x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (e0 + k >= m) break;
          const int from = src[e0 + k];
          const uint8_t* s = recs[from / kRec] + at + from % kRec * step;
          x[k] = byte ? *s : *reinterpret_cast<const uint32_t*>(s);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (e0 + k >= m) break;
          const int to = off + e0 + k;
          uint8_t* d = recs[to / kRec] + at + to % kRec * step;
          if (byte) *d = (uint8_t)x[k];
          else *reinterpret_cast<uint32_t*>(d) = x[k];
        }
      }
    }
    if (part > 0) {
      // two channels a lane, the words of 8 tokens of both beside each other
      const int64_t at = at0 + off_v(D) + ((part - 1) * 64 + lane) * 16;
      uint4 v[2][kWindow];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int w = 0; w < kWindow; ++w)
          if (w >= rec0 && w <= last)
            v[k][w] = *reinterpret_cast<const uint4*>(recs[w] + at + k * 512);
      uint2(&row)[kWindow * 4][32] = rows[warp];
#pragma unroll
      for (int w = 0; w < kWindow; ++w)
        if (w >= rec0 && w <= last) {
          row[w * 4][lane] = make_uint2(v[0][w].x, v[1][w].x);
          row[w * 4 + 1][lane] = make_uint2(v[0][w].y, v[1][w].y);
          row[w * 4 + 2][lane] = make_uint2(v[0][w].z, v[1][w].z);
          row[w * 4 + 3][lane] = make_uint2(v[0][w].w, v[1][w].w);
        }
      // words in order: a word's sources are at or after it
      for (int w = (off + first) >> 3; w <= (off + m - 1) >> 3; ++w) {
        uint2 x = row[w][lane];
        const int e0 = 8 * w - off;
        for (int e = max(e0, first); e < min(e0 + 8, m); ++e) {
          const int from = src[e], to = 4 * (e - e0), turn = 4 * from - to;
          const uint32_t here = 15u << to;
          const uint2 y = row[from >> 3][lane];
          x.x = (x.x & ~here) | (__funnelshift_r(y.x, y.x, turn) & here);
          x.y = (x.y & ~here) | (__funnelshift_r(y.y, y.y, turn) & here);
        }
        row[w][lane] = x;
      }
#pragma unroll
      for (int w = 0; w < kWindow; ++w)
        if (w >= rec0 && w <= rec1) {
          const uint2 a0 = row[w * 4][lane], a1 = row[w * 4 + 1][lane];
          const uint2 a2 = row[w * 4 + 2][lane], a3 = row[w * 4 + 3][lane];
          *reinterpret_cast<uint4*>(recs[w] + at) = make_uint4(a0.x, a1.x, a2.x, a3.x);
          *reinterpret_cast<uint4*>(recs[w] + at + 512) = make_uint4(a0.y, a1.y, a2.y, a3.y);
        }
    }
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
  // A unit of work a warp while the blocks are one wave, else one wave of blocks with
  // more units each (their path is found once), up to eight; a chain moves nothing:
  // one block per sequence writes its length.
  const int64_t units = (int64_t)n_layers * c.Hkv * (1 + c.D / 64);
  const int64_t wave = (int64_t)sm_count() * 4, most = (units + kCommitWarps - 1) / kCommitWarps;
  if (wave == 0) return GDN_ERR_CUDA;
  const int64_t few = wave / c.B > (most + 7) / 8 ? wave / c.B : (most + 7) / 8;
  const dim3 grid(parent == nullptr ? 1 : (unsigned)(most < few ? most : few), c.B);
  switch (c.D) {
    case 64: return launch_pdl(commit_kernel<64>, grid, dim3(kThreads), 0, s, c, layer_stride, n_layers, N,
                                parent, accept, len_out);
    case 128: return launch_pdl(commit_kernel<128>, grid, dim3(kThreads), 0, s, c, layer_stride, n_layers, N,
                                parent, accept, len_out);
    default: return launch_pdl(commit_kernel<256>, grid, dim3(kThreads), 0, s, c, layer_stride, n_layers, N,
                                parent, accept, len_out);
  }
}

}  // namespace gdn
