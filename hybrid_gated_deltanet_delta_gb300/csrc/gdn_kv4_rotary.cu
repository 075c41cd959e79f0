// Append to the 4-bit key/value cache with rotary positions (include/gdn.h): queries and keys
// turned by their positions, the queries written out, the keys quantised as they are written.
//
//   y_i = x_i c - x_j s,   y_j = x_j c + x_i s   for a pair (i, j), each product and the sum
//                                                rounded to fp32
//
// Grid (records a block can touch, Hkv + rows of query blocks, B).  The first Hkv rows append, a
// record a block: the pairs of the record's keys are turned into shared memory, 8 pairs of a
// token a thread, and quantised from there.  A block of the other rows turns the queries of
// q.tokens tokens, all heads: the channels that pass are moved while the tokens' cosines and
// sines, which all heads use, are gathered in shared memory.
//
// Bound by the bytes where tokens are many: 8,192 tokens of 24 and 4 heads of 256 channels, 32
// pairs, bf16, move 243 MB (36 us at the rate of a copy) in 49.5 us: the queries alone take 36 us,
// keys and values alone 19.  In place (95 MB, 14 us) 29.7; f32 (481 MB, 71 us) 86.6, in place (179
// MB, 26 us) 38.1.  Measured on the way there (with 15 us of reading back): angles
// staged for keys too, each item with two divisions 91 us; the queries' loads before the angles
// 77; items of a thread in one place of every row, channels that pass moved without conversion,
// keys turned before they are quantised 70; 2,048 items a block instead of 1,024 64 (512: 94 in
// the version before, 4,096: 68).  A few tokens are bound by the latency of the length, the
// page, axis, position and angle, one after another: one token 3.8 us.
#include "gdn_common.cuh"
#include "gdn_kv4.cuh"
#include "gdn_kv4_append.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

using namespace kv4;

constexpr int kTurnTokens = kRec;  // tokens whose angles fit in shared memory

// The `part`-th record that the block of N tokens of sequence b touches, of head h.
__device__ __forceinline__ Place find_place(const gdn_kv4_cache& c, int N, int b, int h, int part) {
  Place p = {};
  const int len = seq_len(c, b, part == 0 && h == 0 && threadIdx.x == 0);
  p.base = len - N;
  p.t0 = ((p.base > 0 ? p.base : 0) / kRec + part) * kRec;
  if (p.t0 >= len) return p;
  p.lo = p.base > p.t0 ? p.base - p.t0 : 0, p.hi = len - p.t0 < kRec ? len - p.t0 : kRec;
  p.rec = record(c, b, h, p.t0);
  return p;
}

// Position of a node on an axis, -1 where the table or the axes have none.
__device__ __forceinline__ int position(const gdn_rotary& r, int b, int node, int axis) {
  if (axis >= r.n_axes) return -1;
  const int p = r.positions[axis * r.pos_stride_axis + b * r.pos_stride_b + node];
  return p < r.n_positions ? p : -1;
}

// Cosine and sine of a pair at a position; 1 and 0 where there is none (but for such a pair to
// stay as it is takes more: 0 times an infinity is no number, and -0 + 0 is +0).
__device__ __forceinline__ float2 angle_of(const gdn_rotary& r, int pos, int pair) {
  if (pos < 0) return make_float2(1.f, 0.f);
  const float* at = r.cos_sin + 2 * (int64_t)pos * r.pairs + pair;
  return make_float2(__ldg(at), __ldg(at + r.pairs));
}

// Turns 8 pairs: channel k of a with channel k of b or, adjacent, those of a beside each other
// and then those of b.
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&c)[8],
                                     const float (&s)[8], bool adjacent) {
  auto pair = [](float& x, float& y, float c, float s) {
    const float u = x, w = y;
    x = __fsub_rn(__fmul_rn(u, c), __fmul_rn(w, s));
    y = __fadd_rn(__fmul_rn(w, c), __fmul_rn(u, s));
  };
  if (adjacent) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      pair(a[2 * k], a[2 * k + 1], c[k], s[k]);
      pair(b[2 * k], b[2 * k + 1], c[k + 4], s[k + 4]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) pair(a[k], b[k], c[k], s[k]);
  }
}

struct Queries {
  const void* in;
  void* out;
  int64_t in_b, in_n, out_b, out_n;
  int Hq, tokens;  // tokens: of a block
};

// 8 elements as they are held.
template <int DT>
struct Chunk {
  uint4 w[DT == GDN_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < (DT == GDN_F32 ? 2 : 1); ++i) w[i] = static_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(void* p) const {
#pragma unroll
    for (int i = 0; i < (DT == GDN_F32 ? 2 : 1); ++i) static_cast<uint4*>(p)[i] = w[i];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (DT == GDN_F32 ? 2 : 1); ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if constexpr (DT == GDN_F32) {
      const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i]);
    } else {
      const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f;
        if constexpr (DT == GDN_BF16)
          f = make_float2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u));
        else
          f = __half22float2(*reinterpret_cast<const __half2*>(&v[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void round(const float (&x)[8]) {
    if constexpr (DT == GDN_F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                          __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
    } else {
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = Elem<DT>::from(x[2 * k]) | (uint32_t)Elem<DT>::from(x[2 * k + 1]) << 16;
      w[0] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
};

// The pairs of a block's queries where some have no position: one by one, and those left alone.
// (Of its own, so that the usual way does without the registers.)
template <int DT>
static __device__ __noinline__ void turn_some_queries(const gdn_rotary& r, const Queries& q, int D,
                                                      int b, int node0, int count, int missing,
                                                      const float* cs) {
  using T = typename Elem<DT>::T;
  const T* in = static_cast<const T*>(q.in) + b * q.in_b;
  T* out = static_cast<T*>(q.out) + b * q.out_b;
  for (int64_t i = threadIdx.x; i < (int64_t)count * q.Hq * r.pairs; i += kThreads) {
    const int pair = (int)(i % r.pairs), row = (int)(i / r.pairs);
    const int token = row / q.Hq, head = row - token * q.Hq, node = node0 + token;
    const int first = r.adjacent ? 2 * pair : pair, second = first + (r.adjacent ? 1 : r.pairs);
    const T* from = in + node * q.in_n + (int64_t)head * D;
    T* to = out + node * q.out_n + (int64_t)head * D;
    if (token < missing) {
      to[first] = to[second] = 0;
      continue;
    }
    const T u = from[first], w = from[second];
    if (position(r, b, node, r.axis != nullptr ? r.axis[pair] : 0) < 0) {
      to[first] = u, to[second] = w;
      continue;
    }
    const float x = to_float<DT>(u), y = to_float<DT>(w);
    const float c = cs[2 * token * r.pairs + pair], s = cs[(2 * token + 1) * r.pairs + pair];
    to[first] = Elem<DT>::from(__fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)));
    to[second] = Elem<DT>::from(__fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s)));
  }
}

// Of the record's keys (turned, by this thread), the pairs without a position: as they were.
template <int DT>
static __device__ __noinline__ void pass_keys(const gdn_rotary& r, int lo, int hi, int node0,
                                              const typename Elem<DT>::T* k0, int64_t ksn, int b,
                                              float* turned) {
  const int whole = r.pairs >> 3;
  for (int i = threadIdx.x; i < (hi - lo) * whole; i += kThreads) {
    const int t = i / whole, slot = lo + t, chunk = i - t * whole;
    for (int pair = 8 * chunk; pair < 8 * chunk + 8; ++pair) {
      if (position(r, b, node0 + slot, r.axis != nullptr ? r.axis[pair] : 0) >= 0) continue;
      const int first = r.adjacent ? 2 * pair : pair, second = first + (r.adjacent ? 1 : r.pairs);
      turned[slot * 2 * r.pairs + first] = to_float<DT>(k0[slot * ksn + first]);
      turned[slot * 2 * r.pairs + second] = to_float<DT>(k0[slot * ksn + second]);
    }
  }
}

// Rows (token and head) that a thread visits, `step` apart.
struct Rows {
  int token, head, by_token, by_head, Hq;
  __device__ __forceinline__ Rows(int first, int step, int heads) : Hq(heads) {
    token = first / Hq, head = first - token * Hq;
    by_token = step / Hq, by_head = step - by_token * Hq;
  }
  __device__ __forceinline__ void next() {
    token += by_token, head += by_head;
    if (head >= Hq) head -= Hq, ++token;
  }
};

// Threads beside each other that share a row: the power of two from n (1..16) on, as a shift.
__device__ __forceinline__ int lanes_for(int n) { return n <= 1 ? 0 : 32 - __clz(n - 1); }

// The queries of q.tokens tokens, all heads.  An item is two chunks of 8 channels of one row: two
// that pass, moved as they are while the angles are gathered, or two that hold 8 pairs.  In place
// only the latter are touched (and, of a node that does not exist, all).
template <int DT, int D>
__device__ __forceinline__ void turn_queries(const gdn_kv4_cache& c, const gdn_rotary& r,
                                             const Queries& q, int N, int b, int block, float* cs) {
  using T = typename Elem<DT>::T;
  constexpr int U = DT == GDN_F32 ? 2 : 4;  // items in flight
  const int node0 = block * q.tokens;
  if (node0 >= N) return;
  const int count = min(q.tokens, N - node0), whole = r.pairs >> 3;
  const bool in_place = q.in == q.out;
  const T* in = static_cast<const T*>(q.in) + b * q.in_b + node0 * q.in_n;
  T* out = static_cast<T*>(q.out) + b * q.out_b + node0 * q.out_n;
  const int base = seq_len(c, b, false) - N;
  const int missing = base + node0 < 0 ? min(count, -(base + node0)) : 0;  // first tokens
  // cs[token][2][pairs]
  bool bad = false;
  for (int i = threadIdx.x; i < count * r.pairs; i += kThreads) {
    const int token = i / r.pairs, pair = i - token * r.pairs;
    if (token < missing) continue;
    const int pos = position(r, b, node0 + token, r.axis != nullptr ? r.axis[pair] : 0);
    bad |= pos < 0;
    const float2 a = angle_of(r, pos, pair);
    cs[2 * token * r.pairs + pair] = a.x, cs[(2 * token + 1) * r.pairs + pair] = a.y;
  }
  if (bad) report(c.status, GDN_ERR_POSITION_RANGE);
  // a thread has one item of every row that it visits
  {
    const int n = D / 16 - whole, shift = lanes_for(n), item = threadIdx.x & ((1 << shift) - 1);
    const int tokens = item < n ? (in_place ? missing : count) : 0;
    Rows at(threadIdx.x >> shift, kThreads >> shift, q.Hq);
    const int off = (whole + item) * 16;
#pragma unroll 1
    while (at.token < tokens) {
      Chunk<DT> x[U], y[U];
      T* to[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const T* p = in + at.token * q.in_n + at.head * D + off;
        to[u] = at.token < tokens ? out + at.token * q.out_n + at.head * D + off : nullptr;
        x[u].clear(), y[u].clear();
        if (at.token >= missing && at.token < tokens) x[u].load(p), y[u].load(p + 8);
        at.next();
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (to[u] != nullptr) x[u].store(to[u]), y[u].store(to[u] + 8);
    }
  }
  if (__syncthreads_or(bad)) {
    turn_some_queries<DT>(r, q, D, b, node0, count, missing, cs);
  } else {
    const int shift = lanes_for(whole), item = threadIdx.x & ((1 << shift) - 1);
    const int tokens = item < whole ? count : 0, apart = r.adjacent ? 8 : r.pairs;
    Rows at(threadIdx.x >> shift, kThreads >> shift, q.Hq);
    const int off = item * (r.adjacent ? 16 : 8);
#pragma unroll 1
    while (at.token < tokens) {
      Chunk<DT> x[2], y[2];
      T* to[2];
      const float* angle[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const T* p = in + at.token * q.in_n + at.head * D + off;
        to[u] = at.token < tokens ? out + at.token * q.out_n + at.head * D + off : nullptr;
        angle[u] = at.token >= missing ? cs + 2 * at.token * r.pairs + 8 * item : nullptr;
        x[u].clear(), y[u].clear();
        if (at.token >= missing && at.token < tokens) x[u].load(p), y[u].load(p + apart);
        at.next();
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (to[u] == nullptr) continue;
        if (angle[u] != nullptr) {
          float f[8], g[8], co[8], si[8];
          x[u].values(f);
          y[u].values(g);
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            const float4 c4 = *reinterpret_cast<const float4*>(angle[u] + k);
            const float4 s4 = *reinterpret_cast<const float4*>(angle[u] + r.pairs + k);
            co[k] = c4.x, co[k + 1] = c4.y, co[k + 2] = c4.z, co[k + 3] = c4.w;
            si[k] = s4.x, si[k + 1] = s4.y, si[k + 2] = s4.z, si[k + 3] = s4.w;
          }
          turn(f, g, co, si, r.adjacent);
          x[u].round(f);
          y[u].round(g);
        }
        x[u].store(to[u]);
        y[u].store(to[u] + apart);
      }
    }
  }
}

// What a channel's 16 bytes of V codes hold, where the block covers only part of them.
template <int D>
__device__ __forceinline__ uint4 old_v(const Place& p, int ch) {
  return p.lo != 0 || p.hi != kRec ? *reinterpret_cast<const uint4*>(p.rec + off_v(D) + ch * 16)
                                   : make_uint4(0, 0, 0, 0);
}

// V's codes to the record, after a barrier; `old`: what is there, of the thread's channel.
template <int D>
__device__ __forceinline__ void store_v(const Place& p, const uint8_t (*code)[D], uint4 old) {
  static_assert(D <= kThreads, "a channel of V a thread");
  // nibbles of the block in each word of 8 tokens
  uint32_t mine[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int from = min(max(p.lo - 8 * w, 0), 8), to = min(max(p.hi - 8 * w, 0), 8);
    mine[w] = (uint32_t)(((1ull << (4 * to)) - 1) & ~((1ull << (4 * from)) - 1));
  }
  for (int ch = threadIdx.x; ch < D; ch += kThreads) {
    uint4* at = reinterpret_cast<uint4*>(p.rec + off_v(D) + ch * 16);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (code[4 * k][ch] | (uint32_t)code[4 * k + 1][ch] << 8 |
              (uint32_t)code[4 * k + 2][ch] << 16 | (uint32_t)code[4 * k + 3][ch] << 24) & mine[k];
    if (p.lo != 0 || p.hi != kRec) {
      w[0] |= old.x & ~mine[0], w[1] |= old.y & ~mine[1];
      w[2] |= old.z & ~mine[2], w[3] |= old.w & ~mine[3];
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// BLOCKS an SM: registers against blocks in flight.  With 3 one token takes 6.2 us and 128 of
// eight sequences 8.5 (with reading back), a prompt of 8,192 68.3; with 4 6.5, 9.0 and 66.0.
template <int DT, int D, int BLOCKS>
__global__ void __launch_bounds__(kThreads, BLOCKS)
append_rotary_kernel(const __grid_constant__ gdn_kv4_cache c, const __grid_constant__ gdn_rotary r,
                     const __grid_constant__ Queries q, const void* __restrict__ kin,
                     const void* __restrict__ vin, int64_t ksb, int64_t ksn, int64_t vsb,
                     int64_t vsn, int N) {
  constexpr int G = D / 16;  // scale groups
  using T = typename Elem<DT>::T;
  __shared__ __align__(16) uint8_t code[kRec / 2][D];
  extern __shared__ __align__(16) float turned[];  // [token of the record][2 * pairs]
  pdl_enter();
  const int b = blockIdx.z, h = blockIdx.y;
  if (h >= c.Hkv) {
    turn_queries<DT, D>(c, r, q, N, b, (h - c.Hkv) * gridDim.x + blockIdx.x, turned);
    return;
  }
  const Place at = find_place(c, N, b, h, blockIdx.x);
  if (at.hi == 0) return;
  const int pair0 = at.lo >> 1, pairs = ((at.hi + 1) >> 1) - pair0, whole = r.pairs >> 3;
  bool bad = false, off_table = false;
  const T* k0 = static_cast<const T*>(kin) + b * ksb + (at.t0 - at.base) * ksn + (int64_t)h * D;
  const T* v0 = static_cast<const T*>(vin) + b * vsb + (at.t0 - at.base) * vsn + (int64_t)h * D;
  // the keys' pairs
  for (int i = threadIdx.x; i < (at.hi - at.lo) * whole; i += kThreads) {
    const int t = i / whole, slot = at.lo + t, chunk = i - t * whole;
    const int first = r.adjacent ? chunk * 16 : chunk * 8, apart = r.adjacent ? 8 : r.pairs;
    float x[2][8], co[8], si[8];
    load8<DT>(k0 + slot * ksn + first, x[0]);
    load8<DT>(k0 + slot * ksn + first + apart, x[1]);
    int pos[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      pos[k] = position(r, b, at.t0 + slot - at.base,
                        r.axis != nullptr ? r.axis[chunk * 8 + k] : 0);
      off_table |= pos[k] < 0;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float2 a = angle_of(r, pos[k], chunk * 8 + k);
      co[k] = a.x, si[k] = a.y;
    }
    turn(x[0], x[1], co, si, r.adjacent);
    float* y = turned + slot * 2 * r.pairs + first;
    st_f4(y, x[0][0], x[0][1], x[0][2], x[0][3]);
    st_f4(y + 4, x[0][4], x[0][5], x[0][6], x[0][7]);
    st_f4(y + apart, x[1][0], x[1][1], x[1][2], x[1][3]);
    st_f4(y + apart + 4, x[1][4], x[1][5], x[1][6], x[1][7]);
  }
  if (off_table) {
    report(c.status, GDN_ERR_POSITION_RANGE);
    pass_keys<DT>(r, at.lo, at.hi, at.t0 - at.base, k0, ksn, b, turned);
  }
  if (at.rec == nullptr) {
    if (threadIdx.x == 0) report(c.status, GDN_ERR_PAGE_RANGE);
    return;
  }
  const uint4 old = threadIdx.x < D ? old_v<D>(at, threadIdx.x) : make_uint4(0, 0, 0, 0);
  const float inv_k = c.k_scale != nullptr ? 1.0f / c.k_scale[h] : 1.0f;
  const float inv_v = c.v_scale != nullptr ? 1.0f / c.v_scale[h] : 1.0f;
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < 2 * pairs * G; i += kThreads) {
    const bool is_v = i >= pairs * G;
    const int u = is_v ? i - pairs * G : i, g = u % G;
    const T* src = is_v ? v0 : k0;
    const int64_t step = is_v ? vsn : ksn;
    quantise_pair<D>(at, is_v, is_v ? inv_v : inv_k, pair0 + u / G, g, code, bad,
                     [&](int slot, float (&x)[2][8]) {
                       const T* p = src + slot * step + g * 16;
                       const float* y = turned + slot * 2 * r.pairs + g * 16;
#pragma unroll
                       for (int k = 0; k < 2; ++k) {
                         if (!is_v && 2 * g + k < 2 * whole) {
#pragma unroll
                           for (int j = 0; j < 8; j += 4) {
                             const float4 f = *reinterpret_cast<const float4*>(y + 8 * k + j);
                             x[k][j] = f.x, x[k][j + 1] = f.y;
                             x[k][j + 2] = f.z, x[k][j + 3] = f.w;
                           }
                         } else {
                           load8<DT>(p + 8 * k, x[k]);
                         }
                       }
                     });
  }
  __syncthreads();
  store_v<D>(at, code, old);
  if (bad) report(c.status, GDN_ERR_NONFINITE);
}

template <int DT, int D>
int append_rotary_d(const gdn_kv4_cache& c, const gdn_rotary& r, const Queries& q, const void* k,
                    const void* v, int64_t ksb, int64_t ksn, int64_t vsb, int64_t vsn, int N,
                    dim3 grid, bool few, cudaStream_t s) {
  const size_t smem = (size_t)kTurnTokens * 2 * r.pairs * sizeof(float);
  return launch_pdl(few ? append_rotary_kernel<DT, D, 3> : append_rotary_kernel<DT, D, 4>, grid,
                    dim3(kThreads), smem, s, c, r, q, k, v, ksb, ksn, vsb, vsn, N);
}

template <int DT>
int append_rotary_dt(const gdn_kv4_cache& c, const gdn_rotary& r, const Queries& q, const void* k,
                     const void* v, int64_t ksb, int64_t ksn, int64_t vsb, int64_t vsn, int N,
                     dim3 grid, bool few, cudaStream_t s) {
  switch (c.D) {
    case 64: return append_rotary_d<DT, 64>(c, r, q, k, v, ksb, ksn, vsb, vsn, N, grid, few, s);
    case 128: return append_rotary_d<DT, 128>(c, r, q, k, v, ksb, ksn, vsb, vsn, N, grid, few, s);
    default: return append_rotary_d<DT, 256>(c, r, q, k, v, ksb, ksn, vsb, vsn, N, grid, few, s);
  }
}

}  // namespace

int launch_kv4_append_rotary(const gdn_kv4_cache& c, const gdn_rotary& r, const void* q, int64_t qsb,
                             int64_t qsn, int Hq, void* q_out, int64_t osb, int64_t osn,
                             const void* k, const void* v, int dtype, int64_t ksb, int64_t ksn,
                             int64_t vsb, int64_t vsn, int N, cudaStream_t s) {
  const int records = touched(N), sms = sm_count();
  if (sms == 0) return GDN_ERR_CUDA;
  // about 2048 items a block of queries, fewer while the blocks do not fill the GPU twice
  const int64_t items = (int64_t)Hq * c.D / 16;
  int tokens = (int)(items >= 2048 ? 1 : 2048 / items);
  if (tokens > kTurnTokens) tokens = kTurnTokens;
  while (tokens > 1 && (int64_t)c.B * ((N + tokens - 1) / tokens) < 2 * sms) tokens /= 2;
  const int64_t blocks = (N + tokens - 1) / tokens, rows = c.Hkv + (blocks + records - 1) / records;
  const dim3 grid(records, (unsigned)rows, c.B);
  const Queries qs = {q, q_out, qsb, qsn, osb, osn, Hq, tokens};
  // blocks of one wave have an SM to three of them at most
  const bool few = (int64_t)records * rows * c.B <= 3 * (int64_t)sms;
  switch (dtype) {
    case GDN_F32:
      return append_rotary_dt<GDN_F32>(c, r, qs, k, v, ksb, ksn, vsb, vsn, N, grid, few, s);
    case GDN_BF16:
      return append_rotary_dt<GDN_BF16>(c, r, qs, k, v, ksb, ksn, vsb, vsn, N, grid, few, s);
    default:
      return append_rotary_dt<GDN_F16>(c, r, qs, k, v, ksb, ksn, vsb, vsn, N, grid, few, s);
  }
}

}  // namespace gdn
