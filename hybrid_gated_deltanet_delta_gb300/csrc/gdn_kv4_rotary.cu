// Append to the 4-bit key/value cache with rotary positions (include/gdn.h): queries and keys
// turned by their positions, the queries written out, the keys quantised as they are written.
//
//   y_i = x_i c - x_j s,   y_j = x_j c + x_i s   for a pair (i, j), each product and the sum
//                                                rounded to fp32
//
// Grid (records a block can touch, Hkv + rows of query blocks, B).  The first Hkv rows append as
// gdn_kv4_append.cuh does, a record a block; a block of the others turns the queries of
// q_tokens tokens, all heads.  Either first gathers its tokens' cosines and sines, which every
// head of a token uses, into shared memory: each pair goes by the position on its own axis.
#include "gdn_common.cuh"
#include "gdn_kv4.cuh"
#include "gdn_kv4_append.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

using namespace kv4;

constexpr int kTurnTokens = kRec;  // tokens whose angles fit in shared memory

// Cosines and sines of `count` tokens from node `node0` of sequence b on: cs[token][2][pairs].
// Those of a node that does not exist are left as they are.
__device__ __forceinline__ void gather_angles(const gdn_rotary& r, int32_t* status, int b,
                                              int node0, int count, int base, float* cs) {
  bool bad = false;
  for (int i = threadIdx.x; i < count * r.pairs; i += kThreads) {
    const int token = i / r.pairs, pair = i - token * r.pairs, node = node0 + token;
    if (base + node < 0) continue;
    const int axis = r.axis != nullptr ? r.axis[pair] : 0;
    const int pos = axis < r.n_axes
                        ? r.positions[axis * r.pos_stride_axis + b * r.pos_stride_b + node]
                        : -1;
    float c = 1.f, s = 0.f;
    if (pos >= 0 && pos < r.n_positions) {
      const float* at = r.cos_sin + 2 * (int64_t)pos * r.pairs + pair;
      c = __ldg(at), s = __ldg(at + r.pairs);
    } else {
      bad = true;
    }
    float* to = cs + 2 * token * r.pairs + pair;
    to[0] = c, to[r.pairs] = s;
  }
  if (bad) report(status, GDN_ERR_POSITION_RANGE);
}

__device__ __forceinline__ float turn_first(float x, float y, float c, float s) {
  return __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}

__device__ __forceinline__ float turn_second(float x, float y, float c, float s) {
  return __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// Turns 8 channels that hold 4 pairs beside each other; cs: cosines from the first pair on.
__device__ __forceinline__ void turn_adjacent(float (&x)[8], const float* cs, int pairs) {
  const float4 c = *reinterpret_cast<const float4*>(cs);
  const float4 s = *reinterpret_cast<const float4*>(cs + pairs);
  const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = x[2 * k], b = x[2 * k + 1];
    x[2 * k] = turn_first(a, b, c4[k], s4[k]);
    x[2 * k + 1] = turn_second(a, b, c4[k], s4[k]);
  }
}

// Turns a record's keys, 8 channels (chunk `c8` of the head's) of a token at a time.
struct KeyTurn {
  const float* cs;  // of token `slot` of the record: cs[slot][2][pairs]
  int pairs, adjacent;

  template <int DT, typename T>
  __device__ __forceinline__ void apply(float (&x)[8], const T* p, int slot, int c8) const {
    const float* at = cs + 2 * slot * pairs;
    const int whole = pairs >> 3;  // chunks of a half
    if (c8 >= 2 * whole) return;
    if (adjacent) {
      turn_adjacent(x, at + 4 * c8, pairs);
      return;
    }
    const bool first = c8 < whole;
    float y[8];
    load8<DT>(first ? p + pairs : p - pairs, y);
    at += (first ? c8 : c8 - whole) * 8;
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      const float4 c = *reinterpret_cast<const float4*>(at + k);
      const float4 s = *reinterpret_cast<const float4*>(at + pairs + k);
      const float c4[4] = {c.x, c.y, c.z, c.w}, s4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[k + j] = first ? turn_first(x[k + j], y[k + j], c4[j], s4[j])
                         : turn_second(y[k + j], x[k + j], c4[j], s4[j]);
    }
  }
};

// 8 elements at p (16-byte aligned) from fp32.
template <int DT>
__device__ __forceinline__ void store8(void* p, const float (&x)[8]) {
  if constexpr (DT == GDN_F32) {
    st_f4(static_cast<float*>(p), x[0], x[1], x[2], x[3]);
    st_f4(static_cast<float*>(p) + 4, x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = Elem<DT>::from(x[2 * k]) | (uint32_t)Elem<DT>::from(x[2 * k + 1]) << 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

struct Queries {
  const void* in;
  void* out;
  int64_t in_b, in_n, out_b, out_n;
  int Hq, tokens;  // tokens: of a block
};

// 8 elements that this thread alone writes, if anyone does (the queries may be turned in place).
template <int DT>
__device__ __forceinline__ void load8_own(const void* p, float (&x)[8]) {
  if constexpr (DT == GDN_F32) {
    const float4 a = *static_cast<const float4*>(p), b = *(static_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 u = *static_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (DT == GDN_BF16)
        f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      else
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
}

// An item is two chunks of 8 channels of one head: two that hold 8 pairs, or two that pass.  In
// place only the former are touched (and, of a node that does not exist, all).
template <int DT, int D>
__device__ __forceinline__ void turn_queries(const gdn_kv4_cache& c, const gdn_rotary& r,
                                             const Queries& q, int N, int b, int block, float* cs) {
  using T = typename Elem<DT>::T;
  const int node0 = block * q.tokens;
  if (node0 >= N) return;
  const int count = min(q.tokens, N - node0), base = seq_len(c, b, false) - N;
  gather_angles(r, c.status, b, node0, count, base, cs);
  __syncthreads();
  const int whole = r.pairs >> 3;
  const bool in_place = q.in == q.out;
  const int items = in_place ? whole : D / 16, total = count * q.Hq * items;
  const T* in = static_cast<const T*>(q.in) + b * q.in_b;
  T* out = static_cast<T*>(q.out) + b * q.out_b;
  constexpr int U = DT == GDN_F32 ? 1 : 2;  // items in flight
  for (int i0 = threadIdx.x; i0 < total; i0 += U * kThreads) {
    float x[U][2][8];
    int token[U], at[U], first[U], second[U], item[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u * kThreads, total - 1), row = i / items;
      item[u] = i - row * items;
      token[u] = row / q.Hq;
      at[u] = (row - token[u] * q.Hq) * D;
      const bool apart = !r.adjacent && item[u] < whole;
      first[u] = apart ? item[u] * 8 : item[u] * 16;
      second[u] = apart ? first[u] + r.pairs : first[u] + 8;
      const T* p = in + (int64_t)(node0 + token[u]) * q.in_n + at[u];
      load8_own<DT>(p + first[u], x[u][0]);
      load8_own<DT>(p + second[u], x[u][1]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * kThreads >= total) break;
      const float* angle = cs + 2 * token[u] * r.pairs;
      if (base + node0 + token[u] < 0) {
#pragma unroll
        for (int k = 0; k < 16; ++k) x[u][k >> 3][k & 7] = 0.f;
      } else if (item[u] < whole) {
        if (r.adjacent) {
          turn_adjacent(x[u][0], angle + 8 * item[u], r.pairs);
          turn_adjacent(x[u][1], angle + 8 * item[u] + 4, r.pairs);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float cc = angle[8 * item[u] + k], ss = angle[r.pairs + 8 * item[u] + k];
            const float a = x[u][0][k], d = x[u][1][k];
            x[u][0][k] = turn_first(a, d, cc, ss);
            x[u][1][k] = turn_second(a, d, cc, ss);
          }
        }
      }
      T* p = out + (int64_t)(node0 + token[u]) * q.out_n + at[u];
      store8<DT>(p + first[u], x[u][0]);
      store8<DT>(p + second[u], x[u][1]);
    }
  }
  if (in_place && base + node0 < 0) {
    const float zero[8] = {};
    const int rest = D / 8 - 2 * whole, missing = min(count, -(base + node0));
    for (int i = threadIdx.x; i < missing * q.Hq * rest; i += kThreads) {
      const int row = i / rest, tok = row / q.Hq;
      store8<DT>(out + (int64_t)(node0 + tok) * q.out_n + (row - tok * q.Hq) * D +
                     (2 * whole + i - row * rest) * 8, zero);
    }
  }
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 3)
append_rotary_kernel(const __grid_constant__ gdn_kv4_cache c, const __grid_constant__ gdn_rotary r,
                     const __grid_constant__ Queries q, const void* __restrict__ kin,
                     const void* __restrict__ vin, int64_t ksb, int64_t ksn, int64_t vsb,
                     int64_t vsn, int N) {
  extern __shared__ __align__(16) float cs[];
  pdl_enter();
  const int b = blockIdx.z, h = blockIdx.y;
  if (h >= c.Hkv) {
    turn_queries<DT, D>(c, r, q, N, b, (h - c.Hkv) * gridDim.x + blockIdx.x, cs);
    return;
  }
  append_record<DT, D, KeyTurn>(
      c, kin, vin, ksb, ksn, vsb, vsn, N, b, h, blockIdx.x,
      [&](int, int t0, int base, int lo, int hi) {
        gather_angles(r, c.status, b, t0 + lo - base, hi - lo, base, cs + 2 * lo * r.pairs);
        __syncthreads();
        return KeyTurn{cs, r.pairs, r.adjacent};
      });
}

template <int DT>
int append_rotary_d(const gdn_kv4_cache& c, const gdn_rotary& r, const Queries& q, const void* k,
                    const void* v, int64_t ksb, int64_t ksn, int64_t vsb, int64_t vsn, int N,
                    dim3 grid, cudaStream_t s) {
  const size_t smem = (size_t)kTurnTokens * 2 * r.pairs * sizeof(float);
  switch (c.D) {
    case 64:
      return launch_pdl(append_rotary_kernel<DT, 64>, grid, dim3(kThreads), smem, s, c, r, q, k, v,
                        ksb, ksn, vsb, vsn, N);
    case 128:
      return launch_pdl(append_rotary_kernel<DT, 128>, grid, dim3(kThreads), smem, s, c, r, q, k, v,
                        ksb, ksn, vsb, vsn, N);
    default:
      return launch_pdl(append_rotary_kernel<DT, 256>, grid, dim3(kThreads), smem, s, c, r, q, k, v,
                        ksb, ksn, vsb, vsn, N);
  }
}

}  // namespace

int launch_kv4_append_rotary(const gdn_kv4_cache& c, const gdn_rotary& r, const void* q, int64_t qsb,
                             int64_t qsn, int Hq, void* q_out, int64_t osb, int64_t osn,
                             const void* k, const void* v, int dtype, int64_t ksb, int64_t ksn,
                             int64_t vsb, int64_t vsn, int N, cudaStream_t s) {
  const int records = touched(N), sms = sm_count();
  if (sms == 0) return GDN_ERR_CUDA;
  // about 1024 items a block of queries, fewer while the blocks do not fill the GPU twice
  const int64_t items = (int64_t)Hq * c.D / 16;
  int tokens = (int)(items >= 1024 ? 1 : 1024 / items);
  if (tokens > kTurnTokens) tokens = kTurnTokens;
  while (tokens > 1 && (int64_t)c.B * ((N + tokens - 1) / tokens) < 2 * sms) tokens /= 2;
  const int64_t blocks = (N + tokens - 1) / tokens, rows = c.Hkv + (blocks + records - 1) / records;
  if (rows > 65535) return GDN_ERR_UNSUPPORTED;
  const dim3 grid(records, (unsigned)rows, c.B);
  const Queries qs = {q, q_out, qsb, qsn, osb, osn, Hq, tokens};
  switch (dtype) {
    case GDN_F32:
      return append_rotary_d<GDN_F32>(c, r, qs, k, v, ksb, ksn, vsb, vsn, N, grid, s);
    case GDN_BF16:
      return append_rotary_d<GDN_BF16>(c, r, qs, k, v, ksb, ksn, vsb, vsn, N, grid, s);
    default:
      return append_rotary_d<GDN_F16>(c, r, qs, k, v, ksb, ksn, vsb, vsn, N, grid, s);
  }
}

}  // namespace gdn
