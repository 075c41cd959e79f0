// Append to the 4-bit key/value cache: quantise a record's tokens on write (include/gdn.h),
// with the keys as they are (gdn_kv4_cache.cu) or turned by their positions first
// (gdn_kv4_rotary.cu).
#pragma once

#include "gdn_common.cuh"
#include "gdn_kv4.cuh"

namespace gdn {
namespace kv4 {

constexpr int kThreads = 256;

// Records that N tokens can touch, whatever the offset of the first.
inline int touched(int N) { return (int)(((int64_t)N + kRec - 2) / kRec + 1); }

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
struct Codes {
  uint32_t w[2];  // 16 codes
  uint32_t scale;
};

// The larger of a and |x|; NaN if either is.
__device__ __forceinline__ float max_abs(float a, float x) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(x)));
  return d;
}

// Quantises 16 values; `bad` is set by a NaN or an infinity.  The product with
// `inv` is monotone, so the largest |x| gives the largest |y|, and only where that
// passes the bound (or is no number) are the values looked at one by one.
__device__ __forceinline__ Codes quantise(float (&x)[2][8], float inv, bool& bad) {
  float a = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) a = max_abs(a, x[j >> 3][j & 7]);
  bad |= !(a <= 3.4028235e38f);
  a *= fabsf(inv);
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j >> 3][j & 7] *= inv;
  if (!(a <= 2688.f)) {
    a = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float y = x[j >> 3][j & 7];
      y = y == y ? fminf(fmaxf(y, -2688.f), 2688.f) : 0.f;
      a = fmaxf(a, fabsf(y));
      x[j >> 3][j & 7] = y;
    }
  }
  Codes c = {{0, 0}, to_e4m3(a * (1.0f / 6.0f))};
  const float s = e4m3((uint8_t)c.scale);
  const float r = s > 0.f ? 1.0f / s : 0.f;
#pragma unroll
  for (int j = 0; j < 16; j += 2)
    c.w[j >> 3] |= to_e2m1x2(x[j >> 3][j & 7] * r, x[j >> 3][(j & 7) + 1] * r) << (4 * (j & 7));
  return c;
}

// 8 codes of two tokens (a word each) as 8 bytes, the first token in the low halves.
__device__ __forceinline__ uint2 pair_bytes(uint32_t a, uint32_t b) {
  const uint32_t even = (a & 0x0f0f0f0fu) | (b & 0x0f0f0f0fu) << 4;   // channels 0, 2, 4, 6
  const uint32_t odd = (a >> 4 & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);    // channels 1, 3, 5, 7
  return make_uint2(__byte_perm(even, odd, 0x5140), __byte_perm(even, odd, 0x7362));
}

// Keys that are stored as they are given.
struct NoTurn {
  template <int DT, typename T>
  __device__ __forceinline__ void apply(float (&)[8], const T*, int, int) const {}
};

// One thread block's record: the `part`-th that the block of N tokens of sequence b touches, of
// head h.  `make` is given what the record holds of the block and returns what turns the keys,
// 8 channels of a token at a time.
template <int DT, int D, typename Turn, typename Make>
__device__ __forceinline__ void append_record(const gdn_kv4_cache& c, const void* __restrict__ kin,
                                              const void* __restrict__ vin, int64_t ksb,
                                              int64_t ksn, int64_t vsb, int64_t vsn, int N, int b,
                                              int h, int part, Make make) {
  constexpr int G = D / 16;  // scale groups
  using T = typename Elem<DT>::T;
  __shared__ __align__(16) uint8_t code[kRec / 2][D];
  const int len = seq_len(c, b, part == 0 && h == 0 && threadIdx.x == 0);
  const int base = len - N;
  const int t0 = ((base > 0 ? base : 0) / kRec + part) * kRec;  // first token here
  if (t0 >= len) return;
  const int lo = base > t0 ? base - t0 : 0, hi = len - t0 < kRec ? len - t0 : kRec;
  uint8_t* rec = record(c, b, h, t0);
  if (rec == nullptr) {
    if (threadIdx.x == 0) report(c.status, GDN_ERR_PAGE_RANGE);
    return;
  }
  const float inv_k = c.k_scale != nullptr ? 1.0f / c.k_scale[h] : 1.0f;
  const float inv_v = c.v_scale != nullptr ? 1.0f / c.v_scale[h] : 1.0f;
  const Turn turn = make(b, t0, base, lo, hi);
  const int pair0 = lo >> 1, pairs = ((hi + 1) >> 1) - pair0;
  bool bad = false;
  for (int i = threadIdx.x; i < 2 * pairs * G; i += kThreads) {
    const bool is_v = i >= pairs * G;
    const int u = is_v ? i - pairs * G : i, pair = pair0 + u / G, g = u % G;
    const T* src = is_v ? static_cast<const T*>(vin) + b * vsb : static_cast<const T*>(kin) + b * ksb;
    const int64_t step = is_v ? vsn : ksn;
    float x[2][2][8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int slot = 2 * pair + t;
      if (slot >= lo && slot < hi) {
        const T* p = src + (int64_t)(t0 + slot - base) * step + (int64_t)h * D + g * 16;
        load8<DT>(p, x[t][0]);
        load8<DT>(p + 8, x[t][1]);
        if (!is_v) {
          turn.template apply<DT>(x[t][0], p, slot, 2 * g);
          turn.template apply<DT>(x[t][1], p + 8, slot, 2 * g + 1);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[t][j >> 3][j & 7] = 0.f;
      }
    }
    Codes q[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      q[t] = quantise(x[t], is_v ? inv_v : inv_k, bad);
      const int slot = 2 * pair + t;
      if (slot < lo || slot >= hi) continue;
      if (is_v) {
        rec[off_vs(D) + g * kRec + slot] = (uint8_t)q[t].scale;
      } else {
        *reinterpret_cast<uint2*>(rec + (g >> 1) * 512 + slot * 16 + (g & 1) * 8) =
            make_uint2(q[t].w[0], q[t].w[1]);
        rec[off_ks(D) + slot * G + g] = (uint8_t)q[t].scale;
      }
    }
    if (is_v) {
      const uint2 first = pair_bytes(q[0].w[0], q[1].w[0]), second = pair_bytes(q[0].w[1], q[1].w[1]);
      *reinterpret_cast<uint4*>(&code[pair][g * 16]) =
          make_uint4(first.x, first.y, second.x, second.y);
    }
  }
  if (bad) report(c.status, GDN_ERR_NONFINITE);
  __syncthreads();
  // nibbles of the block in each word of 8 tokens
  uint32_t mine[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int from = min(max(lo - 8 * w, 0), 8), to = min(max(hi - 8 * w, 0), 8);
    mine[w] = (uint32_t)(((1ull << (4 * to)) - 1) & ~((1ull << (4 * from)) - 1));
  }
  for (int ch = threadIdx.x; ch < D; ch += kThreads) {
    uint4* at = reinterpret_cast<uint4*>(rec + off_v(D) + ch * 16);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = (code[4 * k][ch] | (uint32_t)code[4 * k + 1][ch] << 8 |
              (uint32_t)code[4 * k + 2][ch] << 16 | (uint32_t)code[4 * k + 3][ch] << 24) & mine[k];
    if (lo != 0 || hi != kRec) {
      const uint4 old = *at;
      w[0] |= old.x & ~mine[0], w[1] |= old.y & ~mine[1];
      w[2] |= old.z & ~mine[2], w[3] |= old.w & ~mine[3];
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace kv4
}  // namespace gdn
