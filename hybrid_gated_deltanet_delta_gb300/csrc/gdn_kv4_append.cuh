// Append to the 4-bit key/value cache: quantise a record's tokens on write (include/gdn.h), the
// keys as they are (gdn_kv4_cache.cu) or turned by their positions first (gdn_kv4_rotary.cu).
#pragma once

#include "gdn_common.cuh"
#include "gdn_kv4.cuh"

namespace gdn {
namespace kv4 {

constexpr int kThreads = 256;

// Records that N tokens can touch, whatever the offset of the first.
inline int touched(int N) { return (int)(((int64_t)N + kRec - 2) / kRec + 1); }

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

// What a block of threads appends to: the `part`-th record that the block of N tokens of
// sequence b touches, of head h.
struct Place {
  uint8_t* rec;  // NULL: the page is not there
  int base, t0;  // positions of node 0 and of the record's first token
  int lo, hi;    // the record's tokens that are the block's; none where it touches fewer records
};

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

// Quantises channels 16*g .. of a pair of tokens; `load(slot, x)` brings in one token's.  K goes
// to the record, V's codes to `code`.
template <int D, typename Load>
__device__ __forceinline__ void quantise_pair(const Place& p, bool is_v, float inv, int pair, int g,
                                              uint8_t (*code)[D], bool& bad, Load load) {
  constexpr int G = D / 16;  // scale groups
  float x[2][2][8];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int slot = 2 * pair + t;
    if (slot >= p.lo && slot < p.hi) {
      load(slot, x[t]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[t][j >> 3][j & 7] = 0.f;
    }
  }
  Codes q[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    q[t] = quantise(x[t], inv, bad);
    const int slot = 2 * pair + t;
    if (slot < p.lo || slot >= p.hi) continue;
    if (is_v) {
      p.rec[off_vs(D) + g * kRec + slot] = (uint8_t)q[t].scale;
    } else {
      *reinterpret_cast<uint2*>(p.rec + (g >> 1) * 512 + slot * 16 + (g & 1) * 8) =
          make_uint2(q[t].w[0], q[t].w[1]);
      p.rec[off_ks(D) + slot * G + g] = (uint8_t)q[t].scale;
    }
  }
  if (is_v) {
    const uint2 first = pair_bytes(q[0].w[0], q[1].w[0]), second = pair_bytes(q[0].w[1], q[1].w[1]);
    *reinterpret_cast<uint4*>(&code[pair][g * 16]) =
        make_uint4(first.x, first.y, second.x, second.y);
  }
}

// What a channel's 16 bytes of V codes hold, where the block covers only part of them.
template <int D>
__device__ __forceinline__ uint4 old_v(const Place& p, int ch) {
  return p.lo != 0 || p.hi != kRec ? *reinterpret_cast<const uint4*>(p.rec + off_v(D) + ch * 16)
                                   : make_uint4(0, 0, 0, 0);
}

// V's codes to the record, after a barrier; `old(ch)`: what is there.
template <int D, typename Old>
__device__ __forceinline__ void store_v(const Place& p, const uint8_t (*code)[D], Old old_of) {
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
      const uint4 old = old_of(ch);
      w[0] |= old.x & ~mine[0], w[1] |= old.y & ~mine[1];
      w[2] |= old.z & ~mine[2], w[3] |= old.w & ~mine[3];
    }
    *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace kv4
}  // namespace gdn
