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
  int lo, hi;    // the record's tokens that are the block's
};

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

}  // namespace kv4
}  // namespace gdn
