// Attention over the 4-bit key/value cache on the fifth-generation tensor cores
// (include/gdn.h; instantiated per head size by gdn_kv4_attn_*.cu).
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q.k_j - m),  c = scale * k_scale * log2 e
//
// evaluated in one pass over the cache with a running reference m per query
// row.  The products are turned round: 128 cached positions are the M rows of
//     S^T [128 positions x rows] = K [128 x D] Q^T [D x rows]
// and the channels are the M rows of
//     O^T [D x rows] += V^T [D x 128] P^T [128 x rows],
// so the 4-bit operand is always the A operand, which tcgen05.mma takes from
// tensor memory: a dequantised value goes from a register straight into TMEM
// and never into shared memory, and the N extent is the number of query rows
// (nodes x heads of the group), from 16 for a decoded token to 96 for a block.
//
// Work.  The tiles of 128 positions of all (sequence, kv head, row tile) items
// are laid end to end and cut into one equal run per block (the block reads
// the lengths itself; the grid depends on the device alone).  A block whose run
// starts or ends inside an item writes that part's O, m and l to the workspace,
// and join_kernel adds the parts in block order; whole items are written at once.
//
// Warps of a block (20), connected by mbarriers only:
//   0-3    K: position = TMEM lane; codes * scale -> binary16 -> TMEM (64 channels a unit)
//   4-7    V: channel = TMEM lane; the same for V^T (32 positions a unit)
//   8-15   softmax, two groups of four, each half of the rows: S^T from TMEM, p to
//          shared memory (B operand), sums in registers, and the item's epilogue
//   16     issues the MMAs        17   bulk copies of records, V scales to binary16
//   18-19  query rows: to binary16, scaled by a power of two per row so that
//          any bf16 magnitude fits, into the B operand's swizzled layout
//
// The reference m is moved only when some p would pass 2^8 (p is at most 65504
// in binary16): the sums and O^T are then multiplied by 2^(old - new), which
// happens on an item's first tile and seldom later, so the usual tile takes
// one FMA, one maximum, one exp2 and one addition per logit and no reduction
// across lanes.  p is rounded to binary16 for the product (2^-11; bf16 would
// give 2^-8); code * scale needs 6 significand bits, so K and V are exact.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "gdn_common.cuh"
#include "gdn_kv4.cuh"
#include "gdn_kv4_attn.h"
#include "gdn_tc.cuh"

namespace gdn {
namespace kv4 {

constexpr int kTile = 128;  // positions of a tile: four records
constexpr int kAttnThreads = 640;
constexpr float kNone = -1e30f;      // reference of a row that has seen nothing
constexpr float kSlack = 8.f;        // log2 of the largest p before m moves
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWaitPolls = 1 << 20;  // bound of every wait

template <int D_, int NT_>
struct AttnCfg {
  static constexpr int D = D_, NT = NT_;
  static constexpr int MB = D == 256 ? 2 : 1;  // 128-channel blocks of O^T
  static constexpr int NH = NT / 2;            // rows of a softmax group
  static constexpr int UNITS = D / 64;         // K units of a tile
  // TMEM columns: K ring, two S^T, O^T, V ring.  The widest case keeps two
  // stages per ring so that S^T can be double buffered.
  static constexpr int KU = 3 * NT + 128 + 64 * MB > 512 - (MB - 1) * NT ? 2 : 4;
  static constexpr int VU = KU;
  static constexpr int cS = 32 * KU, cO = cS + 2 * NT, cV = cO + MB * NT;
  static_assert(cV + VU * 16 * MB <= 512, "TMEM");
  // shared memory
  static constexpr int RAW = 4 * rec_bytes(D);
  static constexpr int QB = NT * D * 2;
  static constexpr int PB = (NT > 64 ? 2 : 1) * kTile * 128;
  static constexpr int VSG = 272;  // bytes between the scale rows of two groups (bank offset)
  static constexpr int VSB = D / 16 * VSG;
  static constexpr int LS = NT * 129 * 4;  // row sums of every lane, over the P buffers
  static constexpr int P2 = 2 * PB > LS ? 2 * PB : (LS + 1023) / 1024 * 1024;
  static constexpr int ROOM = 224 * 1024 - P2 - 2 * VSB - 4096;
  static constexpr int NQ = ROOM - 2 * QB >= 2 * RAW ? 2 : 1;
  static constexpr int NRAW = (ROOM - NQ * QB) / RAW > 4 ? 4 : (ROOM - NQ * QB) / RAW;
  static_assert(NRAW >= 2, "stages");
  static constexpr int oQ = 0, oP = oQ + NQ * QB, oRaw = oP + P2, oVS = oRaw + NRAW * RAW;
  static constexpr int oEnd = oVS + 2 * VSB;
  static constexpr int SMEM = oEnd + 1024;  // + alignment of the swizzled operands
};

struct Row {       // of a query row, beside its operand
  float c;         // logit of S: c * S (log2 units)
  float pad;
  unsigned lo, hi; // chain: node in lo; tree: the positions of the block it sees
};

template <typename C>
struct AttnShared {
  uint64_t raw_full[C::NRAW], raw_empty[C::NRAW];
  uint64_t k_full[C::KU], k_empty[C::KU], v_full[C::VU], v_empty[C::VU];
  uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], vs_full[2], vs_empty[2];
  uint64_t q_full[C::NQ], q_empty[C::NQ], row_full[2], row_empty[2], o_full, o_empty, drain;
  uint32_t tmem;
  int dead;
  AttnSpan span;
  int tile_ok[8];  // records of a tile that could be read, by tile number
  alignas(16) float2 cm[C::NT];  // (c, m) of the rows in work; read two rows a load
  float alpha[C::NT], inv[C::NT];
  float wmax[4][C::NT];
  Row row[2][C::NT];
};

// A wait that ends: false once any wait of the block has run out.
__device__ __forceinline__ bool attn_wait(uint64_t* bar, unsigned parity, volatile int* dead) {
  for (int i = 0; i < kWaitPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && *dead) return false;
  }
  *dead = 1;
  return false;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_addr(bar)) : "memory");
}

// tcgen05.mma kind::f16 with A in TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// binary16 operands, fp32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16, "columns");
  if constexpr (N == 8) tc::tmem_ld8(addr, r);
  else tc::tmem_ld16(addr, r);
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float first, float second) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(second), "f"(first));
  return d;
}

// 8 codes (one word) times the scale pair(s): four f16x2 words.
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t s, uint32_t* out) {
  out[0] = hmul2(e2m1x2<0>(w), s);
  out[1] = hmul2(e2m1x2<1>(w), s);
  out[2] = hmul2(e2m1x2<2>(w), s);
  out[3] = hmul2(e2m1x2<3>(w), s);
}

// Maximum over the warp (NaN wins over every number).
__device__ __forceinline__ float warp_max(float x) {
  int i = __float_as_int(x);
  i ^= (i >> 31) & 0x7fffffff;
  i = __reduce_max_sync(0xffffffffu, i);
  i ^= (i >> 31) & 0x7fffffff;
  return __int_as_float(i);
}

// ---------------------------------------------------------------- segments
// The part of one item that a block works on: tiles [t0, t1) of `tiles`.
struct Seg {
  int b, h, rt, t0, t1, tiles;
  int len, rows, n_lo, n_hi;
};

__device__ __forceinline__ bool attn_tree_bad(const AttnArgs& a, int b) {
  return a.parent != nullptr && !tree_ok(a.parent + (int64_t)b * a.N, a.N);
}

// Length of sequence b as attention counts it (0: skipped).
__device__ __forceinline__ int attn_len(const AttnArgs& a, int b, bool report_it) {
  const int n = seq_len(a.c, b, report_it);
  if (n > 0 && attn_tree_bad(a, b)) {
    if (report_it) report(a.c.status, GDN_ERR_BAD_TREE);
    return 0;
  }
  return n;
}

// Tiles that row tile `rt` of a sequence of `len` positions sees.
__device__ __forceinline__ int attn_tiles(const AttnArgs& a, int len, int rt) {
  int see = len;
  if (a.parent == nullptr) {
    int last = (rt + 1) * a.rows_per_tile - 1;
    if (last >= a.rows_total) last = a.rows_total - 1;
    see = len - a.N + last / a.G + 1;
  }
  return see <= 0 ? 0 : (see + kTile - 1) / kTile;
}

__device__ __forceinline__ int64_t attn_cost(const AttnArgs& a, int len) {
  int64_t t = 0;
  for (int rt = 0; rt < a.row_tiles; ++rt) t += attn_tiles(a, len, rt);
  return t * a.c.Hkv;
}

__device__ __forceinline__ void seg_rows(const AttnArgs& a, Seg& s) {
  const int first = s.rt * a.rows_per_tile;
  s.rows = a.rows_total - first < a.rows_per_tile ? a.rows_total - first : a.rows_per_tile;
  s.n_lo = first / a.G;
  s.n_hi = (first + s.rows - 1) / a.G;
}

// First segment of the block's run; false when the run is empty.
__device__ __forceinline__ bool seg_first(const AttnArgs& a, const AttnSpan& sp, Seg& s,
                                          int64_t& left) {
  left = sp.count;
  if (left <= 0) return false;
  s.b = sp.b, s.h = sp.h, s.rt = sp.rt, s.t0 = sp.t0;
  s.len = attn_len(a, s.b, false);
  s.tiles = attn_tiles(a, s.len, s.rt);
  s.t1 = s.t0 + left < s.tiles ? s.t0 + (int)left : s.tiles;
  left -= s.t1 - s.t0;
  seg_rows(a, s);
  return true;
}

__device__ __forceinline__ bool seg_next(const AttnArgs& a, Seg& s, int64_t& left) {
  if (left <= 0) return false;
  do {
    if (++s.rt == a.row_tiles) {
      s.rt = 0;
      if (++s.h == a.c.Hkv) {
        s.h = 0;
        if (++s.b >= a.c.B) return false;
        s.len = attn_len(a, s.b, false);
      }
    }
    s.tiles = attn_tiles(a, s.len, s.rt);
  } while (s.tiles == 0);
  s.t0 = 0;
  s.t1 = left < s.tiles ? (int)left : s.tiles;
  left -= s.t1;
  seg_rows(a, s);
  return true;
}

// The run of block `part` of `parts`, found by one warp: every sequence's tiles
// are summed, then the one that holds the run's first tile is taken apart.
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs& a, int part, int parts,
                                              bool report_it) {
  const int lane = threadIdx.x & 31;
  int64_t total = 0;
  for (int b0 = 0; b0 < a.c.B; b0 += 32) {
    const int b = b0 + lane;
    int64_t x = b < a.c.B ? attn_cost(a, attn_len(a, b, report_it)) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    total += x;
  }
  AttnSpan sp = {};
  if (parts > total) parts = (int)total;  // no empty runs in between
  if (part >= parts) return sp;
  const int64_t start = total * part / parts, end = total * (part + 1) / parts;
  sp.count = end - start;
  int64_t before = 0;
  for (int b0 = 0; b0 < a.c.B; b0 += 32) {
    const int b = b0 + lane;
    const int64_t mine = b < a.c.B ? attn_cost(a, attn_len(a, b, false)) : 0;
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + x > start);
    if (hit != 0) {
      const int l = __ffs(hit) - 1;
      const int64_t upto = __shfl_sync(0xffffffffu, x, l), its = __shfl_sync(0xffffffffu, mine, l);
      int64_t in = start - before - (upto - its);
      sp.b = b0 + l;
      const int64_t per_head = its / a.c.Hkv;
      sp.h = (int)(in / per_head);
      in -= sp.h * per_head;
      const int len = attn_len(a, sp.b, false);
      for (sp.rt = 0;; ++sp.rt) {
        const int t = attn_tiles(a, len, sp.rt);
        if (in < t) break;
        in -= t;
      }
      sp.t0 = (int)in;
      return sp;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  return sp;
}

// ---------------------------------------------------------------- the kernel
template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = AttnCfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnShared<C> sh;
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* dead = &sh.dead;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NRAW; ++i) mbar_init(&sh.raw_full[i], 1), mbar_init(&sh.raw_empty[i], 9);
    for (int i = 0; i < C::KU; ++i) mbar_init(&sh.k_full[i], 4), mbar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < C::VU; ++i) mbar_init(&sh.v_full[i], 4), mbar_init(&sh.v_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1), mbar_init(&sh.s_empty[i], 8);
      mbar_init(&sh.p_full[i], 8), mbar_init(&sh.p_empty[i], 1);
      mbar_init(&sh.vs_full[i], 1), mbar_init(&sh.vs_empty[i], 4);
      mbar_init(&sh.row_full[i], 2), mbar_init(&sh.row_empty[i], 8);
    }
    for (int i = 0; i < C::NQ; ++i) mbar_init(&sh.q_full[i], 2), mbar_init(&sh.q_empty[i], 1);
    mbar_init(&sh.o_full, 1);
    mbar_init(&sh.o_empty, 8);
    mbar_init(&sh.drain, 1);
    sh.dead = 0;
    mbar_init_fence();
  }
  if (warp == 16) tc::tmem_alloc(&sh.tmem, 512);
  pdl_enter();
  if (warp == 17) {
    const AttnSpan sp = attn_span(a, blockIdx.x, gridDim.x, blockIdx.x == 0);
    if (lane == 0) sh.span = sp;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const AttnSpan span = sh.span;
  Seg s;
  int64_t left;
  bool on = seg_first(a, span, s, left);

  if (warp < 4) {
    // ------------------------------------------------ K -> TMEM
    const uint32_t dst = tmem + ((uint32_t)(warp * 32) << 16);
    int stage = 0, unit = 0;
    unsigned raw_ph = 0, unit_ph = 1;  // an empty ring's first pass does not wait
    for (; on; on = seg_next(a, s, left)) {
      for (int t = s.t0; t < s.t1; ++t) {
        attn_wait(&sh.raw_full[stage], raw_ph, dead);
        const uint8_t* rec = smem + C::oRaw + stage * C::RAW + warp * rec_bytes(D);
        uint32_t s8[D / 64];
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          s8[i] = reinterpret_cast<const uint32_t*>(rec + off_ks(D) + lane * (D / 16))[i];
#pragma unroll
        for (int u = 0; u < C::UNITS; ++u) {
          uint32_t w[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(rec + (2 * u + half) * 512 + lane * 16);
            const uint32_t sc = e4m3x2(s8[u] >> (16 * half));
            const uint32_t s0 = __byte_perm(sc, sc, 0x1010), s1 = __byte_perm(sc, sc, 0x3232);
            dequant8(q4.x, s0, w + 16 * half);
            dequant8(q4.y, s0, w + 16 * half + 4);
            dequant8(q4.z, s1, w + 16 * half + 8);
            dequant8(q4.w, s1, w + 16 * half + 12);
          }
          attn_wait(&sh.k_empty[unit], unit_ph, dead);
          tc::fence_after_sync();
          tmem_st16(dst + unit * 32, w);
          tmem_st16(dst + unit * 32 + 16, w + 16);
          tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.k_full[unit]);
          if (++unit == C::KU) unit = 0, unit_ph ^= 1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.raw_empty[stage]);
        if (++stage == C::NRAW) stage = 0, raw_ph ^= 1;
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------ V^T -> TMEM
    const int quarter = warp - 4;
    const uint32_t dst = tmem + ((uint32_t)(quarter * 32) << 16) + C::cV;
    int stage = 0, unit = 0, vb = 0;
    unsigned vs_ph = 0, unit_ph = 1;
    for (; on; on = seg_next(a, s, left)) {
      for (int t = s.t0; t < s.t1; ++t) {
        attn_wait(&sh.vs_full[vb], vs_ph, dead);  // the records have landed before
        const uint8_t* raw = smem + C::oRaw + stage * C::RAW;
        const uint8_t* vs = smem + C::oVS + vb * C::VSB;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint32_t w[C::MB][16];
#pragma unroll
          for (int mb = 0; mb < C::MB; ++mb) {
            const int ch = mb * 128 + quarter * 32 + lane;
            if (D >= 128 || ch < D) {
              const uint4 q4 =
                  *reinterpret_cast<const uint4*>(raw + r * rec_bytes(D) + off_v(D) + ch * 16);
              const uint4* sp = reinterpret_cast<const uint4*>(vs + (ch >> 4) * C::VSG + r * 64);
              const uint32_t c4[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint4 s4 = sp[i];
                w[mb][4 * i] = hmul2(e2m1x2<0>(c4[i]), s4.x);
                w[mb][4 * i + 1] = hmul2(e2m1x2<1>(c4[i]), s4.y);
                w[mb][4 * i + 2] = hmul2(e2m1x2<2>(c4[i]), s4.z);
                w[mb][4 * i + 3] = hmul2(e2m1x2<3>(c4[i]), s4.w);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) w[mb][i] = 0;
            }
          }
          attn_wait(&sh.v_empty[unit], unit_ph, dead);
          tc::fence_after_sync();
#pragma unroll
          for (int mb = 0; mb < C::MB; ++mb)
            tmem_st16(dst + unit * 16 * C::MB + mb * 16, w[mb]);
          tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.v_full[unit]);
          if (++unit == C::VU) unit = 0, unit_ph ^= 1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.raw_empty[stage]), mbar_arrive(&sh.vs_empty[vb]);
        if (++stage == C::NRAW) stage = 0;
        if (++vb == 2) vb = 0, vs_ph ^= 1;
      }
    }
  } else if (warp < 16) {
    // ------------------------------------------------ softmax and epilogue
    const int group = (warp - 8) >> 2, quarter = warp & 3;
    const int c0 = group * C::NH;                  // first row of the group
    const int gt = (threadIdx.x - 256) & 127;      // thread of the group
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    constexpr int CH = C::NH < 16 ? C::NH : 16;    // columns of one load
    int tile = 0, seg_no = 0;
    for (; on; on = seg_next(a, s, left), ++seg_no) {
      const int base = s.len - a.N;
      const Row* rows = sh.row[seg_no & 1];
      attn_wait(&sh.row_full[seg_no & 1], (seg_no >> 1) & 1, dead);
      float l[C::NH];
#pragma unroll
      for (int i = 0; i < C::NH; ++i) l[i] = 0.f;
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        const int buf = tile & 1;
        const unsigned ph = (tile >> 1) & 1;
        attn_wait(&sh.s_full[buf], ph, dead);
        tc::fence_after_sync();
        if (t == s.t0) {  // the rows' scales came with the queries
          if (gt < C::NH) sh.cm[c0 + gt] = make_float2(rows[c0 + gt].c, kNone);
          tc::named_barrier(1 + group, 128);
        }
        attn_wait(&sh.p_empty[buf], ph ^ 1, dead);
        const int ok = sh.tile_ok[tile & 7];
        const int pos = t * kTile + quarter * 32 + lane, u = pos - base;
        // every row sees the whole tile?
        const bool masked = ok != 15 || (a.parent != nullptr ? t * kTile + kTile > base
                                                             : t * kTile + kTile - 1 > base + s.n_lo);
        const bool gone = !((ok >> quarter) & 1);
        const uint32_t sa = lane_base + C::cS + buf * C::NT + c0;
        uint8_t* prow = smem + C::oP + buf * C::PB + (quarter * 32 + lane) * 128;
        auto hidden = [&](int r) {
          if (gone) return true;
          const Row& w = rows[c0 + r];
          if (a.parent == nullptr) return u > (int)w.lo;
          if (u < 0) return false;
          return u >= 64 || !(((u < 32 ? w.lo : w.hi) >> (u & 31)) & 1);
        };
        // p of all rows with the present references, sums updated; returns the
        // largest exponent seen
        auto pass = [&](bool mask) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < C::NH; k += CH) {
            uint32_t x[CH];
            tmem_load(sa + k, x);
            tc::tmem_wait_ld(x);
            uint32_t p[CH / 2];
#pragma unroll
            for (int i = 0; i < CH; i += 2) {
              const float4 cm = *reinterpret_cast<const float4*>(&sh.cm[c0 + k + i]);
              float y0 = fmaf(__uint_as_float(x[i]), cm.x, -cm.y);
              float y1 = fmaf(__uint_as_float(x[i + 1]), cm.z, -cm.w);
              if (mask) {
                if (hidden(k + i)) y0 = -INFINITY;
                if (hidden(k + i + 1)) y1 = -INFINITY;
              }
              top = fmaxf(top, fmaxf(y0, y1));
              y0 = exp2_fast(y0);
              y1 = exp2_fast(y1);
              l[k + i] += y0;
              l[k + i + 1] += y1;
              p[i / 2] = pack_f16x2(y0, y1);
            }
#pragma unroll
            for (int i = 0; i < CH / 8; ++i) {
              const int col = c0 + k + 8 * i;  // 16-byte chunk of 8 rows, swizzled by position
              uint8_t* at = prow + (col >> 6) * (kTile * 128) +
                            ((((col & 63) >> 3) ^ (lane & 7)) << 4);
              *reinterpret_cast<uint4*>(at) =
                  make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
            }
          }
          return top;
        };
        // takes back what pass() added (a row whose p overflowed held less than
        // 2^-24 of what is to come)
        auto undo = [&](bool mask) {
#pragma unroll
          for (int k = 0; k < C::NH; k += CH) {
            uint32_t x[CH];
            tmem_load(sa + k, x);
            tc::tmem_wait_ld(x);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              const float2 cm = sh.cm[c0 + k + i];
              float y = fmaf(__uint_as_float(x[i]), cm.x, -cm.y);
              if (mask && hidden(k + i)) y = -INFINITY;
              l[k + i] = y > 100.f ? 0.f : l[k + i] - exp2_fast(y);
            }
          }
        };
        // new references: the largest logit so far
        auto raise = [&](bool mask, bool first) {
#pragma unroll
          for (int k = 0; k < C::NH; k += CH) {
            uint32_t x[CH];
            tmem_load(sa + k, x);
            tc::tmem_wait_ld(x);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              float y = __uint_as_float(x[i]) * sh.cm[c0 + k + i].x;
              if (mask && hidden(k + i)) y = -INFINITY;
              y = warp_max(y);
              if (lane == 0) sh.wmax[quarter][c0 + k + i] = y;
            }
          }
          tc::named_barrier(1 + group, 128);
          if (gt < C::NH) {
            const int r = c0 + gt;
            const float old = sh.cm[r].y;
            float m = old;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float w = sh.wmax[q][r];
              m = w > m || w != w ? w : m;
            }
            sh.cm[r].y = m;
            sh.alpha[r] = exp2_fast(old - m);
          }
          tc::named_barrier(1 + group, 128);
          if (!first) {
            // every product into O^T so far is done: the last one freed its P
            attn_wait(&sh.p_empty[buf ^ 1], ((tile - 1) >> 1) & 1, dead);
            tc::fence_after_sync();
#pragma unroll
            for (int k = 0; k < C::NH; ++k) l[k] *= sh.alpha[c0 + k];
            for (int mb = 0; mb < C::MB; ++mb) {
#pragma unroll
              for (int k = 0; k < C::NH; k += 8) {
                const uint32_t oa = lane_base + C::cO + mb * C::NT + c0 + k;
                uint32_t x[8];
                tc::tmem_ld8(oa, x);
                tc::tmem_wait_ld(x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  x[i] = __float_as_uint(__uint_as_float(x[i]) * sh.alpha[c0 + k + i]);
                tmem_st8(oa, x);
              }
            }
            tmem_wait_st();
          }
        };
        const bool first = t == s.t0;
        if (first) raise(masked, true);
        float top = masked ? pass(true) : pass(false);
        if (!first) {
          // NaN logits keep their row NaN and do not count here
          unsigned over = top > kSlack, any;
          asm volatile(
              "{.reg .pred p, q; setp.ne.u32 p, %1, 0;"
              " barrier.cta.red.or.pred q, %2, 128, p; selp.u32 %0, 1, 0, q;}"
              : "=r"(any)
              : "r"(over), "r"(1 + group)
              : "memory");
          if (any) {
            undo(masked);
            raise(masked, false);
            pass(masked);
          }
        }
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.s_empty[buf]), mbar_arrive(&sh.p_full[buf]);
      }
      if (lane == 0) mbar_arrive(&sh.row_empty[seg_no & 1]);
      // ---- epilogue
      const bool whole = s.t0 == 0 && s.t1 == s.tiles;
      attn_wait(&sh.o_full, seg_no & 1, dead);
      tc::fence_after_sync();
      float* sums = reinterpret_cast<float*>(smem + C::oP) + c0 * 129;  // P is free now
#pragma unroll
      for (int k = 0; k < C::NH; ++k) sums[k * 129 + gt] = l[k];
      tc::named_barrier(1 + group, 128);
      const int64_t slot = 2 * (int64_t)blockIdx.x + (seg_no > 0);
      const int row0 = s.rt * a.rows_per_tile;
      if (gt < C::NH) {
        const int r = c0 + gt;
        float total = 0.f;
#pragma unroll 8
        for (int i = 0; i < 128; ++i) total += sums[gt * 129 + i];
        const float m = sh.cm[r].y;
        if (whole) {
          const float vsc = a.c.v_scale != nullptr ? a.c.v_scale[s.h] : 1.f;
          sh.inv[r] = total != 0.f ? vsc / total : 0.f;
          if (a.lse != nullptr && r < s.rows) {
            const int n = (row0 + r) / a.G, g = (row0 + r) % a.G;
            a.lse[((int64_t)s.b * a.N + n) * a.Hq + s.h * a.G + g] =
                total != 0.f ? (m + log2f(total)) * 0.6931471805599453f : -INFINITY;
          }
        } else {
          a.part_ml[slot * NT + r] = make_float2(m, total);
          sh.inv[r] = 1.f;
        }
      }
      tc::named_barrier(3, 256);  // both groups' sums are read: P may be written again
      for (int mb = 0; mb < C::MB; ++mb) {
        const int ch = mb * 128 + quarter * 32 + lane;
#pragma unroll
        for (int k = 0; k < C::NH; k += 8) {
          if (c0 + k >= s.rows) break;
          uint32_t x[8];
          tc::tmem_ld8(lane_base + C::cO + mb * C::NT + c0 + k, x);
          tc::tmem_wait_ld(x);
          if (ch >= D) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = c0 + k + i;
            if (r >= s.rows) break;
            const float o = __uint_as_float(x[i]) * sh.inv[r];
            if (whole) {
              const int n = (row0 + r) / a.G, g = (row0 + r) % a.G;
              const int64_t at = (((int64_t)s.b * a.N + n) * a.Hq + s.h * a.G + g) * D + ch;
              static_cast<uint16_t*>(a.o)[at] =
                  a.bf16 ? Elem<GDN_BF16>::from(o) : Elem<GDN_F16>::from(o);
            } else {
              a.part_o[(slot * NT + r) * D + ch] = o;
            }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_empty);
    }
  } else if (warp == 16) {
    // ------------------------------------------------ MMA issue
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f16(NT, false), id_o = idesc_f16(NT, true);
      const uint32_t q0 = smem_addr(smem + C::oQ), p0 = smem_addr(smem + C::oP);
      int ku = 0, vu = 0, s_tile = 0, o_tile = 0, qs = 0, seg_no = 0;
      unsigned ku_ph = 0, vu_ph = 0, q_ph = 0;
      // S^T of the next tile; `fresh`: the first of a segment, `last`: its queries are done with
      auto issue_s = [&](bool fresh, bool last) {
        const int buf = s_tile & 1;
        if (fresh) attn_wait(&sh.q_full[qs], q_ph, dead);
        attn_wait(&sh.s_empty[buf], ((s_tile >> 1) & 1) ^ 1, dead);
        const uint32_t q = q0 + qs * C::QB;
#pragma unroll 1
        for (int u = 0; u < C::UNITS; ++u) {
          const bool live = attn_wait(&sh.k_full[ku], ku_ph, dead);
          tc::fence_after_sync();
          if (live) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + C::cS + buf * NT, tmem + ku * 32 + k * 8,
                     tc::sdesc_sw128(q + u * NT * 128 + k * 32, 16, 1024), id_s, u > 0 || k > 0);
          }
          tc::mma_commit(&sh.k_empty[ku]);
          if (++ku == C::KU) ku = 0, ku_ph ^= 1;
        }
        tc::mma_commit(&sh.s_full[buf]);
        if (last) {
          tc::mma_commit(&sh.q_empty[qs]);
          if (++qs == C::NQ) qs = 0, q_ph ^= 1;
        }
        ++s_tile;
      };
      auto issue_o = [&](bool fresh, bool last) {
        const int buf = o_tile & 1;
        if (fresh) attn_wait(&sh.o_empty, (seg_no & 1) ^ 1, dead);
        attn_wait(&sh.p_full[buf], (o_tile >> 1) & 1, dead);
        const uint32_t p = p0 + buf * C::PB;
#pragma unroll 1
        for (int r = 0; r < 4; ++r) {
          const bool live = attn_wait(&sh.v_full[vu], vu_ph, dead);
          tc::fence_after_sync();
          if (live) {
#pragma unroll
            for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                mma_ts(tmem + C::cO + mb * NT, tmem + C::cV + (vu * C::MB + mb) * 16 + k * 8,
                       tc::sdesc_sw128(p + (r * 2 + k) * 2048, kTile * 128, 1024), id_o,
                       !(fresh && r == 0 && k == 0));
          }
          tc::mma_commit(&sh.v_empty[vu]);
          if (++vu == C::VU) vu = 0, vu_ph ^= 1;
        }
        tc::mma_commit(&sh.p_empty[buf]);
        if (last) tc::mma_commit(&sh.o_full);
        ++o_tile;
      };
      for (; on; on = seg_next(a, s, left), ++seg_no) {
        issue_s(true, s.t0 + 1 == s.t1);
        for (int t = s.t0; t < s.t1; ++t) {
          if (t + 1 < s.t1) issue_s(false, t + 2 == s.t1);
          issue_o(t == s.t0, t + 1 == s.t1);
        }
      }
      if (*dead) {  // products in flight end before TMEM is given back
        tc::mma_commit(&sh.drain);
        (void)mbar_wait_bounded(&sh.drain, 0, kWaitPolls);
      }
    }
    __syncwarp();
  } else if (warp == 17) {
    // ------------------------------------------------ records in, V scales to binary16
    Seg f = s;  // the copies run ahead of the conversion
    int64_t f_left = left;
    bool f_on = on;
    int f_t = on ? s.t0 : 0, f_tile = 0, stage_f = 0;
    unsigned empty_ph = 1;
    auto fetch = [&]() {
      if (!f_on) return;
      attn_wait(&sh.raw_empty[stage_f], empty_ph, dead);
      int ok = 0;
      const uint8_t* src = nullptr;
      if (lane < 4) {
        const int pos = f_t * kTile + lane * kRec;
        if (pos < f.len) {
          src = record(a.c, f.b, f.h, pos);
          if (src == nullptr) report(a.c.status, GDN_ERR_PAGE_RANGE);
        } else {
          ok = 1;  // nothing to read: hidden by position
        }
        if (src != nullptr) ok = 1;
      }
      const unsigned good = __ballot_sync(0xffffffffu, ok != 0) & 15u;
      const unsigned copies = __ballot_sync(0xffffffffu, src != nullptr);
      if (lane == 0) {
        sh.tile_ok[f_tile & 7] = (int)good;
        mbar_arrive_expect_tx(&sh.raw_full[stage_f], __popc(copies) * rec_bytes(D));
      }
      __syncwarp();
      if (src != nullptr)
        bulk_g2s(smem + C::oRaw + stage_f * C::RAW + lane * rec_bytes(D), src, rec_bytes(D),
                 &sh.raw_full[stage_f]);
      if (++stage_f == C::NRAW) stage_f = 0, empty_ph ^= 1;
      ++f_tile;
      if (++f_t == f.t1) {
        f_on = seg_next(a, f, f_left);
        f_t = f.t0;
      }
    };
    for (int i = 0; i < C::NRAW; ++i) fetch();
    // a stage is filled again one tile later, so that the conversion of the next
    // tile does not wait for the readers of this one
    int stage = 0, vb = 0, tile = 0;
    unsigned raw_ph = 0, vs_ph = 1;
    for (; on; on = seg_next(a, s, left)) {
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        attn_wait(&sh.raw_full[stage], raw_ph, dead);
        attn_wait(&sh.vs_empty[vb], vs_ph, dead);
        const uint8_t* raw = smem + C::oRaw + stage * C::RAW;
        uint8_t* vs = smem + C::oVS + vb * C::VSB;
        const int ok = sh.tile_ok[tile & 7];
        // 8 scales of a group a step; positions past the end count as 0
#pragma unroll 4
        for (int i = lane; i < 4 * (D / 16) * 4; i += 32) {
          const int r = i / (D / 4), g = (i / 4) % (D / 16), o = i & 3;
          const uint2 s8 = *reinterpret_cast<const uint2*>(raw + r * rec_bytes(D) + off_vs(D) +
                                                           g * kRec + o * 8);
          uint32_t w[4] = {e4m3x2(s8.x), e4m3x2(s8.x >> 16), e4m3x2(s8.y), e4m3x2(s8.y >> 16)};
          int n = s.len - (t * kTile + r * kRec + o * 8);  // positions that exist
          if (!((ok >> r) & 1)) n = 0;
          if (n < 8) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = n >= 2 * j + 2 ? w[j] : n == 2 * j + 1 ? (w[j] & 0xffffu) : 0u;
          }
          *reinterpret_cast<uint4*>(vs + g * C::VSG + r * 64 + o * 16) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.vs_full[vb]), mbar_arrive(&sh.raw_empty[stage]);
        if (++stage == C::NRAW) stage = 0, raw_ph ^= 1;
        if (++vb == 2) vb = 0, vs_ph ^= 1;
        if (tile > 0) fetch();
      }
    }
    if (*dead) {  // copies in flight land before the block's memory is given back
      for (int i = 0; i < C::NRAW && i < f_tile; ++i)
        (void)mbar_wait_bounded(&sh.raw_full[i], ((f_tile - i - 1) / C::NRAW) & 1, kWaitPolls);
    }
  } else {
    // ------------------------------------------------ queries
    constexpr int E = D / 32;   // channels of a lane
    const int half = warp - 18;
    int qb = 0, seg_no = 0;
    unsigned ph = 1;
    for (; on; on = seg_next(a, s, left), ++seg_no) {
      attn_wait(&sh.q_empty[qb], ph, dead);
      attn_wait(&sh.row_empty[seg_no & 1], ((seg_no >> 1) & 1) ^ 1, dead);
      const float ks = a.c.k_scale != nullptr ? a.c.k_scale[s.h] : 1.f;
      uint8_t* q = smem + C::oQ + qb * C::QB;
      const int row0 = s.rt * a.rows_per_tile;
      constexpr int BATCH = 8;
      for (int r0 = half; r0 < NT; r0 += 2 * BATCH) {
        uint32_t x[BATCH][E / 2];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const int r = r0 + 2 * j;
#pragma unroll
          for (int i = 0; i < E / 2; ++i) x[j][i] = 0;
          if (r < s.rows) {
            const int n = (row0 + r) / a.G, g = (row0 + r) % a.G;
            const uint16_t* src = static_cast<const uint16_t*>(a.q) + s.b * a.q_stride_b +
                                  n * a.q_stride_n + (int64_t)(s.h * a.G + g) * D + lane * E;
            if constexpr (E == 8) {
              const uint4 v = ld_nc_u4(src);
              x[j][0] = v.x, x[j][1] = v.y, x[j][2] = v.z, x[j][3] = v.w;
            } else if constexpr (E == 4) {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
              x[j][0] = v.x, x[j][1] = v.y;
            } else {
              x[j][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
            }
          }
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const int r = r0 + 2 * j;
          if (r >= NT) break;
          float f[E];
          unsigned big = 0;
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            if (a.bf16) {
              f[2 * i] = __uint_as_float(x[j][i] << 16);
              f[2 * i + 1] = __uint_as_float(x[j][i] & 0xffff0000u);
            } else {
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&x[j][i]));
              f[2 * i] = v.x;
              f[2 * i + 1] = v.y;
            }
            big = max(big, max(__float_as_uint(f[2 * i]) & 0x7fffffffu,
                               __float_as_uint(f[2 * i + 1]) & 0x7fffffffu));
          }
          big = __reduce_max_sync(0xffffffffu, big) >> 23;
          // the row's largest magnitude to [2^8, 2^9); not for zeros, infinities and NaN
          const unsigned up = big == 0 || big == 255 ? 127u : min(262u - big, 252u);
          const float mul = __uint_as_float(up << 23), back = __uint_as_float((254u - up) << 23);
          uint32_t w[E / 2];
#pragma unroll
          for (int i = 0; i < E / 2; ++i) w[i] = pack_f16x2(f[2 * i] * mul, f[2 * i + 1] * mul);
          const int ch = lane * E;
          uint8_t* at = q + (ch >> 6) * (NT * 128) + r * 128 +
                        ((((ch & 63) >> 3) ^ (r & 7)) << 4) + (ch & 7) * 2;
          if constexpr (E == 8) *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
          else if constexpr (E == 4) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
          else *reinterpret_cast<uint32_t*>(at) = w[0];
          if (lane == 0) {
            Row info = {a.scale * back * (ks * kLog2e), 0.f, 0, 0};
            const int n = r < s.rows ? (row0 + r) / a.G : 0;
            if (a.parent == nullptr) {
              info.lo = n;
            } else {
              unsigned long long seen = 0;
              const int32_t* p = a.parent + (int64_t)s.b * a.N;
              for (int m = n; m >= 0; m = p[m]) seen |= 1ull << m;
              info.lo = (unsigned)seen;
              info.hi = (unsigned)(seen >> 32);
            }
            sh.row[seg_no & 1][r] = info;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[qb]), mbar_arrive(&sh.row_full[seg_no & 1]);
      if (++qb == C::NQ) qb = 0, ph ^= 1;
    }
  }
  // every role is done with its loops, hence (bounded) with its copies and products
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *dead) report(a.c.status, GDN_ERR_TIMEOUT);
  if (warp == 16) {
    tc::fence_after_sync();
    tc::tmem_relinquish();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- join
// One block per item: nothing for an item that one block wrote whole, zeros for
// one that sees nothing, else the parts' sum in block order.
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
join_kernel(const __grid_constant__ AttnArgs a, int NT, int parts) {
  __shared__ int64_t red[kJoinWarps][2];
  pdl_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int item = blockIdx.x;
  const int rt = item % a.row_tiles;
  item /= a.row_tiles;
  const int h = item % a.c.Hkv, b = item / a.c.Hkv;
  int64_t total = 0, before = 0;
  for (int i = threadIdx.x; i < a.c.B; i += kJoinWarps * 32) {
    const int64_t x = attn_cost(a, attn_len(a, i, false));
    total += x;
    if (i < b) before += x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) red[warp][0] = total, red[warp][1] = before;
  __syncthreads();
  total = before = 0;
  for (int w = 0; w < kJoinWarps; ++w) total += red[w][0], before += red[w][1];
  if (parts > total) parts = (int)total;
  const int len = attn_len(a, b, false);
  int64_t per_head = 0;
  for (int i = 0; i < a.row_tiles; ++i) {
    const int t = attn_tiles(a, len, i);
    if (i < rt) before += t;
    per_head += t;
  }
  before += h * per_head;
  Seg s = {};
  s.rt = rt;
  seg_rows(a, s);
  const int tiles = attn_tiles(a, len, rt), row0 = rt * a.rows_per_tile;
  int first = 0, last = 0;
  if (tiles > 0) {
    // the blocks that hold the item's first and last tile
    first = (int)(((before + 1) * parts + total - 1) / total) - 1;
    last = (int)(((before + tiles) * parts + total - 1) / total) - 1;
    if (first == last) return;
  }
  const float vsc = a.c.v_scale != nullptr ? a.c.v_scale[h] : 1.f;
  for (int r = warp; r < s.rows; r += kJoinWarps) {
    float acc[D / 32] = {}, sum = 0.f, top = kNone;
    if (tiles > 0) {
      for (int c = first + lane; c <= last; c += 32) {
        const int64_t slot = 2 * (int64_t)c + (total * c / parts < before);
        const float m = a.part_ml[slot * NT + r].x;
        top = m > top || m != m ? m : top;
      }
      top = warp_max(top);
#pragma unroll 4
      for (int c = first; c <= last; ++c) {
        const int64_t slot = 2 * (int64_t)c + (total * c / parts < before);
        const float2 ml = a.part_ml[slot * NT + r];
        const float w = exp2_fast(ml.x - top);
        sum += w * ml.y;
        const float* p = a.part_o + (slot * NT + r) * D + lane;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] += w * p[i * 32];
      }
    }
    const int n = (row0 + r) / a.G, g = (row0 + r) % a.G;
    const int64_t at = ((int64_t)b * a.N + n) * a.Hq + h * a.G + g;
    const float inv = sum != 0.f ? vsc / sum : 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const float o = acc[i] * inv;
      static_cast<uint16_t*>(a.o)[at * D + i * 32 + lane] =
          a.bf16 ? Elem<GDN_BF16>::from(o) : Elem<GDN_F16>::from(o);
    }
    if (a.lse != nullptr && lane == 0)
      a.lse[at] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  }
}

template <int D, int NT>
int attn_launch_nt(const AttnArgs& a, int parts, cudaStream_t s) {
  using C = AttnCfg<D, NT>;
  if (cudaFuncSetAttribute(attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::SMEM) != cudaSuccess) {
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
  }
  const int rc = launch_pdl(attn_kernel<D, NT>, dim3(parts), dim3(kAttnThreads), C::SMEM, s, a);
  if (rc != GDN_OK) return rc;
  return launch_pdl(join_kernel<D>, dim3(a.c.B * a.c.Hkv * a.row_tiles), dim3(kJoinWarps * 32), 0,
                    s, a, NT, parts);
}

template <int D>
int attn_launch_d(const AttnArgs& a, int NT, int parts, cudaStream_t s) {
  switch (NT) {
    case 16: return attn_launch_nt<D, 16>(a, parts, s);
    case 32: return attn_launch_nt<D, 32>(a, parts, s);
    case 64: return attn_launch_nt<D, 64>(a, parts, s);
    default: return attn_launch_nt<D, 96>(a, parts, s);
  }
}

}  // namespace kv4
}  // namespace gdn
