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
// Warps of a block, connected by mbarriers only:
//   4 of K      position = TMEM lane; codes * scale -> binary16 -> TMEM, in units of 64 or
//               128 channels
//   4 of V      channel = TMEM lane; the same for V^T, in units of 32 or 64 positions
//   4 or more of softmax, a group of four for 16 or 32 rows: S^T from TMEM, p to shared
//               memory (B operand), sums in registers, the item's epilogue, and the next
//               item's queries into the B operand (binary16, scaled by powers of two so
//               that any bf16 magnitude fits)
//   1 that issues S^T's products, 1 that issues O^T's (products into one accumulator
//               come from one thread: across threads they have no order)
//   1 or 2 that cut the run into segments and copy the records
//
// The reference m is set 7 under a row's largest logit (so that p = 2^7 there) and
// moved only when some p would pass 2^15 (binary16 ends at 65504): the sums and O^T are
// then multiplied by 2^(old - new), which happens on an item's first tile and seldom
// later, so the usual tile takes one FMA, one maximum, one exp2 and one addition per
// logit and no reduction across lanes.  p is rounded to binary16 for the product: 2^-11
// relative (bf16 would give 2^-8) from 2^-21 of the row's largest p on, and to multiples of
// 2^-31 of it below (their sum l is taken before, in fp32); with m at the largest logit
// itself these were 2^-14 and 2^-24, and a flat tail 17 nats under one large logit was lost.
// code * scale needs 6 significand bits, so K and V are exact.
//
// What bounds it.  With few rows the bytes: a tile of 36.8 KB (D = 256) takes 0.93 us a
// block, 39.6 GB/s an SM of 43.8 measured for a copy; 131072 tokens of 4 heads take
// 37.9 us, 23 us of them the floor, about 5 us before the first tile and 5 us for the last
// item's output and the join.  With 96 rows the softmax warps: 1.6 us a tile, of which 0.5
// us is the exponentials' issue at 80 registers, the tensor pipe 0.8 us; a 2048-token piece
// of a prompt at 8192 tokens takes 362 to 371 us over runs, 975 to 997 TFLOP/s of 1,880
// measured.
// Measured and left out (us for 131072 tokens / the prompt, against the figure of the
// time): the products issued by the K and V warps themselves, 55 / 500 against 50 / 464;
// two streams of tiles, each with softmax warps, 58 / 693 against 50 / 464; steps of two
// tiles with few rows, 41.8 against 39.9; a second group of K and V warps with few rows,
// 170 against 152 for 48 sequences; softmax groups of 24 rows, - / 500 against 401.
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
constexpr float kNone = -3.402823466e38f;  // reference of a row that has seen nothing
// m is set kBelow under the largest logit (log2 units), so that p starts at 2^7, and moves
// when some p passes 2^15 in binary16.
constexpr float kBelow = 7.f;
constexpr unsigned kMostP = 0x7800;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWaitPolls = 1 << 20;  // bound of every wait

template <int D_, int NT_>
struct AttnCfg {
  static constexpr int D = D_, NT = NT_;
  static constexpr int MB = D == 256 ? 2 : 1;  // 128-channel blocks of O^T
  static constexpr int NS = NT < 64 ? 1 : NT / 32;  // softmax groups
  static constexpr int NH = NT / NS;                // rows of one
  static constexpr int ROWS = NT / (4 * NS);        // query rows that a softmax warp brings in
  static constexpr bool COMMON = NT >= 64;          // one scale for all rows (attn_rows)
  static constexpr int wV = 4, wS = 8;  // first warps of the roles
  // warps that copy: with few rows a tile is short (48 sequences: two 85 us, one 103 us),
  // with many the registers of a warp less count more (the prompt: one 407 us, two 417 us)
  static constexpr int wI = wS + 4 * NS, FW = NT < 64 ? 2 : 1;
  static constexpr int THREADS = 32 * (wI + 2 + FW);
  // TMEM columns: two K units (KW columns of 2 channels each), two S^T, O^T, two V units
  // (VW records each).  Large units cost fewer hand-overs; the widest case has no
  // room for them.
  static constexpr bool BIG = 128 + 64 * MB + (2 + MB) * NT <= 512;
  static constexpr int KW = BIG && D >= 128 ? 64 : 32, VW = BIG ? 2 : 1;
  static constexpr int UNITS = D / 2 / KW, VUNITS = 4 / VW;  // of a tile
  static constexpr int KU = 2, VU = 2;
  // of the K and V warps' units: with many rows all roles' loops together strain the
  // instruction cache (a 2048-token piece of a prompt: unrolled 377 us, rolled 365), with
  // few they do less (131072 tokens: unrolled 37.3 us, rolled 38.4)
  static constexpr int UNROLL = NT < 64 ? 8 : 1;
  static constexpr int cS = KW * KU, cO = cS + 2 * NT, cV = cO + MB * NT;
  static_assert(cV + VU * VW * 16 * MB <= 512, "TMEM");
  // shared memory
  static constexpr int HALF = 18 * D;          // of a record: K's or V's codes and scales
  static constexpr int RAW = 4 * HALF;         // a stage of either ring
  static constexpr int QB = NT * D * 2;
  static constexpr int PB = (NT > 64 ? 2 : 1) * kTile * 128;
  static constexpr int VSG = 272;  // bytes between the scale rows of two groups (bank offset)
  static constexpr int VSB = D / 16 * VSG;
  static constexpr int ROOM = (214 * 1024 - QB - 2 * PB - 2 * VSB) / RAW;
  static constexpr int KR = ROOM / 2 > 6 ? 6 : ROOM / 2;
  static constexpr int VR = ROOM - KR > 6 ? 6 : ROOM - KR;
  static_assert(KR >= 2 && VR >= 2, "stages");
  static constexpr int oQ = 0, oP = oQ + QB, oK = oP + 2 * PB, oV = oK + KR * RAW;
  static constexpr int oVS = oV + VR * RAW;
  static constexpr int oEnd = oVS + 2 * VSB;
  static constexpr int SMEM = oEnd + 1024;  // + alignment of the swizzled operands
};

// The part of one item that a block works on: tiles [t0, t1) of `tiles` (t1 = 0: the end).
struct Seg {
  int b, h, t0, t1, tiles, len, row0, rows;
  int last;  // block that holds the item's last tile
};

// What a block's work is measured in: an item's tiles, and kLead more before them
// for what an item costs beside its tiles (its queries, first references and
// output).  Measured: without the lead 48 sequences of 0 to 8192 tokens took 150 us,
// the blocks with many short ones twice the others' time; with 4, 6, 8 and 10 it is
// 80.5, 80.6, 81.9 and 83.7 us, eight verified chains of 16 take 69.8, 68.8, 69.0 and
// 68.9 us, a tree of 22 nodes 45.7, 44.7, 45.2 and 44.3 us.
constexpr int kLead = 6;

// Equal runs of `total` units for at most `parts` blocks: the first `extra` runs
// have one unit more.  (The host keeps the count below 2^31.)
struct Runs {
  int each, extra, parts;
  Runs() = default;
  __device__ __forceinline__ Runs(int total, int n) {
    parts = min(total, n);  // no empty runs in between
    each = parts > 0 ? total / parts : 0;
    extra = total - each * parts;
  }
  __device__ __forceinline__ int start(int part) const { return each * part + min(part, extra); }
  // the run that holds unit x
  __device__ __forceinline__ int of(int x) const {
    const int head = extra * (each + 1);
    return x < head ? x / (each + 1) : extra + (x - head) / each;
  }
};

// Walks the tiles of a block's run, item by item (one warp).
struct Run {
  int b, h, rt, u0, at, left;
  Runs runs;
};

constexpr int kSegs = 16;    // ring of segments
constexpr int kTiles = 32;   // ring of tiles' page checks; copies are fewer tiles ahead
constexpr int kLens = 1024;  // lengths kept in shared memory

template <typename C>
struct AttnShared {
  uint64_t kr_full[C::KR], kr_empty[C::KR], vr_full[C::VR], vr_empty[C::VR];
  uint64_t k_full[C::KU], k_empty[C::KU], v_full[C::VU], v_empty[C::VU];
  uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2];
  uint64_t q_full, o_full, o_empty, drain;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint32_t tmem;
  int dead;
  int tile_ok[2][kTiles];  // records of a tile that could be read, by tile number
  Seg seg[kSegs];
  // of the query rows: c (logit of S: c * S, log2 units), the row of
  // the output from the item's first node and head on, and for trees the
  // positions of the block that the row sees
  alignas(16) float row_c[C::NT];
  alignas(16) int row_at[C::NT];
  uint2 row_path[C::NT];
  uint2 path[64];                   // of each node
  alignas(16) float neg_m[C::NT];   // of the rows in work
  int row_e[C::NT];                 // exponent of a row's largest magnitude
  alignas(16) float alpha[C::NT], inv[C::NT];
  float part[4][C::NT];             // of a softmax group's four warps
  Run run;
  // for the functions that are not inlined: a reference to the kernel's parameters
  // themselves is read through global memory
  AttnArgs args;
  int len[kLens];
};

// A wait that ends: false once any wait of the block has run out.
static __device__ __noinline__ bool attn_wait_on(uint64_t* bar, unsigned parity, volatile int* dead) {
  for (int i = 0; i < kWaitPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 63 && *dead) return false;
  }
  *dead = 1;
  return false;
}

__device__ __forceinline__ bool attn_wait(uint64_t* bar, unsigned parity, volatile int* dead) {
  if (mbar_try_wait(bar, parity)) return true;
  return attn_wait_on(bar, parity, dead);
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_addr(bar)) : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(e));
  return e != 0;
}

// Named barrier over `threads` threads; true for all when `x` holds for any.
__device__ __forceinline__ bool barrier_any(int id, int threads, bool x) {
  uint32_t any;
  asm volatile(
      "{.reg .pred p, q; setp.ne.u32 p, %1, 0;"
      " barrier.cta.red.or.pred q, %2, %3, p; selp.u32 %0, 1, 0, q;}"
      : "=r"(any)
      : "r"((uint32_t)x), "r"(id), "r"(threads)
      : "memory");
  return any != 0;
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

// Pairs of fp32 values in one instruction.
union Pair {
  unsigned long long u;
  float2 f;
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  Pair x, y, z;
  x.f = a, y.f = b, z.f = c;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(z.u) : "l"(x.u), "l"(y.u), "l"(z.u));
  return z.f;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  Pair x, y;
  x.f = a, y.f = b;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(x.u) : "l"(x.u), "l"(y.u));
  return x.f;
}

// Reduces N values (16 or 32) over the warp's lanes: lane i ends with value
// i % N's result.  Each step halves the values that a lane still carries.
template <int N, typename Op>
__device__ __forceinline__ float warp_transpose_reduce(float (&v)[N], Op op) {
  const int lane = threadIdx.x & 31;
  if constexpr (N == 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], 16));
  }
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = upper ? v[i + o] : v[i], give = upper ? v[i] : v[i + o];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  return v[0];
}

__device__ __forceinline__ void st_shared16(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

// 8 codes (one word) times the scale pair(s): four f16x2 words.
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t s, uint32_t* out) {
  out[0] = hmul2(e2m1x2<0>(w), s);
  out[1] = hmul2(e2m1x2<1>(w), s);
  out[2] = hmul2(e2m1x2<2>(w), s);
  out[3] = hmul2(e2m1x2<3>(w), s);
}

// ---------------------------------------------------------------- work
// Length of sequence b as attention counts it (0: skipped).
static __device__ __noinline__ int attn_len(const AttnArgs& a, int b, bool report_it) {
  const int n = seq_len(a.c, b, report_it);
  if (n > 0 && a.parent != nullptr && !tree_ok(a.parent + (int64_t)b * a.N, a.N)) {
    if (report_it) report(a.c.status, GDN_ERR_BAD_TREE);
    return 0;
  }
  return n;
}

// Tiles that row tile `rt` of a sequence of `len` positions sees.
__device__ __forceinline__ int attn_tiles(const AttnArgs& a, int len, int rt) {
  int see = len;
  if (a.parent == nullptr) {
    const int last = min((rt + 1) * a.rows_per_tile, a.rows_total) - 1;
    see = len - a.N + last / a.G + 1;
  }
  return see <= 0 ? 0 : (see + kTile - 1) / kTile;
}

__device__ __forceinline__ int warp_sum(int x) { return __reduce_add_sync(0xffffffffu, x); }

// The lengths the block works with: the first kLens are kept in shared memory.
struct Lens {
  const AttnArgs& a;
  const int* kept;
  __device__ __forceinline__ int operator()(int b) const {
    return b < kLens ? kept[b] : attn_len(a, b, false);
  }
};

// Lengths into shared memory, by all threads: a thread a sequence, or for
// trees a warp a sequence (its lanes check the nodes).  Returns whether any of
// this thread's differs from what was there.
static __device__ __noinline__ bool attn_lens(const AttnArgs& a, int* kept, bool report_it) {
  bool changed = false;
  const int lane = threadIdx.x & 31, n_kept = min(a.c.B, kLens);
  const int unit = a.parent == nullptr ? 1 : 32;  // threads of a sequence
#pragma unroll 1
  for (int b = threadIdx.x / unit; b < n_kept; b += blockDim.x / unit) {
    bool ok = true;
    if (a.parent != nullptr) {
      const volatile int32_t* p = a.parent + (int64_t)b * a.N;
#pragma unroll 1
      for (int n = lane; n < a.N; n += 32) {
        const int up = p[n];
        ok = ok && (n == 0 ? up == -1 : up >= 0 && up < n);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (lane != 0) continue;
    }
    int len = *(const volatile int32_t*)(a.c.kv_len + b);
    if (len < 0 || (int64_t)len > (int64_t)a.c.max_pages * a.c.page_tokens) {
      if (report_it) report(a.c.status, GDN_ERR_ROW_RANGE);
      len = 0;
    }
    if (!ok) {
      if (report_it && len > 0) report(a.c.status, GDN_ERR_BAD_TREE);
      len = 0;
    }
    changed |= kept[b] != len;
    kept[b] = len;
  }
  if (report_it)  // the others' reports (their lengths are looked up when needed)
#pragma unroll 1
    for (int b = kLens + threadIdx.x; b < a.c.B; b += blockDim.x) (void)attn_len(a, b, true);
  return changed;
}

// The same in units of work.
__device__ __forceinline__ int attn_units(const AttnArgs& a, int len, int rt) {
  const int t = attn_tiles(a, len, rt);
  return t > 0 ? t + kLead : 0;
}

// Units of sequence b over all heads, by a whole warp.
__device__ __forceinline__ int warp_cost(const AttnArgs& a, int len) {
  int t = 0;
#pragma unroll 1
  for (int rt = threadIdx.x & 31; rt < a.row_tiles; rt += 32) t += attn_units(a, len, rt);
  return warp_sum(t) * a.c.Hkv;
}

// The run of block `part` of `parts`: the units of all sequences are counted,
// then the sequence that holds the run's first one is taken apart.
static __device__ __noinline__ Run attn_run(const AttnArgs& a, const Lens& lens, int part,
                                            int parts) {
  const int lane = threadIdx.x & 31;
  const bool by_lane = a.row_tiles <= 4;  // a lane a sequence, or the warp a sequence
  const int step = by_lane ? 32 : 1;
  // units of the sequence b0 + lane, or (of all lanes the same) of b0
  auto units = [&](int b0) {
    if (!by_lane) return warp_cost(a, lens(b0));
    int x = 0;
    if (b0 + lane < a.c.B) {
      const int len = lens(b0 + lane);
#pragma unroll 1
      for (int rt = 0; rt < a.row_tiles; ++rt) x += attn_units(a, len, rt);
    }
    return x * a.c.Hkv;
  };
  int total = 0, mine = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.c.B; b0 += step) {
    mine = units(b0);
    total += by_lane ? warp_sum(mine) : mine;
  }
  Run r = {0, 0, 0, 0, 0, 0, Runs(total, parts)};
  if (part >= r.runs.parts) return r;
  r.at = r.runs.start(part);
  r.left = r.runs.start(part + 1) - r.at;
  int before = 0, its = 0;
#pragma unroll 1
  for (int b0 = 0;; b0 += step) {
    if (a.c.B > step) mine = units(b0);  // else it is still there
    int upto = mine;
    if (by_lane) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + upto > r.at);
    if (hit == 0) {
      before += __shfl_sync(0xffffffffu, upto, 31);
      continue;
    }
    const int l = by_lane ? __ffs(hit) - 1 : 0;
    its = __shfl_sync(0xffffffffu, mine, l);
    before += __shfl_sync(0xffffffffu, upto, l) - its;
    r.b = b0 + l;
    break;
  }
  int in = r.at - before;  // of the sequence's `its` tiles
  const int per_head = its / a.c.Hkv, len = lens(r.b);
  r.h = in / per_head;
  in -= r.h * per_head;
#pragma unroll 1
  for (;; ++r.rt) {
    const int t = attn_units(a, len, r.rt);
    if (in < t) break;
    in -= t;
  }
  r.u0 = in;
  return r;
}

// The run's next segment (t1 = 0 when it is at its end).
static __device__ __noinline__ Seg attn_seg(const AttnArgs& a, const Lens& lens, Run& r) {
  Seg s = {};
#pragma unroll 1
  while (r.left > 0 && r.b < a.c.B) {
    const int len = lens(r.b);
    const int tiles = attn_tiles(a, len, r.rt), units = tiles > 0 ? tiles + kLead : 0;
    const int rt = r.rt, h = r.h, b = r.b, end = min(units, r.u0 + r.left), taken = end - r.u0;
    const int t0 = max(r.u0 - kLead, 0), t1 = end - kLead;
    r.u0 = 0;
    r.left -= taken;
    r.at += taken;
    if (++r.rt == a.row_tiles) {
      r.rt = 0;
      if (++r.h == a.c.Hkv) r.h = 0, ++r.b;
    }
    if (t1 <= t0) continue;  // no tiles, or the lead alone
    s.b = b, s.h = h, s.t0 = t0, s.t1 = t1, s.tiles = tiles, s.len = len;
    s.last = t1 < tiles ? r.runs.of(r.at + tiles - t1 - 1) : 0;
    s.row0 = rt * a.rows_per_tile;
    s.rows = min(a.rows_total - s.row0, a.rows_per_tile);
    return s;
  }
  return s;
}

// Rows that see no tile at all: 0 (and -infinity), spread over the blocks; 128 threads.
static __device__ __noinline__ void attn_zero(const AttnArgs& a, const Lens& lens, int D, int tid) {
  const int64_t pairs = (int64_t)a.c.B * a.row_tiles;
#pragma unroll 1
  for (int64_t i = blockIdx.x; i < pairs; i += gridDim.x) {
    const int b = (int)(i / a.row_tiles), rt = (int)(i % a.row_tiles);
    if (attn_tiles(a, lens(b), rt) > 0) continue;
    const int row0 = rt * a.rows_per_tile, rows = min(a.rows_total - row0, a.rows_per_tile);
#pragma unroll 1
    for (int k = 0; k < rows * a.c.Hkv; ++k) {
      const int h = k / rows, r = row0 + k % rows;
      const int64_t at = ((int64_t)b * a.N + r / a.G) * a.Hq + h * a.G + r % a.G;
      if (tid < D / 2) static_cast<uint32_t*>(a.o)[at * (D / 2) + tid] = 0;
      if (a.lse != nullptr && tid == 0) a.lse[at] = -INFINITY;
    }
  }
}

// ---------------------------------------------------------------- queries
// The query rows of a segment go to the B operand at q, ROWS neighbouring rows a
// softmax warp.  They are copied as they are to where the operand goes (the copies
// are this thread's cp.async, not waited for); a lane works out one row's place.
template <int D, int NT>
static __device__ __noinline__ void attn_rows_copy(const AttnArgs& a, int b, int h, int row0,
                                                   int rows, uint8_t* q, int warp) {
  constexpr int E = D / 32, ROWS = AttnCfg<D, NT>::ROWS;  // channels of a lane
  const int lane = threadIdx.x & 31, ch = lane * E, r0 = warp * ROWS;
  const int row = row0 + r0 + lane % ROWS, n = row / a.G;
  const int64_t mine = b * a.q_stride_b + n * a.q_stride_n +
                       (int64_t)(h * a.G + row - n * a.G) * D;
  const uint16_t* src = static_cast<const uint16_t*>(a.q) + ch;
  q += (ch >> 6) * (NT * 128) + (ch & 7) * 2;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + i;
    uint8_t* at = q + r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4);
    const int64_t from = __shfl_sync(0xffffffffu, mine, i);
    if (r < rows) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(smem_addr(at)),
                   "l"(src + from), "n"(E * 2)
                   : "memory");
    } else {
#pragma unroll
      for (int k = 0; k < E / 2; ++k) reinterpret_cast<uint32_t*>(at)[k] = 0;
    }
  }
}

// One lane's channels of a row in the B operand: 4, 8 or 16 bytes.
template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&x)[W]) {
  if constexpr (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = v.x, x[1] = v.y;
  } else {
    x[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <int W>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&x)[W]) {
  if constexpr (W == 4) {
    *reinterpret_cast<uint4*>(p) = make_uint4(x[0], x[1], x[2], x[3]);
  } else if constexpr (W == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(x[0], x[1]);
  } else {
    *reinterpret_cast<uint32_t*>(p) = x[0];
  }
}

// Then each lane turns its own channels into binary16 in place, and what goes
// with the rows is written, a lane a row.  With many rows, all are scaled by one
// power of two where their largest magnitudes lie within 2^8 of each other (the
// smallest row's then is at least 1, so that binary16's fixed point error, 2^-25, is
// below fp32's own), and else each row by its own; returns c of all rows, or 0 where
// rows differ.  One c halves what the softmax reads per row: a 2048-token piece of a
// prompt 385 -> 369 us, eight chains of 16 65.7 -> 63.3 us; with few rows finding it
// costs more (48 uneven sequences 81 -> 83 us), and each row has its own.
template <int D, int NT>
static __device__ __noinline__ float attn_rows(const AttnArgs& a, AttnShared<AttnCfg<D, NT>>& sh,
                                               int b, int row0, int rows, uint8_t* q, int warp,
                                               float to_log2) {
  const int G = a.G, Hq = a.Hq;
  const bool bf16 = a.bf16, tree = a.parent != nullptr;
  constexpr int E = D / 32, ROWS = AttnCfg<D, NT>::ROWS;
  const int lane = threadIdx.x & 31, ch = lane * E, r0 = warp * ROWS;
  q += (ch >> 6) * (NT * 128) + (ch & 7) * 2;
  auto place = [&](int r) { return q + r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4); };
  if (tree) {
    // path of every node: pointers double their reach in each step
    const int32_t* p = a.parent + (int64_t)b * a.N;
    int to[2];
    unsigned long long path[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = lane + 32 * i;
      to[i] = m < a.N ? __ldg(p + m) : -1;
      path[i] = 1ull << m;
    }
#pragma unroll 1
    while (__any_sync(0xffffffffu, to[0] >= 0 || to[1] >= 0)) {
      int next[2];
      unsigned long long more[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int from = to[i] & 31;
        const unsigned long long m0 = __shfl_sync(0xffffffffu, path[0], from);
        const unsigned long long m1 = __shfl_sync(0xffffffffu, path[1], from);
        const int t0 = __shfl_sync(0xffffffffu, to[0], from);
        const int t1 = __shfl_sync(0xffffffffu, to[1], from);
        more[i] = to[i] < 0 ? 0 : to[i] < 32 ? m0 : m1;
        next[i] = to[i] < 0 ? -1 : to[i] < 32 ? t0 : t1;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) path[i] |= more[i], to[i] = next[i];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)  // several warps may write the same values
      sh.path[lane + 32 * i] = make_uint2((unsigned)path[i], (unsigned)(path[i] >> 32));
    __syncwarp();
  }
  const int row = row0 + min(r0 + lane % ROWS, rows - 1), n = row / G;
  cp_async_wait_all();
  uint32_t x[ROWS][E / 2];
  unsigned mine = 0;  // the lane's row's largest magnitude
#pragma unroll
  for (int i = 0; i < ROWS; ++i) load_words<E / 2>(place(r0 + i), x[i]);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    unsigned big = 0;
#pragma unroll
    for (int k = 0; k < E / 2; ++k)  // magnitudes order as integers in either type
      big = max(big, max(x[i][k] & 0x7fffu, (x[i][k] >> 16) & 0x7fffu));
    big = __reduce_max_sync(0xffffffffu, big);
    if (lane % ROWS == i) mine = big;
  }
  const float top = bf16 ? __uint_as_float(mine << 16)
                         : __half2float(__ushort_as_half((unsigned short)mine));
  const int e = (int)(__float_as_uint(top) >> 23);
  int most = 0, least = 255;  // of the rows but those of zeros, infinities and NaN
  if constexpr (AttnCfg<D, NT>::COMMON) {
    if (lane < ROWS) sh.row_e[r0 + lane] = e;
    tc::named_barrier(4, 128 * AttnCfg<D, NT>::NS);
#pragma unroll
    for (int r = lane; r < NT; r += 32) {
      const int o = sh.row_e[r];
      if (o > 0 && o < 255) most = max(most, o), least = min(least, o);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
  }
  const bool same = AttnCfg<D, NT>::COMMON && most - least <= 8;
  // the largest magnitude to [2^8, 2^9)
  const int of = same ? most : e;
  const int up = of == 0 || of == 255 ? 127 : min(262 - of, 252);
  const float mul = __uint_as_float((unsigned)up << 23);
  const float c = to_log2 * __uint_as_float((unsigned)(254 - up) << 23);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const float m = __shfl_sync(0xffffffffu, mul, i);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) {
      float2 f;
      if (bf16) {
        f = make_float2(__uint_as_float(x[i][k] << 16), __uint_as_float(x[i][k] & 0xffff0000u));
      } else {
        f = __half22float2(*reinterpret_cast<const __half2*>(&x[i][k]));
      }
      x[i][k] = pack_f16x2(f.x * m, f.y * m);
    }
    store_words<E / 2>(place(r0 + i), x[i]);
  }
  if (lane < ROWS) {
    const int r = r0 + lane;
    sh.row_c[r] = c;
    sh.row_at[r] = n * Hq + row - n * G;
    if (tree) sh.row_path[r] = sh.path[n];
  }
  fence_proxy_async_smem();
  __syncwarp();
  return same ? c : 0.f;
}

// ---------------------------------------------------------------- the kernel
template <int D, int NT>
__global__ void __launch_bounds__(AttnCfg<D, NT>::THREADS, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = AttnCfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ AttnShared<C> sh;
  uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* dead = &sh.dead;

  static_assert(sizeof(AttnArgs) / 4 <= 64 && 64 <= C::THREADS, "a word a thread");
  if (threadIdx.x < sizeof(AttnArgs) / 4)
    reinterpret_cast<uint32_t*>(&sh.args)[threadIdx.x] =
        reinterpret_cast<const uint32_t*>(&a)[threadIdx.x];
  __syncthreads();
  const AttnArgs& args = sh.args;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KR; ++i)
      mbar_init(&sh.kr_full[i], 1), mbar_init(&sh.kr_empty[i], 4);
    for (int i = 0; i < C::VR; ++i)
      mbar_init(&sh.vr_full[i], 1), mbar_init(&sh.vr_empty[i], 4);
    for (int i = 0; i < C::KU; ++i) mbar_init(&sh.k_full[i], 4), mbar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < C::VU; ++i) mbar_init(&sh.v_full[i], 4), mbar_init(&sh.v_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1), mbar_init(&sh.s_empty[i], 4 * C::NS);
      mbar_init(&sh.p_full[i], 4 * C::NS), mbar_init(&sh.p_empty[i], 1);
    }
    mbar_init(&sh.q_full, 1);
    for (int i = 0; i < kSegs; ++i) mbar_init(&sh.seg_full[i], 1), mbar_init(&sh.seg_empty[i], C::wI + 1 + C::FW);
    mbar_init(&sh.o_full, 1);
    mbar_init(&sh.o_empty, 4 * C::NS);
    mbar_init(&sh.drain, 2);
    sh.dead = 0;
    mbar_init_fence();
  }
  if (warp == C::wI) tc::tmem_alloc(&sh.tmem, 512);
  // The block's run follows from the lengths alone.  It is worked out before the
  // wait on the kernel before this one, from the lengths as they read then, and
  // again after it in the case that one of them has changed (with more sequences
  // than are kept, always).
  const Lens lens = {args, sh.len};
  const bool kept = a.c.B <= kLens;
  (void)attn_lens(args, sh.len, false);
  __syncthreads();
  if (warp == C::wI + 2 && kept) {
    Run run = attn_run(args, lens, blockIdx.x, gridDim.x);
    const Seg first = attn_seg(args, lens, run);
    if (lane == 0) sh.run = run, sh.seg[0] = first;
  }
  __syncthreads();
  pdl_enter();
  // the first segment's queries are on their way while the lengths are read again
  const bool softmax = warp >= C::wS && warp < C::wI;
  auto head_scale = [&](int h) { return a.c.k_scale != nullptr ? a.c.k_scale[h] : 1.f; };
  float k_scale = 1.f;
  if (softmax && kept && sh.seg[0].t1 > 0) {
    k_scale = head_scale(sh.seg[0].h);
    attn_rows_copy<D, NT>(args, sh.seg[0].b, sh.seg[0].h, sh.seg[0].row0, sh.seg[0].rows,
                          smem + C::oQ, warp - C::wS);
  }
  const bool changed = attn_lens(args, sh.len, blockIdx.x == 0);
  tc::fence_before_sync();
  const bool again = __syncthreads_or(changed) || !kept;
  tc::fence_after_sync();
  // all 512 columns are this block's, so its tensor memory begins at address 0, and
  // the addresses below are column numbers known at compile time
  if (sh.tmem != 0) *dead = 1;

  // every warp but the one that cuts them takes the run's segments from the ring
  int seg_no = 0;
  Seg s;
  auto next_seg = [&]() {
    const int i = seg_no & (kSegs - 1);
    if (seg_no > 0 || again)  // the first one is there since before the wait
      attn_wait(&sh.seg_full[i], (seg_no / kSegs) & 1, dead);
    s = sh.seg[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.seg_empty[i]);
    return s.t1 > 0 && !__any_sync(0xffffffffu, *dead);
  };

  if (warp < C::wV) {
    // ------------------------------------------------ K -> TMEM
    // A unit in two halves of 32 channels: the first is on its way to TMEM, and the
    // next one's bytes to registers, while the second is converted.
    const uint32_t dst = (uint32_t)(warp * 32) << 16;
    int stage = 0, unit = 0;
    unsigned raw_ph = 0, unit_ph = 1;  // an empty ring's first pass does not wait
    for (; next_seg(); ++seg_no) {
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t) {
        attn_wait(&sh.kr_full[stage], raw_ph, dead);
        const uint8_t* rec = smem + C::oK + stage * C::RAW + warp * C::HALF + lane * 16;
        const uint8_t* scales = smem + C::oK + stage * C::RAW + warp * C::HALF + 16 * D +
                                lane * (D / 16);
        uint4 q4 = *reinterpret_cast<const uint4*>(rec);
#pragma unroll C::UNROLL
        for (int u = 0; u < C::UNITS; ++u) {
#pragma unroll
          for (int k = 0; k < C::KW / 16; ++k) {  // 32 channels: one 16-byte chunk
            const int chunk = u * (C::KW / 16) + k;
            const uint4 now = q4;
            if (chunk + 1 < D / 32) q4 = *reinterpret_cast<const uint4*>(rec + (chunk + 1) * 512);
            const uint32_t sc =
                e4m3x2(*reinterpret_cast<const uint16_t*>(scales + 2 * chunk));
            const uint32_t g = __byte_perm(sc, sc, 0x1010), h = __byte_perm(sc, sc, 0x3232);
            uint32_t w[16];
            dequant8(now.x, g, w);
            dequant8(now.y, g, w + 4);
            dequant8(now.z, h, w + 8);
            dequant8(now.w, h, w + 12);
            if (k == 0) {
              attn_wait(&sh.k_empty[unit], unit_ph, dead);
              tc::fence_after_sync();
            }
            tmem_st16(dst + unit * C::KW + k * 16, w);
          }
          tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.k_full[unit]);
          if (++unit == C::KU) unit = 0, unit_ph ^= 1;
        }
        if (lane == 0) mbar_arrive(&sh.kr_empty[stage]);
        if (++stage == C::KR) stage = 0, raw_ph ^= 1;
      }
    }
  } else if (warp < C::wS) {
    // ------------------------------------------------ V^T -> TMEM
    const int quarter = warp & 3;
    const uint32_t dst = ((uint32_t)(quarter * 32) << 16) + C::cV;
    const int vt = threadIdx.x - 32 * C::wV;
    attn_zero(args, lens, D, vt);
    int stage = 0, unit = 0, tile = 0;
    unsigned raw_ph = 0, unit_ph = 1;
    for (;; ++seg_no) {
      // all of them go on, or none: they meet at a barrier below
      if (barrier_any(5, 128, !next_seg())) break;
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        attn_wait(&sh.vr_full[stage], raw_ph, dead);
        const uint8_t* raw = smem + C::oV + stage * C::RAW;
        // the tile's scales to binary16, 8 positions of a group a step; those past
        // the end, or on a page that is not there, count as 0
        uint8_t* vs = smem + C::oVS + (tile & 1) * C::VSB;
        const int ok = sh.tile_ok[1][tile & (kTiles - 1)], end = s.len - t * kTile;
        const bool full = ok == 15 && end >= kTile;
#pragma unroll
        for (int i = vt; i < D; i += 128) {
          const int r = i / (D / 4), go = i % (D / 4);
          const uint2 s8 =
              *reinterpret_cast<const uint2*>(raw + r * C::HALF + 16 * D + go * 8);
          uint32_t w[4] = {e4m3x2(s8.x), e4m3x2(s8.x >> 16), e4m3x2(s8.y), e4m3x2(s8.y >> 16)};
          if (!full) {
            const int n = (ok >> r) & 1 ? end - (r * kRec + (go & 3) * 8) : 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = n >= 2 * q + 2 ? w[q] : n == 2 * q + 1 ? (w[q] & 0xffffu) : 0u;
          }
          *reinterpret_cast<uint4*>(vs + (go >> 2) * C::VSG + r * 64 + (go & 3) * 16) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        tc::named_barrier(5, 128);  // also: the other buffer's readers are done
        const int ch = quarter * 32 + lane;
        const bool mine = D >= 128 || ch < D;  // D = 64: the upper lanes hold zeros
        const uint8_t* codes = raw + (mine ? ch * 16 : 0);
        const uint8_t* scales = vs + (ch >> 4) * C::VSG;
        uint4 q4 = *reinterpret_cast<const uint4*>(codes);
#pragma unroll C::UNROLL
        for (int u = 0; u < C::VUNITS; ++u, codes += C::VW * C::HALF, scales += C::VW * 64) {
#pragma unroll
          for (int k = 0; k < C::VW * C::MB; ++k) {  // 128 channels of a record
            const int r = k / C::MB, mb = k % C::MB, next = k + 1;
            const uint32_t c4[4] = {q4.x, q4.y, q4.z, q4.w};
            // the next 16 bytes: the other channel block's, or the next record's
            if (next < C::VW * C::MB || u + 1 < C::VUNITS)
              q4 = *reinterpret_cast<const uint4*>(codes + next / C::MB * C::HALF +
                                                   next % C::MB * 2048);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 s4 = mine ? *reinterpret_cast<const uint4*>(
                                          scales + mb * 8 * C::VSG + r * 64 + i * 16)
                                    : make_uint4(0, 0, 0, 0);
              w[4 * i] = hmul2(e2m1x2<0>(c4[i]), s4.x);
              w[4 * i + 1] = hmul2(e2m1x2<1>(c4[i]), s4.y);
              w[4 * i + 2] = hmul2(e2m1x2<2>(c4[i]), s4.z);
              w[4 * i + 3] = hmul2(e2m1x2<3>(c4[i]), s4.w);
            }
            if (k == 0) {
              attn_wait(&sh.v_empty[unit], unit_ph, dead);
              tc::fence_after_sync();
            }
            tmem_st16(dst + ((unit * C::VW + r) * C::MB + mb) * 16, w);
          }
          tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.v_full[unit]);
          if (++unit == C::VU) unit = 0, unit_ph ^= 1;
        }
        if (lane == 0) mbar_arrive(&sh.vr_empty[stage]);
        if (++stage == C::VR) stage = 0, raw_ph ^= 1;
      }
    }
  } else if (warp < C::wI) {
    // ------------------------------------------------ softmax and epilogue
    const int group = (warp - C::wS) >> 2, quarter = warp & 3;
    const int c0 = group * C::NH;                      // first row of the group
    const int gt = (threadIdx.x - 32 * C::wS) & 127;   // thread of the group
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    int tile = 0;
    if (threadIdx.x == 32 * C::wS) a.join[blockIdx.x] = AttnJoin{};
    // (the segment stays in the ring until its item is written: registers are short)
    auto find_seg = [&](int no) {
      if (no > 0 || again) attn_wait(&sh.seg_full[no & (kSegs - 1)], (no / kSegs) & 1, dead);
      return sh.seg[no & (kSegs - 1)].t1 > 0 && !__any_sync(0xffffffffu, *dead);
    };
    auto fetch_rows = [&](const Seg& n) {
      k_scale = head_scale(n.h);
      attn_rows_copy<D, NT>(args, n.b, n.h, n.row0, n.rows, smem + C::oQ, warp - C::wS);
    };
    bool more = find_seg(0);
    if (again) {
      cp_async_wait_all();  // of the early copy, to the same place
      if (more) fetch_rows(sh.seg[0]);
    }
    for (;; ++seg_no) {
      // all softmax warps go on, or none: they meet at barriers below
      if (barrier_any(4, 128 * C::NS, !more)) break;
      const Seg& e = sh.seg[seg_no & (kSegs - 1)];
      const float c_all =
          attn_rows<D, NT>(args, sh, e.b, e.row0, e.rows, smem + C::oQ, warp - C::wS,
                       a.scale * (k_scale * kLog2e));
      tc::named_barrier(4, 128 * C::NS);
      if (threadIdx.x == 32 * C::wS) mbar_arrive(&sh.q_full);
      if (gt < C::NH) sh.neg_m[c0 + gt] = -kNone;
      tc::named_barrier(1 + group, 128);
      const int base = e.len - a.N, n_lo = e.row0 / a.G;
      float2 l[C::NH / 2];
#pragma unroll
      for (int i = 0; i < C::NH / 2; ++i) l[i] = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int t = e.t0; t < e.t1; ++t, ++tile) {
        const int buf = tile & 1;
        const unsigned ph = (tile >> 1) & 1;
        attn_wait(&sh.s_full[buf], ph, dead);
        tc::fence_after_sync();
        const int ok = sh.tile_ok[0][tile & (kTiles - 1)];
        const uint32_t sa = lane_base + C::cS + buf * C::NT + c0;
        // rows that see this position, where not all rows see all of the tile
        unsigned vis = ~0u;
        if (ok != 15 || (a.parent != nullptr ? (t + 1) * kTile > base
                                             : (t + 1) * kTile - 1 > base + n_lo)) {
          const int u = t * kTile + quarter * 32 + lane - base;
          if (!((ok >> quarter) & 1)) {
            vis = 0;
          } else if (a.parent == nullptr) {
            // nodes rise with the rows: the first row of node u
            const int64_t from = (int64_t)u * a.G - e.row0 - c0;
            vis = from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from;
          } else if (u >= 0) {
            vis = 0;
            if (u < 64)
#pragma unroll 1
              for (int r = 0; r < C::NH; ++r) {
                const uint2 w = sh.row_path[c0 + r];
                vis |= (((u < 32 ? w.x : w.y) >> (u & 31)) & 1) << r;
              }
          }
        }
        const bool masked = __any_sync(0xffffffffu, vis != ~0u);
        attn_wait(&sh.p_empty[buf], ph ^ 1, dead);
        const uint32_t prow = smem_addr(smem) + C::oP + buf * C::PB + (quarter * 32 + lane) * 128;
        uint32_t y[C::NH / 16][16];
        auto load = [&](uint32_t at) {
#pragma unroll
          for (int k = 0; k < C::NH / 16; ++k) tc::tmem_ld16(at + 16 * k, y[k]);
          tc::tmem_wait_ld(y[0]);
          if constexpr (C::NH == 32) tc::tmem_ready(y[1]);
        };
        // The first tile sets the references; a later one is tried with those there
        // are, and done again in the case that some p passed 2^15.
        bool raise = t == e.t0;
#pragma unroll 1
        for (;;) {
          load(sa);
          if (raise) {
            // ---- new references: kBelow under the largest logits so far
            float x[C::NH];
#pragma unroll
            for (int i = 0; i < C::NH; i += 4) {
              const float4 c = *reinterpret_cast<const float4*>(&sh.row_c[c0 + i]);
              const float c4[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x[i + k] = (vis >> (i + k)) & 1
                               ? __uint_as_float(y[(i + k) / 16][(i + k) % 16]) * c4[k]
                               : -INFINITY;
            }
            const float top = warp_transpose_reduce(
                x, [](float p, float q) { return q > p || q != q ? q : p; });
            if (lane < C::NH) sh.part[quarter][c0 + lane] = top;
            tc::named_barrier(1 + group, 128);
            if (gt < C::NH) {
              const int r = c0 + gt;
              const float old = -sh.neg_m[r];
              float m = old;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float w = sh.part[q][r] - kBelow;
                m = w > m || w != w ? w : m;
              }
              sh.neg_m[r] = -m;
              sh.alpha[r] = exp2_fast(old - m);
            }
            tc::named_barrier(1 + group, 128);
            if (t != e.t0) {
              // every product into O^T so far is done: the last one freed its P
              attn_wait(&sh.p_empty[buf ^ 1], ((tile - 1) >> 1) & 1, dead);
              tc::fence_after_sync();
#pragma unroll
              for (int k = 0; k < C::NH / 2; ++k) {
                l[k].x *= sh.alpha[c0 + 2 * k];
                l[k].y *= sh.alpha[c0 + 2 * k + 1];
              }
#pragma unroll 1
              for (int k = 0; k < C::MB * C::NH; k += 8) {
                const int col = c0 + k % C::NH;
                const uint32_t oa = lane_base + C::cO + k / C::NH * C::NT + col;
                uint32_t o[8];
                tc::tmem_ld8(oa, o);
                tc::tmem_wait_ld(o);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  o[i] = __float_as_uint(__uint_as_float(o[i]) * sh.alpha[col + i]);
                tmem_st8(oa, o);
              }
              tmem_wait_st();
            }
            load(sa);
          }
          // ---- p, and P as the B operand
#pragma unroll
          for (int i = 0; i < C::NH; i += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&sh.neg_m[c0 + i]);
            float4 c = make_float4(c_all, c_all, c_all, c_all);
            if (!C::COMMON || c_all == 0.f) c = *reinterpret_cast<const float4*>(&sh.row_c[c0 + i]);
            uint32_t* z = &y[i / 16][i % 16];
            const float2 z0 = fma2(make_float2(__uint_as_float(z[0]), __uint_as_float(z[1])),
                                   make_float2(c.x, c.y), make_float2(m.x, m.y));
            const float2 z1 = fma2(make_float2(__uint_as_float(z[2]), __uint_as_float(z[3])),
                                   make_float2(c.z, c.w), make_float2(m.z, m.w));
            z[0] = __float_as_uint(exp2_fast(z0.x)), z[1] = __float_as_uint(exp2_fast(z0.y));
            z[2] = __float_as_uint(exp2_fast(z1.x)), z[3] = __float_as_uint(exp2_fast(z1.y));
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < C::NH; ++i)
              if (!((vis >> i) & 1)) y[i / 16][i % 16] = 0;
          }
          unsigned top = 0;
#pragma unroll
          for (int k = 0; k < C::NH; k += 8) {
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = k + 2 * i;
              p[i] = pack_f16x2(__uint_as_float(y[at / 16][at % 16]),
                                __uint_as_float(y[at / 16][at % 16 + 1]));
              top = __vmaxu2(top, p[i]);  // p >= 0: ordered as integers
            }
            const int col = c0 + k;  // 16-byte chunk of 8 rows, swizzled by position
            st_shared16(prow + (col >> 6) * (kTile * 128) +
                            ((((col & 63) >> 3) ^ (lane & 7)) << 4), p);
          }
          if (raise) break;
          raise = barrier_any(1 + group, 128, max(top & 0xffffu, top >> 16) > kMostP);
          if (!raise) break;
        }
#pragma unroll
        for (int i = 0; i < C::NH; i += 2)
          l[i / 2] = add2(l[i / 2], make_float2(__uint_as_float(y[i / 16][i % 16]),
                                                __uint_as_float(y[i / 16][i % 16 + 1])));
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.s_empty[buf]), mbar_arrive(&sh.p_full[buf]);
      }
      // S^T's products are done, and Q is free: the next rows are on their way
      // while this item is written
      more = find_seg(seg_no + 1);
      if (more) fetch_rows(sh.seg[(seg_no + 1) & (kSegs - 1)]);
      // ---- epilogue
      const bool whole = e.t0 == 0 && e.t1 == e.tiles;
      const int64_t item = (int64_t)e.b * a.N * a.Hq + e.h * a.G;  // output row of node 0
      const int64_t slot = 2 * (int64_t)blockIdx.x + (seg_no > 0);
      {
        float x[C::NH];
#pragma unroll
        for (int i = 0; i < C::NH / 2; ++i) x[2 * i] = l[i].x, x[2 * i + 1] = l[i].y;
        const float sum = warp_transpose_reduce(x, [](float p, float q) { return p + q; });
        if (lane < C::NH) sh.part[quarter][c0 + lane] = sum;
      }
      if (e.t0 == 0 && !whole)  // at most one: the rest of the item is the next blocks'
        if (threadIdx.x == 32 * C::wS)
          a.join[blockIdx.x] = {item, e.h, e.row0, e.rows, (int)slot, e.last};
      tc::named_barrier(1 + group, 128);
      if (gt < C::NH) {
        const int r = c0 + gt;
        const float total = sh.part[0][r] + sh.part[1][r] + sh.part[2][r] + sh.part[3][r];
        const float m = -sh.neg_m[r];
        float inv = 1.f;
        if (whole) {
          inv = total != 0.f ? (a.c.v_scale != nullptr ? a.c.v_scale[e.h] : 1.f) / total : 0.f;
          if (a.lse != nullptr && r < e.rows)
            a.lse[item + sh.row_at[r]] =
                total != 0.f ? (m + log2f(total)) * 0.6931471805599453f : -INFINITY;
        } else {
          a.part_ml[slot * NT + r] = make_float2(m, total);
        }
        sh.inv[r] = inv;
      }
      attn_wait(&sh.o_full, seg_no & 1, dead);
      tc::fence_after_sync();
      tc::named_barrier(1 + group, 128);
#pragma unroll 1
      for (int mb = 0; mb < C::MB; ++mb) {
        const int ch = mb * 128 + quarter * 32 + lane;
        uint32_t o[C::NH / 16][16];
#pragma unroll
        for (int k = 0; k < C::NH / 16; ++k)
          tc::tmem_ld16(lane_base + C::cO + mb * C::NT + c0 + 16 * k, o[k]);
        tc::tmem_wait_ld(o[0]);
        if constexpr (C::NH == 32) tc::tmem_ready(o[1]);
        if (D < 128 && ch >= D) continue;
        const int rows = e.rows - c0;
        if (whole) {
          uint16_t* out = static_cast<uint16_t*>(a.o) + item * D + ch;
#pragma unroll
          for (int i = 0; i < C::NH; i += 4) {
            const int4 at = *reinterpret_cast<const int4*>(&sh.row_at[c0 + i]);
            const float4 inv = *reinterpret_cast<const float4*>(&sh.inv[c0 + i]);
            const int at_[4] = {at.x, at.y, at.z, at.w};
            const float inv_[4] = {inv.x, inv.y, inv.z, inv.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (i + k >= rows) break;
              const float v = __uint_as_float(o[i / 16][i % 16 + k]) * inv_[k];
              out[(int64_t)at_[k] * D] =
                  a.bf16 ? Elem<GDN_BF16>::from(v) : Elem<GDN_F16>::from(v);
            }
          }
        } else {
          float* out = a.part_o + (slot * NT + c0) * D + ch;
#pragma unroll
          for (int i = 0; i < C::NH; ++i) {
            if (i >= rows) break;
            out[i * D] = __uint_as_float(o[i / 16][i % 16]);
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_empty), mbar_arrive(&sh.seg_empty[seg_no & (kSegs - 1)]);
    }
    cp_async_wait_all();  // (only where a wait ran out are there any)
  } else if (warp == C::wI) {
    // ------------------------------------------------ S^T products (one elected lane)
    constexpr uint32_t id = idesc_f16(NT, false);
    // descriptors advance by 16-byte units in their low word
    const uint64_t desc = tc::sdesc_sw128(smem_addr(smem + C::oQ), 16, 1024);
    int tile = 0, ku = 0;
    unsigned ku_ph = 0;
    for (; next_seg(); ++seg_no) {
      attn_wait(&sh.q_full, seg_no & 1, dead);
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        const int buf = tile & 1;
        attn_wait(&sh.s_empty[buf], ((tile >> 1) & 1) ^ 1, dead);
        const uint32_t d = C::cS + buf * NT;
#pragma unroll 1
        for (int u = 0; u < C::UNITS; ++u) {
          const bool live = attn_wait(&sh.k_full[ku], ku_ph, dead);
          tc::fence_after_sync();
          const uint64_t q = desc + (uint32_t)(u * (C::KW / 32) * NT * 8);
          const uint32_t ka = ku * C::KW;
          if (elect_one() && live) {
#pragma unroll
            for (int k = 0; k < C::KW / 8; ++k)
              mma_ts(d, ka + k * 8, q + (k / 4 * NT * 128 + k % 4 * 32) / 16, id, u > 0 || k > 0);
            tc::mma_commit(&sh.k_empty[ku]);
            if (u + 1 == C::UNITS) tc::mma_commit(&sh.s_full[buf]);
          }
          if (++ku == C::KU) ku = 0, ku_ph ^= 1;
        }
      }
    }
  } else if (warp == C::wI + 1) {
    // ------------------------------------------------ O^T products (one elected lane)
    constexpr uint32_t id = idesc_f16(NT, true);
    const uint64_t desc = tc::sdesc_sw128(smem_addr(smem + C::oP), kTile * 128, 1024);
    int tile = 0, vu = 0;
    unsigned vu_ph = 0;
    for (; next_seg(); ++seg_no) {
      attn_wait(&sh.o_empty, (seg_no & 1) ^ 1, dead);
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        const int buf = tile & 1;
        attn_wait(&sh.p_full[buf], (tile >> 1) & 1, dead);
        const uint64_t p = desc + (uint32_t)(buf * (C::PB >> 4));
#pragma unroll 1
        for (int u = 0; u < C::VUNITS; ++u) {
          const bool live = attn_wait(&sh.v_full[vu], vu_ph, dead);
          tc::fence_after_sync();
          const uint64_t pu = p + (uint32_t)(u * C::VW * 256);
          const uint32_t va = C::cV + vu * C::VW * C::MB * 16;
          if (elect_one() && live) {
#pragma unroll
            for (int r = 0; r < C::VW; ++r)
#pragma unroll
              for (int mb = 0; mb < C::MB; ++mb) {
                const uint32_t d = C::cO + mb * NT, v = va + (r * C::MB + mb) * 16;
                mma_ts(d, v, pu + r * 256, id, t > s.t0 || u > 0 || r > 0);
                mma_ts(d, v + 8, pu + r * 256 + 128, id, 1);
              }
            tc::mma_commit(&sh.v_empty[vu]);
            if (u + 1 == C::VUNITS) {
              tc::mma_commit(&sh.p_empty[buf]);
              if (t + 1 == s.t1) tc::mma_commit(&sh.o_full);
            }
          }
          if (++vu == C::VU) vu = 0, vu_ph ^= 1;
        }
      }
    }
  } else {
    // ------------------------------------------------ the run's segments, the records in
    const bool lead = warp == C::wI + 2, do_k = C::FW == 1 || lead, do_v = C::FW == 1 || !lead;
    Run run = sh.run;
    if (lead && again) run = attn_run(args, lens, blockIdx.x, gridDim.x);
    // lanes 2r and 2r + 1: codes and scales of record r's K half, lanes 8 + 2r and
    // 9 + 2r: of its V half (the first eight lanes where a warp has V alone)
    const int lanes = C::FW == 1 ? 16 : 8;
    const bool is_k = C::FW == 1 ? lane < 8 : lead;
    const int r = (lane & 7) >> 1, part = lane & 1;
    const int from = part == 0 ? (is_k ? 0 : off_v(D)) : (is_k ? off_ks(D) : off_vs(D));
    const int bytes = part == 0 ? 16 * D : 2 * D;
    int k_stage = 0, v_stage = 0, tile = 0;
    unsigned k_ph = 1, v_ph = 1;
    for (;; ++seg_no) {
      if (lead) {
        const bool ready = seg_no == 0 && !again;
        s = ready ? sh.seg[0] : attn_seg(args, lens, run);
        const int i = seg_no & (kSegs - 1);
        // (the ring's first pass: empty, and the first segment's readers may be ahead)
        if (seg_no >= kSegs) attn_wait(&sh.seg_empty[i], ((seg_no / kSegs) & 1) ^ 1, dead);
        if (lane == 0) {
          if (!ready) sh.seg[i] = s;
          mbar_arrive(&sh.seg_full[i]);
        }
        if (s.t1 == 0) break;
      } else if (!next_seg()) {
        break;
      }
      const int32_t* table = a.c.table + (int64_t)s.b * a.c.table_stride;
      const uint8_t* head = static_cast<const uint8_t*>(a.c.pages) + from +
                            (int64_t)s.h * (a.c.page_tokens / kRec) * rec_bytes(D);
      // this lane's position, as an entry of the table and an offset in the page, two
      // tiles ahead of the copies: the page numbers are looked up that early
      int pos = s.t0 * kTile + r * kRec;
      int entry = pos / a.c.page_tokens, off = pos % a.c.page_tokens;
      const int entries = kTile / a.c.page_tokens, rest = kTile % a.c.page_tokens;
      int page[3], offs[3];
      auto look_up = [&](int i, int t) {
        page[i] = lane < lanes && t < s.t1 && t * kTile + r * kRec < s.len ? table[entry] : -1;
        offs[i] = off;
        entry += entries;
        off += rest;
        if (off >= a.c.page_tokens) off -= a.c.page_tokens, ++entry;
      };
      look_up(0, s.t0);
      look_up(1, s.t0 + 1);
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        const bool want = lane < lanes && pos < s.len;  // past the end: nothing to read
        look_up(2, t + 2);
        const bool have = want && page[0] >= 0 && page[0] < a.c.n_pages;
        if (want && !have) report(a.c.status, GDN_ERR_PAGE_RANGE);
        const uint8_t* src = head;
        if (have)
          src += (int64_t)page[0] * a.c.page_stride + offs[0] / kRec * rec_bytes(D);
        pos += kTile;
        page[0] = page[1], offs[0] = offs[1], page[1] = page[2], offs[1] = offs[2];
        const unsigned good = __ballot_sync(0xffffffffu, have || !want);
        const unsigned tx = __popc(__ballot_sync(0xffffffffu, have) & 0x55u) * C::HALF;
        const int ok = (good & 1) | ((good >> 1) & 2) | ((good >> 2) & 4) | ((good >> 3) & 8);
        if (do_k) {
          attn_wait(&sh.kr_empty[k_stage], k_ph, dead);
          if (lane == 0) {
            sh.tile_ok[0][tile & (kTiles - 1)] = ok;
            mbar_arrive_expect_tx(&sh.kr_full[k_stage], tx);
          }
          __syncwarp();
          if (have && is_k)
            bulk_g2s(smem + C::oK + k_stage * C::RAW + r * C::HALF + part * 16 * D, src, bytes,
                     &sh.kr_full[k_stage]);
        }
        if (do_v) {
          attn_wait(&sh.vr_empty[v_stage], v_ph, dead);
          if (lane == 0) {
            sh.tile_ok[1][tile & (kTiles - 1)] = ok;
            mbar_arrive_expect_tx(&sh.vr_full[v_stage], tx);
          }
          __syncwarp();
          if (have && !is_k)
            bulk_g2s(smem + C::oV + v_stage * C::RAW + r * C::HALF + part * 16 * D, src, bytes,
                     &sh.vr_full[v_stage]);
        }
        if (++k_stage == C::KR) k_stage = 0, k_ph ^= 1;
        if (++v_stage == C::VR) v_stage = 0, v_ph ^= 1;
      }
    }
    if (__any_sync(0xffffffffu, *dead)) {  // copies in flight land before the block ends
      for (int i = 0; do_k && i < C::KR && i < tile; ++i)
        (void)mbar_wait_bounded(&sh.kr_full[i], ((tile - i - 1) / C::KR) & 1, kWaitPolls);
      for (int i = 0; do_v && i < C::VR && i < tile; ++i)
        (void)mbar_wait_bounded(&sh.vr_full[i], ((tile - i - 1) / C::VR) & 1, kWaitPolls);
    }
  }
  // every role is done with its loops, hence with its copies and products; after a
  // wait that ran out, products in flight end (bounded) before TMEM is given back
  if ((warp == C::wI || warp == C::wI + 1) && __any_sync(0xffffffffu, *dead)) {
    if (elect_one()) tc::mma_commit(&sh.drain);
    (void)mbar_wait_bounded(&sh.drain, 0, kWaitPolls);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *dead) report(a.c.status, GDN_ERR_TIMEOUT);
  if (warp == C::wI) {
    tc::fence_after_sync();
    tc::tmem_relinquish();
    tc::tmem_dealloc(sh.tmem, 512);
  }
}

// ---------------------------------------------------------------- join
// Grid (blocks of the main kernel, pieces of the rows): the item that block x
// left unfinished, if any: the parts of blocks x .. last, in that order.  A thread
// has four channels, of one row; with few rows (NT = 16) the block's threads share
// one row and take every NP-th part each, else each D/4 of them take a row.  Bound
// by latency: it ends 3.3 us after the last block of the main kernel for eight chains
// (32 items over 152 blocks, 15 MB of parts), 4.6 us for a tree (8 items, 19 parts
// each), 5.2 us for one sequence (4 items, 38 parts each).
constexpr int kJoinThreads = 256;

template <int D, bool ONE_ROW>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const __grid_constant__ AttnArgs a, int NT) {
  constexpr int Q = D / 4, NP = kJoinThreads / Q, STEP = ONE_ROW ? NP : 1;
  __shared__ __align__(16) float acc[ONE_ROW ? NP : 1][D];
  __shared__ float2 sums[NP];
  pdl_enter();
  const AttnJoin j = a.join[blockIdx.x];
  const int quad = threadIdx.x % Q, group = threadIdx.x / Q;
  const int r = ONE_ROW ? blockIdx.y : blockIdx.y * NP + group;
  if (r >= j.rows) return;  // ONE_ROW: all of the block
  const int parts = j.last - (int)blockIdx.x + 1;
  auto at = [&](int i) {
    return (i == 0 ? (int64_t)j.slot : 2 * ((int64_t)blockIdx.x + i)) * NT + r;
  };
  // a running maximum, so that nothing is read twice and the reads overlap
  float top = kNone, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto larger = [](float p, float q) { return q > p || q != q ? q : p; };  // NaN stays
  constexpr int U = 8;
#pragma unroll 1
  for (int i0 = ONE_ROW ? group : 0; i0 < parts; i0 += U * STEP) {
    float2 ml[U];
    float4 p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * STEP;
      ml[u] = make_float2(kNone, 0.f);
      p[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < parts) {
        ml[u] = a.part_ml[at(i)];
        p[u] = __ldcg(reinterpret_cast<const float4*>(a.part_o + at(i) * D) + quad);
      }
    }
    float m = top;
#pragma unroll
    for (int u = 0; u < U; ++u) m = larger(m, ml[u].x);
    const float keep = exp2_fast(top - m);
    top = m;
    sum *= keep;
    o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = exp2_fast(ml[u].x - m);
      sum += w * ml[u].y;
      o.x += w * p[u].x, o.y += w * p[u].y, o.z += w * p[u].z, o.w += w * p[u].w;
    }
  }
  if constexpr (ONE_ROW) {
    *reinterpret_cast<float4*>(&acc[group][quad * 4]) = o;
    if (quad == 0) sums[group] = make_float2(top, sum);
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int g = 0; g < NP; ++g) top = larger(top, sums[g].x);
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    sum = 0.f;
#pragma unroll
    for (int g = 0; g < NP; ++g) {
      const float4 p = *reinterpret_cast<const float4*>(&acc[g][quad * 4]);
      const float w = exp2_fast(sums[g].x - top);
      o.x += w * p.x, o.y += w * p.y, o.z += w * p.z, o.w += w * p.w;
      sum += w * sums[g].y;
    }
  }
  const int row = j.row0 + r;
  const int64_t out = j.item + (int64_t)(row / a.G) * a.Hq + row % a.G;
  const float inv =
      sum != 0.f ? (a.c.v_scale != nullptr ? a.c.v_scale[j.h] : 1.f) / sum : 0.f;
  const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = a.bf16 ? Elem<GDN_BF16>::from(v[i]) : Elem<GDN_F16>::from(v[i]);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + out * D + quad * 4) =
      make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
  if (a.lse != nullptr && quad == 0)
    a.lse[out] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

template <int D, int NT>
int attn_launch_nt(const AttnArgs& a, int parts, cudaStream_t s) {
  using C = AttnCfg<D, NT>;
  if (cudaFuncSetAttribute(attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::SMEM) != cudaSuccess) {
    (void)cudaGetLastError();
    return GDN_ERR_CUDA;
  }
  const int rc = launch_pdl(attn_kernel<D, NT>, dim3(parts), dim3(C::THREADS), C::SMEM, s, a);
  if (rc != GDN_OK) return rc;
  const dim3 block(kJoinThreads);
  if (NT == 16)
    return launch_pdl(join_kernel<D, true>, dim3(parts, a.rows_per_tile), block, 0, s, a, NT);
  constexpr int NP = kJoinThreads / (D / 4);
  return launch_pdl(join_kernel<D, false>, dim3(parts, (a.rows_per_tile + NP - 1) / NP), block, 0,
                    s, a, NT);
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
