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
//   16     issues S^T's MMAs      19   issues O^T's
//   17     the run's segments, bulk copies of records, V scales to binary16
//   18     query rows: to binary16, scaled by a power of two per row so that
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
  int at;          // row of the output, from the item's first node and head on
  unsigned lo, hi; // trees: the positions of the block that the row sees
};

// The part of one item that a block works on: tiles [t0, t1) of `tiles` (t1 = 0: the end).
struct Seg {
  int b, h, t0, t1, tiles, len, row0, rows;
  int last;  // block that holds the item's last tile
};

constexpr int kSegs = 16;    // ring of segments; a block's warps are fewer apart
constexpr int kLens = 1024;  // lengths kept in shared memory

template <typename C>
struct AttnShared {
  uint64_t raw_full[C::NRAW], raw_empty[C::NRAW];
  uint64_t k_full[C::KU], k_empty[C::KU], v_full[C::VU], v_empty[C::VU];
  uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], vs_full[2], vs_empty[2];
  uint64_t q_full[C::NQ], q_empty[C::NQ], row_full[2], row_empty[2], o_full, o_empty, drain;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint32_t tmem;
  int dead;
  int tile_ok[8];  // records of a tile that could be read, by tile number
  alignas(16) float2 cm[C::NT];  // (c, m) of the rows in work; read two rows a load
  alignas(16) Seg seg[kSegs];
  alignas(16) Row row[2][C::NT];
  float alpha[C::NT], inv[C::NT];
  float wmax[4][C::NT];
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

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The lengths the block works with: the first kLens are kept in shared memory.
struct Lens {
  const AttnArgs& a;
  const int* kept;
  __device__ __forceinline__ int operator()(int b) const {
    return b < kLens ? kept[b] : attn_len(a, b, false);
  }
};

// Lengths into shared memory, by all threads: a thread a sequence, or for
// trees a warp a sequence (its lanes check the nodes).
__device__ __forceinline__ void attn_lens(const AttnArgs& a, int* kept, bool report_it) {
  if (a.parent == nullptr) {
#pragma unroll 1
    for (int b = threadIdx.x; b < min(a.c.B, kLens); b += blockDim.x)
      kept[b] = seq_len(a.c, b, report_it);
    return;
  }
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int b = threadIdx.x >> 5; b < min(a.c.B, kLens); b += blockDim.x >> 5) {
    const int32_t* p = a.parent + (int64_t)b * a.N;
    bool ok = true;
    for (int n = lane; n < a.N; n += 32) ok = ok && (n == 0 ? p[n] == -1 : p[n] >= 0 && p[n] < n);
    ok = __all_sync(0xffffffffu, ok);
    if (lane == 0) {
      const int len = seq_len(a.c, b, report_it);
      if (report_it && len > 0 && !ok) report(a.c.status, GDN_ERR_BAD_TREE);
      kept[b] = ok ? len : 0;
    }
  }
  if (report_it)  // the others' reports (their lengths are looked up when needed)
#pragma unroll 1
    for (int b = kLens + threadIdx.x; b < a.c.B; b += blockDim.x) (void)attn_len(a, b, true);
}

// Tiles of sequence b over all heads, by a whole warp.
__device__ __forceinline__ int64_t warp_cost(const AttnArgs& a, int len) {
  int64_t t = 0;
#pragma unroll 1
  for (int rt = threadIdx.x & 31; rt < a.row_tiles; rt += 32) t += attn_tiles(a, len, rt);
  return warp_sum(t) * a.c.Hkv;
}

// Equal runs of `total` tiles for at most `parts` blocks: the first `extra` runs
// have one tile more.
struct Runs {
  int64_t each, extra;
  int parts;
  __device__ __forceinline__ Runs(int64_t total, int n) {
    parts = total < n ? (int)total : n;  // no empty runs in between
    each = parts > 0 ? total / parts : 0;
    extra = total - each * parts;
  }
  __device__ __forceinline__ int64_t start(int part) const {
    return each * part + (part < extra ? part : extra);
  }
  // the run that holds tile x
  __device__ __forceinline__ int of(int64_t x) const {
    const int64_t head = extra * (each + 1);
    return (int)(x < head ? x / (each + 1) : extra + (x - head) / each);
  }
};

// Walks the tiles of a block's run, item by item (one warp).
struct Run {
  int b, h, rt, t0;
  int64_t at, left;
  Runs runs;
};

// The run of block `part` of `parts`: the tiles of all sequences are counted,
// then the sequence that holds the run's first tile is taken apart.
static __device__ __noinline__ Run attn_run(const AttnArgs& a, const Lens& lens, int part, int parts) {
  const int lane = threadIdx.x & 31;
  const bool by_lane = a.row_tiles <= 4;  // a lane a sequence, or the warp a sequence
  int64_t total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.c.B; b0 += by_lane ? 32 : 1) {
    if (by_lane) {
      if (b0 + lane < a.c.B) {
        const int len = lens(b0 + lane);
#pragma unroll 1
        for (int rt = 0; rt < a.row_tiles; ++rt) total += attn_tiles(a, len, rt);
      }
    } else {
      total += warp_cost(a, lens(b0));
    }
  }
  if (by_lane) total = warp_sum(total) * a.c.Hkv;
  const Runs runs(total, parts);
  Run r = {0, 0, 0, 0, 0, 0, runs};
  if (part >= runs.parts) return r;
  const int64_t start = runs.start(part);
  r.at = start;
  r.left = runs.start(part + 1) - start;
  int64_t before = 0, its = 0;
#pragma unroll 1
  for (int b0 = 0;; b0 += by_lane ? 32 : 1) {
    if (by_lane) {
      int64_t mine = 0;
      if (b0 + lane < a.c.B) {
        const int len = lens(b0 + lane);
#pragma unroll 1
        for (int rt = 0; rt < a.row_tiles; ++rt) mine += attn_tiles(a, len, rt);
        mine *= a.c.Hkv;
      }
      int64_t x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + x > start);
      if (hit == 0) {
        before += __shfl_sync(0xffffffffu, x, 31);
        continue;
      }
      const int l = __ffs(hit) - 1;
      its = __shfl_sync(0xffffffffu, mine, l);
      before += __shfl_sync(0xffffffffu, x, l) - its;
      r.b = b0 + l;
    } else {
      its = warp_cost(a, lens(b0));
      if (before + its <= start) {
        before += its;
        continue;
      }
      r.b = b0;
    }
    break;
  }
  int in = (int)(start - before);  // of the sequence's its tiles
  const int per_head = (int)(its / a.c.Hkv), len = lens(r.b);
  r.h = in / per_head;
  in -= r.h * per_head;
#pragma unroll 1
  for (;; ++r.rt) {
    const int t = attn_tiles(a, len, r.rt);
    if (in < t) break;
    in -= t;
  }
  r.t0 = in;
  return r;
}

// The run's next segment (t1 = 0 when it is at its end).
static __device__ __noinline__ Seg attn_seg(const AttnArgs& a, const Lens& lens, Run& r) {
  Seg s = {};
#pragma unroll 1
  while (r.left > 0 && r.b < a.c.B) {
    const int len = lens(r.b);
    const int tiles = attn_tiles(a, len, r.rt);
    const int t0 = r.t0, rt = r.rt, h = r.h, b = r.b;
    r.t0 = 0;
    if (++r.rt == a.row_tiles) {
      r.rt = 0;
      if (++r.h == a.c.Hkv) r.h = 0, ++r.b;
    }
    if (tiles <= t0) continue;
    s.b = b, s.h = h, s.t0 = t0, s.tiles = tiles, s.len = len;
    s.t1 = r.left < tiles - t0 ? t0 + (int)r.left : tiles;
    r.left -= s.t1 - t0;
    r.at += s.t1 - t0;
    s.last = s.t1 < tiles ? r.runs.of(r.at + tiles - s.t1 - 1) : 0;
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
      mbar_init(&sh.row_full[i], 1), mbar_init(&sh.row_empty[i], 8);
    }
    for (int i = 0; i < C::NQ; ++i) mbar_init(&sh.q_full[i], 1), mbar_init(&sh.q_empty[i], 1);
    for (int i = 0; i < kSegs; ++i) mbar_init(&sh.seg_full[i], 1), mbar_init(&sh.seg_empty[i], 19);
    mbar_init(&sh.o_full, 1);
    mbar_init(&sh.o_empty, 8);
    mbar_init(&sh.drain, 2);
    sh.dead = 0;
    mbar_init_fence();
  }
  if (warp == 16) tc::tmem_alloc(&sh.tmem, 512);
  pdl_enter();
  attn_lens(a, sh.len, blockIdx.x == 0);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // all 512 columns are this block's, so its tensor memory begins at address 0
  if (sh.tmem != 0) *dead = 1;
  constexpr uint32_t tmem = 0;

  // every warp but 17 takes the run's segments from the ring
  int seg_no = 0;
  Seg s;
  auto next_seg = [&]() {
    const int i = seg_no & (kSegs - 1);
    attn_wait(&sh.seg_full[i], (seg_no / kSegs) & 1, dead);
    s = sh.seg[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.seg_empty[i]);
    return s.t1 > 0 && !__any_sync(0xffffffffu, *dead);
  };

  if (warp < 4) {
    // ------------------------------------------------ K -> TMEM
    const uint32_t dst = tmem + ((uint32_t)(warp * 32) << 16);
    int stage = 0, unit = 0;
    unsigned raw_ph = 0, unit_ph = 1;  // an empty ring's first pass does not wait
    for (; next_seg(); ++seg_no) {
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t) {
        attn_wait(&sh.raw_full[stage], raw_ph, dead);
        const uint8_t* rec = smem + C::oRaw + stage * C::RAW + warp * rec_bytes(D);
#pragma unroll 1
        for (int u = 0; u < C::UNITS; ++u) {
          const uint32_t s8 =
              *reinterpret_cast<const uint32_t*>(rec + off_ks(D) + lane * (D / 16) + u * 4);
          uint32_t w[32];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint4 q4 = *reinterpret_cast<const uint4*>(rec + (2 * u + half) * 512 + lane * 16);
            const uint32_t sc = e4m3x2(s8 >> (16 * half));
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
        if (lane == 0) mbar_arrive(&sh.raw_empty[stage]);
        if (++stage == C::NRAW) stage = 0, raw_ph ^= 1;
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------ V^T -> TMEM
    const int quarter = warp - 4;
    const uint32_t dst = tmem + ((uint32_t)(quarter * 32) << 16) + C::cV;
    attn_zero(a, Lens{a, sh.len}, D, threadIdx.x - 128);
    int stage = 0, unit = 0, vb = 0;
    unsigned vs_ph = 0, unit_ph = 1;
    for (; next_seg(); ++seg_no) {
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t) {
        attn_wait(&sh.vs_full[vb], vs_ph, dead);  // the records have landed before
        const uint8_t* raw = smem + C::oRaw + stage * C::RAW;
        const uint8_t* vs = smem + C::oVS + vb * C::VSB;
#pragma unroll 1
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
    int tile = 0;
    AttnJoin join = {};
    for (;; ++seg_no) {
      // all eight warps go on, or none: they meet at barriers below
      if (barrier_any(3, 256, !next_seg())) break;
      const int base = s.len - a.N;
      const int n_lo = s.row0 / a.G;
      const Row* rows = sh.row[seg_no & 1];
      attn_wait(&sh.row_full[seg_no & 1], (seg_no >> 1) & 1, dead);
      if (gt < C::NH) sh.cm[c0 + gt] = make_float2(rows[c0 + gt].c, kNone);
      tc::named_barrier(1 + group, 128);
      float l[C::NH];
#pragma unroll
      for (int i = 0; i < C::NH; ++i) l[i] = 0.f;
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        const int buf = tile & 1;
        const unsigned ph = (tile >> 1) & 1;
        attn_wait(&sh.s_full[buf], ph, dead);
        tc::fence_after_sync();
        const int ok = sh.tile_ok[tile & 7];
        const uint32_t sa = lane_base + C::cS + buf * C::NT + c0;
        // rows that see this position, where not all rows see all of the tile
        const bool masked = ok != 15 || (a.parent != nullptr ? (t + 1) * kTile > base
                                                             : (t + 1) * kTile - 1 > base + n_lo);
        unsigned long long vis = ~0ull;
        if (masked) {
          const int u = t * kTile + quarter * 32 + lane - base;
          if (!((ok >> quarter) & 1)) {
            vis = 0;
          } else if (a.parent == nullptr) {
            // nodes rise with the rows: the first row of node u
            const int64_t from = (int64_t)u * a.G - s.row0 - c0;
            vis = from <= 0 ? ~0ull : from >= 64 ? 0ull : ~0ull << from;
          } else if (u >= 0) {
            vis = 0;
            if (u < 64)
#pragma unroll 1
              for (int r = 0; r < C::NH; ++r) {
                const Row& w = rows[c0 + r];
                vis |= (unsigned long long)(((u < 32 ? w.lo : w.hi) >> (u & 31)) & 1) << r;
              }
          }
        }
        // ---- would any p pass 2^kSlack?  (first tile: yes)
        bool raise = t == s.t0;
        if (!raise) {
          float top = -INFINITY;
#pragma unroll 1
          for (int k = 0; k < C::NH; k += CH) {
            uint32_t x[CH];
            tmem_load(sa + k, x);
            tc::tmem_wait_ld(x);
            const unsigned v = (unsigned)(vis >> k);
#pragma unroll
            for (int i = 0; i < CH; i += 2) {
              const float4 cm = *reinterpret_cast<const float4*>(&sh.cm[c0 + k + i]);
              float y0 = fmaf(__uint_as_float(x[i]), cm.x, -cm.y);
              float y1 = fmaf(__uint_as_float(x[i + 1]), cm.z, -cm.w);
              if (masked) {
                y0 = (v >> i) & 1 ? y0 : -INFINITY;
                y1 = (v >> (i + 1)) & 1 ? y1 : -INFINITY;
              }
              top = fmaxf(top, fmaxf(y0, y1));
            }
          }
          raise = barrier_any(1 + group, 128, top > kSlack);  // NaN rows stay NaN without it
        }
        if (raise) {
          // ---- new references: the largest logits so far
#pragma unroll 1
          for (int k = 0; k < C::NH; k += CH) {
            uint32_t x[CH];
            tmem_load(sa + k, x);
            tc::tmem_wait_ld(x);
            const unsigned v = (unsigned)(vis >> k);
            float mine = 0.f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              float y = __uint_as_float(x[i]) * sh.cm[c0 + k + i].x;
              y = warp_max((v >> i) & 1 ? y : -INFINITY);
              if (lane == i) mine = y;
            }
            if (lane < CH) sh.wmax[quarter][c0 + k + lane] = mine;
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
          if (t != s.t0) {
            // every product into O^T so far is done: the last one freed its P
            attn_wait(&sh.p_empty[buf ^ 1], ((tile - 1) >> 1) & 1, dead);
            tc::fence_after_sync();
#pragma unroll
            for (int k = 0; k < C::NH; ++k) l[k] *= sh.alpha[c0 + k];
#pragma unroll 1
            for (int k = 0; k < C::MB * C::NH; k += 8) {
              const int col = c0 + k % C::NH;
              const uint32_t oa = lane_base + C::cO + k / C::NH * C::NT + col;
              uint32_t x[8];
              tc::tmem_ld8(oa, x);
              tc::tmem_wait_ld(x);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                x[i] = __float_as_uint(__uint_as_float(x[i]) * sh.alpha[col + i]);
              tmem_st8(oa, x);
            }
            tmem_wait_st();
          }
        }
        // ---- p, its sums, and P as the B operand
        attn_wait(&sh.p_empty[buf], ph ^ 1, dead);
        uint8_t* prow = smem + C::oP + buf * C::PB + (quarter * 32 + lane) * 128;
#pragma unroll
        for (int k = 0; k < C::NH; k += CH) {
          uint32_t x[CH];
          tmem_load(sa + k, x);
          tc::tmem_wait_ld(x);
          uint32_t p[CH / 2];
          const unsigned v = (unsigned)(vis >> k);
#pragma unroll
          for (int i = 0; i < CH; i += 2) {
            const float4 cm = *reinterpret_cast<const float4*>(&sh.cm[c0 + k + i]);
            float y0 = exp2_fast(fmaf(__uint_as_float(x[i]), cm.x, -cm.y));
            float y1 = exp2_fast(fmaf(__uint_as_float(x[i + 1]), cm.z, -cm.w));
            if (masked) {
              y0 = (v >> i) & 1 ? y0 : 0.f;
              y1 = (v >> (i + 1)) & 1 ? y1 : 0.f;
            }
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
        fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.s_empty[buf]), mbar_arrive(&sh.p_full[buf]);
      }
      // ---- epilogue
      const bool whole = s.t0 == 0 && s.t1 == s.tiles;
      const int64_t item = (int64_t)s.b * a.N * a.Hq + s.h * a.G;  // output row of node 0
      attn_wait(&sh.o_full, seg_no & 1, dead);
      tc::fence_after_sync();
      float* sums = reinterpret_cast<float*>(smem + C::oP) + c0 * 129;  // P is free now
#pragma unroll
      for (int k = 0; k < C::NH; ++k) sums[k * 129 + gt] = l[k];
      tc::named_barrier(1 + group, 128);
      const int64_t slot = 2 * (int64_t)blockIdx.x + (seg_no > 0);
      if (s.t0 == 0 && !whole)  // at most one: the rest of the item is the next blocks'
        join = {item, s.h, s.row0, s.rows, (int)slot, s.last};
      if (gt < C::NH) {
        const int r = c0 + gt;
        float total = 0.f;
#pragma unroll 8
        for (int i = 0; i < 128; ++i) total += sums[gt * 129 + i];
        const float m = sh.cm[r].y;
        if (whole) {
          const float vsc = a.c.v_scale != nullptr ? a.c.v_scale[s.h] : 1.f;
          sh.inv[r] = total != 0.f ? vsc / total : 0.f;
          if (a.lse != nullptr && r < s.rows)
            a.lse[item + rows[r].at] =
                total != 0.f ? (m + log2f(total)) * 0.6931471805599453f : -INFINITY;
        } else {
          a.part_ml[slot * NT + r] = make_float2(m, total);
          sh.inv[r] = 1.f;
        }
      }
      tc::named_barrier(3, 256);  // both groups' sums are read: P may be written again
#pragma unroll 1
      for (int mb = 0; mb < C::MB; ++mb) {
        const int ch = mb * 128 + quarter * 32 + lane;
#pragma unroll 1
        for (int r0 = c0; r0 < c0 + C::NH && r0 < s.rows; r0 += 8) {
          uint32_t x[8];
          tc::tmem_ld8(lane_base + C::cO + mb * C::NT + r0, x);
          tc::tmem_wait_ld(x);
          if (D < 128 && ch >= D) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = r0 + i;
            if (r >= s.rows) break;
            const float o = __uint_as_float(x[i]) * sh.inv[r];
            if (whole)
              static_cast<uint16_t*>(a.o)[(item + rows[r].at) * D + ch] =
                  a.bf16 ? Elem<GDN_BF16>::from(o) : Elem<GDN_F16>::from(o);
            else
              a.part_o[(slot * NT + r) * D + ch] = o;
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_empty), mbar_arrive(&sh.row_empty[seg_no & 1]);
    }
    if (threadIdx.x == 256) a.join[blockIdx.x] = join;
  } else if (warp == 16) {
    // ------------------------------------------------ S^T products (one elected lane)
    constexpr uint32_t id = idesc_f16(NT, false);
    // descriptors advance by 16-byte units in their low word
    const uint64_t desc = tc::sdesc_sw128(smem_addr(smem + C::oQ), 16, 1024);
    int tile = 0, qs = 0, ku = 0;
    unsigned ku_ph = 0, q_ph = 0;
    for (; next_seg(); ++seg_no) {
      attn_wait(&sh.q_full[qs], q_ph, dead);
      const uint64_t q = desc + (uint32_t)(qs * (C::QB >> 4));
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        const int buf = tile & 1;
        attn_wait(&sh.s_empty[buf], ((tile >> 1) & 1) ^ 1, dead);
        const uint32_t d = C::cS + buf * NT;
#pragma unroll
        for (int u = 0; u < C::UNITS; ++u) {
          const int k0 = C::UNITS >= C::KU ? u % C::KU : ku + u;
          const bool live = attn_wait(&sh.k_full[k0], ku_ph ^ (C::UNITS > C::KU && u >= C::KU), dead);
          tc::fence_after_sync();
          if (elect_one() && live) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(d, k0 * 32 + k * 8, q + (u * NT * 128 + k * 32) / 16, id, u > 0 || k > 0);
            tc::mma_commit(&sh.k_empty[k0]);
            if (u + 1 == C::UNITS) {
              tc::mma_commit(&sh.s_full[buf]);
              if (t + 1 == s.t1) tc::mma_commit(&sh.q_empty[qs]);
            }
          }
        }
        if (C::UNITS < C::KU) {
          ku += C::UNITS;
          if (ku == C::KU) ku = 0, ku_ph ^= 1;
        } else if ((C::UNITS / C::KU) & 1) {
          ku_ph ^= 1;
        }
      }
      if (++qs == C::NQ) qs = 0, q_ph ^= 1;
    }
  } else if (warp == 19) {
    // ------------------------------------------------ O^T products (one elected lane)
    constexpr uint32_t id = idesc_f16(NT, true);
    const uint64_t desc = tc::sdesc_sw128(smem_addr(smem + C::oP), kTile * 128, 1024);
    int tile = 0;
    unsigned vu_ph = 0;
    for (; next_seg(); ++seg_no) {
      attn_wait(&sh.o_empty, (seg_no & 1) ^ 1, dead);
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++tile) {
        const int buf = tile & 1;
        attn_wait(&sh.p_full[buf], (tile >> 1) & 1, dead);
        const uint64_t p = desc + (uint32_t)(buf * (C::PB >> 4));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          constexpr int VU = C::VU;
          const int vu = r % VU;
          const bool live = attn_wait(&sh.v_full[vu], vu_ph ^ (r >= VU), dead);
          tc::fence_after_sync();
          if (elect_one() && live) {
#pragma unroll
            for (int mb = 0; mb < C::MB; ++mb) {
              const uint32_t d = C::cO + mb * NT, va = C::cV + (vu * C::MB + mb) * 16;
              mma_ts(d, va, p + r * 256, id, t > s.t0 || r > 0);
              mma_ts(d, va + 8, p + r * 256 + 128, id, 1);
            }
            tc::mma_commit(&sh.v_empty[vu]);
            if (r == 3) {
              tc::mma_commit(&sh.p_empty[buf]);
              if (t + 1 == s.t1) tc::mma_commit(&sh.o_full);
            }
          }
        }
        if ((4 / C::VU) & 1) vu_ph ^= 1;
      }
    }
  } else if (warp == 17) {
    // ------------------------------------------------ segments and records in, V scales to binary16
    const Lens lens = {a, sh.len};
    Run run = attn_run(a, lens, blockIdx.x, gridDim.x);
    Seg f = {};  // the copies run ahead of the conversion
    int f_t = 0, f_seg = 0, f_tile = 0, f_stage = 0;
    bool f_on = true;
    unsigned empty_ph = 1;
    auto fetch = [&]() {
      if (f_t == f.t1 && f_on) {  // publish the next segment
        f = attn_seg(a, lens, run);
        f_t = f.t0;
        f_on = f.t1 > 0;
        const int i = f_seg & (kSegs - 1);
        attn_wait(&sh.seg_empty[i], ((f_seg / kSegs) & 1) ^ 1, dead);
        if (lane == 0) {
          sh.seg[i] = f;
          mbar_arrive(&sh.seg_full[i]);
        }
        ++f_seg;
      }
      if (!f_on) return;
      attn_wait(&sh.raw_empty[f_stage], empty_ph, dead);
      const uint8_t* src = nullptr;
      bool ok = true;  // past the end: nothing to read, hidden by position
      const int pos = f_t * kTile + lane * kRec;
      if (lane < 4 && pos < f.len) {
        src = record(a.c, f.b, f.h, pos);
        ok = src != nullptr;
        if (!ok) report(a.c.status, GDN_ERR_PAGE_RANGE);
      }
      const unsigned good = __ballot_sync(0xffffffffu, ok) & 15u;
      const unsigned copies = __ballot_sync(0xffffffffu, src != nullptr);
      if (lane == 0) {
        sh.tile_ok[f_tile & 7] = (int)good;
        mbar_arrive_expect_tx(&sh.raw_full[f_stage], __popc(copies) * rec_bytes(D));
      }
      __syncwarp();
      if (src != nullptr)
        bulk_g2s(smem + C::oRaw + f_stage * C::RAW + lane * rec_bytes(D), src, rec_bytes(D),
                 &sh.raw_full[f_stage]);
      if (++f_stage == C::NRAW) f_stage = 0, empty_ph ^= 1;
      ++f_tile;
      ++f_t;
    };
    // the conversion follows the copies NRAW - 2 tiles behind, so that it does not
    // wait for the readers of the tile before it
    int stage = 0, vb = 0, tile = 0, t = 0;
    unsigned raw_ph = 0, vs_ph = 1;
    const Seg* c = nullptr;
#pragma unroll 1
    for (int k = 0;; ++k) {
      fetch();
      if (k < C::NRAW - 2) continue;
      if (tile == f_tile) break;
      if (c == nullptr || t == c->t1) {  // the segment of this tile
        c = &sh.seg[seg_no++ & (kSegs - 1)];
        t = c->t0;
      }
      attn_wait(&sh.raw_full[stage], raw_ph, dead);
      attn_wait(&sh.vs_empty[vb], vs_ph, dead);
      const uint8_t* raw = smem + C::oRaw + stage * C::RAW;
      uint8_t* vs = smem + C::oVS + vb * C::VSB;
      const int ok = sh.tile_ok[tile & 7];
      const int end = c->len - t * kTile;
      // 8 scales of a group a step; positions past the end count as 0
#pragma unroll 2
      for (int i = lane; i < 4 * (D / 16) * 4; i += 32) {
        const int r = i / (D / 4), g = (i / 4) % (D / 16), o = i & 3;
        const uint2 s8 = *reinterpret_cast<const uint2*>(raw + r * rec_bytes(D) + off_vs(D) +
                                                         g * kRec + o * 8);
        uint32_t w[4] = {e4m3x2(s8.x), e4m3x2(s8.x >> 16), e4m3x2(s8.y), e4m3x2(s8.y >> 16)};
        const int n = (ok >> r) & 1 ? end - (r * kRec + o * 8) : 0;  // positions that exist
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
      ++t;
      ++tile;
    }
    if (*dead) {  // copies in flight land before the block's memory is given back
      for (int i = 0; i < C::NRAW && i < f_tile; ++i)
        (void)mbar_wait_bounded(&sh.raw_full[i], ((f_tile - i - 1) / C::NRAW) & 1, kWaitPolls);
    }
  } else {
    // ------------------------------------------------ queries
    // Copied as they are to where the operand goes, then each lane turns its own
    // channels into binary16 in place.
    constexpr int E = D / 32;   // channels of a lane
    int qb = 0;
    unsigned ph = 1;
    for (; next_seg(); ++seg_no) {
      attn_wait(&sh.q_empty[qb], ph, dead);
      attn_wait(&sh.row_empty[seg_no & 1], ((seg_no >> 1) & 1) ^ 1, dead);
      const float ks = a.c.k_scale != nullptr ? a.c.k_scale[s.h] : 1.f;
      const int ch = lane * E;
      uint8_t* q = smem + C::oQ + qb * C::QB + (ch >> 6) * (NT * 128) + (ch & 7) * 2;
      const uint16_t* src0 =
          static_cast<const uint16_t*>(a.q) + s.b * a.q_stride_b + (int64_t)s.h * a.G * D + ch;
      int n = s.row0 / a.G, g = s.row0 % a.G;
      const int n0 = n, g0 = g;
#pragma unroll 1
      for (int r = 0; r < NT; ++r) {
        uint8_t* at = q + r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4);
        if (r < s.rows) {
          const uint16_t* src = src0 + n * a.q_stride_n + (int64_t)g * D;
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(smem_addr(at)), "l"(src),
                       "n"(E * 2)
                       : "memory");
        } else if constexpr (E == 8) {
          *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
        } else if constexpr (E == 4) {
          *reinterpret_cast<uint2*>(at) = make_uint2(0, 0);
        } else {
          *reinterpret_cast<uint32_t*>(at) = 0;
        }
        if (++g == a.G) g = 0, ++n;
      }
      cp_async_wait_all();
      n = n0, g = g0;
#pragma unroll 1
      for (int r = 0; r < NT; ++r) {
        uint32_t* at =
            reinterpret_cast<uint32_t*>(q + r * 128 + ((((ch & 63) >> 3) ^ (r & 7)) << 4));
        float f[E];
        unsigned big = 0;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const uint32_t x = at[i];
          if (a.bf16) {
            f[2 * i] = __uint_as_float(x << 16);
            f[2 * i + 1] = __uint_as_float(x & 0xffff0000u);
          } else {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&x));
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
#pragma unroll
        for (int i = 0; i < E / 2; ++i) at[i] = pack_f16x2(f[2 * i] * mul, f[2 * i + 1] * mul);
        if (lane == 0) {
          Row info = {a.scale * back * (ks * kLog2e), n * a.Hq + g, 0, 0};
          if (a.parent != nullptr && r < s.rows) {
            const int32_t* p = a.parent + (int64_t)s.b * a.N;
            unsigned long long seen = 0;
            for (int m = n; m >= 0; m = p[m]) seen |= 1ull << m;
            info.lo = (unsigned)seen;
            info.hi = (unsigned)(seen >> 32);
          }
          sh.row[seg_no & 1][r] = info;
        }
        if (++g == a.G) g = 0, ++n;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full[qb]), mbar_arrive(&sh.row_full[seg_no & 1]);
      if (++qb == C::NQ) qb = 0, ph ^= 1;
    }
  }
  // every role is done with its loops, hence with its copies and products; after a
  // wait that ran out, products in flight end (bounded) before TMEM is given back
  if ((warp == 16 || warp == 19) && __any_sync(0xffffffffu, *dead)) {
    if (elect_one()) tc::mma_commit(&sh.drain);
    (void)mbar_wait_bounded(&sh.drain, 0, kWaitPolls);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && *dead) report(a.c.status, GDN_ERR_TIMEOUT);
  if (warp == 16) {
    tc::fence_after_sync();
    tc::tmem_relinquish();
    tc::tmem_dealloc(sh.tmem, 512);
  }
}

// ---------------------------------------------------------------- join
// Grid (blocks of the main kernel, rows): the item that block x left unfinished,
// if any, row by row: the parts of blocks x .. last, in that order.  A thread
// has four channels of every NP-th part.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 16;      // grid rows; more rows are taken in turn
constexpr int kJoinParts = 1024;   // parts kept in shared memory: as many blocks at most

template <int D>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const __grid_constant__ AttnArgs a, int NT) {
  constexpr int Q = D / 4, NP = kJoinThreads / Q;
  __shared__ float weight[kJoinParts];
  __shared__ float red[kJoinThreads / 32][2];
  __shared__ __align__(16) float acc[NP][D];
  pdl_enter();
  const AttnJoin j = a.join[blockIdx.x];
  const int parts = j.rows > 0 ? j.last - (int)blockIdx.x + 1 : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int quad = threadIdx.x % Q, group = threadIdx.x / Q;
  auto slot = [&](int i) { return i == 0 ? (int64_t)j.slot : 2 * ((int64_t)blockIdx.x + i); };
  const float vsc = a.c.v_scale != nullptr ? a.c.v_scale[j.h] : 1.f;
#pragma unroll 1
  for (int r = blockIdx.y; r < j.rows; r += kJoinRows) {
    float top = kNone;
    for (int i = threadIdx.x; i < parts; i += kJoinThreads) {
      const float m = a.part_ml[slot(i) * NT + r].x;
      top = m > top || m != m ? m : top;
    }
    top = warp_max(top);
    if (lane == 0) red[warp][0] = top;
    __syncthreads();
    for (int w = 0; w < kJoinThreads / 32; ++w) {
      const float m = red[w][0];
      top = m > top || m != m ? m : top;
    }
    float sum = 0.f;
    for (int i = threadIdx.x; i < parts; i += kJoinThreads) {
      const float2 ml = a.part_ml[slot(i) * NT + r];
      const float w = exp2_fast(ml.x - top);
      weight[i] = w;
      sum += w * ml.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) red[warp][1] = sum;
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < kJoinThreads / 32; ++w) sum += red[w][1];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = group; i < parts; i += NP) {
      const float4 p =
          __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot(i) * NT + r) * D) + quad);
      const float w = weight[i];
      o.x += w * p.x, o.y += w * p.y, o.z += w * p.z, o.w += w * p.w;
    }
    *reinterpret_cast<float4*>(&acc[group][quad * 4]) = o;
    __syncthreads();
    const int row = j.row0 + r;
    const int64_t at = j.item + (int64_t)(row / a.G) * a.Hq + row % a.G;
    if (threadIdx.x < D) {
      float x = 0.f;
      for (int g = 0; g < NP; ++g) x += acc[g][threadIdx.x];
      x *= sum != 0.f ? vsc / sum : 0.f;
      static_cast<uint16_t*>(a.o)[at * D + threadIdx.x] =
          a.bf16 ? Elem<GDN_BF16>::from(x) : Elem<GDN_F16>::from(x);
      if (a.lse != nullptr && threadIdx.x == 0)
        a.lse[at] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
    __syncthreads();
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
  return launch_pdl(join_kernel<D>, dim3(parts, min(NT, kJoinRows)), dim3(kJoinThreads), 0, s, a,
                    NT);
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
