// Arguments of the attention kernels over the 4-bit cache (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {
namespace kv4 {

// An item whose tiles end in a later block: what its first block leaves to the join.
struct AttnJoin {
  int64_t item;          // output row of its first node and head
  int h, row0, rows;     // rows = 0: nothing to join
  int slot, last;        // of its own part; block with the last part
};

// What a query row sees of its sequence, and where its result goes.
enum Mode {
  kFull,    // all that its node sees; the output
  kWindow,  // the first `sinks` and the last `window` entries of its node's path; the output
  kShared   // what the sequences of a group share, their rows one after another, and what each
            // has behind it; parts of the output
};

// The first part of a query row's output that a kShared pass leaves: reference and sum, the
// item's first block and its last one (16 bits each), and the row's place in its tile.
struct RowPart {
  float m, l;
  int blocks, row;
};

// Division of 0 <= n < 2^31 by a number that the host knows: (n m / 2^32 + n) / 2^s with
// s = ceil(log2 d), m = 2^32 (2^s - d) / d + 1 rounded down (Granlund and Montgomery, 1994).
// The kernels' few hundred instructions before their first tile are fetched anew in every
// launch, and a division is some twenty of them.
struct Divisor {
  uint32_t m, s;
  Divisor() = default;
  explicit Divisor(uint32_t d) : m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int operator()(int n) const {
    return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> s);
  }
#endif
};

struct AttnArgs {
  gdn_kv4_cache c;
  const void* q;
  int64_t q_stride_b, q_stride_n;
  const int32_t* parent;
  void* o;
  float* lse;
  float* part_o;    // [2 per block][rows][D]
  float2* part_ml;  // [2 per block][rows]: reference and sum
  AttnJoin* join;   // [blocks]
  float scale;
  int N, Hq, G;     // G: query heads of a kv head
  int rows_total, rows_per_tile, row_tiles;
  int bf16;
  Divisor by_G, by_N, by_Hkv, by_page;  // page: its tokens
  int window, sinks;         // kWindow
  // kShared: of the groups and then of the sequences, the shared length and the length (0: it is
  // skipped); a group's sequences and a sequence's first own tile (-1: it is skipped)
  const int32_t *plan_len, *plan_extra;
  const uint32_t* plan_first;  // and the first sequence (in 16 bits) and row of the page table (16)
  int n_groups;
  Divisor by_Hq;
  float* row_o[2];           // [B*N*Hq][D], each row's first own part; and first shared one
  RowPart* row_part[2];      // [B*N*Hq]
};

int attn_launch_64(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int attn_launch_128(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int attn_launch_256(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int window_launch_64(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int window_launch_128(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int window_launch_256(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int shared_launch_64(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int shared_launch_128(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int shared_launch_256(const AttnArgs& a, int NT, int parts, cudaStream_t s);

// Query rows of a tile.  K and V are brought in and dequantised once per row tile, so
// wide ones pay: with tiles of at most 64 rows a 2048-token piece of a prompt takes 431 us,
// eight chains of 16 (96 rows) 79.8 us and a tree of 22 (132 rows, three tiles of 44)
// 42.8 us, with 96 367, 64.0 and 40.7 us (in turn on one box).  Rows are spread evenly over
// the tiles.  More than 96 do not fit tensor memory beside two units of K and V (D = 256).
constexpr int kMaxRows = 96;
inline int round_rows(int rows) {
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : kMaxRows;
}
inline void row_tiles(int rows, int* tiles, int* per_tile) {
  *tiles = (rows + kMaxRows - 1) / kMaxRows;
  *per_tile = (rows + *tiles - 1) / *tiles;
}

}  // namespace kv4

// gdn_kv4_shared.cu: the numbers of AttnArgs that a kShared pass reads, and the sum of the parts
// that it leaves (`rows`: of a slot of part_o).
struct SharedPlan {
  int32_t *len, *extra;
  uint32_t* first;
};
int launch_kv4_shared_plan(const gdn_kv4_cache& c, int N, const int32_t* parent,
                           const int32_t* group, int n_groups, const SharedPlan& plan,
                           cudaStream_t s);
int launch_kv4_shared_join(const kv4::AttnArgs& a, int rows, int blocks, cudaStream_t s);

}  // namespace gdn
