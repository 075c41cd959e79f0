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
};

int attn_launch_64(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int attn_launch_128(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int attn_launch_256(const AttnArgs& a, int NT, int parts, cudaStream_t s);

}  // namespace kv4
}  // namespace gdn
