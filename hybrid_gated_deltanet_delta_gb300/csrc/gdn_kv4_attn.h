// Arguments of the attention kernels over the 4-bit cache (not part of the C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {
namespace kv4 {

struct AttnArgs {
  gdn_kv4_cache c;
  const void* q;
  int64_t q_stride_b, q_stride_n;
  const int32_t* parent;
  void* o;
  float* lse;
  float* part_o;    // [2 per block][rows][D]
  float2* part_ml;  // [2 per block][rows]: reference and sum
  float scale;
  int N, Hq, G;     // G: query heads of a kv head
  int rows_total, rows_per_tile, row_tiles;
  int bf16;
};

// A block's run of tiles.
struct AttnSpan {
  int64_t count;
  int b, h, rt, t0;  // the item and tile that it begins with
};

int attn_launch_64(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int attn_launch_128(const AttnArgs& a, int NT, int parts, cudaStream_t s);
int attn_launch_256(const AttnArgs& a, int NT, int parts, cudaStream_t s);

}  // namespace kv4
}  // namespace gdn
