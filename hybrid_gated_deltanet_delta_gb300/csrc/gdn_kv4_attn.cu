// Host side of the attention over the 4-bit cache: row tiles, grid and workspace
// (the kernels are in gdn_kv4_attn.cuh).
#include "gdn_common.cuh"
#include "gdn_kv4_attn.h"
#include "gdn_launch.h"

namespace gdn {
namespace {

using kv4::AttnArgs;

// Query rows of a tile.  K and V are brought in and dequantised once per row tile, so
// wide ones pay: with tiles of at most 64 rows a 2048-token piece of a prompt takes 431 us,
// eight chains of 16 (96 rows) 79.8 us and a tree of 22 (132 rows, three tiles of 44)
// 42.8 us, with 96 367, 64.0 and 40.7 us (in turn on one box).  Rows are spread evenly over
// the tiles.  More than 96 do not fit tensor memory beside two units of K and V (D = 256).
constexpr int kMaxRows = 96;

int round_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : kMaxRows; }

void row_tiles(int rows, int* tiles, int* per_tile) {
  *tiles = (rows + kMaxRows - 1) / kMaxRows;
  *per_tile = (rows + *tiles - 1) / *tiles;
}

}  // namespace

size_t kv4_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D) {
  int tiles, per_tile;
  row_tiles(N * (Hq / Hkv), &tiles, &per_tile);
  // one block per SM; without a device (a size asked for on the host alone) as for 256
  const int sms = sm_count();
  return (size_t)(sms > 0 ? sms : 256) *
         (2 * round_rows(per_tile) * (D * 4 + 8) + sizeof(kv4::AttnJoin));
}

int launch_kv4_attention(const gdn_kv4_cache& c, const void* q, int dtype, int64_t qsb, int64_t qsn,
                         int N, int Hq, float scale, const int32_t* parent, void* o, float* lse,
                         void* workspace, cudaStream_t s) {
  const int parts = sm_count();  // one block per SM: a block takes the whole of tensor memory
  if (parts == 0) return GDN_ERR_CUDA;
  AttnArgs a = {};
  a.c = c;
  a.q = q;
  a.q_stride_b = qsb;
  a.q_stride_n = qsn;
  a.parent = parent;
  a.o = o;
  a.lse = lse;
  a.scale = scale;
  a.N = N;
  a.Hq = Hq;
  a.G = Hq / c.Hkv;
  a.rows_total = N * a.G;
  row_tiles(a.rows_total, &a.row_tiles, &a.rows_per_tile);
  a.bf16 = dtype == GDN_BF16;
  // the kernels count tiles in 32 bits
  const int64_t tiles = ((int64_t)c.max_pages * c.page_tokens + 127) / 128 + 8;
  if ((int64_t)a.row_tiles * c.B > INT32_MAX / c.Hkv ||
      (int64_t)a.row_tiles * c.B * c.Hkv > INT32_MAX / tiles)
    return GDN_ERR_UNSUPPORTED;
  const int NT = round_rows(a.rows_per_tile);
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)2 * parts * NT * c.D);
  a.join = reinterpret_cast<kv4::AttnJoin*>(a.part_ml + (size_t)2 * parts * NT);
  switch (c.D) {
    case 64: return kv4::attn_launch_64(a, NT, parts, s);
    case 128: return kv4::attn_launch_128(a, NT, parts, s);
    default: return kv4::attn_launch_256(a, NT, parts, s);
  }
}

}  // namespace gdn
