// Host side of the attention over the 4-bit cache: row tiles, grid and workspace
// (the kernels are in gdn_kv4_attn.cuh).
#include "gdn_common.cuh"
#include "gdn_kv4_attn.h"
#include "gdn_launch.h"

namespace gdn {
namespace {

using kv4::AttnArgs;
using kv4::round_rows;
using kv4::row_tiles;

// What all forms of the attention are given.
AttnArgs attn_args(const gdn_kv4_cache& c, const void* q, int dtype, int64_t qsb, int64_t qsn,
                   int N, int Hq, float scale, const int32_t* parent, void* o, float* lse) {
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
  a.by_G = kv4::Divisor(a.G);
  a.by_N = kv4::Divisor(N);
  a.by_Hkv = kv4::Divisor(c.Hkv);
  a.by_page = kv4::Divisor(c.page_tokens);
  return a;
}

// The kernels count tiles in 32 bits.
bool countable(const gdn_kv4_cache& c, int64_t row_tiles) {
  const int64_t tiles = ((int64_t)c.max_pages * c.page_tokens + 127) / 128 + 8;
  return row_tiles <= INT32_MAX / c.Hkv && row_tiles * c.Hkv <= INT32_MAX / tiles;
}

// Workspace of the parts that a pass with one output leaves to its join.
void place_parts(AttnArgs& a, void* workspace, int NT, int parts) {
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)2 * parts * NT * a.c.D);
  a.join = reinterpret_cast<kv4::AttnJoin*>(a.part_ml + (size_t)2 * parts * NT);
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
  AttnArgs a = attn_args(c, q, dtype, qsb, qsn, N, Hq, scale, parent, o, lse);
  if (!countable(c, (int64_t)a.row_tiles * c.B)) return GDN_ERR_UNSUPPORTED;
  const int NT = round_rows(a.rows_per_tile);
  place_parts(a, workspace, NT, parts);
  switch (c.D) {
    case 64: return kv4::attn_launch_64(a, NT, parts, s);
    case 128: return kv4::attn_launch_128(a, NT, parts, s);
    default: return kv4::attn_launch_256(a, NT, parts, s);
  }
}

int launch_kv4_attention_window(const gdn_kv4_cache& c, const void* q, int dtype, int64_t qsb,
                                int64_t qsn, int N, int Hq, float scale, int sinks, int window,
                                const int32_t* parent, void* o, float* lse, void* workspace,
                                cudaStream_t s) {
  const int parts = sm_count();
  if (parts == 0) return GDN_ERR_CUDA;
  AttnArgs a = attn_args(c, q, dtype, qsb, qsn, N, Hq, scale, parent, o, lse);
  if (!countable(c, (int64_t)a.row_tiles * c.B)) return GDN_ERR_UNSUPPORTED;
  // no sequence is longer than the table is wide: positions less a window stay in 32 bits
  const int longest = c.max_pages * c.page_tokens;
  a.window = window < longest ? window : longest;
  a.sinks = sinks < longest ? sinks : longest;
  const int NT = round_rows(a.rows_per_tile);
  place_parts(a, workspace, NT, parts);
  switch (c.D) {
    case 64: return kv4::window_launch_64(a, NT, parts, s);
    case 128: return kv4::window_launch_128(a, NT, parts, s);
    default: return kv4::window_launch_256(a, NT, parts, s);
  }
}

// ---------------------------------------------------------------- shared prompts
namespace {

// Workspace of a call that reads shared pages once: the plan's numbers, each row's first own and
// first shared part, and the parts that go on from another block.
struct SharedSpace {
  SharedPlan plan;
  float *row_o[2], *part_o;
  kv4::RowPart* row_part[2];
  float2* part_ml;
  size_t bytes;
};

SharedSpace shared_space(void* base, int B, int N, int Hq, int D, int n_groups, int sms) {
  const size_t rows = (size_t)B * N * Hq;
  SharedSpace w = {};
  uint8_t* at = static_cast<uint8_t*>(base);
  auto take = [&](size_t bytes) {
    uint8_t* p = at + w.bytes;
    w.bytes += (bytes + 255) / 256 * 256;
    return p;
  };
  auto ints = [&](size_t n) { return reinterpret_cast<int32_t*>(take(4 * n)); };
  const size_t all = (size_t)n_groups + B;
  w.plan.len = ints(all), w.plan.extra = ints(all);
  w.plan.first = reinterpret_cast<uint32_t*>(ints(all));
  for (int i = 0; i < 2; ++i) {
    w.row_o[i] = reinterpret_cast<float*>(take(rows * D * 4));
    w.row_part[i] = reinterpret_cast<kv4::RowPart*>(take(rows * sizeof(kv4::RowPart)));
  }
  w.part_o = reinterpret_cast<float*>(take((size_t)sms * kv4::kMaxRows * D * 4));
  w.part_ml = reinterpret_cast<float2*>(take((size_t)sms * kv4::kMaxRows * 8));
  return w;
}

// Whether rows of several sequences in one tile can save anything: where one sequence's
// rows fill their tiles, reading the prefix once saves bytes that L2 gives anyway.
bool rows_worth_sharing(int N, int G) {
  const int64_t rows = (int64_t)N * G;
  const int64_t tiles = (rows + kv4::kMaxRows - 1) / kv4::kMaxRows;
  return rows <= 2 * kv4::kMaxRows && 4 * tiles * kv4::kMaxRows >= 5 * rows;
}

// And whether it does by the most that there can be to read: plan, longer prologue and join
// cost some 12 us, and the more rows a sequence has the less there is to win.  Measured (shared /
// each sequence for itself, us; W: tiles of 128, and six more an item, of all items at the
// table's width; shared from the bound on; rows of a kv head):
//   rows, D  bound   below it                        above it
//    4, 128  4,594   2,176: 26 / 20, 4,352: 31 / 31  5,248: 27 / 35, 17,536: 34 / 92
//    6, 256  2,469   2,176: 31 / 27                  2,624: 29 / 32, 5,248: 34 / 48
//   24, 256  4,016   2,624: 38 / 36                  4,352: 49 / 53, 10,496: 70 / 102
//   32, 128  9,407   5,248: 49 / 44                  10,496: 72 / 74, 20,992: 112 / 134
//   48, 256  6,079   5,248: 63 / 61                  8,768: 78 / 89, 17,536: 129 / 164
//   66, 256  7,625   5,248: 74 / 75                  8,768: 98 / 111, 17,536: 165 / 199
// The lengths are the device's, so short sequences in a wide table are shared as well: four of
// 700 tokens (6 rows, D 256) take 13.0 us in a table of 16,384 tokens, each for itself, and 17.6
// in one of 32,768 or a million, shared.  (A caller who knows a bound of the lengths gives it as
// max_pages.)
bool worth_sharing(const gdn_kv4_cache& c, int rows, int row_tiles, int n_groups) {
  const int64_t tiles = ((int64_t)c.max_pages * c.page_tokens + 127) / 128 + 6;
  const int64_t most = (int64_t)c.B * c.Hkv * row_tiles * tiles;
  return c.B > n_groups &&
         most * c.D >= 500000 + 22000 * (int64_t)(rows < kv4::kMaxRows ? rows : kv4::kMaxRows);
}

}  // namespace

size_t kv4_attention_shared_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int n_groups) {
  const size_t alone = kv4_attention_workspace_bytes(B, N, Hq, Hkv, D);
  if (!rows_worth_sharing(N, Hq / Hkv)) return alone;
  const int sms = sm_count();
  const size_t shared = shared_space(nullptr, B, N, Hq, D, n_groups, sms > 0 ? sms : 256).bytes;
  return shared > alone ? shared : alone;
}

int launch_kv4_attention_shared(const gdn_kv4_cache& c, const void* q, int dtype, int64_t qsb,
                                int64_t qsn, int N, int Hq, float scale, const int32_t* parent,
                                const int32_t* group, int n_groups, void* o, float* lse,
                                void* workspace, cudaStream_t s) {
  const int parts = sm_count();
  if (parts == 0) return GDN_ERR_CUDA;
  AttnArgs a = attn_args(c, q, dtype, qsb, qsn, N, Hq, scale, parent, o, lse);
  if (!countable(c, (int64_t)a.row_tiles * c.B)) return GDN_ERR_UNSUPPORTED;
  auto alone = [&]() {
    return launch_kv4_attention(c, q, dtype, qsb, qsn, N, Hq, scale, parent, o, lse, workspace, s);
  };
  if (!rows_worth_sharing(N, a.G) || !worth_sharing(c, a.rows_total, a.row_tiles, n_groups))
    return alone();
  // the rows of a group as if they were one sequence's, in tiles as wide as a group of the
  // usual size fills
  const int64_t usual = (int64_t)((c.B + n_groups - 1) / n_groups) * a.rows_total;
  int tiles, per_tile;
  row_tiles((int)usual, &tiles, &per_tile);
  const int NT = round_rows(per_tile);
  // (items of the groups: their rows are the batch's; units of work are up to ten a tile)
  const int64_t items = (int64_t)c.B * a.rows_total / NT + n_groups + (int64_t)a.row_tiles * c.B;
  if (!countable(c, 10 * items)) return alone();
  const SharedSpace w = shared_space(workspace, c.B, N, Hq, c.D, n_groups, parts);
  int rc = launch_kv4_shared_plan(c, N, parent, group, n_groups, w.plan, s);
  if (rc != GDN_OK) return rc;
  a.n_groups = n_groups;
  a.plan_len = w.plan.len;
  a.plan_extra = w.plan.extra;
  a.plan_first = w.plan.first;
  a.by_Hq = kv4::Divisor(Hq);
  for (int i = 0; i < 2; ++i) a.row_o[i] = w.row_o[i], a.row_part[i] = w.row_part[i];
  a.part_o = w.part_o;
  a.part_ml = w.part_ml;
  switch (c.D) {
    case 64: rc = kv4::shared_launch_64(a, NT, parts, s); break;
    case 128: rc = kv4::shared_launch_128(a, NT, parts, s); break;
    default: rc = kv4::shared_launch_256(a, NT, parts, s);
  }
  if (rc != GDN_OK) return rc;
  return launch_kv4_shared_join(a, NT, parts, s);
}

}  // namespace gdn
