// The C ABI (include/gdn.h): argument checks, tile choice and launches.
// Nothing here allocates, synchronises or keeps state between calls.
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>
#include <stdlib.h>

#include <utility>

#include "gdn_common.cuh"
#include "gdn_launch.h"

namespace {

// NVTX range around one entry point, pushed only when GDN_NVTX is set (to
// anything but "0") at the first call; the header-only NVTX calls are no-ops
// unless a profiler injects itself.
bool nvtx_on() {
  static const bool on = [] {
    const char* e = getenv("GDN_NVTX");
    return e != nullptr && e[0] != '\0' && !(e[0] == '0' && e[1] == '\0');
  }();
  return on;
}

struct Range {
  const bool on;
  explicit Range(const char* name) : on(nvtx_on()) {
    if (on) nvtxRangePushA(name);
  }
  ~Range() {
    if (on) nvtxRangePop();
  }
};
#define GDN_RANGE() Range gdn_range_(__func__)

bool ok_ptr16(const void* p) { return p != nullptr && gdn::aligned16(p); }
bool ok_ptr4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Default slab shape for the verify and replay kernels: 16 columns per block
// and one warp per block for a chain: its node loop overlaps each node's
// update with the shuffle tree of the look-ahead sums, which a cross-warp
// exchange would interrupt (measured on the 16-node chain: one warp 13.1 us,
// two row warps 13.4 us per launch).  Tree blocks take whole nodes per warp,
// so the row-warp count applies to chains and replays only.  A replay takes
// the chain's shape, so that a chain committed by replay repeats the verify
// arithmetic bit for bit.
void auto_tile(int* wc, int* nw) {
  *wc = 16;
  *nw = 1;
}

int verify_common(const gdn_verify_args* a, const int32_t* parent, int32_t* depth_out, bool tree,
                  void* stream, void* snap16 = nullptr, bool prep = false) {
  if (a == nullptr) return GDN_ERR_INVALID_ARG;
  if (a->B < 0 || a->N < 1 || a->Hk < 1 || a->Hv < 1 || a->Hv % a->Hk != 0)
    return GDN_ERR_INVALID_ARG;
  if (a->in_dtype != GDN_F32 && a->in_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (a->N > 64 || a->B > 65535 || a->Hv > 65535) return GDN_ERR_UNSUPPORTED;
  if (a->dk != 16 && a->dk != 32 && a->dk != 64 && a->dk != 128) return GDN_ERR_UNSUPPORTED;
  if (a->dv < 16 || a->dv > 1024 || a->dv % 16 != 0) return GDN_ERR_UNSUPPORTED;
  if (a->B == 0) return GDN_OK;
  if (a->n_slots < 1) return GDN_ERR_INVALID_ARG;
  const int64_t head_set = (int64_t)a->Hv * a->dk * a->dv;
  if (a->cache_slot_stride < head_set) return GDN_ERR_INVALID_ARG;
  if (a->cache_slot_stride % 4 != 0) return GDN_ERR_MISALIGNED;
  const void* need16[] = {a->q, a->k, a->v, a->state_cache, a->o};
  for (const void* p : need16) {
    if (p == nullptr) return GDN_ERR_INVALID_ARG;
    if (!gdn::aligned16(p)) return GDN_ERR_MISALIGNED;
  }
  // snapshots may be NULL: nothing is persisted and the accepted state is
  // committed by replay
  if (snap16 == nullptr && a->snapshots != nullptr && !gdn::aligned16(a->snapshots))
    return GDN_ERR_MISALIGNED;
  if (snap16 != nullptr && !gdn::aligned16(snap16)) return GDN_ERR_MISALIGNED;
  if (a->alpha == nullptr || a->beta == nullptr) return GDN_ERR_INVALID_ARG;
  if (tree && parent == nullptr) return GDN_ERR_INVALID_ARG;
  if (tree && a->max_depth < 0) return GDN_ERR_INVALID_ARG;
  const void* need4[] = {a->alpha, a->beta, a->slot, a->status, parent, depth_out};
  for (const void* p : need4)
    if (!ok_ptr4(p)) return GDN_ERR_MISALIGNED;

  int wc = 0, nw = 0;
  auto_tile(&wc, &nw);
  if (a->tile_cols != 0) wc = a->tile_cols;
  if (a->row_warps != 0) nw = a->row_warps;
  else if (!gdn::verify_tile_supported(a->dk, wc, nw)) nw = 1;  // automatic, for a forced width
  if (!gdn::verify_tile_supported(a->dk, wc, nw) || a->dv % wc != 0) return GDN_ERR_UNSUPPORTED;
  return gdn::launch_verify(a, tree ? parent : nullptr, tree ? depth_out : nullptr, wc, nw,
                            static_cast<cudaStream_t>(stream), snap16, prep);
}

int commit_common(const void* snapshots, bool src16, int64_t snap_layer_stride,
                  const int32_t* accept_idx, float* state_cache, int64_t cache_slot_stride,
                  int64_t cache_layer_stride, const int32_t* slot, int32_t n_slots, int32_t B,
                  int32_t N, int32_t Hv, int32_t dk, int32_t dv, int32_t n_layers,
                  int32_t* status, void* stream) {
  if (B < 0 || n_layers < 0 || N < 1 || Hv < 1 || dk < 1 || dv < 1) return GDN_ERR_INVALID_ARG;
  if (snap_layer_stride < 0 || cache_slot_stride < 0 || cache_layer_stride < 0)
    return GDN_ERR_INVALID_ARG;
  if (B > 65535 || n_layers > 65535) return GDN_ERR_UNSUPPORTED;
  if (B == 0 || n_layers == 0) return GDN_OK;
  const int64_t head_set = (int64_t)Hv * dk * dv;
  if (n_slots < 1 || cache_slot_stride < head_set) return GDN_ERR_INVALID_ARG;
  if (head_set % 4 != 0 || snap_layer_stride % 4 != 0 || cache_slot_stride % 4 != 0 ||
      cache_layer_stride % 4 != 0)
    return GDN_ERR_MISALIGNED;
  if (snapshots == nullptr || accept_idx == nullptr || state_cache == nullptr)
    return GDN_ERR_INVALID_ARG;
  if (!ok_ptr16(snapshots) || !ok_ptr16(state_cache)) return GDN_ERR_MISALIGNED;
  if (!ok_ptr4(accept_idx) || !ok_ptr4(slot) || !ok_ptr4(status)) return GDN_ERR_MISALIGNED;
  return gdn::launch_commit(snapshots, src16, snap_layer_stride, accept_idx, state_cache,
                            cache_slot_stride, cache_layer_stride, slot, n_slots, B, N, Hv, dk,
                            dv, n_layers, status, static_cast<cudaStream_t>(stream));
}

int replay_common(const gdn_verify_args* a, const int32_t* parent, const int32_t* accept,
                  void* stream, bool prep = false) {
  if (a == nullptr) return GDN_ERR_INVALID_ARG;
  if (a->B < 0 || a->N < 1 || a->Hk < 1 || a->Hv < 1 || a->Hv % a->Hk != 0)
    return GDN_ERR_INVALID_ARG;
  if (a->in_dtype != GDN_F32 && a->in_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (a->N > 64 || a->B > 65535 || a->Hv > 65535) return GDN_ERR_UNSUPPORTED;
  if (a->dk != 16 && a->dk != 32 && a->dk != 64 && a->dk != 128) return GDN_ERR_UNSUPPORTED;
  if (a->dv < 16 || a->dv > 1024 || a->dv % 16 != 0) return GDN_ERR_UNSUPPORTED;
  if (a->B == 0) return GDN_OK;
  if (a->n_slots < 1) return GDN_ERR_INVALID_ARG;
  const int64_t head_set = (int64_t)a->Hv * a->dk * a->dv;
  if (a->cache_slot_stride < head_set) return GDN_ERR_INVALID_ARG;
  if (a->cache_slot_stride % 4 != 0) return GDN_ERR_MISALIGNED;
  const void* need16[] = {a->k, a->v, a->state_cache};
  for (const void* p : need16) {
    if (p == nullptr) return GDN_ERR_INVALID_ARG;
    if (!gdn::aligned16(p)) return GDN_ERR_MISALIGNED;
  }
  if (a->alpha == nullptr || a->beta == nullptr || accept == nullptr) return GDN_ERR_INVALID_ARG;
  const void* need4[] = {a->alpha, a->beta, a->slot, a->status, parent, accept};
  for (const void* p : need4)
    if (!ok_ptr4(p)) return GDN_ERR_MISALIGNED;
  int wc = 0, nw = 0;
  auto_tile(&wc, &nw);
  if (a->tile_cols != 0) wc = a->tile_cols;
  if (a->row_warps != 0) nw = a->row_warps;
  else if (!gdn::verify_tile_supported(a->dk, wc, nw)) nw = 1;  // automatic, for a forced width
  if (!gdn::verify_tile_supported(a->dk, wc, nw) || a->dv % wc != 0) return GDN_ERR_UNSUPPORTED;
  return gdn::launch_replay(a, parent, accept, wc, nw, static_cast<cudaStream_t>(stream), prep);
}

// Host checks shared by the two prefill entry points.
int prefill_checks(const void* q, const void* k, const void* v, int32_t in_dtype,
                   const float* alpha, const float* beta, int32_t T, int32_t Hk, int32_t Hv,
                   int32_t dk, int32_t dv, int32_t chunk, const float* state, const float* o,
                   const int32_t* status) {
  if (T < 0 || Hk < 1 || Hv < 1 || Hv % Hk != 0) return GDN_ERR_INVALID_ARG;
  if (in_dtype != GDN_F32 && in_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  // the tensor-core form takes bf16 inputs at d_k = d_v = 128, chunk 64 only
  if (dk != 128 || dv != 128 || chunk != 64 || in_dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (Hv > 65535) return GDN_ERR_UNSUPPORTED;
  if (state == nullptr) return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16(state)) return GDN_ERR_MISALIGNED;
  if (!ok_ptr4(status)) return GDN_ERR_MISALIGNED;
  if (T == 0) return GDN_OK;
  const void* need16[] = {q, k, v, o};
  for (const void* p : need16) {
    if (p == nullptr) return GDN_ERR_INVALID_ARG;
    if (!gdn::aligned16(p)) return GDN_ERR_MISALIGNED;
  }
  if (alpha == nullptr || beta == nullptr) return GDN_ERR_INVALID_ARG;
  if (!ok_ptr4(alpha) || !ok_ptr4(beta)) return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

bool kv4_head_size(int32_t D) { return D == 64 || D == 128 || D == 256; }

// Nodes of a block, and nodes times query heads, that the kernels count in 32 bits.
constexpr int32_t kMostNodes = 1 << 24;
bool kv4_rows(int32_t N, int32_t Hq) { return N <= kMostNodes && (int64_t)N * Hq <= (1 << 30); }

int kv4_checks(const gdn_kv4_cache* c, int32_t N) {
  if (c == nullptr) return GDN_ERR_INVALID_ARG;
  if (c->B < 0 || N < 1 || c->Hkv < 1 || c->max_pages < 1 || c->n_pages < 1 || c->page_tokens < 1)
    return GDN_ERR_INVALID_ARG;
  if (!kv4_head_size(c->D) || c->page_tokens % 32 != 0) return GDN_ERR_UNSUPPORTED;
  if (c->B > 65535 || c->Hkv > 65535 || N > kMostNodes) return GDN_ERR_UNSUPPORTED;
  if ((int64_t)c->max_pages * c->page_tokens > 0x7fffffffLL - (1 << 24))
    return GDN_ERR_UNSUPPORTED;
  if (c->table_stride < c->max_pages) return GDN_ERR_INVALID_ARG;
  if (c->page_stride < (int64_t)c->Hkv * (c->page_tokens / 32) * 36 * c->D)
    return GDN_ERR_INVALID_ARG;
  if (c->page_stride % 16 != 0) return GDN_ERR_MISALIGNED;
  if (c->B == 0) return GDN_OK;
  if (c->pages == nullptr || c->table == nullptr || c->kv_len == nullptr)
    return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16(c->pages)) return GDN_ERR_MISALIGNED;
  if (!ok_ptr4(c->table) || !ok_ptr4(c->kv_len) || !ok_ptr4(c->k_scale) ||
      !ok_ptr4(c->v_scale) || !ok_ptr4(c->status))
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

// Whether rows of `extent` elements at b*stride_b + n*stride_n (b < B, n < N) lie apart: of the
// axes longer than one, the one of smaller steps has steps of a row at least, and the other's
// pass all of it.
bool rows_apart(int32_t B, int64_t stride_b, int32_t N, int64_t stride_n, int64_t extent) {
  const auto size = [](int64_t x) { return x < 0 ? 0 - (uint64_t)x : (uint64_t)x; };
  uint64_t step = size(stride_n), wide = size(stride_b);
  int64_t steps = N, others = B;
  if (steps == 1 || (others > 1 && wide < step)) std::swap(step, wide), std::swap(steps, others);
  return steps == 1 || (step >= (uint64_t)extent &&
                        (others == 1 || (wide - extent) / (steps - 1) >= step));
}

// Query rows of a batch, that the join of shared and own parts counts in 31 bits (a block of it
// goes up to 15 past the last).
bool kv4_shared_rows(int32_t B, int32_t N, int32_t Hq) {
  return (int64_t)N * Hq <= 0x7ffffff0 / B;
}

// What every form of the attention checks, but for the size of its workspace.
int kv4_attention_checks(const gdn_kv4_cache* c, const void* q, int32_t dtype, int64_t q_stride_b,
                         int64_t q_stride_n, int32_t N, int32_t Hq, const int32_t* parent,
                         const void* o, const float* lse, const void* workspace) {
  const int st = kv4_checks(c, N);
  if (st != GDN_OK) return st;
  if (Hq < 1 || Hq % c->Hkv != 0) return GDN_ERR_INVALID_ARG;
  if (dtype == GDN_F32) return GDN_ERR_UNSUPPORTED;
  if (dtype != GDN_BF16 && dtype != GDN_F16) return GDN_ERR_INVALID_ARG;
  if (parent != nullptr && N > 64) return GDN_ERR_UNSUPPORTED;
  if (!kv4_rows(N, Hq)) return GDN_ERR_UNSUPPORTED;
  if (c->B == 0) return GDN_OK;
  if (q == nullptr || o == nullptr) return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16(q) || !gdn::aligned16(o) || !gdn::aligned16(workspace))
    return GDN_ERR_MISALIGNED;
  if (q_stride_b % 8 != 0 || q_stride_n % 8 != 0) return GDN_ERR_MISALIGNED;
  if (!ok_ptr4(parent) || !ok_ptr4(lse)) return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

int kv4_pool_checks(const gdn_kv4_pool* p, const int32_t* a, const int32_t* b, int32_t F) {
  if (p == nullptr || F < 0) return GDN_ERR_INVALID_ARG;
  if (p->n_rows < 1 || p->max_pages < 1 || p->n_pages < 1 || p->page_tokens < 1)
    return GDN_ERR_INVALID_ARG;
  if (p->page_tokens % 32 != 0 || F > 65535) return GDN_ERR_UNSUPPORTED;
  if ((int64_t)p->max_pages * p->page_tokens > 0x7fffffffLL - (1 << 24))
    return GDN_ERR_UNSUPPORTED;
  if (p->table_stride < p->max_pages) return GDN_ERR_INVALID_ARG;
  if (F == 0) return GDN_OK;
  if (a == nullptr || b == nullptr || p->table == nullptr || p->kv_len == nullptr ||
      p->ref == nullptr)
    return GDN_ERR_INVALID_ARG;
  if (!ok_ptr4(a) || !ok_ptr4(b) || !ok_ptr4(p->table) || !ok_ptr4(p->kv_len) ||
      !ok_ptr4(p->ref) || !ok_ptr4(p->status))
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

int kv4_reserve_common(const gdn_kv4_pool* p, void* pages, int64_t page_stride,
                       int64_t layer_stride, int32_t n_layers, int32_t Hkv, int32_t D,
                       const int32_t* rows, const int32_t* new_len, int32_t F, int32_t* granted,
                       void* workspace, size_t workspace_bytes, void* stream) {
  const int st = kv4_pool_checks(p, rows, new_len, F);
  if (st != GDN_OK) return st;
  if (Hkv < 1 || n_layers < 1) return GDN_ERR_INVALID_ARG;
  if (!kv4_head_size(D) || n_layers > 65535 || Hkv > 65535) return GDN_ERR_UNSUPPORTED;
  // the plan adds up in 32 bits what all rows ask for, max_pages each at most
  if ((int64_t)F * p->max_pages > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
  const int64_t head = (int64_t)(p->page_tokens / 32) * 36 * D;
  if (page_stride < head * Hkv) return GDN_ERR_INVALID_ARG;
  if (n_layers > 1 && layer_stride < (int64_t)p->n_pages * page_stride)
    return GDN_ERR_INVALID_ARG;
  // the copy's and the plan's indices go on in steps of 4096 past the last one, in 32 bits
  if (head * Hkv / 16 > 0x7ffff000 || p->n_pages > 0x7ffff000) return GDN_ERR_UNSUPPORTED;
  if (page_stride % 16 != 0 || layer_stride % 16 != 0) return GDN_ERR_MISALIGNED;
  if (F == 0) return GDN_OK;
  if (pages == nullptr) return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16(pages) || !gdn::aligned16(workspace) || !ok_ptr4(granted))
    return GDN_ERR_MISALIGNED;
  if (workspace == nullptr || workspace_bytes < gdn::kv4_reserve_workspace_bytes(F))
    return GDN_ERR_WORKSPACE;
  return gdn::launch_kv4_reserve(*p, pages, page_stride, layer_stride, n_layers, Hkv, D, rows,
                                 new_len, F, granted, workspace, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int gdn_replay_accepted(const gdn_verify_args* args, const int32_t* parent,
                        const int32_t* accept_idx, void* stream) {
  GDN_RANGE();
  return replay_common(args, parent, accept_idx, stream);
}

int gdn_verify_chain_prep(const gdn_verify_args* args, void* stream) {
  GDN_RANGE();
  return verify_common(args, nullptr, nullptr, false, stream, nullptr, true);
}

int gdn_verify_tree_prep(const gdn_verify_args* args, const int32_t* parent, int32_t* depth_out,
                         void* stream) {
  GDN_RANGE();
  return verify_common(args, parent, depth_out, true, stream, nullptr, true);
}

int gdn_replay_accepted_prep(const gdn_verify_args* args, const int32_t* parent,
                             const int32_t* accept_idx, void* stream) {
  GDN_RANGE();
  return replay_common(args, parent, accept_idx, stream, true);
}

int gdn_verify_chain(const gdn_verify_args* args, void* stream) {
  GDN_RANGE();
  return verify_common(args, nullptr, nullptr, false, stream);
}

int gdn_verify_tree(const gdn_verify_args* args, const int32_t* parent, int32_t* depth_out,
                    void* stream) {
  GDN_RANGE();
  return verify_common(args, parent, depth_out, true, stream);
}

int gdn_verify_chain_f16(const gdn_verify_args* args, void* snapshots_f16, void* stream) {
  GDN_RANGE();
  if (snapshots_f16 == nullptr) return GDN_ERR_INVALID_ARG;
  return verify_common(args, nullptr, nullptr, false, stream, snapshots_f16);
}

int gdn_verify_tree_f16(const gdn_verify_args* args, const int32_t* parent, int32_t* depth_out,
                        void* snapshots_f16, void* stream) {
  GDN_RANGE();
  if (snapshots_f16 == nullptr) return GDN_ERR_INVALID_ARG;
  return verify_common(args, parent, depth_out, true, stream, snapshots_f16);
}

int gdn_commit_accepted(const float* snapshots, int64_t snap_layer_stride,
                        const int32_t* accept_idx, float* state_cache, int64_t cache_slot_stride,
                        int64_t cache_layer_stride, const int32_t* slot, int32_t n_slots,
                        int32_t B, int32_t N, int32_t Hv, int32_t dk, int32_t dv,
                        int32_t n_layers, int32_t* status, void* stream) {
  GDN_RANGE();
  return commit_common(snapshots, false, snap_layer_stride, accept_idx, state_cache,
                       cache_slot_stride, cache_layer_stride, slot, n_slots, B, N, Hv, dk, dv,
                       n_layers, status, stream);
}

int gdn_commit_accepted_f16(const void* snapshots_f16, int64_t snap_layer_stride,
                            const int32_t* accept_idx, float* state_cache,
                            int64_t cache_slot_stride, int64_t cache_layer_stride,
                            const int32_t* slot, int32_t n_slots, int32_t B, int32_t N,
                            int32_t Hv, int32_t dk, int32_t dv, int32_t n_layers,
                            int32_t* status, void* stream) {
  GDN_RANGE();
  return commit_common(snapshots_f16, true, snap_layer_stride, accept_idx, state_cache,
                       cache_slot_stride, cache_layer_stride, slot, n_slots, B, N, Hv, dk, dv,
                       n_layers, status, stream);
}

int gdn_conv_commit(const void* x, int32_t in_dtype, void* conv_state,
                    int64_t state_slot_stride, const int32_t* slot, int32_t n_slots,
                    const int32_t* parent, const int32_t* accept_idx, int32_t B, int32_t N,
                    int32_t C, int32_t W, int32_t* status, void* stream) {
  GDN_RANGE();
  if (in_dtype != GDN_F32 && in_dtype != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (B < 0 || N < 1 || C < 1 || W < 1 || n_slots < 1) return GDN_ERR_INVALID_ARG;
  if (W > 8 || B > 65535) return GDN_ERR_UNSUPPORTED;
  if (state_slot_stride < (int64_t)C * W) return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  if (x == nullptr || conv_state == nullptr || accept_idx == nullptr) return GDN_ERR_INVALID_ARG;
  const uintptr_t esz = in_dtype == GDN_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(conv_state)) % esz != 0)
    return GDN_ERR_MISALIGNED;
  if (!ok_ptr4(accept_idx) || !ok_ptr4(slot) || !ok_ptr4(parent) || !ok_ptr4(status))
    return GDN_ERR_MISALIGNED;
  return gdn::launch_conv_commit(x, in_dtype == GDN_BF16, conv_state, state_slot_stride, slot,
                                 n_slots, parent, accept_idx, B, N, C, W, status,
                                 static_cast<cudaStream_t>(stream));
}

int gdn_commit_index(const int32_t* accept_idx, int32_t B, int32_t N, int32_t base_slot,
                     int32_t* slot, int32_t* status, void* stream) {
  GDN_RANGE();
  if (B < 0 || N < 1 || base_slot < 0) return GDN_ERR_INVALID_ARG;
  if ((int64_t)base_slot + (int64_t)B * N > 0x7fffffffLL) return GDN_ERR_UNSUPPORTED;
  if (B == 0) return GDN_OK;
  if (accept_idx == nullptr || slot == nullptr) return GDN_ERR_INVALID_ARG;
  if (!ok_ptr4(accept_idx) || !ok_ptr4(slot) || !ok_ptr4(status)) return GDN_ERR_MISALIGNED;
  return gdn::launch_commit_index(accept_idx, B, N, base_slot, slot, status,
                                  static_cast<cudaStream_t>(stream));
}

size_t gdn_prefill_workspace_bytes(int32_t T, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv,
                                   int32_t chunk) {
  if (T < 0 || Hk < 1 || Hv < 1 || dk < 1 || dv < 1 || chunk < 1) return 0;
  return gdn::prefill_workspace_bytes(T, Hk, Hv, dk, dv, chunk);
}

int gdn_prefill_chunked(const void* q, const void* k, const void* v, int32_t in_dtype,
                        const float* alpha, const float* beta, int32_t T, int32_t Hk, int32_t Hv,
                        int32_t dk, int32_t dv, int32_t chunk, float* state, float* o,
                        void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
  GDN_RANGE();
  const int st = prefill_checks(q, k, v, in_dtype, alpha, beta, T, Hk, Hv, dk, dv, chunk, state,
                                o, status);
  if (st != GDN_OK || T == 0) return st;
  const size_t need = gdn::prefill_workspace_bytes(T, Hk, Hv, dk, dv, chunk);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
  if (need > 0 && !gdn::aligned16(workspace)) return GDN_ERR_MISALIGNED;
  return gdn::launch_prefill(q, k, v, true, alpha, beta, T, Hk, Hv, dk, dv, chunk, state, o,
                             workspace, status, static_cast<cudaStream_t>(stream));
}

int gdn_prefill_chunked_noalloc(const void* q, const void* k, const void* v, int32_t in_dtype,
                                const float* alpha, const float* beta, int32_t T, int32_t Hk,
                                int32_t Hv, int32_t dk, int32_t dv, int32_t chunk, float* state,
                                float* o, int32_t* status, void* stream) {
  GDN_RANGE();
  const int st = prefill_checks(q, k, v, in_dtype, alpha, beta, T, Hk, Hv, dk, dv, chunk, state,
                                o, status);
  if (st != GDN_OK || T == 0) return st;
  return gdn::launch_prefill_noalloc(q, k, v, true, alpha, beta, T, Hk, Hv, dk, dv, chunk, state,
                                     o, status, static_cast<cudaStream_t>(stream));
}

int gdn_kv4_append(const gdn_kv4_cache* c, const void* k, const void* v, int32_t dtype,
                   int64_t k_stride_b, int64_t k_stride_n, int64_t v_stride_b,
                   int64_t v_stride_n, int32_t N, void* stream) {
  GDN_RANGE();
  const int st = kv4_checks(c, N);
  if (st != GDN_OK) return st;
  if (dtype != GDN_F32 && dtype != GDN_BF16 && dtype != GDN_F16) return GDN_ERR_INVALID_ARG;
  if (c->B == 0) return GDN_OK;
  if (k == nullptr || v == nullptr) return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16(k) || !gdn::aligned16(v)) return GDN_ERR_MISALIGNED;
  const int64_t unit = dtype == GDN_F32 ? 4 : 8;
  if (k_stride_b % unit != 0 || k_stride_n % unit != 0 || v_stride_b % unit != 0 ||
      v_stride_n % unit != 0)
    return GDN_ERR_MISALIGNED;
  return gdn::launch_kv4_append(*c, k, v, dtype, k_stride_b, k_stride_n, v_stride_b, v_stride_n,
                                N, static_cast<cudaStream_t>(stream));
}

int gdn_kv4_append_rotary(const gdn_kv4_cache* c, const gdn_rotary* r, const void* q,
                          int64_t q_stride_b, int64_t q_stride_n, int32_t Hq, void* q_out,
                          int64_t out_stride_b, int64_t out_stride_n, const void* k, const void* v,
                          int32_t dtype, int64_t k_stride_b, int64_t k_stride_n,
                          int64_t v_stride_b, int64_t v_stride_n, int32_t N, void* stream) {
  GDN_RANGE();
  const int st = kv4_checks(c, N);
  if (st != GDN_OK) return st;
  if (dtype != GDN_F32 && dtype != GDN_BF16 && dtype != GDN_F16) return GDN_ERR_INVALID_ARG;
  if (r == nullptr || Hq < 1 || Hq % c->Hkv != 0) return GDN_ERR_INVALID_ARG;
  if (r->pairs < 1 || r->n_positions < 1 || r->n_axes < 1) return GDN_ERR_INVALID_ARG;
  if (r->adjacent != 0 && r->adjacent != 1) return GDN_ERR_INVALID_ARG;
  if (r->pairs % 8 != 0 || r->pairs > c->D / 2 || Hq > 65535) return GDN_ERR_UNSUPPORTED;
  if (c->Hkv > 65535 - gdn::kRotaryQueryRows) return GDN_ERR_UNSUPPORTED;
  if (c->B == 0) return GDN_OK;
  if (q == nullptr || q_out == nullptr || k == nullptr || v == nullptr || r->cos_sin == nullptr ||
      r->positions == nullptr)
    return GDN_ERR_INVALID_ARG;
  // in place (an axis of one has no steps)
  if (q == q_out &&
      ((c->B > 1 && q_stride_b != out_stride_b) || (N > 1 && q_stride_n != out_stride_n)))
    return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16(q) || !gdn::aligned16(q_out) || !gdn::aligned16(k) || !gdn::aligned16(v) ||
      !gdn::aligned16(r->cos_sin) || !ok_ptr4(r->positions))
    return GDN_ERR_MISALIGNED;
  const int64_t unit = dtype == GDN_F32 ? 4 : 8;
  for (int64_t stride : {q_stride_b, q_stride_n, out_stride_b, out_stride_n, k_stride_b, k_stride_n,
                         v_stride_b, v_stride_n})
    if (stride % unit != 0) return GDN_ERR_MISALIGNED;
  if (!rows_apart(c->B, out_stride_b, N, out_stride_n, (int64_t)Hq * c->D))
    return GDN_ERR_INVALID_ARG;
  return gdn::launch_kv4_append_rotary(*c, *r, q, q_stride_b, q_stride_n, Hq, q_out, out_stride_b,
                                       out_stride_n, k, v, dtype, k_stride_b, k_stride_n,
                                       v_stride_b, v_stride_n, N,
                                       static_cast<cudaStream_t>(stream));
}

int gdn_kv4_read(const gdn_kv4_cache* c, void* k_out, void* v_out, int32_t dtype, int32_t N,
                 void* stream) {
  GDN_RANGE();
  const int st = kv4_checks(c, N);
  if (st != GDN_OK) return st;
  if (dtype != GDN_F32 && dtype != GDN_BF16 && dtype != GDN_F16) return GDN_ERR_INVALID_ARG;
  if (c->B == 0) return GDN_OK;
  if (k_out == nullptr || v_out == nullptr) return GDN_ERR_INVALID_ARG;
  if (!gdn::aligned16(k_out) || !gdn::aligned16(v_out)) return GDN_ERR_MISALIGNED;
  return gdn::launch_kv4_read(*c, k_out, v_out, dtype, N, static_cast<cudaStream_t>(stream));
}

size_t gdn_kv4_attention_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv,
                                         int32_t D) {
  if (B < 1 || N < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || !kv4_head_size(D)) return 0;
  if (B > 65535 || Hkv > 65535 || !kv4_rows(N, Hq)) return 0;
  return gdn::kv4_attention_workspace_bytes(B, N, Hq, Hkv, D);
}

int gdn_kv4_attention(const gdn_kv4_cache* c, const void* q, int32_t dtype, int64_t q_stride_b,
                      int64_t q_stride_n, int32_t N, int32_t Hq, float scale,
                      const int32_t* parent, void* o, float* lse, void* workspace,
                      size_t workspace_bytes, void* stream) {
  GDN_RANGE();
  const int st = kv4_attention_checks(c, q, dtype, q_stride_b, q_stride_n, N, Hq, parent, o, lse,
                                      workspace);
  if (st != GDN_OK || c->B == 0) return st;
  if (workspace == nullptr ||
      workspace_bytes < gdn_kv4_attention_workspace_bytes(c->B, N, Hq, c->Hkv, c->D))
    return GDN_ERR_WORKSPACE;
  return gdn::launch_kv4_attention(*c, q, dtype, q_stride_b, q_stride_n, N, Hq, scale, parent, o,
                                   lse, workspace, static_cast<cudaStream_t>(stream));
}

int gdn_kv4_attention_window(const gdn_kv4_cache* c, const void* q, int32_t dtype,
                             int64_t q_stride_b, int64_t q_stride_n, int32_t N, int32_t Hq,
                             float scale, int32_t sinks, int32_t window, const int32_t* parent,
                             void* o, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream) {
  GDN_RANGE();
  if (window < 1 || sinks < 0) return GDN_ERR_INVALID_ARG;
  const int st = kv4_attention_checks(c, q, dtype, q_stride_b, q_stride_n, N, Hq, parent, o, lse,
                                      workspace);
  if (st != GDN_OK || c->B == 0) return st;
  if (workspace == nullptr ||
      workspace_bytes < gdn_kv4_attention_workspace_bytes(c->B, N, Hq, c->Hkv, c->D))
    return GDN_ERR_WORKSPACE;
  return gdn::launch_kv4_attention_window(*c, q, dtype, q_stride_b, q_stride_n, N, Hq, scale, sinks,
                                          window, parent, o, lse, workspace,
                                          static_cast<cudaStream_t>(stream));
}

size_t gdn_kv4_attention_shared_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv,
                                                int32_t D, int32_t n_groups) {
  if (gdn_kv4_attention_workspace_bytes(B, N, Hq, Hkv, D) == 0) return 0;
  if (n_groups < 1 || n_groups > B || !kv4_shared_rows(B, N, Hq)) return 0;
  return gdn::kv4_attention_shared_workspace_bytes(B, N, Hq, Hkv, D, n_groups);
}

int gdn_kv4_attention_shared(const gdn_kv4_cache* c, const void* q, int32_t dtype,
                             int64_t q_stride_b, int64_t q_stride_n, int32_t N, int32_t Hq,
                             float scale, const int32_t* parent, const int32_t* group,
                             int32_t n_groups, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream) {
  GDN_RANGE();
  const int st = kv4_attention_checks(c, q, dtype, q_stride_b, q_stride_n, N, Hq, parent, o, lse,
                                      workspace);
  if (st != GDN_OK || c->B == 0) return st;
  if (group == nullptr || n_groups < 1 || n_groups > c->B) return GDN_ERR_INVALID_ARG;
  if (!kv4_shared_rows(c->B, N, Hq)) return GDN_ERR_UNSUPPORTED;
  if (!ok_ptr4(group)) return GDN_ERR_MISALIGNED;
  if (workspace == nullptr ||
      workspace_bytes <
          gdn_kv4_attention_shared_workspace_bytes(c->B, N, Hq, c->Hkv, c->D, n_groups))
    return GDN_ERR_WORKSPACE;
  return gdn::launch_kv4_attention_shared(*c, q, dtype, q_stride_b, q_stride_n, N, Hq, scale,
                                          parent, group, n_groups, o, lse, workspace,
                                          static_cast<cudaStream_t>(stream));
}

int gdn_kv4_commit(const gdn_kv4_cache* c, int64_t layer_stride, int32_t n_layers, int32_t N,
                   const int32_t* parent, const int32_t* accept_idx, int32_t* len_out,
                   void* stream) {
  GDN_RANGE();
  const int st = kv4_checks(c, N);
  if (st != GDN_OK) return st;
  if (n_layers < 1) return GDN_ERR_INVALID_ARG;
  if (n_layers > 65535 || (parent != nullptr && N > 64)) return GDN_ERR_UNSUPPORTED;
  if (layer_stride % 16 != 0) return GDN_ERR_MISALIGNED;
  if (n_layers > 1 && layer_stride < (int64_t)c->n_pages * c->page_stride)
    return GDN_ERR_INVALID_ARG;
  if (c->B == 0) return GDN_OK;
  if (accept_idx == nullptr || len_out == nullptr || len_out == c->kv_len)
    return GDN_ERR_INVALID_ARG;
  if (!ok_ptr4(parent) || !ok_ptr4(accept_idx) || !ok_ptr4(len_out)) return GDN_ERR_MISALIGNED;
  return gdn::launch_kv4_commit(*c, layer_stride, n_layers, N, parent, accept_idx, len_out,
                                static_cast<cudaStream_t>(stream));
}

int gdn_kv4_release(const gdn_kv4_pool* p, const int32_t* rows, const int32_t* keep_len,
                    int32_t F, void* stream) {
  GDN_RANGE();
  const int st = kv4_pool_checks(p, rows, keep_len, F);
  if (st != GDN_OK || F == 0) return st;
  return gdn::launch_kv4_release(*p, rows, keep_len, F, static_cast<cudaStream_t>(stream));
}

int gdn_kv4_fork(const gdn_kv4_pool* p, const int32_t* src, const int32_t* dst, int32_t F,
                 void* stream) {
  GDN_RANGE();
  const int st = kv4_pool_checks(p, src, dst, F);
  if (st != GDN_OK || F == 0) return st;
  return gdn::launch_kv4_fork(*p, src, dst, F, static_cast<cudaStream_t>(stream));
}

size_t gdn_kv4_reserve_workspace_bytes(int32_t F) {
  return F < 1 ? 0 : gdn::kv4_reserve_workspace_bytes(F);
}

int gdn_kv4_reserve(const gdn_kv4_pool* p, void* pages, int64_t page_stride,
                    int64_t layer_stride, int32_t n_layers, int32_t Hkv, int32_t D,
                    const int32_t* rows, const int32_t* new_len, int32_t F, void* workspace,
                    size_t workspace_bytes, void* stream) {
  GDN_RANGE();
  return kv4_reserve_common(p, pages, page_stride, layer_stride, n_layers, Hkv, D, rows, new_len,
                            F, nullptr, workspace, workspace_bytes, stream);
}

int gdn_kv4_reserve_granted(const gdn_kv4_pool* p, void* pages, int64_t page_stride,
                            int64_t layer_stride, int32_t n_layers, int32_t Hkv, int32_t D,
                            const int32_t* rows, const int32_t* new_len, int32_t F,
                            int32_t* granted, void* workspace, size_t workspace_bytes,
                            void* stream) {
  GDN_RANGE();
  if (F > 0 && granted == nullptr) return GDN_ERR_INVALID_ARG;
  return kv4_reserve_common(p, pages, page_stride, layer_stride, n_layers, Hkv, D, rows, new_len,
                            F, granted, workspace, workspace_bytes, stream);
}

const char* gdn_status_string(int status) {
  switch (status) {
    case GDN_OK: return "GDN_OK";
    case GDN_ERR_INVALID_ARG: return "GDN_ERR_INVALID_ARG";
    case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED";
    case GDN_ERR_MISALIGNED: return "GDN_ERR_MISALIGNED";
    case GDN_ERR_CUDA: return "GDN_ERR_CUDA";
    case GDN_ERR_BAD_TREE: return "GDN_ERR_BAD_TREE";
    case GDN_ERR_ACCEPT_RANGE: return "GDN_ERR_ACCEPT_RANGE";
    case GDN_ERR_SLOT_RANGE: return "GDN_ERR_SLOT_RANGE";
    case GDN_ERR_WORKSPACE: return "GDN_ERR_WORKSPACE";
    case GDN_ERR_SCRATCH_LIMIT: return "GDN_ERR_SCRATCH_LIMIT";
    case GDN_ERR_TIMEOUT: return "GDN_ERR_TIMEOUT";
    case GDN_ERR_PAGE_RANGE: return "GDN_ERR_PAGE_RANGE";
    case GDN_ERR_POOL_EMPTY: return "GDN_ERR_POOL_EMPTY";
    case GDN_ERR_ROW_RANGE: return "GDN_ERR_ROW_RANGE";
    case GDN_ERR_NONFINITE: return "GDN_ERR_NONFINITE";
    case GDN_ERR_POSITION_RANGE: return "GDN_ERR_POSITION_RANGE";
    default: return "GDN_ERR_UNKNOWN";
  }
}

int gdn_version(void) { return GDN_VERSION; }

}  // extern "C"
