/*
 * gdn.h -- C ABI of the GB300 (sm_103a) gated delta-rule verification library.
 *
 * The library runs the Gated DeltaNet recurrence of a hybrid (linear +
 * full attention) model over a speculative verification block and commits
 * the accepted state:
 *
 *     S_n = alpha_n * S_src(n) * (I - beta_n k_n k_n^T) + beta_n v_n k_n^T
 *     o_n = S_n q_n
 *
 * ("TokenSpeed hits 580 tok/s", section "Why Qwen3.5 is hard to serve fast":
 * a fixed d x d state per head, updated per token and queried by q.)
 * S_src(n) is the previous position for a causal chain ("Photon 2.6",
 * section "Speculative verification in a megakernel") and the parent node
 * for a best-first draft tree ("Qwen3.6 27B: From 20 t/s to 184 t/s",
 * DFlash section, steps 3-4).  Every node's state is persisted so that a
 * rejected suffix needs no work ("We got 207 tok/s with Qwen3.5-27B on an
 * RTX 3090", list "Key wins", persist-write kernel), and the accepted node's
 * state is committed into the recurrent-state cache ("Photon 2.6", section
 * "Handling recurrent state").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - The state of one value head is stored TRANSPOSED: H[i][j] = S[j][i],
 *    an fp32 row-major d_k x d_v matrix (i over d_k, j over d_v).
 *  - Value head h reads q/k head h / (Hv / Hk) (contiguous groups).
 *  - No scaling is applied to q; fold any 1/sqrt(d_k) into q beforehand.
 *    q and k are used as given (callers L2-normalise them upstream).
 *  - Every pointer argument is DEVICE memory of the current CUDA device,
 *    allocated and owned by the caller, unless stated otherwise.  The library
 *    allocates nothing and never synchronises: work is enqueued on `stream`
 *    (a cudaStream_t; NULL = the legacy default stream) and the call returns
 *    once it is launched.  It keeps no mutable state between calls, with one
 *    exception: the built-in scratch array of gdn_prefill_chunked_noalloc
 *    (see there for how concurrent calls of that entry point race).
 *  - Profiling ranges: with the environment variable GDN_NVTX set to a value
 *    other than "0" when the library is loaded, every entry point pushes an
 *    NVTX range named after itself for the duration of the host call (so a
 *    timeline tool shows where each launch was issued); unset, the check
 *    costs one branch per call.
 *  - Kernels are launched with programmatic dependent launch allowed: each
 *    kernel starts by waiting until the kernel before it on the stream has
 *    completed and its memory is visible, then lets the next kernel begin
 *    launching.  Stream order is kept for every read and write.  Before that
 *    wait a kernel only issues L2 prefetch hints for lines it will read
 *    (which never change memory), or reads arrays of lengths and parents that
 *    it reads again after it and then goes by.  A kernel of the caller's that
 *    follows one of ours with the same launch attribute must itself wait
 *    before reading our outputs (griddepcontrol.wait), as programmatic launch
 *    requires.
 *  - All pointers must be 16-byte aligned; element strides are in elements.
 *  - Host-detected errors return a negative gdn_status before anything is
 *    launched.  Errors that depend on device data (a malformed tree, an
 *    out-of-range accept index or slot) are written to the optional device
 *    word `status` (first error wins; the caller zeroes it) and the affected
 *    sequence is skipped; kernels never trap and never wait on other blocks (but
 *    for those of their own cluster, which the hardware runs together).
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_VERSION 3

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARG = -1,   /* null pointer, negative or inconsistent size */
  GDN_ERR_UNSUPPORTED = -2,   /* a size outside what the kernels implement */
  GDN_ERR_MISALIGNED = -3,    /* pointer not 16-byte aligned, or stride not a multiple of 4 */
  GDN_ERR_CUDA = -4,          /* the launch itself failed */
  GDN_ERR_BAD_TREE = -5,      /* device: parent[0] != -1 or parent[n] outside [0, n) */
  GDN_ERR_ACCEPT_RANGE = -6,  /* device: accept index outside [0, N) */
  GDN_ERR_SLOT_RANGE = -7,    /* device: slot outside [0, n_slots) */
  GDN_ERR_WORKSPACE = -8,     /* workspace missing or smaller than required */
  GDN_ERR_SCRATCH_LIMIT = -9, /* problem too large for the built-in scratch of the _noalloc call */
  GDN_ERR_TIMEOUT = -10,      /* device: a bounded wait on an asynchronous copy or tensor-core
                                 operation expired; that call's outputs are not valid */
  GDN_ERR_PAGE_RANGE = -11,   /* device: a page-table entry outside [0, n_pages) */
  GDN_ERR_POOL_EMPTY = -12,   /* device: fewer free pages than a row needs */
  GDN_ERR_ROW_RANGE = -13,    /* device: a row outside the table, a length below 0 or beyond the
                                 table's width, or a branch onto a row that is not empty */
  GDN_ERR_NONFINITE = -14,    /* device: a NaN or infinity was given to the 4-bit cache */
  GDN_ERR_POSITION_RANGE = -15 /* device: a rotary position outside the table of angles, or a
                                 pair's axis outside the axes given */
} gdn_status;

/* GDN_F16 (IEEE binary16) is taken by the gdn_kv4_* calls only. */
typedef enum gdn_dtype {
  GDN_F32 = 0,
  GDN_BF16 = 1,
  GDN_F16 = 2
} gdn_dtype;

/*
 * Arguments of one verify call (one GDN layer, B sequences, N nodes each).
 *
 *   q, k          [B][N][Hk][dk]  in_dtype (GDN_F32 or GDN_BF16)
 *   v             [B][N][Hv][dv]  in_dtype
 *   alpha, beta   [B][N][Hv]      fp32 gates (decay alpha, write strength beta)
 *   state_cache   recurrent-state cache, READ ONLY here: the state of
 *                 sequence b, head h starts at
 *                 state_cache + slot[b]*cache_slot_stride + h*dk*dv.
 *                 It may be the snapshots buffer itself (index-table
 *                 commit, gdn_commit_index): each sequence's state is read
 *                 before any of its nodes is written
 *   slot          [B] int32 cache slot per sequence; NULL means slot[b] = b
 *   n_slots       number of valid slots (slot[b] is checked against it)
 *   snapshots     [B][N][Hv][dk][dv] fp32 output: S_n of every node.  May be
 *                 NULL (chain or tree): nothing is persisted and the accepted
 *                 state is committed by replay (gdn_replay_accepted)
 *   o             [B][N][Hv][dv] fp32 output
 *   status        optional device int32 error word (see above)
 *   tile_cols, row_warps
 *                 0 = automatic; otherwise the d_v columns owned by one
 *                 thread block (8 or 16) and the warps that split its d_k
 *                 rows (1, or 2 for 16 columns with d_k = 64 or 128).  A
 *                 performance hint: results are identical up to the order
 *                 in which the column sums are added, and a replay commit
 *                 repeats a chain verify bit for bit only with the same
 *                 tile.  GDN_ERR_UNSUPPORTED for any other combination.
 *   max_depth     tree verify only: 0 = no cap; otherwise a sequence whose
 *                 tree has a node deeper than max_depth (the root has depth 1)
 *                 is skipped and GDN_ERR_BAD_TREE is written to `status`.
 *                 Ignored by the chain and replay calls.
 *
 * Supported sizes: dk in {16, 32, 64, 128}; dv a multiple of 16, <= 1024;
 * 1 <= N <= 64; Hv a multiple of Hk; B >= 0 (B = 0 launches nothing).
 */
typedef struct gdn_verify_args {
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;
  const float* beta;
  const float* state_cache;
  const int32_t* slot;
  float* snapshots;
  float* o;
  int32_t* status;
  int64_t cache_slot_stride;
  int32_t n_slots;
  int32_t B;
  int32_t N;
  int32_t Hk;
  int32_t Hv;
  int32_t dk;
  int32_t dv;
  int32_t in_dtype;
  int32_t tile_cols;
  int32_t row_warps;
  int32_t max_depth;
} gdn_verify_args;

/*
 * Causal-chain verification (DFlash block: the last committed token plus the
 * drafts).  Node n starts from node n-1's state; node 0 from the cache.
 * Writes every node's state to `snapshots` (when not NULL) and its output to
 * `o`.
 */
int gdn_verify_chain(const gdn_verify_args* args, void* stream);

/*
 * Tree verification (DDTree block).  parent [B][N] int32 with parent[b][0] = -1
 * (the root, i.e. the last committed token, starts from the cache) and
 * 0 <= parent[b][n] < n otherwise (nodes in topological order).  Node n starts
 * from its parent's state.  depth_out [B][N] int32 (optional, may be NULL)
 * receives each node's depth, root = 1.  A sequence whose parent array breaks
 * the rule, or whose tree is deeper than args->max_depth (when not 0), is
 * skipped and GDN_ERR_BAD_TREE is written to args->status (its depth_out row
 * is still written when the parent array itself is valid).  With
 * args->snapshots == NULL (a block committed by gdn_replay_accepted) the
 * block is verified by one lower-triangular solve per slab instead of the
 * node-by-node walk, and only o (and depth_out) is written; the outputs agree
 * with the walk's up to floating-point rounding.
 */
int gdn_verify_tree(const gdn_verify_args* args, const int32_t* parent, int32_t* depth_out,
                    void* stream);

/*
 * Commit the accepted node of every sequence, for n_layers layers at once:
 *
 *   state_cache[l][slot[b]][h] = snapshots[l][b][accept_idx[b]][h]
 *
 * Layer l of the snapshots starts at snapshots + l*snap_layer_stride and is
 * laid out [B][N][Hv][dk][dv]; layer l of the cache starts at
 * state_cache + l*cache_layer_stride, slot s at + s*cache_slot_stride, head h
 * at + h*dk*dv.  For a chain with accept length L, accept_idx = L - 1.
 * The copy is bit-exact.  An accept index outside [0, N) or a slot outside
 * [0, n_slots) skips that sequence and is reported through `status`.
 * snapshots and state_cache must not overlap, and the slot[] entries of one
 * call must be distinct (two sequences committing into one slot race, and
 * the slot then holds either state).
 */
int gdn_commit_accepted(const float* snapshots, int64_t snap_layer_stride,
                        const int32_t* accept_idx, float* state_cache, int64_t cache_slot_stride,
                        int64_t cache_layer_stride, const int32_t* slot, int32_t n_slots,
                        int32_t B, int32_t N, int32_t Hv, int32_t dk, int32_t dv,
                        int32_t n_layers, int32_t* status, void* stream);

/*
 * Verification and replay from raw projections (input preparation fused into
 * the recurrence kernel).  The same calls as gdn_verify_chain,
 * gdn_verify_tree and gdn_replay_accepted, except that
 *   q, k          are the raw projections: each (node, q/k head) vector is
 *                 L2-normalised in the kernel (a zero vector stays zero);
 *   alpha, beta   hold the gate pre-activations a, b: the kernel uses
 *                 alpha = exp(-softplus(a)) = 1 / (1 + e^a) and
 *                 beta = sigmoid(b) = 1 / (1 + e^-b).
 * These are the maps the block's inputs are defined by (q and k L2-normalised
 * per head, alpha from exp(-softplus), beta from sigmoid).  Results equal the
 * plain calls on the prepared inputs up to floating-point rounding.
 */
int gdn_verify_chain_prep(const gdn_verify_args* args, void* stream);
int gdn_verify_tree_prep(const gdn_verify_args* args, const int32_t* parent, int32_t* depth_out,
                         void* stream);
int gdn_replay_accepted_prep(const gdn_verify_args* args, const int32_t* parent,
                             const int32_t* accept_idx, void* stream);

/*
 * Verification with 16-bit persisted states ("We got 207 tok/s with
 * Qwen3.5-27B on an RTX 3090", list "Key wins": an f16 intermediate cache at
 * half the bandwidth, "at the same tree budget").  The same as
 * gdn_verify_chain / gdn_verify_tree, except that every node's state is
 * written to `snapshots_f16` [B][N][Hv][dk][dv] as IEEE binary16, rounded to
 * nearest even from the fp32 state the kernel forms (args->snapshots is not
 * used).
 *   chain: the recurrence and the outputs o are unchanged; only the
 *          persisted copies are rounded.
 *   tree:  the tree is walked depth level by depth level (the warps of a
 *          block take a level's nodes round robin, in index order).  A node
 *          continues from its parent's exact fp32 state when the warp that
 *          formed the parent takes the node next, or when the parent is one
 *          of the first three nodes of its depth (in index order) that have
 *          children (those stay in shared memory); otherwise it continues
 *          from the parent's binary16 snapshot, as an f16 intermediate cache
 *          does.  The root starts from the fp32 cache.
 */
int gdn_verify_chain_f16(const gdn_verify_args* args, void* snapshots_f16, void* stream);
int gdn_verify_tree_f16(const gdn_verify_args* args, const int32_t* parent, int32_t* depth_out,
                        void* snapshots_f16, void* stream);

/*
 * gdn_commit_accepted for binary16 snapshots: the accepted node's state is
 * widened exactly to fp32 into the cache (so the committed state carries one
 * binary16 rounding per block).  Strides are in elements; same checks and
 * status reporting as gdn_commit_accepted.
 */
int gdn_commit_accepted_f16(const void* snapshots_f16, int64_t snap_layer_stride,
                            const int32_t* accept_idx, float* state_cache,
                            int64_t cache_slot_stride, int64_t cache_layer_stride,
                            const int32_t* slot, int32_t n_slots, int32_t B, int32_t N,
                            int32_t Hv, int32_t dk, int32_t dv, int32_t n_layers,
                            int32_t* status, void* stream);

/*
 * Convolution-history commit ("Photon 2.6", section "Handling recurrent
 * state": the convolution history is committed to the same boundary as the
 * recurrent state).  A short causal convolution before the recurrence keeps,
 * per cache slot and channel, the last W raw inputs (oldest first):
 *
 *   conv_state  slot s, channel c at conv_state + s*state_slot_stride + c*W,
 *               W consecutive elements (in_dtype)
 *   x           [B][N][C] raw inputs of the block's nodes (in_dtype)
 *
 * For every sequence b the history is advanced in place over the accepted
 * path (chain: nodes 0 .. accept_idx[b], parent == NULL; tree: the ancestors
 * of accept_idx[b] from the root, parent [B][N] as in gdn_verify_tree): the
 * new history is the last W elements of [old history, x of the path nodes].
 * The copy is bit-exact.  1 <= W <= 8.  A bad accept index, slot or parent
 * array skips that sequence and is reported through `status`.  The slot[]
 * entries of one call must be distinct: the history is rewritten in place,
 * and two sequences sharing a slot race on it.
 */
int gdn_conv_commit(const void* x, int32_t in_dtype, void* conv_state,
                    int64_t state_slot_stride, const int32_t* slot, int32_t n_slots,
                    const int32_t* parent, const int32_t* accept_idx, int32_t B, int32_t N,
                    int32_t C, int32_t W, int32_t* status, void* stream);

/*
 * Index-table commit ("TokenSpeed hits 580 tok/s", section "How they actually
 * got there": move pointers, not data -- the persisted states form a draft
 * region and a small index table says which one is current).  No state is
 * copied: the slot table is pointed at the accepted node's snapshot,
 *
 *   slot[b] = base_slot + b*N + accept_idx[b]
 *
 * so that a verify call given the snapshots buffer [B][N][Hv][dk][dv] of this
 * block as its state_cache (cache_slot_stride = Hv*dk*dv, n_slots >=
 * base_slot + B*N) starts every sequence from its accepted node; base_slot
 * places the block's region inside a larger slot space.  That verify may
 * write its own snapshots into the same buffer.  An accept index outside
 * [0, N) leaves slot[b] unchanged and is reported through `status`.
 */
int gdn_commit_index(const int32_t* accept_idx, int32_t B, int32_t N, int32_t base_slot,
                     int32_t* slot, int32_t* status, void* stream);

/*
 * Checkpoint-and-replay commit ("Photon 2.6", section "Handling recurrent
 * state": keep the state from before the block and re-run the accepted
 * tokens instead of persisting every node).  For every sequence b the
 * recurrence is run again over the accepted path, starting from the cached
 * state, and the result replaces the cached state in place:
 *
 *   state_cache[slot[b]][h] <- S_{accept_idx[b]} of the block
 *
 * The path is nodes 0 .. accept_idx[b] for a chain (parent == NULL; accept
 * length L = accept_idx + 1) and the ancestors of accept_idx[b] from the root
 * for a tree (parent [B][N] as in gdn_verify_tree).  Uses k, v, alpha, beta,
 * state_cache, slot, n_slots, status and the sizes of `args` (args->q,
 * snapshots and o are not used and may be NULL); here state_cache is read and
 * written.  The state equals snapshots[b][accept_idx[b]] of a verify call on
 * the same inputs up to floating-point rounding.  An accept index outside
 * [0, N), a slot outside [0, n_slots) or a bad parent array skips that
 * sequence and is reported through args->status.  Two sequences must not
 * share a slot.
 */
int gdn_replay_accepted(const gdn_verify_args* args, const int32_t* parent,
                        const int32_t* accept_idx, void* stream);

/*
 * Chunked prefill of one sequence of T tokens: the same recurrence, evaluated
 * chunk by chunk in the WY / UT-transform form on tensor cores.
 *
 *   q, k   [T][Hk][dk]  bf16;  v [T][Hv][dv] bf16
 *   alpha, beta [T][Hv] fp32
 *   state  [Hv][dk][dv] fp32, in: the state before token 0, out: after token T-1
 *   o      [T][Hv][dv] fp32 output
 *   workspace  device scratch of at least gdn_prefill_workspace_bytes(...) bytes,
 *              owned by the caller, contents need not be initialised
 *   status optional device int32 error word (first error wins; the caller
 *          zeroes it): GDN_ERR_TIMEOUT if a bounded wait of the kernel on its
 *          own asynchronous copies or tensor-core work expired.  The kernel
 *          then stops early; the state of the affected heads is written as
 *          NaN, and o is not valid.
 *
 * Supported: dk = dv = 128, chunk = 64, in_dtype = GDN_BF16, T >= 0 (any T;
 * the last chunk may be partial); any other size or dtype returns
 * GDN_ERR_UNSUPPORTED before anything is launched.  GDN_ERR_WORKSPACE if the
 * workspace is NULL or too small.  Two kernels run on `stream`: a parallel
 * pass over (chunk, q/k head) that fills the workspace, then the sequential
 * pass over the chunks of each value head; the workspace may be reused once
 * the call's work has finished on the stream.
 */
size_t gdn_prefill_workspace_bytes(int32_t T, int32_t Hk, int32_t Hv, int32_t dk, int32_t dv,
                                   int32_t chunk);

int gdn_prefill_chunked(const void* q, const void* k, const void* v, int32_t in_dtype,
                        const float* alpha, const float* beta, int32_t T, int32_t Hk, int32_t Hv,
                        int32_t dk, int32_t dv, int32_t chunk, float* state, float* o,
                        void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * gdn_prefill_chunked without a workspace argument, for callers that cannot
 * allocate device memory themselves: for example a plugin whose host engine
 * owns every device allocation and offers it no allocator, or a code path
 * where the implicit synchronisation of cudaMalloc is not acceptable and no
 * buffer was reserved up front.  (The source pages have no counterpart to this
 * call; it is an addition of this library.)
 *
 * The call computes exactly what gdn_prefill_chunked computes, with the same
 * arguments minus `workspace`/`workspace_bytes`; the scratch it needs lives in
 * a device array built into the library of GDN_PREFILL_NOALLOC_SCRATCH_BYTES
 * (16 MiB) per GPU that loads the library, held until the process exits.
 * Limit: ceil(T/64) * Hv * 33280 bytes must fit, i.e. ceil(T/64) * Hv <= 504
 * (T <= 640 tokens at 48 value heads); larger problems return
 * GDN_ERR_SCRATCH_LIMIT without launching anything.  The library allocates
 * nothing here: no cudaMalloc, cudaFree or allocating library routine.
 *
 * Every call looks up the device address of the scratch array on the current
 * device (cudaGetSymbolAddress, a host-side query that is repeated each time
 * so that a reset device or a new context is never handed a stale address).
 * The first such lookup on a device loads the library's device code there;
 * make that first call before any stream capture.  All calls share the one
 * array, which keeps
 * the previous call's contents (nothing in it needs clearing: the first kernel
 * of a call writes every byte the second kernel reads).  Calls that overlap on
 * the GPU -- on different streams, or from different host threads -- race on
 * the shared scratch and must be serialised by the caller.
 */
#define GDN_PREFILL_NOALLOC_SCRATCH_BYTES (16u << 20)

int gdn_prefill_chunked_noalloc(const void* q, const void* k, const void* v, int32_t in_dtype,
                                const float* alpha, const float* beta, int32_t T, int32_t Hk,
                                int32_t Hv, int32_t dk, int32_t dv, int32_t chunk, float* state,
                                float* o, int32_t* status, void* stream);

/*
 * ---------------------------------------------------------------------------
 * 4-bit key/value cache of the full-attention layers
 * ---------------------------------------------------------------------------
 * A hybrid model keeps one full-attention layer for every three recurrent
 * ones.  The calls below give those layers the same speculative step as the
 * recurrent ones have: the block's keys and values are appended to a paged
 * cache held in 4 bits ("We got 207 tok/s with Qwen3.5-27B on an RTX 3090":
 * a KV cache quantised on write, 128K context), the block's queries attend
 * over it under the causal or the ancestor mask, the accepted path is
 * committed, and sequences share and free pages.
 *
 * Values.  A stored value is  code * scale * head_scale:  a 4-bit e2m1 code
 * (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; bit 3 is the sign), an e4m3
 * scale shared by 16 consecutive channels of one token, and an fp32 scale per
 * kv head (k_scale, v_scale; 1 where the pointer is NULL).  code * scale is
 * exact in binary16.
 *
 * Pages.  `pages` holds n_pages pages, page_stride bytes apart; a page holds
 * page_tokens tokens (a multiple of 32) of Hkv heads as
 * [Hkv][page_tokens/32] records of 36*D bytes.  A record is 32 tokens of one
 * head:
 *     K codes   [D/32][32 tokens][16 bytes]  byte i: channels 2i (low half), 2i+1
 *     V codes   [D][16 bytes]                byte i: tokens 2i (low half), 2i+1
 *     K scales  [32 tokens][D/16]            e4m3
 *     V scales  [D/16][32 tokens]            e4m3
 * Position p of sequence b is token p % page_tokens of page
 * table[b][p / page_tokens].
 *
 * Blocks.  kv_len[b] counts the block: node n of a block of N nodes is at
 * position kv_len[b] - N + n.  Nodes at negative positions do not exist (so
 * shorter blocks, and sequences of length 0, are given right-aligned in one
 * call): they are not written, read back as 0, and attend over nothing.
 *
 * Supported sizes: D in {64, 128, 256}; page_tokens a multiple of 32; any
 * Hkv >= 1, B >= 0, N >= 1.  Page starts are 16-byte aligned (page_stride a
 * multiple of 16).  A sequence with a length below 0 or above
 * max_pages*page_tokens is taken to have length 0, and GDN_ERR_ROW_RANGE is
 * reported; positions on a page number outside [0, n_pages) are left out (not
 * written, read as 0, not attended over), and GDN_ERR_PAGE_RANGE is reported.
 */
typedef struct gdn_kv4_cache {
  void* pages;
  const int32_t* table;  /* [B] rows of max_pages entries, table_stride entries apart */
  const int32_t* kv_len; /* [B] */
  const float* k_scale;  /* [Hkv] or NULL */
  const float* v_scale;  /* [Hkv] or NULL */
  int32_t* status;       /* optional device error word */
  int64_t page_stride;   /* bytes */
  int64_t table_stride;  /* entries */
  int32_t n_pages;
  int32_t page_tokens;
  int32_t max_pages;
  int32_t B;
  int32_t Hkv;
  int32_t D;
} gdn_kv4_cache;

/*
 * Append: quantise k and v [B][N][Hkv][D] (dtype GDN_F32, GDN_BF16 or GDN_F16;
 * the two strides of each in elements, multiples of 16 bytes; heads and
 * channels contiguous) into positions kv_len[b] - N .. kv_len[b] - 1.  With
 * y = x * (1 / head_scale), saturated at +-2688, and a = max |y| over the 16
 * channels, the scale is a * (1/6) rounded to e4m3 and the code y * (1 / scale)
 * rounded to e2m1, both to nearest even and saturating (every operation in
 * fp32; a scale that rounds to 0 gives codes of 0).  A NaN is stored as 0, an
 * infinity at +-2688, and GDN_ERR_NONFINITE is reported: what the cache holds
 * is always finite.  Pages written to must not be shared by two sequences of
 * the call (see gdn_kv4_reserve).
 */
int gdn_kv4_append(const gdn_kv4_cache* c, const void* k, const void* v, int32_t dtype,
                   int64_t k_stride_b, int64_t k_stride_n, int64_t v_stride_b,
                   int64_t v_stride_n, int32_t N, void* stream);

/*
 * Append with rotary positions: the queries q [B][N][Hq][D] and the keys of the block are turned
 * by their positions on one or several axes (text: one; images and video: time, height and
 * width), the queries are written to q_out, and keys and values appended as gdn_kv4_append does.
 *
 *   pairs        rotated pairs of a head: a multiple of 8, at most D/2; channels from 2*pairs on
 *                pass as they are
 *   adjacent     0: pair i is channels i and pairs + i; 1: channels 2i and 2i + 1
 *   cos_sin      [n_positions][2][pairs] fp32: the cosines, then the sines of a position (so the
 *                frequencies and their scaling are the caller's, in any precision)
 *   positions    position of node n of sequence b on axis a at
 *                positions[a*pos_stride_axis + b*pos_stride_b + n]
 *   axis         [pairs] bytes: the axis that a pair goes by (sections one after another,
 *                interleaved, or any other order); NULL: all go by axis 0
 *
 * A pair (i, j) with the cosine c and sine s of its axis' position becomes
 *     y_i = x_i c - x_j s,   y_j = x_j c + x_i s
 * in fp32, each product and the sum rounded to nearest even, nothing fused; q_out is y rounded
 * once to dtype, and the cache takes the keys' y unrounded.  So the stored codes and q_out are
 * fixed to the operation.
 *
 * q_out [B][N][Hq][D] is either q itself (with q's strides on axes longer than one: the queries
 * are turned in place, and channels that pass are not touched) or overlaps none of q, k and v;
 * its rows of Hq*D lie apart (the smaller of its strides is at least Hq*D, and the other passes
 * all of those rows), else GDN_ERR_INVALID_ARG.  q, k, v and q_out share a dtype (GDN_F32,
 * GDN_BF16 or GDN_F16); strides in elements, multiples of 16 bytes.  Nodes that do not exist give
 * q_out = 0, and their positions are not looked at.  A position outside [0, n_positions), or a
 * pair's axis outside [0, n_axes), leaves the node's pairs on that axis as they are (an infinity's
 * or a NaN's partner and the sign of a zero too), and GDN_ERR_POSITION_RANGE is reported.  A NaN
 * or infinity in a key is treated as gdn_kv4_append treats what the rotation makes of it.  Hq is a
 * multiple of Hkv, at most 65535, and Hkv at most 65503.
 */
typedef struct gdn_rotary {
  const float* cos_sin;
  const int32_t* positions;
  const uint8_t* axis;
  int64_t pos_stride_axis;
  int64_t pos_stride_b;
  int32_t n_positions;
  int32_t n_axes;
  int32_t pairs;
  int32_t adjacent;
} gdn_rotary;

int gdn_kv4_append_rotary(const gdn_kv4_cache* c, const gdn_rotary* r, const void* q,
                          int64_t q_stride_b, int64_t q_stride_n, int32_t Hq, void* q_out,
                          int64_t out_stride_b, int64_t out_stride_n, const void* k, const void* v,
                          int32_t dtype, int64_t k_stride_b, int64_t k_stride_n,
                          int64_t v_stride_b, int64_t v_stride_n, int32_t N, void* stream);

/*
 * Read back: the stored values of positions kv_len[b] - N .. kv_len[b] - 1 into
 * k_out and v_out [B][N][Hkv][D] (contiguous; rounded once to dtype).
 */
int gdn_kv4_read(const gdn_kv4_cache* c, void* k_out, void* v_out, int32_t dtype, int32_t N,
                 void* stream);

/*
 * Attention of the block's N query nodes over the cache (the block's own keys
 * and values having been appended):
 *     o[b][n][h] = sum_j p_j v_j,   p = softmax_j(scale * q[b][n][h] . k_j)
 * over the positions j that node n sees: all before the block, and in the
 * block the nodes up to n (parent == NULL, any N: a decoded token, a draft
 * chain, a piece of a prompt) or n's ancestors and n itself (parent [B][N] as in
 * gdn_verify_tree, N <= 64).  Query head h reads kv head h / (Hq / Hkv).
 *   q    [B][N][Hq][D] GDN_BF16 or GDN_F16, strides in elements (multiples of
 *        8), heads and channels contiguous
 *   o    [B][N][Hq][D] contiguous, q's dtype
 *   lse  optional [B][N][Hq] fp32: log sum_j exp(scale * q . k_j)
 * A node that sees nothing gives o = 0 and lse = -infinity.  A sequence whose
 * parent array is malformed is taken to have length 0 and GDN_ERR_BAD_TREE is
 * reported.  The workspace (gdn_kv4_attention_workspace_bytes, on the current
 * device) need not be initialised and may be reused once the call's work has
 * finished on the stream; the size depends on the sizes given here only, not on
 * the lengths, and is 0 for sizes that the call refuses.  The probabilities are
 * rounded to binary16 for the product with v (2^-11 of each down to 2^-21 of their
 * row's largest, 2^-32 of that below; their sum is taken before); queries are held
 * as binary16, scaled by powers of two (exact down to 2^-14 of their row's largest
 * element, within 2^-25 of it below); sums and the running maximum are fp32.  The
 * order of the sums depends on the lengths and the device alone: repeated calls
 * give the same bits.
 * GDN_ERR_UNSUPPORTED when B * Hkv * N * (Hq / Hkv) / 96 times max_pages *
 * page_tokens / 128 would not fit 31 bits (work is counted in tiles of 128
 * positions).  A wait inside the kernel that runs out is reported as
 * GDN_ERR_TIMEOUT; the outputs are then undefined.
 */
size_t gdn_kv4_attention_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv,
                                         int32_t D);

int gdn_kv4_attention(const gdn_kv4_cache* c, const void* q, int32_t dtype, int64_t q_stride_b,
                      int64_t q_stride_n, int32_t N, int32_t Hq, float scale,
                      const int32_t* parent, void* o, float* lse, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * gdn_kv4_attention through a sliding window that leaves the first tokens visible.  Of the
 * entries of its path (the positions before the block, then the block's nodes up to it or its
 * ancestors, and itself: the i-th ancestor from the root is entry kv_len[b] - N + i), a node
 * that is entry e sees the entries f with
 *     f > e - window   or   f < sinks,
 * so its own window's last entry is itself.  window >= 1, sinks >= 0; a window as long as the
 * sequence gives gdn_kv4_attention's result.  In a tree the window runs along each node's own
 * path.  Only tiles that some row sees are read.  Everything else, the workspace and its size
 * (gdn_kv4_attention_workspace_bytes) among it, is as for gdn_kv4_attention.
 */
int gdn_kv4_attention_window(const gdn_kv4_cache* c, const void* q, int32_t dtype,
                             int64_t q_stride_b, int64_t q_stride_n, int32_t N, int32_t Hq,
                             float scale, int32_t sinks, int32_t window, const int32_t* parent,
                             void* o, float* lse, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * gdn_kv4_attention for sequences that share pages (branches of a prompt, gdn_kv4_fork): what
 * the sequences of a group have in common is read, and multiplied, once for all of them.
 *
 *   group  [n_groups + 1] int32, device: group g is sequences group[g] .. group[g+1] - 1 of the
 *          batch (so branches of one prompt stand beside each other); 1 <= n_groups <= B.
 *          Sequences before group[0] and from group[n_groups] on share with nobody
 *
 * How much a group shares follows from the table: the positions before the blocks that lie on
 * the same pages, from the first position on and in whole tiles of 128, in all sequences of the
 * group that share a tile with the first of it.  A group that shares nothing is right as well,
 * and a sequence that is skipped does not count.  Offsets that are not ascending within [0, B]
 * are reported (GDN_ERR_ROW_RANGE), and nothing is shared then.  Where sharing cannot pay by the
 * sizes (the rows of a sequence fill the tensor cores' tiles by themselves, the table's width
 * leaves little to read, there are as many groups as sequences, or the work counted in tenths of
 * tiles would not fit 31 bits) every sequence is read for itself, and the offsets are not looked
 * at.  The sizes are what the host is given: where the lengths are short for the table's width
 * (max_pages * page_tokens), gdn_kv4_attention, or a max_pages that the lengths need, is faster.
 *
 * The result is gdn_kv4_attention's up to the order of the sums, which depends on the lengths,
 * the table, the groups and the device alone.  The workspace
 * (gdn_kv4_attention_shared_workspace_bytes; 0 for sizes that the call refuses) grows with B*N*Hq;
 * two calls that may overlap (two streams, two captured graphs) need one each.
 * GDN_ERR_UNSUPPORTED also when B * N * Hq does not fit 31 bits.  Everything else is as for
 * gdn_kv4_attention.
 */
size_t gdn_kv4_attention_shared_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv,
                                                int32_t D, int32_t n_groups);

int gdn_kv4_attention_shared(const gdn_kv4_cache* c, const void* q, int32_t dtype,
                             int64_t q_stride_b, int64_t q_stride_n, int32_t N, int32_t Hq,
                             float scale, const int32_t* parent, const int32_t* group,
                             int32_t n_groups, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * Commit the accepted path of a block, for n_layers layers at once (layer l's
 * pages at pages + l*layer_stride bytes, one table and length for all).  The
 * path is nodes 0 .. accept_idx[b] (parent == NULL) or the ancestors of
 * accept_idx[b] from the root (parent [B][N], N <= 64); its i-th node's keys
 * and values are moved to position kv_len[b] - N + i, codes and scales
 * unchanged, and len_out[b] = kv_len[b] - N + (nodes on the path).  Positions
 * from len_out[b] on keep unspecified contents.  len_out must not be kv_len.
 * A block with kv_len[b] < N, a bad accept index or a malformed parent array, or
 * one that has nodes to move and lies, in whole or in part, on a page number
 * outside the pool, leaves the sequence as it is in every layer (len_out[b] =
 * kv_len[b]) and is reported (GDN_ERR_ROW_RANGE, GDN_ERR_ACCEPT_RANGE,
 * GDN_ERR_BAD_TREE, GDN_ERR_PAGE_RANGE).  Pages that nodes are moved in must not
 * be held by another sequence as well: gdn_kv4_reserve gives a row its own before
 * the block is appended; branch it (gdn_kv4_fork) after the commit, not between.
 */
int gdn_kv4_commit(const gdn_kv4_cache* c, int64_t layer_stride, int32_t n_layers, int32_t N,
                   const int32_t* parent, const int32_t* accept_idx, int32_t* len_out,
                   void* stream);

/*
 * The page pool: a table of n_rows sequences, their lengths, and for every page
 * the number of table entries that hold it (ref[p]; 0 = free).  A row of length
 * n holds its first ceil(n / page_tokens) entries; the others are -1.  All of it
 * is device memory that the three calls below read and update on the stream, so
 * a captured step can branch and free sequences without the host.  The rows
 * named by one call must be distinct (fork: the dst rows; a dst row is not a
 * src row).  A row that cannot be served is left as it is and reported:
 * GDN_ERR_ROW_RANGE for a row, length or branch that is out of range, and
 * GDN_ERR_PAGE_RANGE for a page number outside [0, n_pages) among the pages that
 * the call has to look at (fork: all of the source's; release: those given up;
 * reserve: a partly filled last one).
 */
typedef struct gdn_kv4_pool {
  int32_t* table;  /* [n_rows] rows of max_pages entries, table_stride entries apart */
  int32_t* kv_len; /* [n_rows] */
  int32_t* ref;    /* [n_pages] */
  int32_t* status;
  int64_t table_stride;
  int32_t n_rows;
  int32_t max_pages;
  int32_t n_pages;
  int32_t page_tokens;
} gdn_kv4_pool;

/* Truncate rows[i] to keep_len[i] tokens (0 frees it; a keep_len of the row's length or more
 * changes nothing): the pages past it lose a holder and their entries become -1. */
int gdn_kv4_release(const gdn_kv4_pool* p, const int32_t* rows, const int32_t* keep_len,
                    int32_t F, void* stream);

/* Branch row src[i] onto the empty row dst[i]: the same pages, one more holder each. */
int gdn_kv4_fork(const gdn_kv4_pool* p, const int32_t* src, const int32_t* dst, int32_t F,
                 void* stream);

/*
 * Grow rows[i] to new_len[i] tokens (no less than its length), taking the
 * lowest-numbered free pages in the order of the rows.  Where the row's last
 * page is partly filled and had other holders when the call began, the row gets
 * a page of its own first: the records that hold tokens are copied, in all
 * n_layers layers (copy-on-write), and the old page loses a holder.  A row that
 * does not fit, and every row after it that needs pages, is left as it is:
 * GDN_ERR_POOL_EMPTY.  Afterwards positions below new_len[i] from the old
 * length on may be appended to, in the rows that were served (where some may not
 * be, gdn_kv4_reserve_granted says which).  GDN_ERR_UNSUPPORTED when F * max_pages would
 * not fit 31 bits (the pages that the rows ask for are added up).
 */
size_t gdn_kv4_reserve_workspace_bytes(int32_t F);

int gdn_kv4_reserve(const gdn_kv4_pool* p, void* pages, int64_t page_stride,
                    int64_t layer_stride, int32_t n_layers, int32_t Hkv, int32_t D,
                    const int32_t* rows, const int32_t* new_len, int32_t F, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * gdn_kv4_reserve that also says which rows were served: granted[i] = new_len[i]
 * for those, -1 for the others.
 *
 * A row that was refused keeps its length, and its last page may have other
 * holders; a block appended at that length would overwrite the row's last N
 * tokens, theirs too.  A step that goes on without the host therefore takes the
 * block's lengths from `granted`: given as kv_len of gdn_kv4_append, _attention and
 * _commit (with the table's rows in the order of rows[]), a -1 is skipped and
 * reported by each (GDN_ERR_ROW_RANGE, after GDN_ERR_POOL_EMPTY in a status word that
 * they share): nothing is written, the output is 0, len_out is -1.  That -1 as
 * keep_len of gdn_kv4_release leaves the row as it is.
 */
int gdn_kv4_reserve_granted(const gdn_kv4_pool* p, void* pages, int64_t page_stride,
                            int64_t layer_stride, int32_t n_layers, int32_t Hkv, int32_t D,
                            const int32_t* rows, const int32_t* new_len, int32_t F,
                            int32_t* granted, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Human-readable name of a gdn_status value (static string, never NULL). */
const char* gdn_status_string(int status);

/* GDN_VERSION of the loaded library. */
int gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
