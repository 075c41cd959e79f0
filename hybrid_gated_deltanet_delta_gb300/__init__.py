"""GB300 gated delta-rule verification library: Python binding.

A thin ctypes layer over libgdn.so (C ABI in include/gdn.h).  It only
marshals arguments: torch tensors in, raw device pointers and sizes out, the
current torch CUDA stream as the launch stream.  Every step of the path runs
in the library's CUDA kernels; there is no CPU or PyTorch fallback, and the
functions raise if the library is missing or a call fails.

Entry points (same names as the C ABI):
  gdn_verify_chain, gdn_verify_chain_f16, gdn_verify_tree, gdn_verify_tree_f16,
  gdn_commit_accepted,
  gdn_commit_accepted_f16, gdn_commit_index, gdn_conv_commit,
  gdn_replay_accepted,
  gdn_prefill_chunked, gdn_prefill_workspace_bytes, gdn_prefill_chunked_noalloc
  the 4-bit key/value cache of the full-attention layers: gdn_kv4_append,
  gdn_kv4_read, gdn_kv4_attention, gdn_kv4_commit, and its page pool:
  gdn_kv4_release, gdn_kv4_fork, gdn_kv4_reserve (gdn_kv4_reserve_granted)
and, for serving loops that issue the same call every step, bound calls
(bind_verify_chain, bind_verify_tree, bind_commit_accepted,
bind_replay_accepted, bind_prefill_chunked, bind_kv4_*): the arguments are marshalled once
and each call is one ctypes call.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libgdn.so")

GDN_OK = 0
GDN_ERR_INVALID_ARG = -1
GDN_ERR_UNSUPPORTED = -2
GDN_ERR_MISALIGNED = -3
GDN_ERR_CUDA = -4
GDN_ERR_BAD_TREE = -5
GDN_ERR_ACCEPT_RANGE = -6
GDN_ERR_SLOT_RANGE = -7
GDN_ERR_WORKSPACE = -8
GDN_ERR_SCRATCH_LIMIT = -9
GDN_ERR_TIMEOUT = -10
GDN_ERR_PAGE_RANGE = -11
GDN_ERR_POOL_EMPTY = -12
GDN_ERR_ROW_RANGE = -13
GDN_ERR_NONFINITE = -14
PREFILL_NOALLOC_SCRATCH_BYTES = 16 << 20

GDN_F32 = 0
GDN_BF16 = 1
GDN_F16 = 2

_lib = None


class GdnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


class VerifyArgs(ctypes.Structure):
    """Mirror of gdn_verify_args."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("alpha", ctypes.c_void_p), ("beta", ctypes.c_void_p),
        ("state_cache", ctypes.c_void_p), ("slot", ctypes.c_void_p),
        ("snapshots", ctypes.c_void_p), ("o", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("cache_slot_stride", ctypes.c_int64), ("n_slots", ctypes.c_int32),
        ("B", ctypes.c_int32), ("N", ctypes.c_int32), ("Hk", ctypes.c_int32),
        ("Hv", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32), ("tile_cols", ctypes.c_int32),
        ("row_warps", ctypes.c_int32), ("max_depth", ctypes.c_int32),
    ]


class Kv4Cache(ctypes.Structure):
    """Mirror of gdn_kv4_cache."""
    _fields_ = [
        ("pages", ctypes.c_void_p), ("table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("status", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64), ("table_stride", ctypes.c_int64),
        ("n_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("B", ctypes.c_int32), ("Hkv", ctypes.c_int32),
        ("D", ctypes.c_int32),
    ]


class Kv4Pool(ctypes.Structure):
    """Mirror of gdn_kv4_pool."""
    _fields_ = [
        ("table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("ref", ctypes.c_void_p),
        ("status", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
        ("n_rows", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int32),
        ("page_tokens", ctypes.c_int32),
    ]


def load(path: str | None = None):
    """Load libgdn.so (built by __graft_entry__.build()); raise if it is absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libgdn.so not found at {p}: build it first "
                           "(python -m hybrid_gated_deltanet_delta_gb300.build)")
    lib = ctypes.CDLL(p)
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.gdn_verify_chain.argtypes = [ctypes.POINTER(VerifyArgs), P]
    lib.gdn_verify_chain.restype = ctypes.c_int
    lib.gdn_verify_tree.argtypes = [ctypes.POINTER(VerifyArgs), P, P, P]
    lib.gdn_verify_tree.restype = ctypes.c_int
    lib.gdn_commit_accepted.argtypes = [P, i64, P, P, i64, i64, P, i32, i32, i32, i32, i32, i32,
                                        i32, P, P]
    lib.gdn_commit_accepted.restype = ctypes.c_int
    lib.gdn_verify_chain_prep.argtypes = [ctypes.POINTER(VerifyArgs), P]
    lib.gdn_verify_chain_prep.restype = ctypes.c_int
    lib.gdn_verify_tree_prep.argtypes = [ctypes.POINTER(VerifyArgs), P, P, P]
    lib.gdn_verify_tree_prep.restype = ctypes.c_int
    lib.gdn_replay_accepted_prep.argtypes = [ctypes.POINTER(VerifyArgs), P, P, P]
    lib.gdn_replay_accepted_prep.restype = ctypes.c_int
    lib.gdn_verify_chain_f16.argtypes = [ctypes.POINTER(VerifyArgs), P, P]
    lib.gdn_verify_chain_f16.restype = ctypes.c_int
    lib.gdn_verify_tree_f16.argtypes = [ctypes.POINTER(VerifyArgs), P, P, P, P]
    lib.gdn_verify_tree_f16.restype = ctypes.c_int
    lib.gdn_commit_accepted_f16.argtypes = [P, i64, P, P, i64, i64, P, i32, i32, i32, i32, i32,
                                            i32, i32, P, P]
    lib.gdn_commit_accepted_f16.restype = ctypes.c_int
    lib.gdn_conv_commit.argtypes = [P, i32, P, i64, P, i32, P, P, i32, i32, i32, i32, P, P]
    lib.gdn_conv_commit.restype = ctypes.c_int
    lib.gdn_commit_index.argtypes = [P, i32, i32, i32, P, P, P]
    lib.gdn_commit_index.restype = ctypes.c_int
    lib.gdn_replay_accepted.argtypes = [ctypes.POINTER(VerifyArgs), P, P, P]
    lib.gdn_replay_accepted.restype = ctypes.c_int
    lib.gdn_prefill_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.gdn_prefill_workspace_bytes.restype = sz
    lib.gdn_prefill_chunked.argtypes = [P, P, P, i32, P, P, i32, i32, i32, i32, i32, i32, P, P,
                                        P, sz, P, P]
    lib.gdn_prefill_chunked.restype = ctypes.c_int
    lib.gdn_prefill_chunked_noalloc.argtypes = [P, P, P, i32, P, P, i32, i32, i32, i32, i32, i32,
                                                P, P, P, P]
    lib.gdn_prefill_chunked_noalloc.restype = ctypes.c_int
    C, L = ctypes.POINTER(Kv4Cache), ctypes.POINTER(Kv4Pool)
    lib.gdn_kv4_append.argtypes = [C, P, P, i32, i64, i64, i64, i64, i32, P]
    lib.gdn_kv4_append.restype = ctypes.c_int
    lib.gdn_kv4_read.argtypes = [C, P, P, i32, i32, P]
    lib.gdn_kv4_read.restype = ctypes.c_int
    lib.gdn_kv4_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    lib.gdn_kv4_attention_workspace_bytes.restype = sz
    lib.gdn_kv4_attention.argtypes = [C, P, i32, i64, i64, i32, i32, ctypes.c_float, P, P, P, P,
                                      sz, P]
    lib.gdn_kv4_attention.restype = ctypes.c_int
    lib.gdn_kv4_commit.argtypes = [C, i64, i32, i32, P, P, P, P]
    lib.gdn_kv4_commit.restype = ctypes.c_int
    lib.gdn_kv4_release.argtypes = [L, P, P, i32, P]
    lib.gdn_kv4_release.restype = ctypes.c_int
    lib.gdn_kv4_fork.argtypes = [L, P, P, i32, P]
    lib.gdn_kv4_fork.restype = ctypes.c_int
    lib.gdn_kv4_reserve_workspace_bytes.argtypes = [i32]
    lib.gdn_kv4_reserve_workspace_bytes.restype = sz
    lib.gdn_kv4_reserve.argtypes = [L, P, i64, i64, i32, i32, i32, P, P, i32, P, sz, P]
    lib.gdn_kv4_reserve.restype = ctypes.c_int
    lib.gdn_kv4_reserve_granted.argtypes = [L, P, i64, i64, i32, i32, i32, P, P, i32, P, P, sz, P]
    lib.gdn_kv4_reserve_granted.restype = ctypes.c_int
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_version.argtypes = []
    lib.gdn_version.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def status_string(code: int) -> str:
    try:
        return load().gdn_status_string(int(code)).decode()
    except RuntimeError:
        return f"status {code}"


# ------------------------------------------------------------- marshalling
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(code, where):
    if code != GDN_OK:
        raise GdnError(code, where)


def _dtype_code(t):
    import torch

    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def make_verify_args(q, k, v, alpha, beta, state_cache, snapshots, o, *, slot=None, n_slots=None,
                     status=None, cache_slot_stride=None, tile_cols=0, row_warps=0,
                     max_depth=0):
    """Build a gdn_verify_args from tensors.  q, k [B,N,Hk,dk]; v [B,N,Hv,dv];
    alpha, beta [B,N,Hv] fp32; state_cache [n_slots,Hv,dk,dv] fp32 (or any
    buffer with `cache_slot_stride`); snapshots [B,N,Hv,dk,dv] fp32 or None
    (a chain committed by replay); o [B,N,Hv,dv] fp32.  q and o may be None for
    gdn_replay_accepted."""
    B, N, Hk, dk = k.shape
    Hv, dv = v.shape[2], v.shape[3]
    for t in (q, k, v, alpha, beta, state_cache, snapshots, o):
        _need(t is None or t.is_contiguous(), "all tensors must be contiguous")
    _need((q is None or q.shape == k.shape) and v.shape[:2] == (B, N), "q/k/v shapes disagree")
    _need((q is None or q.dtype == k.dtype) and k.dtype == v.dtype,
          "q, k and v must share a dtype")
    if cache_slot_stride is None:
        cache_slot_stride = Hv * dk * dv
    if n_slots is None:
        n_slots = state_cache.numel() // cache_slot_stride
    def ptr(t):
        return None if t is None else t.data_ptr()

    return VerifyArgs(
        q=ptr(q), k=k.data_ptr(), v=v.data_ptr(), alpha=alpha.data_ptr(),
        beta=beta.data_ptr(), state_cache=state_cache.data_ptr(), slot=ptr(slot),
        snapshots=ptr(snapshots), o=ptr(o), status=ptr(status),
        cache_slot_stride=cache_slot_stride, n_slots=n_slots, B=B, N=N, Hk=Hk, Hv=Hv, dk=dk,
        dv=dv, in_dtype=_dtype_code(k), tile_cols=tile_cols, row_warps=row_warps,
        max_depth=max_depth)


def gdn_verify_chain(q, k, v, alpha, beta, state_cache, snapshots, o, *, slot=None, n_slots=None,
                     status=None, cache_slot_stride=None, tile_cols=0, row_warps=0, stream=None,
                     prep=False):
    """Causal-chain verification; writes snapshots and o (see include/gdn.h).
    prep=True: q, k are raw projections and alpha, beta gate pre-activations
    (gdn_verify_chain_prep)."""
    a = make_verify_args(q, k, v, alpha, beta, state_cache, snapshots, o, slot=slot,
                         n_slots=n_slots, status=status, cache_slot_stride=cache_slot_stride,
                         tile_cols=tile_cols, row_warps=row_warps)
    fn = load().gdn_verify_chain_prep if prep else load().gdn_verify_chain
    _check(fn(ctypes.byref(a), _stream(stream)),
           "gdn_verify_chain_prep" if prep else "gdn_verify_chain")


def gdn_verify_chain_f16(q, k, v, alpha, beta, state_cache, snapshots_f16, o, *, slot=None,
                         n_slots=None, status=None, cache_slot_stride=None, tile_cols=0,
                         row_warps=0, stream=None):
    """Chain verification persisting every node's state as float16 (RNE) in
    snapshots_f16 [B,N,Hv,dk,dv]; outputs unchanged (see include/gdn.h)."""
    import torch

    _need(snapshots_f16.dtype == torch.float16 and snapshots_f16.is_contiguous(),
          "snapshots_f16 must be a contiguous float16 tensor")
    a = make_verify_args(q, k, v, alpha, beta, state_cache, None, o, slot=slot,
                         n_slots=n_slots, status=status, cache_slot_stride=cache_slot_stride,
                         tile_cols=tile_cols, row_warps=row_warps)
    _check(load().gdn_verify_chain_f16(ctypes.byref(a), _ptr(snapshots_f16), _stream(stream)),
           "gdn_verify_chain_f16")


def gdn_verify_tree_f16(q, k, v, alpha, beta, state_cache, snapshots_f16, o, parent, *,
                        depth_out=None, slot=None, n_slots=None, status=None,
                        cache_slot_stride=None, tile_cols=0, row_warps=0, max_depth=0,
                        stream=None):
    """Tree verification persisting every node's state as float16 (RNE) in
    snapshots_f16 [B,N,Hv,dk,dv]; outputs unchanged (see include/gdn.h)."""
    import torch

    _need(snapshots_f16.dtype == torch.float16 and snapshots_f16.is_contiguous(),
          "snapshots_f16 must be a contiguous float16 tensor")
    _need(parent.is_contiguous() and tuple(parent.shape) == tuple(k.shape[:2]),
          "parent must be a contiguous [B,N] int32 tensor")
    a = make_verify_args(q, k, v, alpha, beta, state_cache, None, o, slot=slot,
                         n_slots=n_slots, status=status, cache_slot_stride=cache_slot_stride,
                         tile_cols=tile_cols, row_warps=row_warps, max_depth=max_depth)
    _check(load().gdn_verify_tree_f16(ctypes.byref(a), _ptr(parent), _ptr(depth_out),
                                      _ptr(snapshots_f16), _stream(stream)),
           "gdn_verify_tree_f16")


def gdn_verify_tree(q, k, v, alpha, beta, state_cache, snapshots, o, parent, *, depth_out=None,
                    slot=None, n_slots=None, status=None, cache_slot_stride=None, tile_cols=0,
                    row_warps=0, max_depth=0, stream=None, prep=False):
    """Tree verification; parent [B,N] int32 (see include/gdn.h).  max_depth > 0
    skips (and reports through `status`) any sequence whose tree is deeper.
    prep=True: raw projections and gate pre-activations (gdn_verify_tree_prep)."""
    _need(parent.is_contiguous() and tuple(parent.shape) == tuple(q.shape[:2]),
          "parent must be a contiguous [B,N] int32 tensor")
    a = make_verify_args(q, k, v, alpha, beta, state_cache, snapshots, o, slot=slot,
                         n_slots=n_slots, status=status, cache_slot_stride=cache_slot_stride,
                         tile_cols=tile_cols, row_warps=row_warps, max_depth=max_depth)
    fn = load().gdn_verify_tree_prep if prep else load().gdn_verify_tree
    _check(fn(ctypes.byref(a), _ptr(parent), _ptr(depth_out), _stream(stream)),
           "gdn_verify_tree_prep" if prep else "gdn_verify_tree")


def gdn_commit_accepted(snapshots, accept_idx, state_cache, *, B, N, Hv, dk, dv, n_layers=1,
                        snap_layer_stride=0, cache_slot_stride=None, cache_layer_stride=0,
                        slot=None, n_slots=None, status=None, stream=None):
    """state_cache[l][slot[b]][h] = snapshots[l][b][accept_idx[b]][h] for every layer
    (fp32 snapshots; float16 ones go through gdn_commit_accepted_f16)."""
    if cache_slot_stride is None:
        cache_slot_stride = Hv * dk * dv
    if n_slots is None:
        n_slots = (state_cache.numel() - (n_layers - 1) * cache_layer_stride) // cache_slot_stride
    fn = load().gdn_commit_accepted
    name = "gdn_commit_accepted"
    if snapshots.dtype != state_cache.dtype:
        fn, name = load().gdn_commit_accepted_f16, "gdn_commit_accepted_f16"
    _check(fn(_ptr(snapshots), snap_layer_stride, _ptr(accept_idx), _ptr(state_cache),
              cache_slot_stride, cache_layer_stride, _ptr(slot), n_slots, B, N, Hv, dk, dv,
              n_layers, _ptr(status), _stream(stream)), name)


def gdn_commit_accepted_f16(snapshots_f16, accept_idx, state_cache, **kw):
    """gdn_commit_accepted from float16 snapshots, widened into the fp32 cache."""
    import torch

    _need(snapshots_f16.dtype == torch.float16, "snapshots_f16 must be float16")
    gdn_commit_accepted(snapshots_f16, accept_idx, state_cache, **kw)


def gdn_conv_commit(x, conv_state, accept_idx, *, parent=None, slot=None, n_slots=None,
                    state_slot_stride=None, status=None, stream=None):
    """Convolution-history commit in place: x [B,N,C] raw inputs of the block
    (bfloat16 or float32), conv_state [n_slots,C,W] of the same dtype; the
    history becomes the last W elements of [history, x of the accepted path]."""
    B, N, C = x.shape
    W = conv_state.shape[-1]
    _need(x.is_contiguous() and conv_state.is_contiguous(), "tensors must be contiguous")
    _need(x.dtype == conv_state.dtype, "x and conv_state must share a dtype")
    if state_slot_stride is None:
        state_slot_stride = C * W
    if n_slots is None:
        n_slots = conv_state.numel() // state_slot_stride
    _check(load().gdn_conv_commit(_ptr(x), _dtype_code(x), _ptr(conv_state), state_slot_stride,
                                  _ptr(slot), n_slots, _ptr(parent), _ptr(accept_idx), B, N, C,
                                  W, _ptr(status), _stream(stream)), "gdn_conv_commit")


def gdn_commit_index(accept_idx, slot, *, N, base_slot=0, status=None, stream=None):
    """Index-table commit: slot[b] = base_slot + b*N + accept_idx[b] (int32
    device tensors of B entries), so that the next verify reads its state from
    this block's snapshots buffer."""
    _need(accept_idx.is_contiguous() and slot.is_contiguous() and
          accept_idx.numel() == slot.numel(), "accept_idx and slot must be [B] int32")
    _check(load().gdn_commit_index(_ptr(accept_idx), accept_idx.numel(), N, base_slot, _ptr(slot),
                                   _ptr(status), _stream(stream)), "gdn_commit_index")


def gdn_replay_accepted(k, v, alpha, beta, state_cache, accept_idx, *, parent=None, slot=None,
                        n_slots=None, status=None, cache_slot_stride=None, tile_cols=0,
                        row_warps=0, stream=None, prep=False):
    """Checkpoint-and-replay commit: state_cache[slot[b]] <- the state of node
    accept_idx[b], recomputed over the accepted path from the cached state
    (chain when parent is None; parent [B,N] int32 for a tree)."""
    if parent is not None:
        _need(parent.is_contiguous() and tuple(parent.shape) == tuple(k.shape[:2]),
              "parent must be a contiguous [B,N] int32 tensor")
    _need(accept_idx.is_contiguous() and accept_idx.numel() == k.shape[0],
          "accept_idx must be a contiguous [B] int32 tensor")
    a = make_verify_args(None, k, v, alpha, beta, state_cache, None, None, slot=slot,
                         n_slots=n_slots, status=status, cache_slot_stride=cache_slot_stride,
                         tile_cols=tile_cols, row_warps=row_warps)
    fn = load().gdn_replay_accepted_prep if prep else load().gdn_replay_accepted
    _check(fn(ctypes.byref(a), _ptr(parent), _ptr(accept_idx), _stream(stream)),
           "gdn_replay_accepted_prep" if prep else "gdn_replay_accepted")


def gdn_prefill_workspace_bytes(T, Hk, Hv, dk, dv, chunk=64) -> int:
    return int(load().gdn_prefill_workspace_bytes(T, Hk, Hv, dk, dv, chunk))


def gdn_prefill_chunked(q, k, v, alpha, beta, state, o, workspace=None, *, chunk=64,
                        status=None, stream=None):
    """Chunked prefill of one sequence: q, k [T,Hk,dk]; v [T,Hv,dv]; alpha, beta [T,Hv];
    state [Hv,dk,dv] fp32 in/out; o [T,Hv,dv] fp32; workspace a uint8 device tensor of
    gdn_prefill_workspace_bytes(...) bytes (or None when that is 0); status an
    optional int32 device word that receives GDN_ERR_TIMEOUT if a bounded wait
    inside the kernel expired."""
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().gdn_prefill_chunked(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(alpha),
                                      _ptr(beta), T, Hk, Hv, dk, dv, chunk, _ptr(state), _ptr(o),
                                      _ptr(workspace), wbytes, _ptr(status), _stream(stream)),
           "gdn_prefill_chunked")


def gdn_prefill_chunked_noalloc(q, k, v, alpha, beta, state, o, *, chunk=64, status=None,
                                stream=None):
    """gdn_prefill_chunked on the library's built-in device scratch, for callers
    that cannot allocate device memory (no workspace argument).  Problems whose
    workspace would exceed PREFILL_NOALLOC_SCRATCH_BYTES raise GdnError with
    GDN_ERR_SCRATCH_LIMIT; calls that overlap on the GPU share the scratch and
    must be serialised by the caller."""
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    _check(load().gdn_prefill_chunked_noalloc(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q),
                                              _ptr(alpha), _ptr(beta), T, Hk, Hv, dk, dv, chunk,
                                              _ptr(state), _ptr(o), _ptr(status),
                                              _stream(stream)),
           "gdn_prefill_chunked_noalloc")


# ------------------------------------------------------- bound calls (serving)
class BoundCall:
    """One entry point with its arguments marshalled once.

    A serving loop that issues the same call every step (the same buffers,
    refilled in place) binds it once; each call then costs a single ctypes
    call: no shape checks, no argument struct built, no stream lookup.  The
    tensors given at binding time are kept alive by this object and must keep
    their addresses and shapes; the stream is fixed at binding time.  A
    non-zero status from the library raises GdnError, as the plain functions
    do."""

    __slots__ = ("_fn", "_name", "_args", "_keep")

    def __init__(self, fn, name, args, keep):
        self._fn, self._name, self._args, self._keep = fn, name, tuple(args), keep

    def __call__(self):
        code = self._fn(*self._args)
        if code != GDN_OK:
            raise GdnError(code, self._name)


def bind_verify_chain(q, k, v, alpha, beta, state_cache, snapshots, o, *, snapshots_f16=None,
                      stream=None, **kw):
    """gdn_verify_chain (or, with snapshots_f16, gdn_verify_chain_f16) bound
    to these buffers; keyword arguments as for gdn_verify_chain."""
    a = make_verify_args(q, k, v, alpha, beta, state_cache, snapshots, o, **kw)
    s = _stream(stream)
    if snapshots_f16 is not None:
        return BoundCall(load().gdn_verify_chain_f16, "gdn_verify_chain_f16",
                         (ctypes.byref(a), _ptr(snapshots_f16), s),
                         (a, q, k, v, alpha, beta, state_cache, snapshots_f16, o))
    return BoundCall(load().gdn_verify_chain, "gdn_verify_chain", (ctypes.byref(a), s),
                     (a, q, k, v, alpha, beta, state_cache, snapshots, o))


def bind_verify_tree(q, k, v, alpha, beta, state_cache, snapshots, o, parent, *, depth_out=None,
                     snapshots_f16=None, stream=None, **kw):
    """gdn_verify_tree (or, with snapshots_f16, gdn_verify_tree_f16) bound to
    these buffers; keyword arguments as for gdn_verify_tree."""
    _need(parent.is_contiguous() and tuple(parent.shape) == tuple(k.shape[:2]),
          "parent must be a contiguous [B,N] int32 tensor")
    a = make_verify_args(q, k, v, alpha, beta, state_cache, snapshots, o, **kw)
    s = _stream(stream)
    if snapshots_f16 is not None:
        return BoundCall(load().gdn_verify_tree_f16, "gdn_verify_tree_f16",
                         (ctypes.byref(a), _ptr(parent), _ptr(depth_out), _ptr(snapshots_f16), s),
                         (a, q, k, v, alpha, beta, state_cache, snapshots_f16, o, parent,
                          depth_out))
    return BoundCall(load().gdn_verify_tree, "gdn_verify_tree",
                     (ctypes.byref(a), _ptr(parent), _ptr(depth_out), s),
                     (a, q, k, v, alpha, beta, state_cache, snapshots, o, parent, depth_out))


def bind_commit_accepted(snapshots, accept_idx, state_cache, *, B, N, Hv, dk, dv, n_layers=1,
                         snap_layer_stride=0, cache_slot_stride=None, cache_layer_stride=0,
                         slot=None, n_slots=None, status=None, stream=None):
    """gdn_commit_accepted (gdn_commit_accepted_f16 for float16 snapshots)
    bound to these buffers."""
    if cache_slot_stride is None:
        cache_slot_stride = Hv * dk * dv
    if n_slots is None:
        n_slots = (state_cache.numel() - (n_layers - 1) * cache_layer_stride) // cache_slot_stride
    fn, name = load().gdn_commit_accepted, "gdn_commit_accepted"
    if snapshots.dtype != state_cache.dtype:
        fn, name = load().gdn_commit_accepted_f16, "gdn_commit_accepted_f16"
    args = (_ptr(snapshots), snap_layer_stride, _ptr(accept_idx), _ptr(state_cache),
            cache_slot_stride, cache_layer_stride, _ptr(slot), n_slots, B, N, Hv, dk, dv,
            n_layers, _ptr(status), _stream(stream))
    return BoundCall(fn, name, args, (snapshots, accept_idx, state_cache, slot, status))


def bind_replay_accepted(k, v, alpha, beta, state_cache, accept_idx, *, parent=None, stream=None,
                         **kw):
    """gdn_replay_accepted bound to these buffers."""
    a = make_verify_args(None, k, v, alpha, beta, state_cache, None, None, **kw)
    return BoundCall(load().gdn_replay_accepted, "gdn_replay_accepted",
                     (ctypes.byref(a), _ptr(parent), _ptr(accept_idx), _stream(stream)),
                     (a, k, v, alpha, beta, state_cache, accept_idx, parent))


def bind_prefill_chunked(q, k, v, alpha, beta, state, o, workspace=None, *, chunk=64,
                         status=None, stream=None):
    """gdn_prefill_chunked bound to these buffers."""
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(alpha), _ptr(beta), T, Hk, Hv, dk,
            dv, chunk, _ptr(state), _ptr(o), _ptr(workspace), wbytes, _ptr(status),
            _stream(stream))
    return BoundCall(load().gdn_prefill_chunked, "gdn_prefill_chunked", args,
                     (q, k, v, alpha, beta, state, o, workspace, status))


# ------------------------------------------- the 4-bit key/value cache
# Every function builds one BoundCall (checks and marshalling) and calls it; the
# bind_kv4_* functions return it.
def _dtype16(t):
    import torch

    if t.dtype == torch.float16:
        return GDN_F16
    return _dtype_code(t)


def _i32(t, shape, what):
    import torch

    _need(t is None or (t.dtype == torch.int32 and t.is_contiguous() and
                        tuple(t.shape) == tuple(shape)),
          f"{what} must be a contiguous int32 tensor of shape {tuple(shape)}")


def _kv4_pages(pages):
    """(n_layers, n_pages, Hkv, page_tokens, D, page_stride, layer_stride) of a
    pages tensor [n_pages,Hkv,page_tokens/32,36*D] (or with a layer dimension in
    front), uint8; the last three dimensions contiguous."""
    import torch

    _need(pages.dtype == torch.uint8 and pages.dim() in (4, 5),
          "pages must be uint8 [n_pages,Hkv,page_tokens/32,36*D], or [n_layers,...]")
    n_pages, Hkv, recs, rec = pages.shape[-4:]
    _need(rec % 36 == 0 and pages.stride()[-3:] == (recs * rec, rec, 1),
          "a page must be contiguous records of 36*D bytes")
    layers = pages.shape[0] if pages.dim() == 5 else 1
    return (layers, n_pages, Hkv, recs * 32, rec // 36, pages.stride(-4),
            pages.stride(0) if pages.dim() == 5 else 0)


def _kv4_table(table):
    import torch

    _need(table.dtype == torch.int32 and table.dim() == 2 and table.stride(1) == 1,
          "table must be int32 [rows,max_pages] with contiguous rows")


def _kv4_cache(pages, table, kv_len, k_scale, v_scale, status):
    import torch

    _, n_pages, Hkv, page_tokens, D, page_stride, _ = _kv4_pages(pages)
    B = kv_len.numel()
    _kv4_table(table)
    _need(table.shape[0] == B, "table and kv_len must have one row per sequence")
    _i32(kv_len, (B,), "kv_len")
    for t in (k_scale, v_scale):
        _need(t is None or (t.dtype == torch.float32 and t.is_contiguous() and t.numel() == Hkv),
              "k_scale and v_scale must be contiguous float32 [Hkv]")

    def ptr(t):
        return None if t is None else t.data_ptr()

    return Kv4Cache(pages=ptr(pages), table=ptr(table), kv_len=ptr(kv_len), k_scale=ptr(k_scale),
                    v_scale=ptr(v_scale), status=ptr(status), page_stride=page_stride,
                    table_stride=table.stride(0), n_pages=n_pages, page_tokens=page_tokens,
                    max_pages=table.shape[1], B=B, Hkv=Hkv, D=D)


def _rows(t, c, what):
    """Batch and node strides of [B,N,H,D] with contiguous heads and channels."""
    _need(t.dim() == 4 and t.shape[0] == c.B and t.shape[3] == c.D, f"{what} must be [B,N,H,D]")
    _need(t.stride(3) == 1 and (t.shape[2] == 1 or t.stride(2) == c.D),
          f"{what}'s heads and channels must be contiguous")
    return t.stride(0), t.stride(1)


def bind_kv4_append(k, v, pages, table, kv_len, *, k_scale=None, v_scale=None, status=None,
                    stream=None):
    """gdn_kv4_append bound to these buffers."""
    _need(pages.dim() == 4, "append takes one layer's pages")
    c = _kv4_cache(pages, table, kv_len, k_scale, v_scale, status)
    ks, vs = _rows(k, c, "k"), _rows(v, c, "v")
    _need(k.shape == v.shape and k.shape[2] == c.Hkv and k.dtype == v.dtype,
          "k and v must share a shape [B,N,Hkv,D] and a dtype")
    return BoundCall(load().gdn_kv4_append, "gdn_kv4_append",
                     (ctypes.byref(c), _ptr(k), _ptr(v), _dtype16(k), *ks, *vs, k.shape[1],
                      _stream(stream)),
                     (c, k, v, pages, table, kv_len, k_scale, v_scale, status))


def gdn_kv4_append(k, v, pages, table, kv_len, **kw):
    """Quantise k, v [B,N,Hkv,D] (float32, bfloat16 or float16; any batch and
    node strides) into positions kv_len[b]-N .. kv_len[b]-1 of the 4-bit cache.

    pages uint8 [n_pages,Hkv,page_tokens/32,36*D]; table int32 [B,max_pages];
    kv_len int32 [B]; k_scale, v_scale optional float32 [Hkv]; status an optional
    int32 device word (see include/gdn.h)."""
    bind_kv4_append(k, v, pages, table, kv_len, **kw)()


def bind_kv4_read(pages, table, kv_len, k_out, v_out, *, k_scale=None, v_scale=None, status=None,
                  stream=None):
    """gdn_kv4_read bound to these buffers."""
    _need(pages.dim() == 4, "read takes one layer's pages")
    c = _kv4_cache(pages, table, kv_len, k_scale, v_scale, status)
    _rows(k_out, c, "k_out")
    _need(k_out.shape == v_out.shape and k_out.dtype == v_out.dtype and
          k_out.shape[2] == c.Hkv and k_out.is_contiguous() and v_out.is_contiguous(),
          "k_out and v_out must be contiguous [B,N,Hkv,D] of one dtype")
    return BoundCall(load().gdn_kv4_read, "gdn_kv4_read",
                     (ctypes.byref(c), _ptr(k_out), _ptr(v_out), _dtype16(k_out), k_out.shape[1],
                      _stream(stream)),
                     (c, pages, table, kv_len, k_out, v_out, k_scale, v_scale, status))


def gdn_kv4_read(pages, table, kv_len, k_out, v_out, **kw):
    """The stored values of positions kv_len[b]-N .. kv_len[b]-1 into k_out and
    v_out [B,N,Hkv,D]; keyword arguments as for gdn_kv4_append."""
    bind_kv4_read(pages, table, kv_len, k_out, v_out, **kw)()


def gdn_kv4_attention_workspace_bytes(B, N, Hq, Hkv, D) -> int:
    return int(load().gdn_kv4_attention_workspace_bytes(B, N, Hq, Hkv, D))


def bind_kv4_attention(q, pages, table, kv_len, o, workspace, *, scale, parent=None, lse=None,
                       k_scale=None, v_scale=None, status=None, stream=None):
    """gdn_kv4_attention bound to these buffers."""
    import torch

    _need(pages.dim() == 4, "attention takes one layer's pages")
    c = _kv4_cache(pages, table, kv_len, k_scale, v_scale, status)
    qs = _rows(q, c, "q")
    B, N, Hq, _ = q.shape
    _need(o.shape == q.shape and o.dtype == q.dtype and o.is_contiguous(),
          "o must be a contiguous tensor of q's shape and dtype")
    _i32(parent, (B, N), "parent")
    _need(lse is None or (lse.dtype == torch.float32 and lse.is_contiguous() and
                          tuple(lse.shape) == (B, N, Hq)), "lse must be float32 [B,N,Hq]")
    return BoundCall(load().gdn_kv4_attention, "gdn_kv4_attention",
                     (ctypes.byref(c), _ptr(q), _dtype16(q), *qs, N, Hq, scale, _ptr(parent),
                      _ptr(o), _ptr(lse), _ptr(workspace),
                      workspace.numel() * workspace.element_size(), _stream(stream)),
                     (c, q, pages, table, kv_len, o, workspace, parent, lse, k_scale, v_scale,
                      status))


def gdn_kv4_attention(q, pages, table, kv_len, o, workspace, **kw):
    """o[b,n,h] = softmax(scale * q[b,n,h] . k) v over the cached positions that
    node n sees: all before the block, and within it the nodes up to n, or n's
    ancestors and itself where parent [B,N] is given (N <= 64).

    q, o [B,N,Hq,D] bfloat16 or float16 (q with any batch and node strides);
    workspace a uint8 tensor of gdn_kv4_attention_workspace_bytes(...) bytes;
    scale a float; lse an optional float32 [B,N,Hq]; the others as for
    gdn_kv4_append."""
    bind_kv4_attention(q, pages, table, kv_len, o, workspace, **kw)()


def bind_kv4_commit(pages, table, kv_len, accept_idx, len_out, *, N, parent=None, status=None,
                    stream=None):
    """gdn_kv4_commit bound to these buffers."""
    c = _kv4_cache(pages, table, kv_len, None, None, status)
    _i32(accept_idx, (c.B,), "accept_idx")
    _i32(len_out, (c.B,), "len_out")
    _i32(parent, (c.B, N), "parent")
    layers, layer_stride = (pages.shape[0], pages.stride(0)) if pages.dim() == 5 else (1, 0)
    return BoundCall(load().gdn_kv4_commit, "gdn_kv4_commit",
                     (ctypes.byref(c), layer_stride, layers, N, _ptr(parent), _ptr(accept_idx),
                      _ptr(len_out), _stream(stream)),
                     (c, pages, table, kv_len, accept_idx, len_out, parent, status))


def gdn_kv4_commit(pages, table, kv_len, accept_idx, len_out, **kw):
    """Move the accepted path of every block of N nodes to the block's start, in
    every layer of pages [n_layers,n_pages,Hkv,page_tokens/32,36*D], and write
    the committed lengths to len_out [B] (not kv_len itself).  accept_idx [B];
    parent [B,N] for trees, None for chains (whose path is in place already)."""
    bind_kv4_commit(pages, table, kv_len, accept_idx, len_out, **kw)()


def _kv4_pool(table, kv_len, ref, page_tokens, status):
    _kv4_table(table)
    n_rows = table.shape[0]
    _i32(kv_len, (n_rows,), "kv_len")
    _i32(ref, (ref.numel(),), "ref")
    return Kv4Pool(table=table.data_ptr(), kv_len=kv_len.data_ptr(), ref=ref.data_ptr(),
                   status=None if status is None else status.data_ptr(),
                   table_stride=table.stride(0), n_rows=n_rows, max_pages=table.shape[1],
                   n_pages=ref.numel(), page_tokens=page_tokens)


def bind_kv4_release(table, kv_len, ref, rows, keep_len, *, page_tokens, status=None,
                     stream=None):
    """gdn_kv4_release bound to these buffers."""
    p = _kv4_pool(table, kv_len, ref, page_tokens, status)
    _i32(rows, (rows.numel(),), "rows")
    _i32(keep_len, (rows.numel(),), "keep_len")
    return BoundCall(load().gdn_kv4_release, "gdn_kv4_release",
                     (ctypes.byref(p), _ptr(rows), _ptr(keep_len), rows.numel(),
                      _stream(stream)), (p, table, kv_len, ref, rows, keep_len, status))


def gdn_kv4_release(table, kv_len, ref, rows, keep_len, **kw):
    """Truncate rows[i] of the page table to keep_len[i] tokens (0 frees the
    row).  table int32 [n_rows,max_pages], kv_len int32 [n_rows], ref int32
    [n_pages] (holders of each page; 0 = free); page_tokens a keyword."""
    bind_kv4_release(table, kv_len, ref, rows, keep_len, **kw)()


def bind_kv4_fork(table, kv_len, ref, src, dst, *, page_tokens, status=None, stream=None):
    """gdn_kv4_fork bound to these buffers."""
    p = _kv4_pool(table, kv_len, ref, page_tokens, status)
    _i32(src, (src.numel(),), "src")
    _i32(dst, (src.numel(),), "dst")
    return BoundCall(load().gdn_kv4_fork, "gdn_kv4_fork",
                     (ctypes.byref(p), _ptr(src), _ptr(dst), src.numel(), _stream(stream)),
                     (p, table, kv_len, ref, src, dst, status))


def gdn_kv4_fork(table, kv_len, ref, src, dst, **kw):
    """Branch row src[i] onto the empty row dst[i]: both hold the same pages."""
    bind_kv4_fork(table, kv_len, ref, src, dst, **kw)()


def gdn_kv4_reserve_workspace_bytes(F) -> int:
    return int(load().gdn_kv4_reserve_workspace_bytes(F))


def bind_kv4_reserve(pages, table, kv_len, ref, rows, new_len, workspace, *, granted=None,
                     status=None, stream=None):
    """gdn_kv4_reserve (or, with granted, gdn_kv4_reserve_granted) bound to these buffers."""
    layers, n_pages, Hkv, page_tokens, D, page_stride, layer_stride = _kv4_pages(pages)
    p = _kv4_pool(table, kv_len, ref, page_tokens, status)
    _need(p.n_pages == n_pages, "ref must have one entry per page")
    _i32(rows, (rows.numel(),), "rows")
    _i32(new_len, (rows.numel(),), "new_len")
    _i32(granted, (rows.numel(),), "granted")
    fn, name, more = load().gdn_kv4_reserve, "gdn_kv4_reserve", ()
    if granted is not None:
        fn, name, more = load().gdn_kv4_reserve_granted, "gdn_kv4_reserve_granted", (_ptr(granted),)
    return BoundCall(fn, name,
                     (ctypes.byref(p), _ptr(pages), page_stride, layer_stride, layers, Hkv, D,
                      _ptr(rows), _ptr(new_len), rows.numel(), *more, _ptr(workspace),
                      workspace.numel() * workspace.element_size(), _stream(stream)),
                     (p, pages, table, kv_len, ref, rows, new_len, workspace, granted, status))


def gdn_kv4_reserve(pages, table, kv_len, ref, rows, new_len, workspace, **kw):
    """Grow rows[i] to new_len[i] tokens with the lowest-numbered free pages; a
    partly filled last page that has other holders is copied first, in every
    layer of pages.  workspace: gdn_kv4_reserve_workspace_bytes(len(rows)).

    granted, an optional int32 [len(rows)], gets new_len[i] for a row that was
    served and -1 for one that was not.  Given as kv_len of append, attention and
    commit it keeps a row that found no page, and those that share its pages, as
    they are (see include/gdn.h)."""
    bind_kv4_reserve(pages, table, kv_len, ref, rows, new_len, workspace, **kw)()
