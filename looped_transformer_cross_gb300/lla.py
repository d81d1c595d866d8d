"""Thin Python binding of liblla.so (include/lla.h): argument marshalling only.

Every step of the computation runs in the library's CUDA kernels.  PyTorch is
used for device memory and the current stream; tensors are passed by pointer.
If the library is missing, loading raises — there is no fallback.

Names follow the C ABI: :func:`encode` = ``lla_encode``, :func:`decode_attn` =
``lla_decode_attn``, :func:`workspace_size`, :func:`rope_table`,
:func:`device_status`, :func:`status_string`.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "liblla.so")

(LLA_OK, LLA_ERR_INVALID_ARG, LLA_ERR_UNSUPPORTED, LLA_ERR_CUDA, LLA_ERR_TIMEOUT, LLA_ERR_DEVICE_ARG,
 LLA_ERR_RANGE) = range(7)
LLA_BF16, LLA_F32 = 0, 1
LLA_PER_HEAD, LLA_2D = 0, 1
LLA_ROPE_HALF, LLA_ROPE_INTERLEAVED = 0, 1
LLA_ROPE_PLAIN, LLA_ROPE_LINEAR, LLA_ROPE_BASE, LLA_ROPE_BY_PARTS = range(4)
LLA_TREE_MAX_NODES = 128


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("d_head", ctypes.c_int),
                ("r_k", ctypes.c_int), ("r_v", ctypes.c_int), ("variant", ctypes.c_int),
                ("dtype", ctypes.c_int), ("rope_base", ctypes.c_float), ("rope_style", ctypes.c_int)]


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("B", ctypes.c_int),
                ("L_max", ctypes.c_int64)]


class PagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("B", ctypes.c_int), ("max_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_pages", ctypes.c_int64)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double), ("original_len", ctypes.c_int64),
                ("fast", ctypes.c_double), ("slow", ctypes.c_double)]


class Q4Cache(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("B", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int64)]


class Tree(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("n_tok", ctypes.c_int), ("max_nodes", ctypes.c_int),
                ("tok_start", ctypes.c_void_p), ("parent", ctypes.c_void_p), ("pos", ctypes.c_void_p)]


class LogitRulesC(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("hist_len", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p),
                ("max_history", ctypes.c_int), ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("bias_token", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("max_bias", ctypes.c_int), ("allowed", ctypes.c_void_p), ("allowed_row", ctypes.c_void_p),
                ("n_masks", ctypes.c_int)]


class LLAError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s: %s (status %d)" % (what, status_string(status), status))
        self.status = status


_lib = None
_lock = threading.Lock()


def lib():
    """Load liblla.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            L = ctypes.CDLL(LIB_PATH)
            vp, i32p, fp = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
            pd = ctypes.POINTER(Dims)
            L.lla_encode.argtypes = [pd, vp, vp, ctypes.c_int, i32p, i32p, vp, vp, fp, fp, Cache,
                                     vp, ctypes.c_size_t, vp]
            L.lla_encode.restype = ctypes.c_int
            L.lla_decode_attn.argtypes = [pd, ctypes.c_int, vp, Cache, i32p, i32p, vp, vp, fp, fp,
                                          fp, fp, ctypes.c_int64, fp, fp, vp, ctypes.c_size_t, vp]
            L.lla_decode_attn.restype = ctypes.c_int
            L.lla_workspace_size.argtypes = [pd, ctypes.c_int, ctypes.c_int64, ctypes.c_int]
            L.lla_workspace_size.restype = ctypes.c_size_t
            L.lla_rope_table.argtypes = [pd, ctypes.c_int64, fp, fp]
            L.lla_rope_table.restype = ctypes.c_int
            L.lla_device_status.argtypes = [vp, vp, ctypes.c_int]
            L.lla_device_status.restype = ctypes.c_int
            L.lla_status_string.argtypes = [ctypes.c_int]
            L.lla_status_string.restype = ctypes.c_char_p
            L.lla_window_attn.argtypes = [pd, ctypes.c_int, ctypes.c_int, vp, vp, vp, i32p, i32p, i32p,
                                          fp, fp, ctypes.c_int64, fp, fp, vp, ctypes.c_size_t, vp]
            L.lla_window_attn.restype = ctypes.c_int
            L.lla_decoupled_workspace_size.argtypes = [pd, ctypes.c_int, ctypes.c_int, ctypes.c_int64]
            L.lla_decoupled_workspace_size.restype = ctypes.c_size_t
            L.lla_decode_attn_decoupled.argtypes = [pd, ctypes.c_int, ctypes.c_int, vp, Cache, vp, i32p, i32p, vp, vp,
                                                    fp, fp, fp, fp, ctypes.c_int64, fp, fp, vp, ctypes.c_size_t, vp]
            L.lla_decode_attn_decoupled.restype = ctypes.c_int
            L.lla_encode_paged.argtypes = [pd, vp, vp, ctypes.c_int, i32p, i32p, vp, vp, fp, fp, PagedCache,
                                           vp, ctypes.c_size_t, vp]
            L.lla_encode_paged.restype = ctypes.c_int
            L.lla_decode_attn_paged.argtypes = [pd, ctypes.c_int, vp, PagedCache, i32p, i32p, vp, vp, fp, fp,
                                                fp, fp, ctypes.c_int64, fp, fp, vp, ctypes.c_size_t, vp]
            L.lla_decode_attn_paged.restype = ctypes.c_int
            L.lla_decode_attn_noalloc.argtypes = [pd, ctypes.c_int, vp, Cache, i32p, i32p, vp, vp, fp, fp,
                                                  fp, fp, ctypes.c_int64, fp, fp, vp]
            L.lla_decode_attn_noalloc.restype = ctypes.c_int
            L.lla_evict_window.argtypes = [pd, Cache, i32p, ctypes.c_int, ctypes.c_int, vp, ctypes.c_size_t, vp]
            L.lla_evict_window.restype = ctypes.c_int
            i32, i64, sz, i64p = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
            pq = ctypes.POINTER(Q4Cache)
            L.lla_rope_table_scaled.argtypes = [pd, ctypes.POINTER(RopeScaling), i64, i64, fp, fp, vp]
            L.lla_rope_table_scaled.restype = ctypes.c_int
            L.lla_rope_apply.argtypes = [pd, vp, i64, i64, vp, i64, i64, i32, i32, i32, i32, i32, i32p, fp, fp, i64,
                                         ctypes.c_float, i32, vp, sz, vp]
            L.lla_rope_apply.restype = ctypes.c_int
            L.lla_page_plan.argtypes = [i32, i32, i32, i64, i32p, i32p, i32p, i32, i32p, i32p, i32p, i32p, i32p, i32,
                                        i32p, i32p, i64p, i32p, vp, sz, vp]
            L.lla_page_plan.restype = ctypes.c_int
            L.lla_q4_row_bytes.argtypes = [pd]
            L.lla_q4_row_bytes.restype = sz
            L.lla_q4_store.argtypes = [pd, vp, vp, i32, i64p, pq, vp, sz, vp]
            L.lla_q4_store.restype = ctypes.c_int
            L.lla_q4_load.argtypes = [pd, i64p, i32, pq, vp, vp, vp, sz, vp]
            L.lla_q4_load.restype = ctypes.c_int
            L.lla_q4_workspace_size.argtypes = [pd, i32, i64]
            L.lla_q4_workspace_size.restype = sz
            L.lla_decode_attn_q4.argtypes = [pd, i32, vp, pq, i32p, i32p, vp, vp, fp, fp, fp, fp, i64, vp, fp,
                                             vp, sz, vp]
            L.lla_decode_attn_q4.restype = ctypes.c_int
            pt, pr = ctypes.POINTER(Tree), ctypes.POINTER(LogitRulesC)
            after = [i32p, vp, vp, fp, fp, fp, fp, i64, vp, fp, vp, sz, vp]
            L.lla_tree_workspace_size.argtypes = [pd, i32, i32, i64]
            L.lla_tree_workspace_size.restype = sz
            L.lla_tree_attn.argtypes = [pd, i32, pt, vp, i64, vp, i64, vp, i64, Cache] + after
            L.lla_tree_attn.restype = ctypes.c_int
            L.lla_tree_attn_paged.argtypes = [pd, i32, pt, vp, i64, vp, i64, vp, i64, PagedCache] + after
            L.lla_tree_attn_paged.restype = ctypes.c_int
            L.lla_tree_kernel.argtypes = [pd, i32]
            L.lla_tree_kernel.restype = ctypes.c_char_p
            L.lla_logits_workspace_size.argtypes = [i32, i32]
            L.lla_logits_workspace_size.restype = sz
            L.lla_logits_adjust.argtypes = [pt, i32p, i32, vp, i64, i32, pr, vp, i64, i32p, fp, vp, sz, vp]
            L.lla_logits_adjust.restype = ctypes.c_int
            L.lla_tree_accept.argtypes = [pt, i32p, i32p, i32p, i32p, i32p, i32p, i32p, i32p, i32p, vp, sz, vp]
            L.lla_tree_accept.restype = ctypes.c_int
            L.lla_decode_kernel.argtypes = [pd]
            L.lla_decode_kernel.restype = ctypes.c_char_p
            L.lla_decoupled_kernel.argtypes = [pd, ctypes.c_int]
            L.lla_decoupled_kernel.restype = ctypes.c_char_p
            L.lla_abi_version.argtypes = []
            L.lla_abi_version.restype = ctypes.c_int
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().lla_status_string(int(status)).decode()


def decode_kernel(dm: Dims) -> Optional[str]:
    """Kernel family lla_decode_attn runs for these dims ("tile", "small-rank",
    "pair-2d", "fp32"), or None if they are invalid or unsupported."""
    r = lib().lla_decode_kernel(ctypes.byref(dm))
    return None if r is None else r.decode()


def decoupled_kernel(dm: Dims, d_rope: int = 64) -> Optional[str]:
    """Kernel family lla_decode_attn_decoupled runs for these dims ("small-rank",
    "tile", "fp32"), or None if they are invalid or unsupported."""
    r = lib().lla_decoupled_kernel(ctypes.byref(dm), int(d_rope))
    return None if r is None else r.decode()


def dims(T, H, r_k, r_v, d_head=128, variant=LLA_PER_HEAD, dtype=LLA_BF16, rope_base=10000.0,
         rope_style=LLA_ROPE_HALF) -> Dims:
    return Dims(T, H, d_head, r_k, r_v, variant, dtype, float(rope_base), rope_style)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to liblla must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, what: str):
    if status != LLA_OK:
        raise LLAError(status, what)


def workspace_size(dm: Dims, B: int, L_max: int, max_N: int = 0) -> int:
    n = lib().lla_workspace_size(ctypes.byref(dm), int(B), int(L_max), int(max_N))
    if n == 0:
        raise LLAError(LLA_ERR_INVALID_ARG, "lla_workspace_size")
    return n


def make_workspace(dm: Dims, B: int, L_max: int, max_N: int = 0, device="cuda") -> torch.Tensor:
    """A zero-filled workspace buffer of the required size (status word cleared)."""
    return torch.zeros(workspace_size(dm, B, L_max, max_N), dtype=torch.uint8, device=device)


def rope_table(dm: Dims, n_pos: int):
    """(cos, sin) fp32 CPU tensors [n_pos][d/2] from lla_rope_table (fp64 on the host)."""
    c = torch.empty((int(n_pos), dm.d_head // 2), dtype=torch.float32)
    s = torch.empty_like(c)
    _check(lib().lla_rope_table(ctypes.byref(dm), int(n_pos), _ptr(c), _ptr(s)), "lla_rope_table")
    return c, s


def encode(dm: Dims, x_k, x_v, seq_idx, pos, w_down_k, w_down_v, mu_k, mu_v, cache_k, cache_v,
           workspace, stream=None):
    """lla_encode: latents of N tokens into cache slots (seq_idx[n], pos[n])."""
    N = int(seq_idx.shape[0])
    B = int(cache_k.shape[0])
    L_max = int(cache_k.shape[2] if dm.variant == LLA_PER_HEAD else cache_k.shape[1])
    cache = Cache(ctypes.c_void_p(cache_k.data_ptr()), ctypes.c_void_p(cache_v.data_ptr()), B, L_max)
    st = lib().lla_encode(ctypes.byref(dm), _ptr(x_k), _ptr(x_v), N, _ptr(seq_idx), _ptr(pos),
                          _ptr(w_down_k), _ptr(w_down_v), _ptr(mu_k), _ptr(mu_v), cache,
                          _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "lla_encode")


def decode_attn(dm: Dims, loop_t: int, q, cache_k, cache_v, seq_lens, q_pos, w_up_k, w_up_v,
                mu_k, mu_v, rope_cos, rope_sin, out, lse, workspace, stream=None):
    """lla_decode_attn: one layer, loop ``loop_t``, all heads and sequences, into out / lse."""
    B = int(cache_k.shape[0])
    L_max = int(cache_k.shape[2] if dm.variant == LLA_PER_HEAD else cache_k.shape[1])
    cache = Cache(ctypes.c_void_p(cache_k.data_ptr()), ctypes.c_void_p(cache_v.data_ptr()), B, L_max)
    st = lib().lla_decode_attn(ctypes.byref(dm), int(loop_t), _ptr(q), cache, _ptr(seq_lens),
                               _ptr(q_pos), _ptr(w_up_k), _ptr(w_up_v), _ptr(mu_k), _ptr(mu_v),
                               _ptr(rope_cos), _ptr(rope_sin), int(rope_cos.shape[0]), _ptr(out),
                               _ptr(lse), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "lla_decode_attn")


def paged_cache(pool_k, pool_v, block_table, page_size: int) -> PagedCache:
    """The lla_paged_cache of pools [num_pages][H][page_size][r] and a block table
    [B][max_pages] (int32, device)."""
    B, max_pages = int(block_table.shape[0]), int(block_table.shape[1])
    return PagedCache(ctypes.c_void_p(pool_k.data_ptr()), ctypes.c_void_p(pool_v.data_ptr()),
                      ctypes.c_void_p(block_table.data_ptr()), B, max_pages, int(page_size),
                      int(pool_k.shape[0]))


def encode_paged(dm: Dims, x_k, x_v, seq_idx, pos, w_down_k, w_down_v, mu_k, mu_v, pool_k, pool_v,
                 block_table, page_size: int, workspace, stream=None):
    """lla_encode_paged: latents of N tokens into paged slots (seq_idx[n], pos[n])."""
    N = int(seq_idx.shape[0])
    st = lib().lla_encode_paged(ctypes.byref(dm), _ptr(x_k), _ptr(x_v), N, _ptr(seq_idx), _ptr(pos),
                                _ptr(w_down_k), _ptr(w_down_v), _ptr(mu_k), _ptr(mu_v),
                                paged_cache(pool_k, pool_v, block_table, page_size),
                                _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "lla_encode_paged")


def decode_attn_paged(dm: Dims, loop_t: int, q, pool_k, pool_v, block_table, page_size: int, seq_lens,
                      q_pos, w_up_k, w_up_v, mu_k, mu_v, rope_cos, rope_sin, out, lse, workspace,
                      stream=None):
    """lla_decode_attn_paged: lla_decode_attn over a paged cache (pools [num_pages][H][page_size][r],
    block table [B][max_pages])."""
    st = lib().lla_decode_attn_paged(ctypes.byref(dm), int(loop_t), _ptr(q),
                                     paged_cache(pool_k, pool_v, block_table, page_size), _ptr(seq_lens),
                                     _ptr(q_pos), _ptr(w_up_k), _ptr(w_up_v), _ptr(mu_k), _ptr(mu_v),
                                     _ptr(rope_cos), _ptr(rope_sin), int(rope_cos.shape[0]), _ptr(out),
                                     _ptr(lse), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "lla_decode_attn_paged")


def evict_window(dm: Dims, cache_k, cache_v, seq_lens, sink: int, window: int, workspace, stream=None):
    """lla_evict_window: keep each sequence's `sink` first and `window` newest latents
    (moved in order to slots sink..), rewriting seq_lens in place."""
    B = int(cache_k.shape[0])
    L_max = int(cache_k.shape[2] if dm.variant == LLA_PER_HEAD else cache_k.shape[1])
    cache = Cache(ctypes.c_void_p(cache_k.data_ptr()), ctypes.c_void_p(cache_v.data_ptr()), B, L_max)
    st = lib().lla_evict_window(ctypes.byref(dm), cache, _ptr(seq_lens), int(sink), int(window), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "lla_evict_window")


def window_attn(dm: Dims, q, k_win, v_win, win_len, win_pos, q_pos, rope_cos, rope_sin, out, lse,
                workspace, stream=None):
    """lla_window_attn: exact attention over each sequence's window of recent tokens
    (k_win / v_win [B][H][W][d], keys before RoPE, token w at position win_pos[b] + w),
    merged in place into ``out`` / ``lse`` holding lla_decode_attn's latent result."""
    B, W = int(k_win.shape[0]), int(k_win.shape[2])
    st = lib().lla_window_attn(ctypes.byref(dm), B, W, _ptr(q), _ptr(k_win), _ptr(v_win), _ptr(win_len),
                               _ptr(win_pos), _ptr(q_pos), _ptr(rope_cos), _ptr(rope_sin),
                               int(rope_cos.shape[0]), _ptr(out), _ptr(lse), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "lla_window_attn")


def decoupled_workspace(dm: Dims, d_rope: int, B: int, L_max: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for lla_decode_attn_decoupled."""
    n = lib().lla_decoupled_workspace_size(ctypes.byref(dm), int(d_rope), int(B), int(L_max))
    if n == 0:
        raise LLAError(LLA_ERR_INVALID_ARG, "lla_decoupled_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def decode_attn_decoupled(dm: Dims, loop_t: int, q, cache_k, cache_v, k_rope, seq_lens, q_pos, w_up_k,
                          w_up_v, mu_k, mu_v, rope_cos, rope_sin, out, lse, workspace, stream=None):
    """lla_decode_attn_decoupled: absorbed decoupled-RoPE decode (content on the latents,
    a d_rope = k_rope.shape[3] rotary branch); q is [B][H][d + d_rope]."""
    B, L_max = int(cache_k.shape[0]), int(cache_k.shape[2])
    cache = Cache(ctypes.c_void_p(cache_k.data_ptr()), ctypes.c_void_p(cache_v.data_ptr()), B, L_max)
    st = lib().lla_decode_attn_decoupled(ctypes.byref(dm), int(loop_t), int(k_rope.shape[3]), _ptr(q), cache,
                                         _ptr(k_rope), _ptr(seq_lens), _ptr(q_pos), _ptr(w_up_k), _ptr(w_up_v),
                                         _ptr(mu_k), _ptr(mu_v), _ptr(rope_cos), _ptr(rope_sin),
                                         int(rope_cos.shape[0]), _ptr(out), _ptr(lse), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "lla_decode_attn_decoupled")


def device_status(workspace, stream=None, clear=True) -> int:
    """Synchronise and read (then clear) the kernels' status word in ``workspace``."""
    return int(lib().lla_device_status(_ptr(workspace), _stream(stream), 1 if clear else 0))


class Decoder:
    """Convenience holder of one layer's codec parameters and a RoPE table on the device.

    ``__call__`` runs ``lla_decode_attn`` for loop t and returns (out, lse).
    """

    def __init__(self, dm: Dims, w_up_k, w_up_v, mu_k, mu_v, B: int, L_max: int, device="cuda"):
        self.dm = dm
        self.w_up_k, self.w_up_v, self.mu_k, self.mu_v = w_up_k, w_up_v, mu_k, mu_v
        n = max(int(L_max), 128)
        c, s = rope_table(dm, n)
        self.rope_cos, self.rope_sin = c.to(device), s.to(device)
        self.workspace = make_workspace(dm, B, L_max, device=device)

    def __call__(self, loop_t, q, cache_k, cache_v, seq_lens, q_pos, out=None, lse=None, stream=None):
        B, H = q.shape[0], q.shape[1]
        if out is None:
            out = torch.empty((B, H, self.dm.d_head), dtype=torch.float32, device=q.device)
        if lse is None:
            lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
        decode_attn(self.dm, loop_t, q, cache_k, cache_v, seq_lens, q_pos, self.w_up_k,
                    self.w_up_v, self.mu_k, self.mu_v, self.rope_cos, self.rope_sin, out, lse,
                    self.workspace, stream)
        return out, lse


def decode_attn_noalloc(dm: Dims, loop_t: int, q, cache_k, cache_v, seq_lens, q_pos, w_up_k,
                        w_up_v, mu_k, mu_v, rope_cos, rope_sin, out, lse, stream=None):
    """lla_decode_attn_noalloc: lla_decode_attn with the library's fixed device scratch
    instead of a caller workspace, for callers that cannot allocate device memory.
    Calls that overlap on the GPU race on that scratch; make the first call on a
    device before any stream capture."""
    f = lib().lla_decode_attn_noalloc
    B = int(cache_k.shape[0])
    L_max = int(cache_k.shape[2] if dm.variant == LLA_PER_HEAD else cache_k.shape[1])
    cache = Cache(ctypes.c_void_p(cache_k.data_ptr()), ctypes.c_void_p(cache_v.data_ptr()), B, L_max)
    st = f(ctypes.byref(dm), int(loop_t), _ptr(q), cache, _ptr(seq_lens), _ptr(q_pos), _ptr(w_up_k),
           _ptr(w_up_v), _ptr(mu_k), _ptr(mu_v), _ptr(rope_cos), _ptr(rope_sin),
           int(rope_cos.shape[0]), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "lla_decode_attn_noalloc")


# ---------------------------------------------------------------- RoPE operators, page plans, the 4-bit cache
#
# These calls check what they are given (types, shapes, one device) before they pass
# pointers on, and run on the tensors' own device: its current stream unless `stream` is
# given.  A step's calls are short, so the checks that pass cost little: one comparison
# per property, and the wording of an error only once something does not fit.

def _need(cond: bool, what: str):
    if not cond:
        raise ValueError(what)


def _misfit(name: str, t, dtype, index, shape):
    """Raise the error that names what does not fit of an argument tensor."""
    _need(isinstance(t, torch.Tensor), name + " must be a tensor")
    _need(t.dtype == dtype, "%s must be %s, not %s" % (name, dtype, t.dtype))
    _need(t.is_cuda, "%s is on %s: a CUDA device is needed" % (name, t.device))
    _need(t.get_device() == index, "%s is on %s, not on cuda:%d" % (name, t.device, index))
    _need(shape is None or t.shape == shape, "%s has shape %s, not %s" % (name, tuple(t.shape), shape))
    _need(t.is_contiguous(), name + " must be contiguous")
    raise ValueError(name + " does not fit")


def _arg(name: str, t, dtype, index: int, shape):
    """Address of an argument tensor of this type, device, shape and contiguous."""
    try:
        if t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _misfit(name, t, dtype, index, shape)


def _device_of(name: str, t) -> int:
    _need(isinstance(t, torch.Tensor), name + " must be a tensor")
    index = t.get_device()
    _need(index >= 0, "%s is on %s: a CUDA device is needed" % (name, t.device))
    return index


def _space(t, index: int):
    """Address and bytes of a workspace."""
    _need(isinstance(t, torch.Tensor) and t.get_device() == index and t.is_contiguous(),
          "the workspace must be a contiguous tensor on cuda:%d" % index)
    return t.data_ptr(), t.numel() * t.element_size()


def _storage(dm: Dims):
    return torch.bfloat16 if dm.dtype == LLA_BF16 else torch.float32


def _run(what: str, f, index: int, stream, *args):
    """Call f(*args, stream) with device ``index`` current; raise for a status that is not ok."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        _need(stream.device.index == index, "the stream is of %s, not of cuda:%d" % (stream.device, index))
        raw = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        status = f(*args, raw)
    else:
        with torch.cuda.device(index):
            status = f(*args, raw)
    if status != LLA_OK:
        raise LLAError(status, what)


_SCALINGS = {"plain": LLA_ROPE_PLAIN, "linear": LLA_ROPE_LINEAR, "base": LLA_ROPE_BASE, "by_parts": LLA_ROPE_BY_PARTS}


def rope_scaling(kind="plain", factor=1.0, original_len=0, fast=32.0, slow=1.0) -> RopeScaling:
    """An lla_rope_scaling: ``kind`` is "plain", "linear", "base" or "by_parts"."""
    _need(kind in _SCALINGS, "unknown scaling %r" % (kind,))
    return RopeScaling(_SCALINGS[kind], float(factor), int(original_len), float(fast), float(slow))


def rope_table_scaled(dm: Dims, n_pos: int, scaling: Optional[RopeScaling] = None, pos0: int = 0, cos=None, sin=None,
                      device=None, stream=None):
    """lla_rope_table_scaled: (cos, sin) fp32 [n_pos][d_head/2] built on the GPU, for positions
    pos0 .. pos0 + n_pos - 1."""
    shape = (int(n_pos), dm.d_head // 2)
    _need((cos is None) == (sin is None), "give both outputs or neither")
    if cos is None:
        cos = torch.empty(shape, dtype=torch.float32, device="cuda" if device is None else device)
        sin = torch.empty_like(cos)
    dev = _device_of("cos", cos)
    _run("lla_rope_table_scaled", lib().lla_rope_table_scaled, dev, stream, ctypes.byref(dm),
         None if scaling is None else ctypes.byref(scaling), pos0, n_pos, _arg("cos", cos, torch.float32, dev, shape),
         _arg("sin", sin, torch.float32, dev, shape))
    return cos, sin


def rope_apply(dm: Dims, x, pos, rope_cos, rope_sin, out=None, offset: int = 0, scale: float = 1.0,
               inverse: bool = False, workspace=None, stream=None):
    """lla_rope_apply: rotate 2 * rope_cos.shape[1] elements of every head's vector of ``x``
    [N][heads][d_x], from element ``offset`` on; ``out`` may be ``x`` (in place) and is
    returned.  Token and head strides are free, a head's vector is contiguous."""
    dev = _device_of("x", x)
    _need(x.dim() == 3, "x must be [N][heads][d_x]")
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    sd, shape = _storage(dm), x.shape
    N, heads, d_x = shape
    xs, os = x.stride(), out.stride()
    if not (x.dtype is sd and out.dtype is sd and out.get_device() == dev and out.shape == shape and
            (d_x <= 1 or xs[2] == 1 and os[2] == 1)):
        raise ValueError("x and out must be %s of one shape on one device, each head's vector contiguous" % (sd,))
    table = rope_cos.shape
    _need(len(table) == 2, "rope_cos must be [rope_len][d_rope / 2]")
    ws, wb = _space(workspace, dev)
    _run("lla_rope_apply", lib().lla_rope_apply, dev, stream, ctypes.byref(dm), x.data_ptr(), xs[0], xs[1], out.data_ptr(),
         os[0], os[1], N, heads, d_x, offset, 2 * table[1], _arg("pos", pos, torch.int32, dev, (N,)),
         _arg("rope_cos", rope_cos, torch.float32, dev, table), _arg("rope_sin", rope_sin, torch.float32, dev, table),
         table[0], scale, 1 if inverse else 0, ws, wb)
    return out


class PagePlan:
    """Output arrays and status word of lla_page_plan for B requests and at most ``n_tok``
    new tokens; calling it plans one step into them (``block_table`` is updated in place).

    ``seq_lens`` [B], ``tok_start`` [B + 1], ``granted`` [B], ``seq_idx``, ``pos``, ``slots``
    (int64) [n_tok], ``counts`` [2] (the next call's ``free_head``; tokens granted).
    """

    def __init__(self, B: int, n_tok: int, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.B, self.n_tok = int(B), int(n_tok)
        self.seq_lens, self.granted = torch.empty(self.B, **i32), torch.empty(self.B, **i32)
        self.tok_start, self.counts = torch.empty(self.B + 1, **i32), torch.empty(2, **i32)
        self.seq_idx, self.pos = torch.empty(self.n_tok, **i32), torch.empty(self.n_tok, **i32)
        self.slots = torch.empty(self.n_tok, dtype=torch.int64, device=device)
        self.workspace = torch.zeros(256, dtype=torch.uint8, device=device)

    def __call__(self, page_size: int, num_pages: int, ctx_lens, new_lens, free_pages, block_table, free_head=None,
                 stream=None):
        dev, B, i32 = self.counts.get_device(), self.B, torch.int32
        table = block_table.shape
        _need(len(table) == 2 and table[0] == B, "block_table must be [%d][max_pages]" % B)
        free = free_pages.shape
        _need(len(free) == 1, "free_pages must be one-dimensional")
        _run("lla_page_plan", lib().lla_page_plan, dev, stream, B, page_size, table[1], num_pages,
             _arg("ctx_lens", ctx_lens, i32, dev, (B,)), _arg("new_lens", new_lens, i32, dev, (B,)),
             _arg("free_pages", free_pages, i32, dev, free), free[0],
             None if free_head is None else _arg("free_head", free_head, i32, dev, (1,)),
             _arg("block_table", block_table, i32, dev, table), self.seq_lens.data_ptr(), self.tok_start.data_ptr(),
             self.granted.data_ptr(), self.n_tok, self.seq_idx.data_ptr(), self.pos.data_ptr(), self.slots.data_ptr(),
             self.counts.data_ptr(), self.workspace.data_ptr(), 256)
        return self


def q4_row_bytes(dm: Dims) -> int:
    """Bytes of one token-head's row of the 4-bit cache."""
    n = lib().lla_q4_row_bytes(ctypes.byref(dm))
    if n == 0:
        raise LLAError(LLA_ERR_UNSUPPORTED, "lla_q4_row_bytes")
    return int(n)


def q4_pool(dm: Dims, num_pages: int, page_size: int, device="cuda") -> torch.Tensor:
    """A zeroed 4-bit pool [num_pages][H][page_size][row bytes] (uint8)."""
    return torch.zeros((int(num_pages), dm.H, int(page_size), q4_row_bytes(dm)), dtype=torch.uint8, device=device)


def q4_workspace(dm: Dims, B: int, L_max: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for lla_decode_attn_q4 (L_max = max_pages * page_size)."""
    with torch.cuda.device(device):
        n = lib().lla_q4_workspace_size(ctypes.byref(dm), int(B), int(L_max))
    if n == 0:
        raise LLAError(LLA_ERR_INVALID_ARG, "lla_q4_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _q4_cache(L, dm: Dims, pool, dev: int, block_table=None) -> Q4Cache:
    shape = pool.shape
    _need(len(shape) == 4 and shape[1] == dm.H and shape[3] == L.lla_q4_row_bytes(ctypes.byref(dm)),
          "the pool must be [num_pages][%d][page_size][row bytes], not %s" % (dm.H, tuple(shape)))
    rows = _arg("pool", pool, torch.uint8, dev, shape)
    if block_table is None:
        return Q4Cache(rows, None, 0, 1, shape[2], shape[0])
    table = block_table.shape
    _need(len(table) == 2, "block_table must be [B][max_pages]")
    return Q4Cache(rows, _arg("block_table", block_table, torch.int32, dev, table), table[0], table[1], shape[2], shape[0])


def _q4_latents(dm: Dims, c_k, c_v, slots, dev: int):
    """Addresses of c_k [N][H][r_k], c_v [N][H][r_v] and slots [N], and N."""
    N, sd = slots.shape[0], _storage(dm)
    return (_arg("c_k", c_k, sd, dev, (N, dm.H, dm.r_k)), _arg("c_v", c_v, sd, dev, (N, dm.H, dm.r_v)),
            _arg("slots", slots, torch.int64, dev, (N,)), N)


def q4_store(dm: Dims, c_k, c_v, slots, pool, workspace, stream=None):
    """lla_q4_store: latents c_k [N][H][r_k], c_v [N][H][r_v] rounded to 4 bits into the
    pool's rows at ``slots`` [N] (int64, as lla_page_plan makes them)."""
    dev, L = _device_of("pool", pool), lib()
    c = _q4_cache(L, dm, pool, dev)
    pk, pv, ps, N = _q4_latents(dm, c_k, c_v, slots, dev)
    ws, wb = _space(workspace, dev)
    _run("lla_q4_store", L.lla_q4_store, dev, stream, ctypes.byref(dm), pk, pv, N, ps, ctypes.byref(c), ws, wb)


def q4_load(dm: Dims, slots, pool, c_k, c_v, workspace, stream=None):
    """lla_q4_load: the latents that the pool's rows at ``slots`` stand for, into c_k, c_v."""
    dev, L = _device_of("pool", pool), lib()
    c = _q4_cache(L, dm, pool, dev)
    pk, pv, ps, N = _q4_latents(dm, c_k, c_v, slots, dev)
    ws, wb = _space(workspace, dev)
    _run("lla_q4_load", L.lla_q4_load, dev, stream, ctypes.byref(dm), ps, N, ctypes.byref(c), pk, pv, ws, wb)


def decode_attn_q4(dm: Dims, loop_t: int, q, pool, block_table, seq_lens, q_pos, w_up_k, w_up_v, mu_k, mu_v, rope_cos,
                   rope_sin, out, lse, workspace, stream=None):
    """lla_decode_attn_q4: latent-store decode attention over a 4-bit paged cache, into ``out``
    [B][H][d] (storage dtype) and, unless None, ``lse`` [B][H] (fp32)."""
    dev, L = _device_of("pool", pool), lib()
    c = _q4_cache(L, dm, pool, dev, block_table)
    sd, T, H, d, f32, i32 = _storage(dm), dm.T, dm.H, dm.d_head, torch.float32, torch.int32
    vec, one = (c.B, H, d), (c.B,)
    table = rope_cos.shape
    _need(len(table) == 2 and table[1] == d // 2, "rope_cos must be [rope_len][%d]" % (d // 2))
    ws, wb = _space(workspace, dev)
    _run("lla_decode_attn_q4", L.lla_decode_attn_q4, dev, stream, ctypes.byref(dm), loop_t, _arg("q", q, sd, dev, vec),
         ctypes.byref(c), _arg("seq_lens", seq_lens, i32, dev, one), _arg("q_pos", q_pos, i32, dev, one),
         _arg("w_up_k", w_up_k, sd, dev, (T, H, d, dm.r_k)), _arg("w_up_v", w_up_v, sd, dev, (T, H, d, dm.r_v)),
         _arg("mu_k", mu_k, f32, dev, (H, T * d)), _arg("mu_v", mu_v, f32, dev, (H, T * d)),
         _arg("rope_cos", rope_cos, f32, dev, table), _arg("rope_sin", rope_sin, f32, dev, table), table[0],
         _arg("out", out, sd, dev, vec), None if lse is None else _arg("lse", lse, f32, dev, (c.B, H)), ws, wb)


# ---------------------------------------------------------------- verifying drafted tokens

class DraftTree:
    """An lla_tree: the drafted tokens (nodes) of B sequences.

    ``tok_start`` [B + 1], ``parent`` [n_tok] and, for tree_attn, ``pos`` [n_tok] are int32
    tensors on one device, kept alive (and read at every call) here; ``max_nodes`` is the most
    nodes that a sequence has, at most LLA_TREE_MAX_NODES."""

    def __init__(self, tok_start, parent, max_nodes: int, pos=None):
        dev = self.dev = _device_of("tok_start", tok_start)
        _need(tok_start.dim() == 1 and tok_start.shape[0] >= 1, "tok_start must be [B + 1]")
        _need(isinstance(parent, torch.Tensor) and parent.dim() == 1, "parent must be [n_tok]")
        self.B, self.n_tok, self.max_nodes = tok_start.shape[0] - 1, parent.shape[0], int(max_nodes)
        _need(1 <= self.max_nodes <= LLA_TREE_MAX_NODES, "max_nodes must be in 1..%d" % LLA_TREE_MAX_NODES)
        self.tok_start, self.parent, self.pos = tok_start, parent, pos
        one = (self.n_tok,)
        self.c = Tree(self.B, self.n_tok, self.max_nodes, _arg("tok_start", tok_start, torch.int32, dev, (self.B + 1,)),
                      _arg("parent", parent, torch.int32, dev, one),
                      None if pos is None else _arg("pos", pos, torch.int32, dev, one))
        self.ref = ctypes.byref(self.c)


def tree_kernel(dm: Dims, page_size: int = 0) -> Optional[str]:
    """Kernel family of tree_attn (page_size 0) and tree_attn_paged for these dims ("tensor",
    "plain"), or None if they are invalid or unsupported."""
    r = lib().lla_tree_kernel(ctypes.byref(dm), int(page_size))
    return None if r is None else r.decode()


def tree_workspace(dm: Dims, tree: DraftTree, L_max: int) -> torch.Tensor:
    """A zeroed workspace for lla_tree_attn (L_max: the cache's, or max_pages * page_size)."""
    with torch.cuda.device(tree.dev):
        n = lib().lla_tree_workspace_size(ctypes.byref(dm), tree.B, tree.max_nodes, int(L_max))
    if n == 0:
        raise LLAError(LLA_ERR_UNSUPPORTED, "lla_tree_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=tree.tok_start.device)


def _node_vectors(name: str, t, dtype, dev: int, shape):
    """Address and token stride of q, k or v [n_tok][H][d], each token's [H][d] contiguous."""
    n, H, d = shape
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape:
            s0, s1, s2 = t.stride()
            if s2 == 1 and (s1 == d or H == 1):
                # (torch leaves the stride of a single token open)
                return t.data_ptr(), s0 if n > 1 else H * d
    except AttributeError:
        pass
    raise ValueError("%s must be %s of shape %s on cuda:%d, each token's vectors contiguous" % (name, dtype, shape, dev))


def _tree_attn(what, f, dm, loop_t, tree, q, k, v, cache, B, seq_lens, w_up_k, w_up_v, mu_k, mu_v, rope_cos, rope_sin,
               out, lse, workspace, stream):
    dev, sd, T, H, d, f32, n = tree.dev, _storage(dm), dm.T, dm.H, dm.d_head, torch.float32, tree.n_tok
    if tree.pos is None or B != tree.B:
        raise ValueError("the tree has no positions" if tree.pos is None else
                         "the cache is for %d sequences, the tree for %d" % (B, tree.B))
    vec, table, mu = (n, H, d), rope_cos.shape, (H, T * d)
    if len(table) != 2 or table[1] != d // 2:
        raise ValueError("rope_cos must be [rope_len][%d]" % (d // 2))
    qp, qs = _node_vectors("q", q, sd, dev, vec)
    kp, ks = _node_vectors("k", k, sd, dev, vec)
    vp, vs = _node_vectors("v", v, sd, dev, vec)
    ws, wb = _space(workspace, dev)
    _run(what, f, dev, stream, ctypes.byref(dm), loop_t, tree.ref, qp, qs, kp, ks, vp, vs, cache,
         _arg("seq_lens", seq_lens, torch.int32, dev, (B,)), _arg("w_up_k", w_up_k, sd, dev, (T, H, d, dm.r_k)),
         _arg("w_up_v", w_up_v, sd, dev, (T, H, d, dm.r_v)), _arg("mu_k", mu_k, f32, dev, mu),
         _arg("mu_v", mu_v, f32, dev, mu), _arg("rope_cos", rope_cos, f32, dev, table),
         _arg("rope_sin", rope_sin, f32, dev, table), table[0], _arg("out", out, sd, dev, vec),
         None if lse is None else _arg("lse", lse, f32, dev, (n, H)), ws, wb)


def tree_attn(dm: Dims, loop_t: int, tree: DraftTree, q, k, v, cache_k, cache_v, seq_lens, w_up_k, w_up_v, mu_k, mu_v,
              rope_cos, rope_sin, out, lse, workspace, stream=None):
    """lla_tree_attn: every node of ``tree`` attends to its sequence's cached latents and to the nodes
    on its path.  q, k, v [n_tok][H][d] (token stride free) of loop ``loop_t``, before RoPE; ``out``
    [n_tok][H][d] (storage dtype), ``lse`` [n_tok][H] (fp32) or None."""
    sd, dev, shape = _storage(dm), tree.dev, cache_k.shape
    if len(shape) != 4:
        raise ValueError("cache_k must be [B][H][L_max][r_k]")
    B, L_max, H = shape[0], shape[2], dm.H
    cache = Cache(_arg("cache_k", cache_k, sd, dev, (B, H, L_max, dm.r_k)),
                  _arg("cache_v", cache_v, sd, dev, (B, H, L_max, dm.r_v)), B, L_max)
    _tree_attn("lla_tree_attn", lib().lla_tree_attn, dm, loop_t, tree, q, k, v, cache, B, seq_lens, w_up_k, w_up_v, mu_k,
               mu_v, rope_cos, rope_sin, out, lse, workspace, stream)


def tree_attn_paged(dm: Dims, loop_t: int, tree: DraftTree, q, k, v, pool_k, pool_v, block_table, page_size: int,
                    seq_lens, w_up_k, w_up_v, mu_k, mu_v, rope_cos, rope_sin, out, lse, workspace, stream=None):
    """lla_tree_attn_paged: tree_attn over pools [num_pages][H][page_size][r] and a block table
    [B][max_pages]."""
    sd, dev, H, table = _storage(dm), tree.dev, dm.H, block_table.shape
    if len(pool_k.shape) != 4 or len(table) != 2:
        raise ValueError("pools must be [num_pages][H][page_size][r], block_table [B][max_pages]")
    num = pool_k.shape[0]
    cache = PagedCache(_arg("pool_k", pool_k, sd, dev, (num, H, page_size, dm.r_k)),
                       _arg("pool_v", pool_v, sd, dev, (num, H, page_size, dm.r_v)),
                       _arg("block_table", block_table, torch.int32, dev, table), table[0], table[1], page_size, num)
    _tree_attn("lla_tree_attn_paged", lib().lla_tree_attn_paged, dm, loop_t, tree, q, k, v, cache, table[0], seq_lens,
               w_up_k, w_up_v, mu_k, mu_v, rope_cos, rope_sin, out, lse, workspace, stream)


class LogitRules:
    """An lla_logit_rules: what the requests of a step impose on their logits.  Tensors are kept
    alive (and read at every call) here.

    ``history`` [B][max_history], ``hist_len``, ``prompt_len`` [B] (int32; prompt_len None: no
    prompt part), ``repetition``, ``presence``, ``frequency`` [B] (fp32 or None), ``bias_token``
    (int32, negative: unused) and ``bias`` (fp32) [B][max_bias], ``allowed`` [n_masks][ceil(vocab / 32)]
    (int32 words of bits) with ``allowed_row`` [n_tok] (int32, negative: no mask)."""

    def __init__(self, history=None, hist_len=None, prompt_len=None, repetition=None, presence=None, frequency=None,
                 bias_token=None, bias=None, allowed=None, allowed_row=None):
        given = (history, hist_len, prompt_len, repetition, presence, frequency, bias_token, bias, allowed, allowed_row)
        self.keep = given
        self.dev = next((_device_of("a rule", t) for t in given if t is not None), None)
        _need((history is None) == (hist_len is None), "give history and hist_len or neither")
        _need(history is not None or prompt_len is None, "prompt_len needs a history")
        _need((bias_token is None) == (bias is None), "give bias_token and bias or neither")
        _need((allowed is None) == (allowed_row is None), "give allowed and allowed_row or neither")
        for name, t in (("history", history), ("bias_token", bias_token), ("allowed", allowed)):
            _need(t is None or t.dim() == 2, name + " must have two dimensions")
        i32, f32 = torch.int32, torch.float32
        per = next((t.shape[0] for t in (history, repetition, presence, frequency, bias_token) if t is not None), None)
        self.B = per
        self.n_tok = None if allowed_row is None else allowed_row.shape[0]
        self.words = None if allowed is None else allowed.shape[1]

        def p(name, t, dtype, shape):
            return None if t is None else _arg(name, t, dtype, self.dev, shape)

        cols = lambda t: 0 if t is None else t.shape[1]  # noqa: E731
        self.c = LogitRulesC(p("history", history, i32, (per, cols(history))), p("hist_len", hist_len, i32, (per,)),
                             p("prompt_len", prompt_len, i32, (per,)), cols(history), p("repetition", repetition, f32, (per,)),
                             p("presence", presence, f32, (per,)), p("frequency", frequency, f32, (per,)),
                             p("bias_token", bias_token, i32, (per, cols(bias_token))),
                             p("bias", bias, f32, (per, cols(bias_token))), cols(bias_token),
                             None if allowed is None else p("allowed", allowed, i32, tuple(allowed.shape)),
                             p("allowed_row", allowed_row, i32, (self.n_tok,)), 0 if allowed is None else allowed.shape[0])
        self.ref = ctypes.byref(self.c)


def logits_workspace(tree: DraftTree, vocab: int) -> torch.Tensor:
    """A zeroed workspace for lla_logits_adjust."""
    n = lib().lla_logits_workspace_size(tree.n_tok, int(vocab))
    if n == 0:
        raise LLAError(LLA_ERR_UNSUPPORTED, "lla_logits_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=tree.tok_start.device)


_LOGIT_TYPES = {torch.bfloat16: LLA_BF16, torch.float32: LLA_F32}


def logits_adjust(tree: DraftTree, token, logits, rules: LogitRules, out=None, best=None, lse=None, workspace=None,
                  stream=None):
    """lla_logits_adjust: ``rules`` on the rows of ``logits`` [n_tok][vocab] (bf16 or fp32, row
    stride free), into ``out`` (may be ``logits``), each row's best token into ``best`` [n_tok] (int32)
    and its log-sum-exp into ``lse`` [n_tok] (fp32); at least one of the three.  ``token`` [n_tok]
    (int32) are the nodes' tokens."""
    dev, n = tree.dev, tree.n_tok
    shape, dtype = logits.shape, logits.dtype
    if len(shape) != 2 or shape[0] != n or logits.get_device() != dev or dtype not in _LOGIT_TYPES:
        raise ValueError("logits must be bfloat16 or float32 [%d][vocab] on cuda:%d" % (n, dev))
    V = shape[1]
    xs, os = logits.stride(), (V, 1) if out is None else out.stride()
    if not (out is None or out.dtype is dtype and out.get_device() == dev and out.shape == shape):
        raise ValueError("out must be like logits")
    if V > 1 and (xs[1] != 1 or os[1] != 1):
        raise ValueError("each row of logits and out must be contiguous")
    if rules.dev not in (None, dev) or rules.B not in (None, tree.B) or rules.n_tok not in (None, n) or \
            rules.words not in (None, (V + 31) // 32):
        raise ValueError("the rules are for %s sequences, %s tokens and masks of %s words on cuda:%s; the call has %d, %d, %d "
                         "and cuda:%d" % (rules.B, rules.n_tok, rules.words, rules.dev, tree.B, n, (V + 31) // 32, dev))
    # (torch leaves the stride of a single row open)
    ws, wb = _space(workspace, dev)
    _run("lla_logits_adjust", lib().lla_logits_adjust, dev, stream, tree.ref, _arg("token", token, torch.int32, dev, (n,)),
         _LOGIT_TYPES[dtype], logits.data_ptr(), xs[0] if n > 1 else V, V, rules.ref,
         None if out is None else out.data_ptr(), os[0] if n > 1 else V,
         None if best is None else _arg("best", best, torch.int32, dev, (n,)),
         None if lse is None else _arg("lse", lse, torch.float32, dev, (n,)), ws, wb)


class TreeAccept:
    """Output arrays and status word of lla_tree_accept for ``tree``; calling it walks down the tree.

    ``count``, ``next_token``, ``seq_lens`` [B], ``path``, ``seq_idx``, ``pos`` [n_tok] (int32; the
    last two as lla_encode takes them, which skips entries of -1).

    Entries of no sequence (behind tok_start[B], or of a sequence that does not fit) are -1 at first, and a call leaves
    them as they are: after one with more nodes they name its slots.  With ``clear`` every call sets them to -1 before it
    walks, as a step needs that hands all n_tok entries on and whose number of nodes varies (a captured one)."""

    def __init__(self, tree: DraftTree, clear: bool = False):
        i32 = dict(dtype=torch.int32, device=tree.tok_start.device)
        self.tree, self.clear = tree, bool(clear)
        self.count, self.next_token, self.seq_lens = (torch.empty(tree.B, **i32) for _ in range(3))
        self._entries = torch.full((3, (tree.n_tok + 63) // 64 * 64), -1, **i32)        # (rows on 256 bytes)
        self.path, self.seq_idx, self.pos = self._entries[:, :tree.n_tok].unbind()
        self.workspace = torch.zeros(256, dtype=torch.uint8, device=tree.tok_start.device)

    def __call__(self, token, chosen, ctx_lens, stream=None):
        t, i32 = self.tree, torch.int32
        one = (t.n_tok,)
        if self.clear:
            if stream is None:
                self._entries.fill_(-1)
            else:
                with torch.cuda.stream(stream):
                    self._entries.fill_(-1)
        _run("lla_tree_accept", lib().lla_tree_accept, t.dev, stream, t.ref, _arg("token", token, i32, t.dev, one),
             _arg("chosen", chosen, i32, t.dev, one), _arg("ctx_lens", ctx_lens, i32, t.dev, (t.B,)),
             self.count.data_ptr(), self.next_token.data_ptr(), self.seq_lens.data_ptr(), self.path.data_ptr(),
             self.seq_idx.data_ptr(), self.pos.data_ptr(), self.workspace.data_ptr(), 256)
        return self
