"""The view-cache operators: torch tensors in, C-ABI calls out.

As in ``api.py`` every function checks placement, type and layout of its tensors,
turns them into pointers and strides and calls the entry point of the same name in
``include/gsa.h``.  Tensors of one call live on one device, which need not be the
current one; ``stream`` defaults to that device's current stream.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from ._lib import GsaCache, GsaViewBatch, check, load
from .api import BF16, F32, I32, WS_HEADER_BYTES


@dataclass(frozen=True)
class ViewBatch:
    """Sizes of a batch of views that share a cache (``gsa_view_batch``)."""

    n_views: int
    n_q: int
    n_own: int
    n_prefix: int
    n_heads: int
    n_kv_heads: int = 0  # 0: as many as query heads
    max_q: int = -1      # most queries of a view; -1: n_q
    max_own: int = -1    # most own tokens of a view; -1: n_own
    causal: bool = False
    head_dim: int = 64
    scale: float = 0.0
    wait_limit_ns: int = 0

    def c(self) -> GsaViewBatch:
        return GsaViewBatch(self.n_views, self.n_heads, self.n_kv_heads or self.n_heads, self.head_dim, self.n_q,
                            self.n_own, self.n_prefix, self.n_q if self.max_q < 0 else self.max_q,
                            self.n_own if self.max_own < 0 else self.max_own, int(self.causal), float(self.scale),
                            self.wait_limit_ns, 0, 0, 0, 0, 0, 0)


def view_workspace_size(batch: ViewBatch) -> int:
    n = ctypes.c_size_t()
    check(load().view_workspace_size(ctypes.byref(batch.c()), ctypes.byref(n)), "view_workspace_size")
    return n.value


def _new_workspace(n: int, device, stream) -> torch.Tensor:
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    with torch.cuda.device(ws.device):
        st = torch.cuda.current_stream() if stream is None else stream
        check(load().gsa_workspace_init(ws.data_ptr(), st.cuda_stream), "gsa_workspace_init")
    return ws


def new_view_workspace(batch: ViewBatch, device=None, stream=None) -> torch.Tensor:
    """Zero-headed workspace for prefix_attn and key_weights.  Calls that share it must be ordered."""
    return _new_workspace(view_workspace_size(batch), device, stream)


class _Call:
    """Checks the tensors of one call: all on one device, the right types and layouts."""

    def __init__(self, ws: torch.Tensor):
        if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        self.ws = ws
        self.device = ws.device
        self.ws_bytes = ws.numel() * ws.element_size()
        if self.ws_bytes < WS_HEADER_BYTES:
            raise ValueError(f"workspace holds {self.ws_bytes} bytes, needs {WS_HEADER_BYTES}")

    def _tensor(self, t, dtype, name):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the workspace on {self.device}")

    def rows(self, t, n, heads, dim, name):
        """Pointer and token stride of [n][heads][dim] bf16 with dense heads; None when n is 0."""
        if n == 0:
            return None, 0
        self._tensor(t, BF16, name)
        if t.shape != (n, heads, dim):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(n, heads, dim)}")
        s = t.stride()
        if s[2] != 1 or (heads > 1 and s[1] != dim):
            raise ValueError(f"{name} must have its heads side by side, got strides {s}")
        return t.data_ptr(), s[0] if n > 1 else 0

    def flat(self, t, dtype, shape, name, optional=False):
        """Pointer of a contiguous tensor."""
        if t is None and optional:
            return None
        self._tensor(t, dtype, name)
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)} strides {t.stride()}")
        return t.data_ptr()

    def table(self, t, dtype, heads, least, name, optional=False):
        """Pointer and row stride of [heads][>= least] with dense rows."""
        if t is None and optional:
            return None, 0
        self._tensor(t, dtype, name)
        if t.dim() != 2 or t.shape[0] != heads or t.shape[1] < least or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{name} must be [{heads}, >= {least}] with dense rows, got {tuple(t.shape)} strides {t.stride()}")
        return t.data_ptr(), t.stride(0) if heads > 1 else t.shape[1]

    def run(self, fn, where, stream, *args):
        if torch.cuda.current_device() == self.device.index:
            st = torch.cuda.current_stream() if stream is None else stream
            check(fn(*args, st.cuda_stream), where)
        else:
            with torch.cuda.device(self.device):
                st = torch.cuda.current_stream() if stream is None else stream
                check(fn(*args, st.cuda_stream), where)


def prefix_attn(batch: ViewBatch, q, k_prefix, v_prefix, k_own, v_own, q_off, own_off, out, lse, ws,
                stream=None) -> None:
    """Attention of a batch of views to one shared prefix and to their own tokens (gsa.h).

    q, out [n_q, H, 64], keys and values [n, Hk, 64] bf16, any token stride that is a multiple of 8;
    q_off, own_off [n_views + 1] int32; lse [n_q, H] float32 or None.  Tensors of no tokens may be None.
    """
    c, b = _Call(ws), batch.c()
    D, H, Hk = batch.head_dim, b.n_heads, b.n_kv_heads
    pq, b.q_stride = c.rows(q, b.n_q, H, D, "q")
    pkp, b.k_prefix_stride = c.rows(k_prefix, b.n_prefix, Hk, D, "k_prefix")
    pvp, b.v_prefix_stride = c.rows(v_prefix, b.n_prefix, Hk, D, "v_prefix")
    pko, b.k_own_stride = c.rows(k_own, b.n_own, Hk, D, "k_own")
    pvo, b.v_own_stride = c.rows(v_own, b.n_own, Hk, D, "v_own")
    pout, b.out_stride = c.rows(out, b.n_q, H, D, "out")
    offs = (b.n_views + 1,)
    c.run(load().prefix_attn, "prefix_attn", stream, ctypes.byref(b), pq, pkp, pvp, pko, pvo,
          c.flat(q_off, I32, offs, "q_off"), c.flat(own_off, I32, offs, "own_off"), pout,
          c.flat(lse, F32, (b.n_q, H), "lse", True), ws.data_ptr(), c.ws_bytes)


def key_weights(batch: ViewBatch, q, k_prefix, k_own, q_off, own_off, lse, acc, acc_out, decay: float, ws,
                stream=None) -> None:
    """Adds the attention every key received (the column sums of prefix_attn's weights, given its lse) to an account.

    acc_out [Hk, >= n_prefix + n_own] float32 gets decay * acc + the sums for the cached tokens and the sums for the
    own tokens behind them; acc [Hk, >= n_prefix] may be None (zeros) or acc_out itself.
    """
    c, b = _Call(ws), batch.c()
    D, H, Hk = batch.head_dim, b.n_heads, b.n_kv_heads
    pq, b.q_stride = c.rows(q, b.n_q, H, D, "q")
    pkp, b.k_prefix_stride = c.rows(k_prefix, b.n_prefix, Hk, D, "k_prefix")
    pko, b.k_own_stride = c.rows(k_own, b.n_own, Hk, D, "k_own")
    offs = (b.n_views + 1,)
    pout, out_stride = c.table(acc_out, F32, Hk, b.n_prefix + b.n_own, "acc_out")
    pacc, acc_stride = c.table(acc, F32, Hk, b.n_prefix, "acc", True)
    c.run(load().key_weights, "key_weights", stream, ctypes.byref(b), pq, pkp, pko, c.flat(q_off, I32, offs, "q_off"),
          c.flat(own_off, I32, offs, "own_off"), c.flat(lse, F32, (b.n_q, H), "lse"), pacc, acc_stride, pout, out_stride,
          decay, ws.data_ptr(), c.ws_bytes)


def _cache(n_kv_heads: int, n_tokens: int, n_keep: int, recent_from: int = 0) -> GsaCache:
    return GsaCache(n_kv_heads, 64, n_tokens, n_keep, recent_from, 0, 0, n_tokens)


def cache_workspace_size(n_kv_heads: int, n_tokens: int, n_keep: int) -> int:
    n = ctypes.c_size_t()
    check(load().cache_workspace_size(ctypes.byref(_cache(n_kv_heads, n_tokens, n_keep)), ctypes.byref(n)),
          "cache_workspace_size")
    return n.value


def new_cache_workspace(n_kv_heads: int, n_tokens: int, n_keep: int, device=None, stream=None) -> torch.Tensor:
    """Zero-headed workspace for cache_evict.  Calls that share it must be ordered."""
    return _new_workspace(cache_workspace_size(n_kv_heads, n_tokens, n_keep), device, stream)


def cache_evict(n_tokens: int, n_keep: int, recent_from: int, k, v, acc, ids, acc_out, ids_out, ws,
                stream=None) -> None:
    """Shrinks a cache to the n_keep tokens of each head with the largest account (gsa.h).

    k, v [>= n_tokens, Hk, 64] bf16 are changed in place; acc, acc_out float32 and ids, ids_out int32 are
    [Hk, >= n_tokens] with one row stride.  Afterwards the first n_keep slots of k, v, acc_out and ids_out are the cache.
    Tokens whose number is recent_from or more rank first.
    """
    c = _Call(ws)
    for t, name in ((k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3 or t.shape[0] < n_tokens:
            raise ValueError(f"{name} must be [>= {n_tokens}, heads, 64]")
    Hk = k.shape[1]
    b = _cache(Hk, n_tokens, n_keep, recent_from)
    pk, b.k_stride = c.rows(k[:n_tokens], n_tokens, Hk, 64, "k")
    pv, b.v_stride = c.rows(v[:n_tokens], n_tokens, Hk, 64, "v")
    tables = [c.table(t, dt, Hk, n_tokens, name) for t, dt, name in
              ((acc, F32, "acc"), (ids, I32, "ids"), (acc_out, F32, "acc_out"), (ids_out, I32, "ids_out"))]
    if len({s for _, s in tables}) != 1:
        raise ValueError(f"acc, ids, acc_out and ids_out must have one row stride, got {[s for _, s in tables]}")
    b.w_stride = tables[0][1]
    c.run(load().cache_evict, "cache_evict", stream, ctypes.byref(b), pk, pv, *[p for p, _ in tables], ws.data_ptr(),
          c.ws_bytes)
