"""The view-cache operators: torch tensors in, C-ABI calls out.

As in ``api.py`` every function checks placement, type and layout of its tensors,
turns them into pointers and strides and calls the entry point of the same name in
``include/gsa.h``.  Tensors of one call live on one device, which need not be the
current one; ``stream`` defaults to that device's current stream.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from functools import cached_property

import torch

from ._lib import GsaCache, GsaViewBatch, check, load
from .api import BF16, F32, I32, WS_HEADER_BYTES, check_device_error


_LEAST, _MOST = -2 ** 31, 2 ** 31 - 1  # ctypes would cut off what is larger


@dataclass(frozen=True)
class ViewBatch:
    """Sizes of a batch of views that share a cache (``gsa_view_batch``).

    The work is laid out for n_views views of max_q queries and max_own own tokens: the defaults fit any batch, and
    take longer where there are many views.
    """

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
        for name, x in vars(self).items():
            if isinstance(x, int) and not _LEAST <= x <= _MOST:
                raise ValueError(f"{name} = {x} does not fit 32 bits")
        return GsaViewBatch(self.n_views, self.n_heads, self.n_kv_heads or self.n_heads, self.head_dim, self.n_q,
                            self.n_own, self.n_prefix, self.n_q if self.max_q < 0 else self.max_q,
                            self.n_own if self.max_own < 0 else self.max_own, int(self.causal), float(self.scale),
                            self.wait_limit_ns, 0, 0, 0, 0, 0, 0)

    @cached_property
    def _bytes(self) -> bytes:
        return bytes(self.c())

    def copy_c(self) -> GsaViewBatch:
        """A structure of its own for one call, which fills in the strides."""
        return GsaViewBatch.from_buffer_copy(self._bytes)


def view_workspace_size(batch: ViewBatch) -> int:
    n = ctypes.c_size_t()
    check(load().view_workspace_size(ctypes.byref(batch.c()), ctypes.byref(n)), "view_workspace_size")
    return n.value


def _new_workspace(n: int, device, stream) -> torch.Tensor:
    if stream is not None:
        # memory of that stream: what the current one has freed may still be in use by its kernels
        with torch.cuda.stream(stream):
            return _new_workspace(n, device, None)
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    with torch.cuda.device(ws.device):
        check(load().gsa_workspace_init(ws.data_ptr(), torch.cuda.current_stream().cuda_stream), "gsa_workspace_init")
    return ws


def new_view_workspace(batch: ViewBatch, device=None, stream=None) -> torch.Tensor:
    """Zero-headed workspace for prefix_attn and key_weights.  Calls that share it must be ordered."""
    return _new_workspace(view_workspace_size(batch), device, stream)


def _workspace(ws) -> tuple[int, int, int]:
    """Device index, pointer and bytes of a workspace."""
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    n = ws.numel() * ws.element_size()
    if n < WS_HEADER_BYTES:
        raise ValueError(f"workspace holds {n} bytes, needs {WS_HEADER_BYTES}")
    return ws.get_device(), ws.data_ptr(), n


def _refuse(t, dtype, dev, name, want):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the workspace on cuda:{dev}")
    raise ValueError(f"{name} must be {want}, got shape {tuple(t.shape)} strides {t.stride()}")


def _rows(t, n, heads, dev, name, exact=True):
    """Pointer and token stride of bf16 [n][heads][64] whose heads lie side by side; (None, 0) when n is 0.

    With ``exact`` false the tensor may hold more than n tokens.  Tokens that share memory (an expanded tensor's,
    whose stride is 0) are refused: the C ABI's stride 0 is a dense layout."""
    if n == 0:
        return None, 0
    if isinstance(t, torch.Tensor) and t.dtype is BF16 and t.get_device() == dev:
        if t.shape == (n, heads, 64) and t.is_contiguous():
            return t.data_ptr(), 0
        if t.dim() == 3:
            tokens, h, dim = t.shape
            s0, s1, s2 = t.stride()
            if ((tokens == n or (not exact and tokens > n)) and h == heads and dim == 64 and s2 == 1 and (s1 == 64 or h == 1)
                    and (s0 >= 64 * h or tokens == 1)):
                return t.data_ptr(), s0 if tokens > 1 else 0
    _refuse(t, BF16, dev, name, f"[{'' if exact else '>= '}{n}, {heads}, 64] with its heads side by side")


def _flat(t, dtype, shape, dev, name, optional=False):
    """Pointer of a contiguous tensor."""
    if t is None and optional:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, dev, name, f"contiguous {shape}")


def _table(t, dtype, heads, least, dev, name, optional=False):
    """Pointer and row stride of [heads][>= least] with dense rows."""
    if t is None and optional:
        return None, 0
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == 2:
        h, n = t.shape
        s0, s1 = t.stride()
        if h == heads and n >= least and (s1 == 1 or n <= 1):
            return t.data_ptr(), s0 if h > 1 else n
    _refuse(t, dtype, dev, name, f"[{heads}, >= {least}] with dense rows")


def _run(fn, where, dev, stream, *args) -> None:
    if torch.cuda.current_device() == dev:
        st = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
        status = fn(*args, st)
    else:
        with torch.cuda.device(dev):
            st = torch.cuda.current_stream() if stream is None else stream
            status = fn(*args, st.cuda_stream)
    if status:
        check(status, where)


def prefix_attn(batch: ViewBatch, q, k_prefix, v_prefix, k_own, v_own, q_off, own_off, out, lse, ws,
                stream=None) -> None:
    """Attention of a batch of views to one shared prefix and to their own tokens (gsa.h).

    q, out [n_q, H, 64], keys and values [n, Hk, 64] bf16, any token stride that is a multiple of 8;
    q_off, own_off [n_views + 1] int32; lse [n_q, H] float32 or None.  Tensors of no tokens may be None.
    """
    dev, pws, ws_bytes = _workspace(ws)
    b = batch.copy_c()
    n_q, n_prefix, n_own, H, Hk = b.n_q, b.n_prefix, b.n_own, b.n_heads, b.n_kv_heads
    pq, b.q_stride = _rows(q, n_q, H, dev, "q")
    pkp, b.k_prefix_stride = _rows(k_prefix, n_prefix, Hk, dev, "k_prefix")
    pvp, b.v_prefix_stride = _rows(v_prefix, n_prefix, Hk, dev, "v_prefix")
    pko, b.k_own_stride = _rows(k_own, n_own, Hk, dev, "k_own")
    pvo, b.v_own_stride = _rows(v_own, n_own, Hk, dev, "v_own")
    pout, b.out_stride = _rows(out, n_q, H, dev, "out")
    offs = (b.n_views + 1,)
    _run(load().prefix_attn, "prefix_attn", dev, stream, ctypes.byref(b), pq, pkp, pvp, pko, pvo,
         _flat(q_off, I32, offs, dev, "q_off"), _flat(own_off, I32, offs, dev, "own_off"), pout,
         _flat(lse, F32, (n_q, H), dev, "lse", True), pws, ws_bytes)


def key_weights(batch: ViewBatch, q, k_prefix, k_own, q_off, own_off, lse, acc, acc_out, decay: float, ws,
                stream=None) -> None:
    """Adds the attention every key received (the column sums of prefix_attn's weights, given its lse) to an account.

    acc_out [Hk, >= n_prefix + n_own] float32 gets decay * acc + the sums for the cached tokens and the sums for the
    own tokens behind them; acc [Hk, >= n_prefix] may be None (zeros) or acc_out itself.
    """
    dev, pws, ws_bytes = _workspace(ws)
    b = batch.copy_c()
    n_q, n_prefix, n_own, H, Hk = b.n_q, b.n_prefix, b.n_own, b.n_heads, b.n_kv_heads
    pq, b.q_stride = _rows(q, n_q, H, dev, "q")
    pkp, b.k_prefix_stride = _rows(k_prefix, n_prefix, Hk, dev, "k_prefix")
    pko, b.k_own_stride = _rows(k_own, n_own, Hk, dev, "k_own")
    offs = (b.n_views + 1,)
    pout, out_stride = _table(acc_out, F32, Hk, n_prefix + n_own, dev, "acc_out")
    pacc, acc_stride = _table(acc, F32, Hk, n_prefix, dev, "acc", True)
    _run(load().key_weights, "key_weights", dev, stream, ctypes.byref(b), pq, pkp, pko,
         _flat(q_off, I32, offs, dev, "q_off"), _flat(own_off, I32, offs, dev, "own_off"),
         _flat(lse, F32, (n_q, H), dev, "lse"), pacc, acc_stride, pout, out_stride, decay, pws, ws_bytes)


def _cache(n_kv_heads: int, n_tokens: int, n_keep: int, recent_from: int, k_stride: int, v_stride: int,
           w_stride: int) -> GsaCache:
    if not (_LEAST <= n_kv_heads <= _MOST and _LEAST <= n_tokens <= _MOST and _LEAST <= n_keep <= _MOST
            and _LEAST <= recent_from <= _MOST):
        raise ValueError(f"n_kv_heads, n_tokens, n_keep or recent_from of {(n_kv_heads, n_tokens, n_keep, recent_from)} "
                         "does not fit 32 bits")
    return GsaCache(n_kv_heads, 64, n_tokens, n_keep, recent_from, k_stride, v_stride, w_stride)


def cache_workspace_size(n_kv_heads: int, n_tokens: int, n_keep: int) -> int:
    n = ctypes.c_size_t()
    b = _cache(n_kv_heads, n_tokens, n_keep, 0, 0, 0, n_tokens)
    check(load().cache_workspace_size(ctypes.byref(b), ctypes.byref(n)), "cache_workspace_size")
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
    dev, pws, ws_bytes = _workspace(ws)
    Hk = k.shape[1] if isinstance(k, torch.Tensor) and k.dim() == 3 else 0
    pk, k_stride = _rows(k, n_tokens, Hk, dev, "k", False)
    pv, v_stride = _rows(v, n_tokens, Hk, dev, "v", False)
    pa, stride = _table(acc, F32, Hk, n_tokens, dev, "acc")
    pi, s1 = _table(ids, I32, Hk, n_tokens, dev, "ids")
    pao, s2 = _table(acc_out, F32, Hk, n_tokens, dev, "acc_out")
    pio, s3 = _table(ids_out, I32, Hk, n_tokens, dev, "ids_out")
    if Hk > 1 and not stride == s1 == s2 == s3:
        raise ValueError(f"acc, ids, acc_out and ids_out must have one row stride, got {(stride, s1, s2, s3)}")
    b = _cache(Hk, n_tokens, n_keep, recent_from, k_stride, v_stride, stride)
    _run(load().cache_evict, "cache_evict", dev, stream, ctypes.byref(b), pk, pv, pa, pi, pao, pio, pws, ws_bytes)


class ViewCache:
    """Keys and values of the views seen so far, with their account: the operators in the order of a stream of views.

    ``step`` attends a batch of views to the cache and to their own tokens, adds up who was looked at and appends the
    tokens; ``evict`` shrinks the cache.  Everything runs on the current stream of ``device``.  Tokens are numbered in
    the order of their coming, up to 2^31 - 1 of them; a ``step`` that is refused leaves the cache as it was.
    """

    def __init__(self, capacity: int, n_heads: int, n_kv_heads: int = 0, device="cuda", scale: float = 0.0):
        self.capacity, self.n_heads, self.n_kv_heads, self.scale = capacity, n_heads, n_kv_heads or n_heads, scale
        self.k = torch.empty(capacity, self.n_kv_heads, 64, dtype=BF16, device=device)
        self.v = torch.empty_like(self.k)
        # accounts and token numbers, and where the next call leaves them
        self.acc = torch.zeros(self.n_kv_heads, capacity, dtype=F32, device=device)
        self.ids = torch.zeros(self.n_kv_heads, capacity, dtype=I32, device=device)
        self._acc, self._ids = torch.zeros_like(self.acc), torch.zeros_like(self.ids)
        self.n = 0        # tokens in the cache
        self.next_id = 0  # tokens ever appended
        self._ws = None

    def _workspace(self, n_bytes: int) -> torch.Tensor:
        old = self._ws
        if old is None or old.numel() < n_bytes:
            self._ws = _new_workspace(n_bytes, self.k.device, None)
            if old is not None:
                # errors that nobody has asked for yet
                self._ws[:WS_HEADER_BYTES].copy_(old[:WS_HEADER_BYTES])
                # earlier steps may have used it on another stream than the one it came from
                old.record_stream(torch.cuda.current_stream(old.device))
        return self._ws

    @torch.no_grad()  # copies of tensors that require gradients would tie every step's graph to the cache
    def step(self, q, k, v, lens=None, decay: float = 1.0) -> torch.Tensor:
        """Attention of the views (``lens`` tokens each; all of them one view by default) to the cache and to their
        own tokens, q [n, H, 64], k and v [n, Hk, 64]; then the tokens join the cache."""
        n = q.shape[0]
        lens = [n] if lens is None else list(lens)
        if not lens or min(lens) < 0 or sum(lens) != n:
            raise ValueError(f"views of {lens} tokens, q has {n}")
        if self.n + n > self.capacity:
            raise ValueError(f"{self.n} + {n} tokens do not fit a cache of {self.capacity}")
        if self.next_id + n > _MOST:
            raise ValueError(f"{self.next_id} tokens were appended: {n} more have no number of 32 bits")
        at = [0]
        for x in lens:
            at.append(at[-1] + x)
        off = torch.tensor(at, dtype=I32, device=self.k.device)
        batch = ViewBatch(n_views=len(lens), n_q=n, n_own=n, n_prefix=self.n, n_heads=self.n_heads,
                          n_kv_heads=self.n_kv_heads, max_q=max(lens), max_own=max(lens), scale=self.scale)
        ws = self._workspace(view_workspace_size(batch))
        out = torch.empty(n, self.n_heads, 64, dtype=BF16, device=self.k.device)
        lse = torch.empty(n, self.n_heads, dtype=F32, device=self.k.device)
        kp, vp = self.k[:self.n], self.v[:self.n]
        prefix_attn(batch, q, kp, vp, k, v, off, off, out, lse, ws)
        key_weights(batch, q, kp, k, off, off, lse, self.acc, self.acc, decay, ws)
        self.k[self.n:self.n + n].copy_(k)
        self.v[self.n:self.n + n].copy_(v)
        self.ids[:, self.n:self.n + n] = torch.arange(self.next_id, self.next_id + n, dtype=I32, device=self.k.device)
        self.n += n
        self.next_id += n
        return out

    def evict(self, n_keep: int, recent: int = 0) -> None:
        """Keeps ``n_keep`` tokens a head: the ``recent`` newest, then those with the largest account."""
        if n_keep >= self.n:
            return
        ws = self._workspace(cache_workspace_size(self.n_kv_heads, self.n, n_keep))
        cache_evict(self.n, n_keep, max(self.next_id - recent, 0), self.k, self.v, self.acc, self.ids, self._acc, self._ids, ws)
        self.acc, self._acc = self._acc, self.acc
        self.ids, self._ids = self._ids, self.ids
        self.n = n_keep

    def check_device_error(self) -> None:
        """Raises if a kernel of an earlier call reported an error (synchronises)."""
        if self._ws is not None:
            with torch.cuda.device(self.k.device):
                check_device_error(self._ws)
