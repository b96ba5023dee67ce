"""A paged key/value cache held in 4 bits, and attention over it (include/marlin.h).

    cache = Kv4Cache(n_pages, kv_heads, head_dim, page_size)       # once
    batch = Kv4Batch(page_table, lengths, q_start, tokens, max_q)  # once per step
    ws = Kv4Workspace(batch, heads, cache)                         # once, for the largest batch
    kv4_append(k, v, cache, batch, ws)                             # the new tokens' keys and values
    o = kv4_attention(q, cache, batch, ws)                         # fp16 [tokens, heads, head_dim]
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import _binding, _Handle, _on_current_device
from ._binding import MarlinError


class Kv4Cache(_Handle):
    """n_pages pages of page_size tokens of every key head, keys and values in
    4 bits (head_dim + 8 bytes per token and head)."""
    _fields = ("buf", "n_pages", "kv_heads", "head_dim", "page_size")

    def __init__(self, n_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device=None):
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError("a cache lives on a CUDA device")
        self.n_pages, self.kv_heads, self.head_dim, self.page_size = n_pages, kv_heads, head_dim, page_size
        self.buf = torch.zeros(_binding.kv_cache_bytes(n_pages, kv_heads, head_dim, page_size), dtype=torch.uint8,
                               device=dev)
        self._check()

    def _check(self):
        self.nbytes = _binding.kv_cache_bytes(self.n_pages, self.kv_heads, self.head_dim, self.page_size)
        _need_bytes(self.buf, "the cache's buf", self.nbytes)
        self._device = self.buf.get_device()
        self._scale = 1.0 / math.sqrt(self.head_dim)
        self._args = (self.buf.data_ptr(), self.n_pages, self.kv_heads, self.head_dim, self.page_size)
        return self._args


@dataclass
class Kv4Batch(_Handle):
    """One step's requests.  page_table int32 [B, pages], lengths int32 [B]
    (cached tokens, the new ones included), q_start int32 [B + 1] (the new
    tokens of request b are rows q_start[b] .. q_start[b+1] - 1, its last
    positions); tokens = q_start[B] rows in all, at most max_q of one request.
    The tensors are read by the kernels at each call: they may be updated in
    place between steps, or replaced (not resized in place)."""
    page_table: torch.Tensor
    lengths: torch.Tensor
    q_start: torch.Tensor
    tokens: int
    max_q: int = 1
    _fields = ("page_table", "lengths", "q_start", "tokens", "max_q")

    def __post_init__(self):
        self._check()

    def _check(self):
        for name in ("page_table", "lengths", "q_start"):
            t = getattr(self, name)
            if not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
        B = self.lengths.shape[0] if self.lengths.dim() == 1 else -1
        if (self.page_table.dim() != 2 or self.page_table.shape[0] != B or tuple(self.q_start.shape) != (B + 1,)
                or self.tokens < 0 or self.max_q < 0):
            raise ValueError("expected page_table [B, pages], lengths [B], q_start [B + 1], tokens >= 0, max_q >= 0")
        if not self.page_table.device == self.lengths.device == self.q_start.device:
            raise ValueError("page_table, lengths and q_start must be on one device")
        self._device = self.lengths.get_device()
        self._args = (self.page_table.data_ptr(), self.page_table.shape[1], self.lengths.data_ptr(),
                      self.q_start.data_ptr(), B, self.tokens)
        return self._args


class Kv4Workspace(_Handle):
    """Device workspace of the cache's calls for this number of query heads and
    batches of up to this one's requests and tokens; zeroed once."""
    _fields = ("buf",)

    def __init__(self, batch: Kv4Batch, heads: int, cache: Kv4Cache):
        dev = cache.buf.device
        nbytes = _binding.kv_workspace_bytes(heads, cache.kv_heads, cache.head_dim, batch.lengths.shape[0],
                                             batch.tokens, dev.index)
        self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
        self._check()

    def _check(self):
        _need_bytes(self.buf, "the workspace's buf", 256)
        self.nbytes, self._device = self.buf.numel(), self.buf.get_device()
        self._args = (self.buf.data_ptr(), self.nbytes)
        return self._args

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()


def _need_bytes(t: torch.Tensor, name: str, nbytes: int) -> None:
    if not t.is_cuda or t.dtype != torch.uint8 or not t.is_contiguous() or t.numel() < nbytes:
        raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor of at least {nbytes} bytes")


def _explain(name: str, t: torch.Tensor, tokens: int, heads, cache: Kv4Cache) -> None:
    """Raises for a tensor that is not fp16 [tokens, heads, head_dim] on the cache's device."""
    if not t.is_cuda or t.dtype != torch.float16:
        raise ValueError(f"{name} must be an fp16 CUDA tensor, got {t.dtype} on {t.device}")
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != cache.head_dim or (heads and t.shape[1] != heads):
        raise ValueError(f"{name}: expected [{tokens}, {heads or 'heads'}, {cache.head_dim}], got {tuple(t.shape)}")
    if t.stride(2) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def _on_device(cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace, *named) -> int:
    """The current device, on which every tensor of a call has to be."""
    cur = torch._C._cuda_getDevice()
    if not (cache._device == batch._device == ws._device == cur and all(t.get_device() == cur for _, t in named)):
        _on_current_device(("cache", cache.buf), ("page_table", batch.page_table), ("workspace", ws.buf), *named)
    return cur


def kv4_append(k: torch.Tensor, v: torch.Tensor, cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace) -> None:
    """Quantise the batch's new keys and values, fp16 [tokens, kv_heads,
    head_dim] (views of one QKV product are fine), into the cache, on the
    current stream."""
    cached, rows, work = cache._args or cache._check(), batch._args or batch._check(), ws._args or ws._check()
    want = (batch.tokens, cache.kv_heads, cache.head_dim)
    ks, vs = k.stride(), v.stride()
    for name, t, st in (("k", k, ks), ("v", v, vs)):
        if t.dtype is not torch.float16 or t.shape != want or st[2] != 1 or not t.is_cuda:
            _explain(name, t, batch.tokens, cache.kv_heads, cache)
    cur = _on_device(cache, batch, ws, ("k", k), ("v", v))
    rc = (_binding._lib or _binding.load()).marlin_kv_append(
        k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], *cached, *rows, work[0],
        torch._C._cuda_getCurrentRawStream(cur))
    if rc:
        raise MarlinError(rc, "marlin_kv_append")


def kv4_read(cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace):
    """(k, v), fp16 [tokens, kv_heads, head_dim]: the values the cache holds for
    the batch's new tokens."""
    cached, rows, work = cache._args or cache._check(), batch._args or batch._check(), ws._args or ws._check()
    cur = _on_device(cache, batch, ws)
    shape = (batch.tokens, cache.kv_heads, cache.head_dim)
    k = torch.empty(shape, dtype=torch.float16, device=cache.buf.device)
    v = torch.empty_like(k)
    rc = (_binding._lib or _binding.load()).marlin_kv_read(
        k.data_ptr(), v.data_ptr(), *cached, *rows, work[0], torch._C._cuda_getCurrentRawStream(cur))
    if rc:
        raise MarlinError(rc, "marlin_kv_read")
    return k, v


def kv4_attention_into(q: torch.Tensor, cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace, out: torch.Tensor,
                       scale: float | None = None, window: int = 0) -> torch.Tensor:
    """out[tokens, heads, head_dim] = causal attention of the batch's new tokens
    over the cache, which holds their own keys and values already.  scale:
    1 / sqrt(head_dim) by default; window > 0: a token sees that many positions,
    its own included.  Rows that no request owns are left alone (kv4_attention's
    are not initialised)."""
    cached, rows, work = cache._args or cache._check(), batch._args or batch._check(), ws._args or ws._check()
    qs, shape = q.stride(), q.shape
    if (q.dtype is not torch.float16 or len(shape) != 3 or shape[0] != batch.tokens or shape[2] != cache.head_dim
            or qs[2] != 1 or not q.is_cuda):
        _explain("q", q, batch.tokens, None, cache)
    if out.dtype is not torch.float16 or out.shape != shape or not out.is_contiguous() or not out.is_cuda:
        _explain("out", out, batch.tokens, shape[1], cache)
        raise ValueError("out must be contiguous")
    cur = _on_device(cache, batch, ws, ("q", q), ("out", out))
    rc = (_binding._lib or _binding.load()).marlin_kv_attention(
        q.data_ptr(), qs[0], qs[1], shape[1], *cached, *rows, batch.max_q,
        cache._scale if scale is None else scale, window, out.data_ptr(), *work,
        torch._C._cuda_getCurrentRawStream(cur))
    if rc:
        raise MarlinError(rc, "marlin_kv_attention")
    return out


def kv4_attention(q: torch.Tensor, cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace, scale: float | None = None,
                  window: int = 0) -> torch.Tensor:
    out = torch.empty(q.shape, dtype=torch.float16, device=q.device)
    return kv4_attention_into(q, cache, batch, ws, out, scale, window)
