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

from . import _binding, _on_current_device, _stream
from ._binding import MarlinError


class Kv4Cache:
    """n_pages pages of page_size tokens of every key head, keys and values in
    4 bits (head_dim + 8 bytes per token and head)."""

    def __init__(self, n_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device=None):
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError("a cache lives on a CUDA device")
        self.nbytes = _binding.kv_cache_bytes(n_pages, kv_heads, head_dim, page_size)
        self.n_pages, self.kv_heads, self.head_dim, self.page_size = n_pages, kv_heads, head_dim, page_size
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=dev)


@dataclass
class Kv4Batch:
    """One step's requests.  page_table int32 [B, pages], lengths int32 [B]
    (cached tokens, the new ones included), q_start int32 [B + 1] (the new
    tokens of request b are rows q_start[b] .. q_start[b+1] - 1, its last
    positions); tokens = q_start[B] rows in all, at most max_q of one request.
    The tensors are read by the kernels at each call: they may be updated in
    place between steps."""
    page_table: torch.Tensor
    lengths: torch.Tensor
    q_start: torch.Tensor
    tokens: int
    max_q: int = 1

    def __post_init__(self):
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
        self._args = (self.page_table.data_ptr(), self.page_table.shape[1], self.lengths.data_ptr(),
                      self.q_start.data_ptr(), B, self.tokens)


class Kv4Workspace:
    """Device workspace of the cache's calls for this number of query heads and
    batches of up to this one's requests and tokens; zeroed once."""

    def __init__(self, batch: Kv4Batch, heads: int, cache: Kv4Cache):
        dev = cache.buf.device
        self.nbytes = _binding.kv_workspace_bytes(heads, cache.kv_heads, cache.head_dim, batch.lengths.shape[0],
                                                  batch.tokens, dev.index)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=dev)

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()


def _check_heads(t: torch.Tensor, name: str, tokens: int, heads: int | None, cache: Kv4Cache) -> None:
    if not t.is_cuda or t.dtype != torch.float16:
        raise ValueError(f"{name} must be an fp16 CUDA tensor, got {t.dtype} on {t.device}")
    if t.dim() != 3 or t.shape[0] != tokens or t.shape[2] != cache.head_dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name}: expected [{tokens}, {heads or 'heads'}, {cache.head_dim}], got {tuple(t.shape)}")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")


def kv4_append(k: torch.Tensor, v: torch.Tensor, cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace) -> None:
    """Quantise the batch's new keys and values, fp16 [tokens, kv_heads,
    head_dim] (views of one QKV product are fine), into the cache, on the
    current stream."""
    table, max_pages, lengths, q_start, B, T = batch._args
    _check_heads(k, "k", T, cache.kv_heads, cache)
    _check_heads(v, "v", T, cache.kv_heads, cache)
    _on_current_device(("k", k), ("v", v), ("cache", cache.buf), ("page_table", batch.page_table), ("workspace", ws.buf))
    rc = _binding.load().marlin_kv_append(
        k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), cache.buf.data_ptr(),
        cache.n_pages, cache.kv_heads, cache.head_dim, cache.page_size, table, max_pages, lengths, q_start, B, T,
        ws.ptr, _stream() or None)
    if rc != _binding.OK:
        raise MarlinError(rc, "marlin_kv_append")


def kv4_read(cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace):
    """(k, v), fp16 [tokens, kv_heads, head_dim]: the values the cache holds for
    the batch's new tokens."""
    table, max_pages, lengths, q_start, B, T = batch._args
    _on_current_device(("cache", cache.buf), ("page_table", batch.page_table), ("workspace", ws.buf))
    k = torch.empty((T, cache.kv_heads, cache.head_dim), dtype=torch.float16, device=cache.buf.device)
    v = torch.empty_like(k)
    rc = _binding.load().marlin_kv_read(
        k.data_ptr(), v.data_ptr(), cache.buf.data_ptr(), cache.n_pages, cache.kv_heads, cache.head_dim,
        cache.page_size, table, max_pages, lengths, q_start, B, T, ws.ptr, _stream() or None)
    if rc != _binding.OK:
        raise MarlinError(rc, "marlin_kv_read")
    return k, v


def kv4_attention_into(q: torch.Tensor, cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace, out: torch.Tensor,
                       scale: float | None = None, window: int = 0) -> torch.Tensor:
    """out[tokens, heads, head_dim] = causal attention of the batch's new tokens
    over the cache, which holds their own keys and values already.  scale:
    1 / sqrt(head_dim) by default; window > 0: a token sees that many positions,
    its own included."""
    table, max_pages, lengths, q_start, B, T = batch._args
    _check_heads(q, "q", T, None, cache)
    _check_heads(out, "out", T, q.shape[1], cache)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    _on_current_device(("q", q), ("cache", cache.buf), ("page_table", batch.page_table), ("workspace", ws.buf),
                       ("out", out))
    rc = _binding.load().marlin_kv_attention(
        q.data_ptr(), q.stride(0), q.stride(1), q.shape[1], cache.buf.data_ptr(), cache.n_pages, cache.kv_heads,
        cache.head_dim, cache.page_size, table, max_pages, lengths, q_start, B, T, batch.max_q,
        1.0 / math.sqrt(cache.head_dim) if scale is None else scale, window, out.data_ptr(), ws.ptr, ws.nbytes,
        _stream() or None)
    if rc != _binding.OK:
        raise MarlinError(rc, "marlin_kv_attention")
    return out


def kv4_attention(q: torch.Tensor, cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace, scale: float | None = None,
                  window: int = 0) -> torch.Tensor:
    out = torch.empty(q.shape, dtype=torch.float16, device=q.device)
    return kv4_attention_into(q, cache, batch, ws, out, scale, window)
