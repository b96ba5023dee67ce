"""A paged key/value cache held in 4 bits, and attention over it (include/marlin.h).

    cache = Kv4Cache(n_pages, kv_heads, head_dim, page_size)       # once
    batch = Kv4Batch(page_table, lengths, q_start, tokens, max_q)  # once per step
    ws = Kv4Workspace(batch, heads, cache)                         # once, for the largest batch
    kv4_append(k, v, cache, batch, ws)                             # the new tokens' keys and values
    o = kv4_attention(q, cache, batch, ws)                         # fp16 [tokens, heads, head_dim]
"""
from __future__ import annotations

import math
import sys
from array import array
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
        # what caches that a call takes together have in common, in a form that is quick to compare
        self._like = sys.intern(repr((self._device, *self._args[1:])))
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


def _need_i32(t: torch.Tensor, name: str, shape) -> None:
    if t.shape != shape or t.dtype is not torch.int32 or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor {list(shape)}, got {t.dtype} {list(t.shape)} "
                         f"on {t.device}")


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


# ---- drafted trees ------------------------------------------------------------------------------

def kv4_tree(parents: torch.Tensor, batch: Kv4Batch, ws: Kv4Workspace):
    """(mask, positions) of the batch's new tokens, where those of a request are a tree: parents int32
    [tokens], each token's parent among its request's new tokens (0 is the first), which comes before it,
    negative for none.  mask int32 [tokens, words], words = max_q / 32 rounded up: bit j (of word j / 32) of a row is
    set where the request's j-th new token is the row's own or one of its ancestors.  positions int32
    [tokens]: the cached tokens before the new ones and the row's ancestors, counted.  Rows that no request
    owns are not initialised.  (A token takes a step for every ancestor, and all rows the words of the longest request:
    long runs without branches, as prompts are, belong to kv4_attention.)"""
    rows, work = batch._args or batch._check(), ws._args or ws._check()
    _need_i32(parents, "parents", (batch.tokens,))
    cur = torch._C._cuda_getDevice()
    if not batch._device == ws._device == parents.get_device() == cur:
        _on_current_device(("page_table", batch.page_table), ("workspace", ws.buf), ("parents", parents))
    words = max(1, (batch.max_q + 31) // 32)
    mask = torch.empty((batch.tokens, words), dtype=torch.int32, device=parents.device)
    positions = torch.empty((batch.tokens,), dtype=torch.int32, device=parents.device)
    rc = (_binding._lib or _binding.load()).marlin_kv_tree(
        parents.data_ptr(), rows[2], rows[3], rows[4], rows[5], words, mask.data_ptr(), positions.data_ptr(), work[0],
        torch._C._cuda_getCurrentRawStream(cur))
    if rc:
        raise MarlinError(rc, "marlin_kv_tree")
    return mask, positions


def kv4_tree_attention_into(q: torch.Tensor, cache: Kv4Cache, batch: Kv4Batch, tree: torch.Tensor, ws: Kv4Workspace,
                            out: torch.Tensor, scale: float | None = None, window: int = 0) -> torch.Tensor:
    """out[tokens, heads, head_dim] = attention of the batch's new tokens over the cache, which holds their own keys and
    values already: a token sees the cached tokens before the new ones, and of its request's new ones those whose bit is
    set in its row of tree (int32 [tokens, words], as kv4_tree makes it, or any other).  scale: 1 / sqrt(head_dim) by
    default; window > 0: of the tokens before the new ones a row sees those among the last `window` up to its position,
    which is the number of them and of the new tokens that it sees, less 1.  New tokens are hidden by their bits alone: to
    hide ancestors `window` or more levels up, leave their bits out.  Rows that no request owns are left alone
    (kv4_tree_attention's are not initialised)."""
    cached, rows, work = cache._args or cache._check(), batch._args or batch._check(), ws._args or ws._check()
    qs, shape = q.stride(), q.shape
    if (q.dtype is not torch.float16 or len(shape) != 3 or shape[0] != batch.tokens or shape[2] != cache.head_dim
            or qs[2] != 1 or not q.is_cuda):
        _explain("q", q, batch.tokens, None, cache)
    if out.dtype is not torch.float16 or out.shape != shape or not out.is_contiguous() or not out.is_cuda:
        _explain("out", out, batch.tokens, shape[1], cache)
        raise ValueError("out must be contiguous")
    if tree.dim() != 2:
        raise ValueError(f"tree: expected [{batch.tokens}, words], got {tuple(tree.shape)}")
    _need_i32(tree, "tree", (batch.tokens, tree.shape[1]))
    cur = _on_device(cache, batch, ws, ("q", q), ("out", out), ("tree", tree))
    rc = (_binding._lib or _binding.load()).marlin_kv_tree_attention(
        q.data_ptr(), qs[0], qs[1], shape[1], *cached, *rows, batch.max_q, tree.data_ptr(), tree.shape[1],
        cache._scale if scale is None else scale, window, out.data_ptr(), *work,
        torch._C._cuda_getCurrentRawStream(cur))
    if rc:
        raise MarlinError(rc, "marlin_kv_tree_attention")
    return out


def kv4_tree_attention(q: torch.Tensor, cache: Kv4Cache, batch: Kv4Batch, tree: torch.Tensor, ws: Kv4Workspace,
                       scale: float | None = None, window: int = 0) -> torch.Tensor:
    out = torch.empty(q.shape, dtype=torch.float16, device=q.device)
    return kv4_tree_attention_into(q, cache, batch, tree, ws, out, scale, window)


# ---- rotary positions ----------------------------------------------------------------------------

class Kv4Rope(_Handle):
    """Cosines and sines of rotary positions, once per model: cos, sin fp32 [positions, rot / 2], the entry for a
    position and a pair of channels; rot, a multiple of head_dim / 8, is how many channels of a head are rotated, its first.
    interleaved: pair j is channels (2 j, 2 j + 1), else (j, j + rot / 2).  axes: for positions on up to 4 axes (time,
    height, width) the axis of each pair, rot / 2 numbers; None for one axis."""
    _fields = ("table", "rot", "interleaved", "axes")

    def __init__(self, cos: torch.Tensor, sin: torch.Tensor, axes=None, interleaved: bool = False):
        if (not cos.is_cuda or cos.dtype != torch.float32 or cos.dim() != 2 or sin.shape != cos.shape
                or sin.dtype != torch.float32 or sin.device != cos.device):
            raise ValueError("cos and sin must be fp32 CUDA tensors [positions, rot / 2] on one device")
        self.table = torch.stack([cos, sin], dim=-1).contiguous()
        self.rot, self.interleaved = 2 * cos.shape[1], bool(interleaved)
        self.axes = None if axes is None else tuple(int(a) for a in axes)
        self._check()

    @classmethod
    def from_theta(cls, rot: int, positions: int, theta: float = 10000.0, axes=None, interleaved: bool = False, device=None):
        """Angles position * theta^(-2 j / rot) for pair j, in 64 bits up to their cosines and sines."""
        if rot <= 0 or rot % 2:
            raise ValueError(f"rot: expected an even number of channels, got {rot}")
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        freq = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        angle = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * freq
        return cls(angle.cos().float(), angle.sin().float(), axes, interleaved)

    def _check(self):
        t = self.table
        if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous() or t.dim() != 3 or t.shape[1:] != (self.rot // 2, 2):
            raise ValueError("the rope's table must be a contiguous fp32 CUDA tensor [positions, rot / 2, 2]")
        if t.shape[0] < 1 or t.shape[1] < 1:
            raise ValueError("the rope's table is empty")
        axes = self.axes if self.axes is not None else (0,) * (self.rot // 2)
        if len(axes) != self.rot // 2 or any(a < 0 or a > 3 for a in axes):
            raise ValueError(f"axes: expected {self.rot // 2} numbers from 0 to 3")
        self.n_axes = max(axes) + 1
        self._device = t.get_device()
        self._args = (t.data_ptr(), t.shape[0], self.rot, int(self.interleaved), bytes(axes))
        return self._args


def _rows_apart(t: torch.Tensor) -> bool:
    """Whether no two of the rows [tokens, heads] share an element, tokens or heads outermost."""
    (T, H, D), (ts, hs, _) = t.shape, t.stride()
    inside = lambda inner, n, outer, m: (n <= 1 or inner >= D) and (m <= 1 or outer >= (n - 1) * inner + D)  # noqa: E731
    return inside(hs, H, ts, T) or inside(ts, T, hs, H)


def kv4_rope_append_into(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, rope: Kv4Rope,
                         cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace, out: torch.Tensor) -> torch.Tensor:
    """Rotate the batch's queries q, fp16 [tokens, heads, head_dim], and keys k, fp16 [tokens, kv_heads, head_dim], by
    their positions, and quantise the rotated keys and the values v into the cache (as kv4_append does: the rotated
    keys are rounded to fp16 first).  The rotated queries go to out, shaped like q (q itself, or anything that
    overlaps neither q, k nor v, its rows apart).  positions int32 [axes, tokens], or [tokens] for one axis: rows of the rope's
    table.  q, k, v and out may be views whose last dimension is contiguous (of one QKV product).  Rows that no
    request owns are left alone."""
    cached, rows, work = cache._args or cache._check(), batch._args or batch._check(), ws._args or ws._check()
    angles = rope._args or rope._check()
    qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
    T, shape, f16 = batch.tokens, q.shape, torch.float16
    new = (T, cache.kv_heads, cache.head_dim)
    if (k.shape != new or v.shape != new or len(shape) != 3 or shape[0] != T or shape[2] != new[2] or out.shape != shape
            or not (q.dtype is k.dtype is v.dtype is out.dtype is f16) or not (qs[2] == ks[2] == vs[2] == os[2] == 1)
            or not (q.is_cuda and k.is_cuda and v.is_cuda and out.is_cuda)):
        for name, t, heads in (("q", q, None), ("k", k, new[1]), ("v", v, new[1]), ("out", out, shape[1] if len(shape) == 3 else None)):
            _explain(name, t, T, heads, cache)
    if (os[1] < new[2] or os[0] < (shape[1] - 1) * os[1] + new[2]) and not _rows_apart(out):
        raise ValueError("out's rows overlap")
    _need_i32(positions, "positions", (T,) if rope.n_axes == 1 and positions.dim() == 1 else (rope.n_axes, T))
    cur = torch._C._cuda_getDevice()
    if not (cache._device == batch._device == ws._device == rope._device == q.get_device() == k.get_device()
            == v.get_device() == out.get_device() == positions.get_device() == cur):
        _on_device(cache, batch, ws, ("q", q), ("k", k), ("v", v), ("out", out), ("positions", positions), ("rope", rope.table))
    rc = (_binding._lib or _binding.load()).marlin_kv_rope_append(
        q.data_ptr(), qs[0], qs[1], shape[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
        positions.data_ptr(), rope.n_axes, *angles, out.data_ptr(), os[0], os[1], *cached, *rows, work[0],
        torch._C._cuda_getCurrentRawStream(cur))
    if rc:
        raise MarlinError(rc, "marlin_kv_rope_append")
    return out


def kv4_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, rope: Kv4Rope,
                    cache: Kv4Cache, batch: Kv4Batch, ws: Kv4Workspace) -> torch.Tensor:
    """kv4_rope_append_into with the rotated queries in a new tensor."""
    out = torch.empty(q.shape, dtype=torch.float16, device=q.device)
    return kv4_rope_append_into(q, k, v, positions, rope, cache, batch, ws, out)


# ---- moving what the caches hold -----------------------------------------------------------------

def _layers(caches, ws: Kv4Workspace, *named):
    """The addresses of the layers' caches (one or several alike), what they share, and the current device."""
    caches = (caches,) if isinstance(caches, Kv4Cache) else tuple(caches)
    at = [(c._args or c._check())[0] for c in caches]
    like = [c._like for c in caches]
    if not at or like.count(like[0]) != len(at):
        raise ValueError("no caches" if not at else
                         "the caches must be alike: device, pages, key heads, head_dim and page size")
    cur = torch._C._cuda_getDevice()
    if caches[0]._device != cur or ws._device != cur or any(t.get_device() != cur for _, t in named):
        _on_current_device(*(("cache", c.buf) for c in caches), ("workspace", ws.buf), *named)
    return array("Q", at), len(at), caches[0]._args[1:], cur


def kv4_compact(caches, batch: Kv4Batch, index: torch.Tensor, kept: torch.Tensor, ws: Kv4Workspace,
                into: torch.Tensor | None = None) -> torch.Tensor:
    """Keep some of each request's new tokens, in the caches of all layers (one Kv4Cache or a sequence of them, all
    alike): with first = lengths[b] - new tokens, position first + i takes what position first + index[q_start[b] + i]
    holds, for i < kept[b].  index int32 [tokens], kept int32 [B].  Returns the new lengths, int32 [B]: first + kept.

    into None: the tokens stay in their pages, and index must ascend within a request (one that does not is left as it
    was, and reported).  into int32 [B, pages]: the kept tokens' pages, which the caller owns and which are none of
    those that are read; index may then name any of the new tokens, in any order.  Other positions are not touched.
    Pages that requests share must hold none of the positions that are written."""
    rows, work = batch._args or batch._check(), ws._args or ws._check()
    B = rows[4]
    _need_i32(index, "index", (batch.tokens,))
    _need_i32(kept, "kept", (B,))
    named = [("page_table", batch.page_table), ("index", index), ("kept", kept)]
    if into is not None:
        if into.dim() != 2:
            raise ValueError(f"into: expected [{B}, pages], got {tuple(into.shape)}")
        _need_i32(into, "into", (B, into.shape[1]))
        named.append(("into", into))
    at, count, shape, cur = _layers(caches, ws, *named)
    lengths = torch.empty((B,), dtype=torch.int32, device=index.device)
    rc = (_binding._lib or _binding.load()).marlin_kv_compact(
        at.buffer_info()[0], count, *shape, rows[0], rows[1], None if into is None else into.data_ptr(),
        0 if into is None else into.shape[1], rows[2], rows[3], index.data_ptr(), kept.data_ptr(), lengths.data_ptr(), B,
        batch.tokens, batch.max_q, work[0], torch._C._cuda_getCurrentRawStream(cur))
    if rc:
        raise MarlinError(rc, "marlin_kv_compact")
    return lengths


def kv4_copy_pages(caches, src: torch.Tensor, dst: torch.Tensor, ws: Kv4Workspace) -> None:
    """Page dst[i] takes what page src[i] holds, in the caches of all layers (one Kv4Cache or a sequence of them, all
    alike); a pair whose source is negative is left out.  src, dst int32 [pairs].  A page that is written must be named
    once only, as source or destination, in a call."""
    work = ws._args or ws._check()
    if src.dim() != 1:
        raise ValueError(f"src: expected [pairs], got {tuple(src.shape)}")
    _need_i32(src, "src", src.shape)
    _need_i32(dst, "dst", src.shape)
    at, count, shape, cur = _layers(caches, ws, ("src", src), ("dst", dst))
    rc = (_binding._lib or _binding.load()).marlin_kv_copy_pages(
        at.buffer_info()[0], count, *shape, src.data_ptr(), dst.data_ptr(), src.shape[0], work[0],
        torch._C._cuda_getCurrentRawStream(cur))
    if rc:
        raise MarlinError(rc, "marlin_kv_copy_pages")


class Kv4Pages:
    """Which pages of the caches are free, and how many requests hold each of the others (on the host)."""

    def __init__(self, n_pages: int, page_size: int):
        self.page_size = page_size
        self._free = list(range(n_pages - 1, -1, -1))
        self._holders = [0] * n_pages

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def take(self, n: int) -> list[int]:
        """n pages that no one holds."""
        if n < 0 or n > len(self._free):
            raise ValueError(f"{n} pages asked for, {len(self._free)} are free")
        pages = [self._free.pop() for _ in range(n)]
        for page in pages:
            self._holders[page] = 1
        return pages

    def fork(self, pages, length: int):
        """(pages, copies) of a request that goes on from another's first `length` tokens: it shares the pages that
        these fill, and has one of its own for the rest of them; copies lists that (from, to), for kv4_copy_pages."""
        full, rest = divmod(length, self.page_size)
        if length < 0 or full + (rest > 0) > len(pages):
            raise ValueError(f"{length} tokens do not fit {len(pages)} pages")
        self._need_held(pages[:full + (rest > 0)])
        own = self.take(1) if rest else []
        for page in pages[:full]:
            self._holders[page] += 1
        return list(pages[:full]) + own, [(pages[full], own[0])] if rest else []

    def free(self, pages) -> None:
        """A request's pages, which it no longer holds; those that no one else holds are free again."""
        self._need_held(pages)
        for page in pages:
            self._holders[page] -= 1
            if self._holders[page] == 0:
                self._free.append(page)

    def shared(self, page: int) -> bool:
        """Whether several requests hold the page: none of them may write into it."""
        return self._holders[page] > 1

    def _need_held(self, pages) -> None:
        count = {}
        for page in pages:
            count[page] = count.get(page, 0) + 1
        for page, n in count.items():
            if not 0 <= page < len(self._holders) or self._holders[page] < n:
                raise ValueError(f"page {page} is not held")
