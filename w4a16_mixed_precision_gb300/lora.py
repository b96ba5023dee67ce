"""Low-rank adapters of many requests beside a shared W4A16 product:

    y[m] = x[m] . dequant(W) + scaling[a] * (x[m] . A[a]^T) . B[a]^T,  a = index[m] (none if negative).

One call (marlin_lora_gemm) per projection; see include/marlin.h.
"""
from __future__ import annotations

import torch

from . import PackedWeights, Workspace, _binding, _Handle, _need_cuda, _need_dense, _on_current_device
from ._binding import MarlinError

MAX_RANK = 128


class LoraBank(_Handle):
    """The adapters of one projection, on the device: a fp16 [n, r, K], b fp16
    [n, N, r], scaling fp32 [n].  A rank that is not a multiple of 8 is padded
    with zeros (a copy).  n, r (padded), K and N follow from the tensors, which
    may be updated in place or replaced between calls (not resized in place)."""
    _fields = ("a", "b", "scaling")

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scaling: torch.Tensor):
        self.a, self.b, self.scaling = a, b, scaling
        self._check()

    def __setattr__(self, name, value):
        if name in ("n", "r", "K", "N"):
            raise AttributeError(f"{name} follows from the adapters' tensors")
        super().__setattr__(name, value)

    def _check(self):
        a, b, scaling = self.a, self.b, self.scaling
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError(f"expected a [n, r, K] and b [n, N, r], got {tuple(a.shape)} and {tuple(b.shape)}")
        if tuple(scaling.shape) != (a.shape[0],):
            raise ValueError(f"expected scaling [{a.shape[0]}], got {tuple(scaling.shape)}")
        for name, t, dtype in (("a", a, torch.float16), ("b", b, torch.float16), ("scaling", scaling, torch.float32)):
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dtype != dtype:
                raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not a.device == b.device == scaling.device:
            raise ValueError("a, b and scaling must be on one device")
        n, r, K = a.shape
        if not 0 < n or not 0 < r <= MAX_RANK:
            raise ValueError(f"at least one adapter, of a rank up to {MAX_RANK}, is wanted: got {n} of rank {r}")
        pad = -r % 8
        if pad:
            a, b = torch.nn.functional.pad(a, (0, 0, 0, pad)), torch.nn.functional.pad(b, (0, pad))
        self.a, self.b, self.scaling = a.contiguous(), b.contiguous(), scaling.contiguous()
        self.__dict__.update(n=n, r=r + pad, K=K, N=b.shape[1])
        self._device = self.a.get_device()
        self._args = (self.a.data_ptr(), self.b.data_ptr(), self.scaling.data_ptr(), n, self.r)
        return self._args

    @classmethod
    def stack(cls, adapters) -> "LoraBank":
        """From (a [r, K], b [N, r], scaling) of each adapter; lower ranks are padded with zeros."""
        adapters = list(adapters)
        if not adapters:
            raise ValueError("at least one adapter is wanted")
        r = max(a.shape[0] for a, _, _ in adapters)
        pad = torch.nn.functional.pad
        return cls(torch.stack([pad(a, (0, 0, 0, r - a.shape[0])) for a, _, _ in adapters]),
                   torch.stack([pad(b, (0, r - b.shape[1])) for _, b, _ in adapters]),
                   torch.tensor([float(s) for _, _, s in adapters], dtype=torch.float32, device=adapters[0][0].device))


class LoraWorkspace(Workspace):
    """Device workspace of lora_gemm for up to max_M rows and adapters of rank r,
    zeroed once; serves gemm with the same shapes too."""

    def __init__(self, max_M: int, K: int, N: int, group: int, r: int, device=None):
        self.r = r + -r % 8
        super().__init__(max_M, K, N, group, device)

    def _bytes(self, M: int, K: int, N: int, group: int, device: int) -> int:
        return _binding.lora_workspace_bytes(M, K, N, group, self.r, device)


def lora_gemm_into(x: torch.Tensor, w: PackedWeights, bank: LoraBank, index: torch.Tensor, ws: LoraWorkspace,
                   y: torch.Tensor) -> torch.Tensor:
    """y[M, N] = x[M, K] . dequant(W) + the part of each row's adapter, fp16, on
    the current stream.  index: int32 [M], negative for no adapter."""
    _need_dense(w)
    adapters = bank._args or bank._check()
    f16, K = torch.float16, w.K
    M = x.shape[0]
    if x.dtype is not f16 or y.dtype is not f16 or index.dtype is not torch.int32 or not (
            x.is_contiguous() and y.is_contiguous() and index.is_contiguous()):
        _need_cuda(x, "x", f16)
        _need_cuda(y, "y", f16)
        _need_cuda(index, "index", torch.int32)
    if x.shape != (M, K) or K != bank.K or w.N != bank.N or y.shape != (M, w.N) or index.shape != (M,):
        raise ValueError("shape mismatch")
    cur = torch._C._cuda_getDevice()
    if not (x.get_device() == y.get_device() == index.get_device() == w.buf.get_device() == bank._device
            == ws.buf.get_device() == cur):
        for name, t in (("x", x), ("y", y), ("index", index)):
            _need_cuda(t, name)
        _on_current_device(("x", x), ("weights", w.buf), ("adapters", bank.a), ("index", index), ("workspace", ws.buf),
                           ("y", y))
    rc = (_binding._lib or _binding.load()).marlin_lora_gemm(
        x.data_ptr(), w.codes_ptr, w.scales_ptr, w.zeros_ptr, *adapters[:3], index.data_ptr(), *adapters[3:],
        y.data_ptr(), M, K, w.N, w.group, ws.buf.data_ptr(), ws.nbytes, torch._C._cuda_getCurrentRawStream(cur))
    if rc:
        raise MarlinError(rc, "marlin_lora_gemm")
    return y


def lora_gemm(x: torch.Tensor, w: PackedWeights, bank: LoraBank, index: torch.Tensor,
              ws: LoraWorkspace) -> torch.Tensor:
    y = torch.empty((x.shape[0], w.N), dtype=torch.float16, device=x.device)
    return lora_gemm_into(x, w, bank, index, ws, y)
