"""Weights in the 2:4 layout are refused where the dense layout is read (its kernels would read K N / 2
bytes of codes from a buffer that holds three quarters of that).  No GPU needed: the refusal comes first."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("name", ["gemm", "gemm_into", "gemm_host", "lora_gemm", "lora_gemm_into"])
def test_sparse_weights_are_refused(name):
    import w4a16_mixed_precision_gb300 as w4
    M, K, N = 2, 256, 128
    nbytes, off_m, off_s, off_z = w4._binding.sparse_packed_layout(K, N, 128, False)
    w = w4.SparsePackedWeights(torch.zeros(nbytes, dtype=torch.uint8), K, N, 128, False, off_m, off_s, off_z, 0)
    x, y = torch.zeros((M, K), dtype=torch.float16), torch.zeros((M, N), dtype=torch.float16)
    ws = SimpleNamespace(buf=torch.zeros(256, dtype=torch.uint8), ptr=0, nbytes=256)
    bank, index = SimpleNamespace(K=K, N=N, _device=-1), torch.zeros(M, dtype=torch.int32)
    args = {"gemm": (x, w, ws), "gemm_into": (x, w, ws, y), "gemm_host": (x, x, w, ws, y, y),
            "lora_gemm": (x, w, bank, index, ws), "lora_gemm_into": (x, w, bank, index, ws, y)}[name]
    with pytest.raises(ValueError, match="2:4"):
        getattr(w4, name)(*args)
