"""Offsets that are not ascending: the products report them and compute nothing. (Counted as they are,
their row tiles would have no bound but groups x rows, and a large enough sum none at all.)"""
import pytest
import torch

from mixture_experts_layer_29_b200 import abi, mx4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("bad", [[0, 70, 30, 70], [0, 900, 0, 900], [0, 1000, -5, 900]])
def test_descending_offsets_compute_nothing(cuda_device, fmt, bad):
    rows, K, I = (70 if max(bad) == 70 else 900), 256, 128
    a = mx4.allocate(fmt, rows, K, 3, torch.tensor(bad, dtype=torch.int32, device="cuda"))
    a.codes.zero_()
    a.scales.zero_()
    w = mx4.quantize_weight(torch.ones(3, 2 * I, K, device="cuda"), fmt)
    d = mx4.quantize_weight(torch.ones(3, K, I, device="cuda"), fmt)
    for dtype in (torch.bfloat16, torch.float32):
        out = torch.full((rows, 2 * I), 5.0, device="cuda", dtype=dtype)
        ws = mx4.gemm_workspace()
        mx4.grouped_gemm(a, w, out, ws)
        assert abi.read_device_status(ws) == -6 and bool((out == 5.0).all())
        out = torch.full((rows, K), 5.0, device="cuda", dtype=dtype)
        ws = mx4.ffn_workspace(a, w)
        mx4.grouped_ffn(a, w, d, out, ws)
        assert abi.read_device_status(ws) == -6 and bool((out == 5.0).all())
