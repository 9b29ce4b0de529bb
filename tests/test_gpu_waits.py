"""Waits of the block norms' gradients and of the 4-bit products that run out: the call reports
MOE_ERR_TIMEOUT, ends soon after the waits' limit, and the next one gives the clean run's bits. (The host
tells the kernel not to load one place of its ring, so nothing is in flight on it.)"""
import time

import pytest
import torch

from mixture_experts_layer_29_b200 import abi, mx4, norm

pytestmark = pytest.mark.gpu
NORM, PRODUCT = 2, 3


def stalled(which, call):
    """Runs call() once with the testing hook set; returns the seconds it took."""
    torch.cuda.synchronize()
    abi.set_tuning(abi.TUNE_TEST_STALL, which)
    try:
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    finally:
        armed = abi.get_tuning(abi.TUNE_TEST_STALL)
        abi.set_tuning(abi.TUNE_TEST_STALL, 0)
    assert armed == 0                       # one shot: taken by that launch
    return took


@pytest.mark.parametrize("T,H,parts", [(5, 768, "both"), (4000, 6144, "both"), (4000, 2048, "post"), (600, 4096, "pre")])
def test_norm_gradients_wait_that_runs_out(cuda_device, T, H, parts):
    """4000 tokens: some 27 and more per CTA. The one whose first token is missing gives up at once, not after
    a wait for each of them."""
    g = torch.Generator(device="cuda").manual_seed(H)
    rows = lambda: torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)     # noqa: E731
    d = norm.make_desc(T, H)
    w, rstd = torch.ones(H, device="cuda"), torch.ones(T, device="cuda")
    post, pre = parts != "pre", parts != "post"
    ins = [rows(), rows() if pre else None, rows() if pre else None, rows() if post else None, w if post else None,
           None, w if pre else None, rstd if post else None, rstd if pre else None]
    outs = [rows(), rows() if post else None, w.clone() if post else None, None, w.clone() if pre else None]
    ws = norm.workspace(d)
    call = lambda: norm.block_norm_backward(d, *ins, *outs, ws)     # noqa: E731
    call()
    assert abi.read_device_status(ws) == 0
    want = [o if o is None else o.clone() for o in outs]
    took = stalled(NORM, call)
    assert abi.read_device_status(ws) == -7 and 1.5 < took < 4, took
    call()
    assert abi.read_device_status(ws) == 0
    assert all(o is None or torch.equal(o, v) for o, v in zip(outs, want))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows", [90, 900])                     # one CTA per tile, and CTA pairs
@pytest.mark.parametrize("what", ["bf16", "fp32", "ffn"])
def test_product_wait_that_runs_out(cuda_device, fmt, rows, what):
    """Two groups, many tiles; thirteen stages along K, more than either ring has."""
    groups, K, I = 2, 3200, 1024
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, K, device="cuda", generator=g).to(torch.bfloat16)
    off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    a = mx4.quantize(x, mx4.allocate(fmt, rows, K, groups, off))
    w = mx4.quantize_weight(torch.randn(groups, 2 * I, K, device="cuda", generator=g) * 0.02, fmt)
    d = mx4.quantize_weight(torch.randn(groups, K, I, device="cuda", generator=g) * 0.02, fmt)
    if what == "ffn":
        out, ws = torch.empty(rows, K, device="cuda"), mx4.ffn_workspace(a, w)
        call = lambda: mx4.grouped_ffn(a, w, d, out, ws)                                        # noqa: E731
    else:
        out = torch.empty(rows, 2 * I, device="cuda", dtype=torch.bfloat16 if what == "bf16" else torch.float32)
        ws = mx4.gemm_workspace()
        call = lambda: mx4.grouped_gemm(a, w, out, ws)                                          # noqa: E731
    call()
    assert abi.read_device_status(ws) == 0
    want = out.clone()
    took = stalled(PRODUCT, call)
    assert abi.read_device_status(ws) == -7 and 1.5 < took < 8, took
    call()
    assert abi.read_device_status(ws) == 0 and torch.equal(out, want)
