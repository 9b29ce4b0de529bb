"""The grouped FFN where each CTA, or pair, has several tiles: the accumulators take turns, the rings of
operands and scales go round, and the staging rows of the epilogue are used again."""
import pytest
import torch

import mx4_reference as ref
from mixture_experts_layer_29_b200 import abi, mx4
from test_gpu_mx4 import BF16_HALF, dev, factor, ffn_reference, gen, offsets_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("counts", [[1500, 3, 0, 2200, 700, 1100],       # pairs: 31 x 8 tiles for at most 74
                                    [40, 64, 1, 0, 13, 30] * 8])         # 40 x 8 tiles for 148 CTAs
def test_ffn_of_many_tiles(cuda_device, fmt, counts):
    H, I = 2048, 1024                                                    # eight stages; four for the down product
    groups, off = len(counts), offsets_of(counts)
    rows = off[-1]
    t, th, tw = factor(fmt, 1, 2.0 ** -7), factor(fmt, 1, 2.0 ** -9), factor(fmt, groups, 2.0 ** -11)
    per = 1.0 if tw is None else tw[:, None, None]
    x = torch.randn(rows, H, device="cuda", generator=gen(7)).to(torch.bfloat16)
    wgu = torch.randn(groups, 2 * I, H, device="cuda", generator=gen(8)) * H ** -0.5
    wd = torch.randn(groups, H, I, device="cuda", generator=gen(9)) * I ** -0.5
    qg, qd = mx4.quantize_weight(wgu, fmt, tw), mx4.quantize_weight(wd, fmt, tw)
    a = mx4.quantize(x, mx4.allocate(fmt, rows, H, groups, dev(off), t))
    ws = mx4.ffn_workspace(a, qg)
    out = mx4.grouped_ffn(a, qg, qd, torch.empty(rows, H, device="cuda", dtype=torch.bfloat16), ws, th)
    assert abi.read_device_status(ws) == 0
    for g in range(groups):                                              # one group's weights at a time in 64 bits
        r = slice(off[g], off[g + 1])
        if not counts[g]:
            continue
        one = None if tw is None else tw[g:g + 1]
        gu = ref.quantize(wgu[g:g + 1], fmt, 1.0 if one is None else one)[2]
        y, tol, near = ffn_reference(x[r], gu[:, :I], gu[:, I:], ref.quantize(wd[g:g + 1], fmt, 1.0 if one is None else one)[2],
                                     [0, counts[g]], fmt, t, th, one)
        assert near < 1e-2
        tol = tol * (1 + BF16_HALF) + y.abs() * BF16_HALF
        bad = (out[r].double() - y).abs() > tol
        assert not bool(bad.any()), (g, int(bad.sum()), bad.nonzero()[:4].tolist())
