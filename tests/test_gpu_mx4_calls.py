"""Calls of the 4-bit operators that the documentation allows and that stand apart from the usual ones:
uniform groups, the most groups and picks, a layer with an output scale."""
import pytest
import torch

import mx4_reference as ref
from mixture_experts_layer_29_b200 import abi, mx4
from mixture_experts_layer_29_b200 import workloads as wl
from test_gpu_block import make_layer, small
from test_gpu_mx4 import BF16_HALF, dev, factor, gen, offsets_of, small_checkpoint

pytestmark = pytest.mark.gpu
FORMATS = ["mxfp4", "nvfp4"]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("groups,each", [(3, 1), (5, 40), (2, 300), (4, 192), (1, 70)])
def test_uniform_groups_of_rows(cuda_device, fmt, groups, each):
    """Groups without offsets: the same bits as with them, through every call."""
    H, I, rows = 256, 128, groups * each
    x = torch.randn(rows, H, device="cuda", generator=gen(rows)).to(torch.bfloat16)
    t = factor(fmt)
    off = dev([g * each for g in range(groups + 1)])
    a, b = mx4.allocate(fmt, rows, H, groups, None, t), mx4.allocate(fmt, rows, H, groups, off, t)
    for m in (a, b):
        m.scales.zero_()
        mx4.quantize(x, m)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    w = mx4.quantize_weight(torch.randn(groups, 2 * I, H, device="cuda", generator=gen(1)), fmt)
    d = mx4.quantize_weight(torch.randn(groups, H, I, device="cuda", generator=gen(2)), fmt)
    out = []
    for m in (a, b):
        y, z, v = (torch.empty(rows, n, device="cuda") for n in (2 * I, H, H))
        ws = mx4.ffn_workspace(m, w)
        mx4.grouped_gemm(m, w, y, ws)
        mx4.grouped_ffn(m, w, d, z, ws)
        mx4.dequantize(m, v)
        assert abi.read_device_status(ws) == 0
        out.append((y, z, v))
    assert all(torch.equal(p, q) for p, q in zip(*out))
    # and by picks: row t of x to the row of its own number, and to none
    c = mx4.allocate(fmt, rows, H, groups, None, t)
    c.scales.zero_()
    row_of = torch.stack([torch.arange(rows), torch.full((rows,), -1)], 1).to(torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx4.quantize(x, c, row_of, status)
    assert torch.equal(a.codes, c.codes) and torch.equal(a.scales, c.scales) and int(status) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [[0] * 1023 + [5], [2] + [0] * 511 + [90] + [0] * 511, [1, 0, 3, 0] * 256, [70] * 1024])
def test_the_most_groups_are_exact(cuda_device, fmt, counts):
    groups, off, N, K = 1024, offsets_of(counts), 136, 256
    code, byte, a = small_checkpoint((off[-1], K), fmt, 3)
    wc, wb, w = small_checkpoint((groups, N, K), fmt, 4)
    m = mx4.allocate(fmt, off[-1] + 3, K, groups, dev(off))
    m.codes[: off[-1]] = ref.pack(code)
    m.codes[off[-1]:] = 0x77
    m.scales.fill_(0xFF)                        # NaN wherever a row's scale is not
    m.scales[ref.scale_index(off, K, fmt, "cuda")] = byte
    out = torch.full((off[-1] + 3, N), 3.0, device="cuda")
    ws = mx4.gemm_workspace()
    mx4.grouped_gemm(m, mx4.from_checkpoint(fmt, ref.pack(wc), wb), out, ws)
    y, _ = ref.grouped(a, w, off)
    assert abi.read_device_status(ws) == 0 and torch.equal(out[: off[-1]].double(), y) and bool((out[off[-1]:] == 3.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_tokens_with_the_most_picks(cuda_device, fmt):
    """32 picks of 1024 groups: every one gets the token's row."""
    tokens, picks, K, groups = 9, 32, 384, 1024
    g = torch.Generator().manual_seed(2)
    expert = torch.stack([torch.randperm(groups, generator=g)[:picks] for _ in range(tokens)])
    flat, order = expert.flatten().sort(stable=True)
    row_of = torch.empty(tokens * picks, dtype=torch.int32)
    row_of[order] = torch.arange(tokens * picks, dtype=torch.int32)
    off = offsets_of(torch.bincount(flat, minlength=groups).tolist())
    x = torch.randn(tokens, K, device="cuda", generator=gen(3))
    a, b = (mx4.allocate(fmt, tokens * picks, K, groups, dev(off)) for _ in range(2))
    for m in (a, b):
        m.scales.zero_()
    mx4.quantize(x, a, row_of.view(tokens, picks).cuda())
    mx4.quantize(x[(order // picks).cuda()], b)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("combine", ["fused", "deterministic"])
@pytest.mark.parametrize("scale", [2.5, 0.0])
def test_layer_with_an_output_scale(cuda_device, fmt, combine, scale):
    cfg = small(50).with_(ffn_out_scale=scale)
    plain, _ = make_layer(cfg.with_(ffn_out_scale=1.0), fmt, "deterministic")
    layer, _ = make_layer(cfg, fmt, combine)
    x = wl.draw_tokens(cfg, "cuda")
    out, idx, gate, _, _ = layer.forward(x)
    plain.forward(x)
    want = layer.zgate.double()[:, None] * x.double()
    mag = want.abs()
    for k in range(cfg.K):
        r = plain.row_of.view(50, cfg.K)[:, k].long()
        term = torch.where((r >= 0)[:, None], scale * gate[:, k].double()[:, None] * plain.y[r.clamp(min=0)].double(), 0.0)
        want, mag = want + term, mag + term.abs()
    # rows rounded to bf16 in `plain`, sums in fp32 in any order, the result rounded to bf16
    tol = want.abs() * 1.01 * BF16_HALF + mag * (1.01 * BF16_HALF + (cfg.K + 4) * 2.0 ** -24)
    assert bool(((out.double() - want).abs() <= tol).all())
