"""The 4-bit layer and the norms as a program runs them: a whole block against float64, captured
into a graph and replayed, on another stream, and several at once."""
import pytest
import torch

import mx4_reference as ref
from mixture_experts_layer_29_b200 import abi, mx4, norm
from mixture_experts_layer_29_b200 import workloads as wl
from test_gpu_mx4 import BF16_HALF, ffn_reference

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def small(T, n_ffn=12, n_zero=4, K=3, H=256, I=128):
    return wl.CONFIGS["proxy_bf16"].with_(T=T, H=H, I=I, n_ffn=n_ffn, n_zero=n_zero, K=K, w_std=0.06)


def scales(fmt):
    if fmt == "mxfp4":
        return None, None, None
    one = lambda v: torch.full((1,), v, device="cuda")     # noqa: E731
    return one(2.0 ** -7), one(2.0 ** -9), 2.0 ** -11


def make_layer(cfg, fmt, combine, seed=0):
    w = wl.draw_weights(cfg, "cuda", seed=seed)
    tx, th, tw = scales(fmt)
    tw = None if tw is None else torch.full((cfg.n_ffn,), tw, device="cuda")
    layer = mx4.Mx4MoELayer(abi.shape_of(cfg, combine), w.w_router, w.bias, mx4.quantize_weight(w.w_gate_up, fmt, tw),
                            mx4.quantize_weight(w.w_down, fmt, tw), abi.Pid(0.01, 0.001, 0.0, 0.6), tx, th)
    return layer, w


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T", [1, 37, 400])
def test_layer_against_float64(cuda_device, fmt, T):
    cfg = small(T)
    det, w = make_layer(cfg, fmt, "deterministic")
    x = wl.draw_tokens(cfg, "cuda")
    out, idx, gate, counts, hist = det.forward(x)
    out = out.clone()
    assert abi.read_device_status(det.ws) == 0 and abi.read_device_status(det.scratch) == 0
    # the routing is the bf16 layer's
    plain = abi.MoELayer(abi.shape_of(cfg, "deterministic"), w.w_router, w.bias, w.w_gate_up, w.w_down)
    _, pidx, pgate, pcounts, _ = plain.forward(x)
    assert torch.equal(idx, pidx) and torch.equal(gate, pgate) and torch.equal(counts, pcounts)
    off = det.offsets.tolist()
    R = off[-1]
    tx, th, tw = scales(fmt)
    per = 1.0 if tw is None else torch.full((cfg.n_ffn, 1, 1), tw, device="cuda")
    gu = ref.quantize(w.w_gate_up, fmt, per)[2]
    y, tol, _ = ffn_reference(x[det.perm_token[:R].long()], gu[:, :cfg.I], gu[:, cfg.I:],
                              ref.quantize(w.w_down, fmt, per)[2], off, fmt, tx, th, tw)
    ty = tol * (1 + BF16_HALF) + y.abs() * BF16_HALF
    assert ((det.y[:R].double() - y).abs() <= ty).all()
    # the combine of the rows that the layer stored: K + 1 fp32 additions, rounded to bf16
    want = det.zgate.double()[:, None] * x.double()
    mag = want.abs()
    for k in range(cfg.K):
        r = det.row_of.view(T, cfg.K)[:, k].long()
        term = torch.where((r >= 0)[:, None], gate[:, k].double()[:, None] * det.y[r.clamp(min=0)].double(), 0.0)
        want, mag = want + term, mag + term.abs()
    assert ((out.double() - want).abs() <= want.abs() * BF16_HALF + mag * (cfg.K + 3) * U).all()
    # the fused combine adds unrounded rows
    fus, _ = make_layer(cfg, fmt, "fused")
    of = fus.forward(x)[0]
    terms = torch.zeros_like(want)
    for k in range(cfg.K):
        r = det.row_of.view(T, cfg.K)[:, k].long()
        terms += torch.where((r >= 0)[:, None], gate[:, k].double()[:, None] * det.y[r.clamp(min=0)].double().abs(), 0.0)
    assert ((of.double() - want).abs() <= want.abs() * 1.01 * BF16_HALF + terms * 1.01 * BF16_HALF + mag * (cfg.K + 4) * U).all()
    stats = det.update_bias()
    assert torch.isfinite(stats).all()


def test_tokens_that_pick_identity_experts_only(cuda_device):
    cfg = small(24)
    layer, _ = make_layer(cfg, "mxfp4", "fused")
    layer.bias.zero_()          # selection adds it to p: 0.1 would beat a small p of an identity expert
    x = wl.draw_tokens(cfg, "cuda")
    logits = wl.draw_forced_logits(24, cfg.n_ffn, cfg.n_zero, range(24), "cuda")
    out = layer.forward(x, logits)[0]
    assert int(layer.offsets[-1]) == 0
    want = layer.zgate[:, None] * x.float()
    assert torch.equal(out, want.to(torch.bfloat16))


def make_block(cfg, fmt="mxfp4", seed=0):
    layer, w = make_layer(cfg, fmt, "deterministic", seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 50)
    vec = lambda n: torch.randn(n, device="cuda", generator=g) * 0.1 + 1.0     # noqa: E731
    blk = norm.MoEBlock(layer, vec(cfg.H), vec(cfg.H), vec(cfg.T), "token", 1e-5, 0.5)
    return blk, vec(cfg.H)


def test_two_blocks_in_a_row(cuda_device):
    """Each block's norm after it is joined with the norm before the next one: the same bits as
    norms of their own, and the residual stream against float64 of the layers' outputs."""
    cfg = small(33)
    a, wb = make_block(cfg, seed=1)
    b, wn = make_block(cfg, seed=2)
    b.w_pre = wb
    res = wl.draw_tokens(cfg, "cuda", seed=9)
    r1, n1 = a.forward(res, b.w_pre)
    r2, n2 = b.forward(r1, wn, normed=n1)
    # the same with separate norms
    c, _ = make_block(cfg, seed=2)
    c.w_pre = wb
    r3, none = c.forward(r1.clone())
    assert none is None and torch.equal(r3, r2)
    out = b.layer.out.double()
    n = b.w_post.double() * out * torch.rsqrt((out * out).mean(1, keepdim=True) + 1e-5)
    add = 0.5 * b.gate.double()[:, None] * n
    want = r1.double() + add
    assert ((r2.double() - want).abs() <= want.abs() * (BF16_HALF + U) + add.abs() * 44 * U).all()
    q = r2.double()
    n = wn.double() * q * torch.rsqrt((q * q).mean(1, keepdim=True) + 1e-5)
    assert ((n2.double() - n).abs() <= n.abs() * (BF16_HALF * 1.01 + 44 * U)).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_captured_block_replays_on_new_inputs(cuda_device, fmt):
    cfg = small(64)
    blk, wn = make_block(cfg, fmt)
    res = wl.draw_tokens(cfg, "cuda", seed=1)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        blk.forward(res, wn)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, n = blk.forward(res, wn)
    for seed in (2, 3, 2):
        res.copy_(wl.draw_tokens(cfg, "cuda", seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        got = r.clone(), n.clone()
        want = blk.forward(res, wn)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_backward_replays(cuda_device):
    T, H = 77, 512
    d = norm.make_desc(T, H, "bf16", "channel", 1e-5, 0.5)
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = lambda: torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)     # noqa: E731
    vec = lambda n: torch.randn(n, device="cuda", generator=g)                          # noqa: E731
    x, b, wp, ga, wn = rows(), rows(), vec(H), vec(H), vec(H)
    res, n, rb, rr = rows(), rows(), vec(T), vec(T)
    dr, dn = rows(), rows()
    outs = [rows(), rows(), vec(H), vec(H), vec(H)]
    ws = norm.workspace(d)

    def step():
        norm.block_norm(d, x, b, wp, ga, wn, res, n, rb, rr)
        norm.block_norm_backward(d, dr, dn, res, b, wp, ga, wn, rb, rr, *outs, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    b.copy_(rows())
    for o in outs:
        o.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    step()
    assert all(torch.equal(u, v) for u, v in zip(got, outs))


def test_streams_and_calls_at_once(cuda_device):
    """Two products on two streams, each with its own workspace, and a layer on a third, against
    the same calls one after another."""
    fmt, groups, H, I = "nvfp4", 6, 512, 256
    counts = [70, 0, 1, 200, 9, 64]
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    wgu = mx4.quantize_weight(torch.randn(groups, 2 * I, H, device="cuda", generator=g) * 0.05, fmt)
    wd = mx4.quantize_weight(torch.randn(groups, H, I, device="cuda", generator=g) * 0.05, fmt)
    xs = [torch.randn(off[-1], H, device="cuda", generator=g) for _ in range(3)]
    mats = [mx4.allocate(fmt, off[-1], H, groups, o) for _ in xs]
    wss = [mx4.ffn_workspace(m, wgu) for m in mats]
    outs = [torch.empty(off[-1], H, device="cuda") for _ in xs]
    want = []
    for x, m, ws, out in zip(xs, mats, wss, outs):
        mx4.quantize(x, m)
        want.append(mx4.grouped_ffn(m, wgu, wd, out, ws).clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for out in outs:
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for x, m, ws, out, st in zip(xs, mats, wss, outs, streams):
            mx4.quantize(x, m, stream=st)                      # named, not the current one
            mx4.grouped_ffn(m, wgu, wd, out, ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert all(abi.read_device_status(ws) == 0 for ws in wss)


def test_python_refuses_wrong_tensors(cuda_device):
    m = mx4.allocate("mxfp4", 8, 256)
    x = torch.zeros(8, 256, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        mx4.quantize(x[:7], m)
    with pytest.raises(ValueError, match="adjacent"):
        mx4.quantize(torch.zeros(256, 8, device="cuda").T, m)
    with pytest.raises(ValueError, match="cpu"):
        mx4.quantize(x.cpu(), m)
    with pytest.raises(ValueError, match="float16"):
        mx4.quantize(x.half(), m)
    with pytest.raises(abi.MoEError, match="ALIGNMENT"):
        mx4.quantize(torch.zeros(8, 258, device="cuda")[:, :256], m)
    w = mx4.quantize_weight(torch.zeros(1, 128, 256, device="cuda"), "mxfp4")
    with pytest.raises(ValueError, match="out"):
        mx4.grouped_gemm(m, w, torch.zeros(8, 127, device="cuda"), mx4.gemm_workspace())
    with pytest.raises(abi.MoEError, match="WORKSPACE"):
        mx4.grouped_gemm(m, w, torch.zeros(8, 128, device="cuda"), mx4.gemm_workspace()[:16])
    d = norm.make_desc(4, 256)
    e = torch.zeros(4, 256, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="normed"):
        norm.block_norm(d, e, None, None, None, torch.ones(256, device="cuda"), None, e[:3])
    with pytest.raises(abi.MoEError, match="INVALID"):
        norm.block_norm(d, e, None, None, None, None, None, None)
    cfg = small(8)
    with pytest.raises(ValueError, match="bf16 layer"):
        mx4.Mx4MoELayer(abi.make_shape(8, 256, 128, 12, 4, 3, "fp32"), None, None, None, None)
    with pytest.raises(ValueError, match="w_gate_up"):
        mx4.Mx4MoELayer(abi.shape_of(cfg), None, None, w, w)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("counts,H,I", [([1500, 3, 0, 2200, 700, 1100], 1536, 1024), ([40, 64, 1, 0, 13, 30] * 8, 1536, 1024)])
def test_calls_back_to_back_agree(cuda_device, fmt, counts, H, I):
    """Launches that overlap their predecessors' ends, with nothing between them: every one gives the
    first one's bits, captured and not. Six and four stages per tile, more tiles than CTAs."""
    groups = len(counts)
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(off[-1], H, device="cuda", generator=g).to(torch.bfloat16)
    wgu = mx4.quantize_weight(torch.randn(groups, 2 * I, H, device="cuda", generator=g) * 0.05, fmt)
    wd = mx4.quantize_weight(torch.randn(groups, H, I, device="cuda", generator=g) * 0.05, fmt)
    a = mx4.allocate(fmt, off[-1], H, groups, o)
    ws, wg = mx4.ffn_workspace(a, wgu), mx4.gemm_workspace()
    first = torch.empty(off[-1], H, dtype=torch.bfloat16, device="cuda")
    gu = torch.empty(off[-1], 2 * I, dtype=torch.bfloat16, device="cuda")
    mx4.quantize(x, a)
    mx4.grouped_ffn(a, wgu, wd, first, ws)
    mx4.grouped_gemm(a, wgu, gu, wg)
    torch.cuda.synchronize()
    outs = [torch.zeros_like(first) for _ in range(24)]
    gus = [torch.zeros_like(gu) for _ in range(8)]

    def step():
        for i, out in enumerate(outs):
            if i % 3 == 0:
                mx4.quantize(x, a)
            mx4.grouped_ffn(a, wgu, wd, out, ws)
        for out in gus:
            mx4.grouped_gemm(a, wgu, out, wg)

    step()
    torch.cuda.synchronize()
    assert all(torch.equal(out, first) for out in outs) and all(torch.equal(out, gu) for out in gus)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for out in outs + gus:
        out.zero_()
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, first) for out in outs) and all(torch.equal(out, gu) for out in gus)
    assert abi.read_device_status(ws) == 0 and abi.read_device_status(wg) == 0


@pytest.mark.parametrize("T,H,dtype", [(900, 6144, "bf16"), (2000, 768, "fp32"), (700, 8192, "fp32")])
def test_norm_gradients_back_to_back_agree(cuda_device, T, H, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    d = norm.make_desc(T, H, dtype, "token", 1e-5, 0.5)
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = lambda: torch.randn(T, H, device="cuda", generator=g).to(dt)     # noqa: E731
    vec = lambda n: torch.rand(n, device="cuda", generator=g) + 0.5        # noqa: E731
    args = [rows(), rows(), rows(), rows(), vec(H), vec(T), vec(H), vec(T), vec(T)]
    outs = [[torch.zeros_like(args[0]), torch.zeros_like(args[0]), vec(H), vec(T), vec(H)] for _ in range(20)]
    ws = norm.workspace(d)
    for o in outs:
        norm.block_norm_backward(d, *args, *o, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for o in outs for u, v in zip(o, outs[0]))
    assert abi.read_device_status(ws) == 0
