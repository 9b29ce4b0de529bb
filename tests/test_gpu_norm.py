"""The block norms on the GPU against float64, their gradients against the formula's and against
differences, and one call against two."""
import pytest
import torch

from mixture_experts_layer_29_b200 import norm

pytestmark = pytest.mark.gpu
EPS = 1e-5
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24                      # half a step of fp32, relative


def draw(T, H, dtype, gate, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + T + H)

    def rows(std):
        return (torch.randn(T, H, device="cuda", generator=g) * std).to(dtype)

    def vec(n, mean):
        return torch.randn(n, device="cuda", generator=g) * 0.2 + mean

    s = dict(residual=rows(2.0), block=rows(0.5), w_post=vec(H, 1.0), w_pre=vec(H, 1.0),
             gate={"none": None, "token": vec(T, 0.5), "channel": vec(H, 0.5)}[gate],
             d_res=rows(1.0), d_norm=rows(1.0))
    if T > 1:
        s["block"][0] = 0.0                            # a norm of nothing
    return s


def name(dtype):
    return "bf16" if dtype == torch.bfloat16 else "fp32"


def gate64(gate, kind):
    if gate is None:
        return 1.0
    return gate.double()[:, None] if kind == "token" else gate.double()[None, :]


def run(d, s, dtype, post=True, pre=True, block=True):
    e = lambda: torch.empty(d.T, d.H, dtype=dtype, device="cuda")  # noqa: E731
    v = lambda: torch.empty(d.T, device="cuda")                    # noqa: E731
    o = dict(res=e() if block else None, n=e() if pre else None,
             rb=v() if block and post else None, rr=v() if pre else None)
    norm.block_norm(d, s["residual"], s["block"] if block else None, s["w_post"] if block and post else None,
                    s["gate"] if block else None, s["w_pre"] if pre else None, o["res"], o["n"], o["rb"], o["rr"])
    return o


def rms(x):
    return torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


SHAPES = [(1, 128), (3, 16), (37, 768), (5, 6144), (2, 8208), (4, 8192), (3, 16384), (300, 1040), (700, 768)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_forward(cuda_device, T, H, dtype, gate):
    s = draw(T, H, dtype, gate)
    d = norm.make_desc(T, H, name(dtype), gate, EPS, 0.5)
    o = run(d, s, dtype)
    b = s["block"].double()
    n1 = s["w_post"].double() * b * rms(b)
    add = 0.5 * gate64(s["gate"], gate) * n1
    r = s["residual"].double() + add
    # rstd: a sum of H squares (each thread adds at most 32, then two butterflies: 48 roundings),
    # halved by the square root, and 4 roundings; then 5 products and one sum
    tol = (add.abs() * 40 * U + r.abs() * U) * 1.01 + r.abs() * HALF[dtype]
    assert ((o["res"].double() - r).abs() <= tol).all()
    q = o["res"].double()                      # n2 is the norm of the stream as it is stored
    n2 = s["w_pre"].double() * q * rms(q)
    tol = n2.abs() * (40 * U * 1.01 + HALF[dtype])
    assert ((o["n"].double() - n2).abs() <= tol).all()
    assert ((o["rb"].double() - rms(b)[:, 0]).abs() <= rms(b)[:, 0] * 32 * U).all()
    assert ((o["rr"].double() - rms(q)[:, 0]).abs() <= rms(q)[:, 0] * 32 * U).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_call_is_two_calls_and_in_place(cuda_device, dtype):
    T, H = 19, 784
    s = draw(T, H, dtype, "channel")
    d = norm.make_desc(T, H, name(dtype), "channel", EPS, 0.7)
    o = run(d, s, dtype)
    first = run(d, s, dtype, pre=False)
    assert torch.equal(first["res"], o["res"])
    plain = norm.make_desc(T, H, name(dtype), "none", EPS, 1.0)
    n, rr = torch.empty_like(o["n"]), torch.empty_like(o["rr"])
    norm.block_norm(plain, first["res"], None, None, None, s["w_pre"], None, n, None, rr)
    assert torch.equal(n, o["n"]) and torch.equal(rr, o["rr"])
    res = s["residual"].clone()
    norm.block_norm(d, res, s["block"], s["w_post"], s["gate"], s["w_pre"], res, n)
    assert torch.equal(res, o["res"]) and torch.equal(n, o["n"])


def backward(d, s, o, dtype, post=True, pre=True, block=True, d_res=True, ws=None):
    T, H = d.T, d.H
    e = lambda: torch.full((T, H), 9.0, dtype=dtype, device="cuda")      # noqa: E731
    v = lambda n: torch.full((n,), 9.0, device="cuda")                   # noqa: E731
    gate = s["gate"] if block else None
    g = dict(d_residual=e(), d_block=e() if block else None, d_w_post=v(H) if block and post else None,
             d_gate=None if gate is None else v(gate.numel()), d_w_pre=v(H) if pre else None)
    norm.block_norm_backward(d, s["d_res"] if d_res else None, s["d_norm"] if pre else None,
                             (o["res"] if block else s["residual"]) if pre else None, s["block"] if block else None,
                             s["w_post"] if block and post else None, gate, s["w_pre"] if pre else None, o["rb"], o["rr"],
                             g["d_residual"], g["d_block"], g["d_w_post"], g["d_gate"], g["d_w_pre"],
                             norm.workspace(d) if ws is None else ws)
    return g


def formula(d, s, o, gate, scale, post=True, pre=True, block=True, d_res=True):
    """The gradients in float64 and, for each, the sum of the magnitudes that went into it."""
    H = d.H
    out, mag = {}, {}
    g = s["d_res"].double() if d_res else torch.zeros_like(s["d_norm"].double())
    m = g.abs()
    if pre:
        x, r, dn = (o["res"] if block else s["residual"]).double(), o["rr"].double()[:, None], s["d_norm"].double()
        xh, c = x * r, dn * s["w_pre"].double()
        g = g + r * (c - xh * (c * xh).mean(1, keepdim=True))
        m = m + r * (c.abs() + xh.abs() * (c * xh).abs().mean(1, keepdim=True))
        out["d_w_pre"], mag["d_w_pre"] = (dn * xh).sum(0), (dn * xh).abs().sum(0)
    out["d_residual"], mag["d_residual"] = g, m
    if block:
        b = s["block"].double()
        rb = o["rb"].double()[:, None] if post else 1.0
        wp = s["w_post"].double() if post else 1.0
        bh, gt = b * rb, scale * gate64(s["gate"], gate)
        up, mup = g * gt, m * abs(gt) if isinstance(gt, float) else m * gt.abs()
        if post:
            out["d_w_post"], mag["d_w_post"] = (up * bh).sum(0), (mup * bh.abs()).sum(0)
        if s["gate"] is not None:
            by = 1 if gate == "token" else 0
            out["d_gate"], mag["d_gate"] = scale * (g * bh * wp).sum(by), abs(scale) * (m * (bh * wp).abs()).sum(by)
        c, mc = up * wp, mup * (wp.abs() if post else 1.0)
        if post:
            out["d_block"] = rb * (c - bh * (c * bh).mean(1, keepdim=True))
            mag["d_block"] = rb * (mc + bh.abs() * (mc * bh.abs()).mean(1, keepdim=True))
        else:
            out["d_block"], mag["d_block"] = c, mc
    return out, mag


def check(got, want, mag, dtype, T):
    for k, w in want.items():
        v = got[k]
        # sums over H: 48 roundings, sums over T: at most T plus the CTAs' partial sums; a
        # dozen products and sums of the terms besides
        n = 140 + (T if v.dim() == 1 else 0)
        tol = mag[k] * n * U + (w.abs() * HALF[dtype] if v.dim() == 2 else w.abs() * U)
        assert ((v.double() - w).abs() <= tol * 1.01).all(), (k, ((v.double() - w).abs() / tol).max())
    for k, v in got.items():
        assert (v is None) == (k not in want), k


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_backward_is_the_formula(cuda_device, T, H, dtype, gate):
    s = draw(T, H, dtype, gate)
    d = norm.make_desc(T, H, name(dtype), gate, EPS, 0.5)
    o = run(d, s, dtype)
    got = backward(d, s, o, dtype)
    want, mag = formula(d, s, o, gate, 0.5)
    check(got, want, mag, dtype, T)
    again = backward(d, s, o, dtype)
    assert all(v is None or torch.equal(v, again[k]) for k, v in got.items())


@pytest.mark.parametrize("parts", [dict(post=False), dict(pre=False), dict(block=False), dict(d_res=False),
                                   dict(post=False, pre=False), dict(block=False, d_res=False)])
@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_parts_left_out(cuda_device, parts, gate):
    T, H, dtype = 21, 528, torch.bfloat16
    block, post, pre = parts.get("block", True), parts.get("post", True), parts.get("pre", True)
    if not block and gate != "none":
        gate = "none"
    s = draw(T, H, dtype, gate)
    d = norm.make_desc(T, H, "bf16", gate, EPS, 0.5)
    o = run(d, s, dtype, post, pre, block)
    if block and not post:
        add = 0.5 * gate64(s["gate"], gate) * s["block"].double()
        r = s["residual"].double() + add
        assert ((o["res"].double() - r).abs() <= r.abs() * HALF[dtype] + 4 * U * (add.abs() + r.abs())).all()
    got = backward(d, s, o, dtype, post, pre, block, parts.get("d_res", True))
    want, mag = formula(d, s, o, gate, 0.5, post, pre, block, parts.get("d_res", True))
    check(got, want, mag, dtype, T)


def test_backward_against_differences(cuda_device):
    """d/de of <d_res, res> + <d_norm, n2> along random directions, by central differences in
    float64 of the forward's formula, fp32 operator."""
    T, H, dtype = 6, 64, torch.float32
    s = draw(T, H, dtype, "channel")
    d = norm.make_desc(T, H, "fp32", "channel", EPS, 0.5)
    o = run(d, s, dtype)
    got = backward(d, s, o, dtype)

    def loss(p):
        b = p["block"]
        r = p["residual"] + 0.5 * p["gate"][None] * p["w_post"] * b * rms(b)
        return (s["d_res"].double() * r).sum() + (s["d_norm"].double() * p["w_pre"] * r * rms(r)).sum()

    p = {k: s[k].double() for k in ("residual", "block", "w_post", "w_pre", "gate")}
    p["block"][0] = s["block"][0] = 0.25 * torch.randn(H, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    o = run(d, s, dtype)
    got = backward(d, s, o, dtype)
    p["block"] = s["block"].double()
    for k in p:
        u = torch.randn(p[k].shape, device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(3))
        h = 1e-5
        num = (loss({**p, k: p[k] + h * u}) - loss({**p, k: p[k] - h * u})) / (2 * h)
        ana = (got["d_" + k].double() * u).sum()
        mag = (got["d_" + k].double() * u).abs().sum()
        # fp32 gradients (140 roundings of their terms, whose cancellation a factor 8 covers)
        # and the differences' own h^2 term
        assert (num - ana).abs() <= mag * (140 * 8 * U + 1e-7), k


def test_no_tokens(cuda_device):
    d = norm.make_desc(0, 256, "bf16", "channel", EPS, 1.0)
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(0, device="cuda")
    w = torch.ones(256, device="cuda")
    norm.block_norm(d, e, e, w, w, w, e, e, v, v)
    sums = [torch.full((256,), 5.0, device="cuda") for _ in range(3)]
    norm.block_norm_backward(d, e, e, e, e, w, w, w, v, v, e, e, sums[0], sums[1], sums[2], norm.workspace(d))
    assert all((x == 0).all() for x in sums)


@pytest.mark.parametrize("T,H", [(301, 6160), (160, 8192), (151, 8208), (149, 12288), (7, 12304), (150, 16384),
                                 (2047, 2048), (2048, 2048), (2100, 1040), (2050, 4096), (2049, 3344)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["token", "channel"])
def test_backward_of_wide_rows_and_several_tokens_per_block(cuda_device, T, H, dtype, gate):
    """Widths on both sides of the ones at which threads hold one vector more, or rows stop going
    through shared memory; more tokens than the card has SMs."""
    test_backward_is_the_formula(None, T, H, dtype, gate)


def test_offsets_past_32_bits(cuda_device):
    """More than 2^31 elements: the last tokens' rows are those of a small batch of them."""
    T, H, last = 351_000, 6144, 400          # more than two tokens per SM: the same CTAs for both
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(H, device="cuda", generator=g) + 1.0
    z = lambda: torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")      # noqa: E731
    ins = [z() for _ in range(4)]                                           # residual, block, their gradients
    for x in ins:
        x[-last:] = torch.randn(last, H, device="cuda", generator=g).to(torch.bfloat16)
    results = []
    for n in (T, last):
        d = norm.make_desc(n, H, "bf16", "none", EPS, 0.5)
        res, blk, d_res, d_norm = (x[-n:].contiguous() for x in ins)
        e = lambda: torch.empty(n, H, dtype=torch.bfloat16, device="cuda")  # noqa: E731, B023
        v = lambda: torch.empty(n, device="cuda")                           # noqa: E731, B023
        out, normed, rb, rr, dr, db = e(), e(), v(), v(), e(), e()
        norm.block_norm(d, res, blk, w, None, w, out, normed, rb, rr)
        dw, dp = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        norm.block_norm_backward(d, d_res, d_norm, out, blk, w, None, w, rb, rr, dr, db, dw, None, dp, norm.workspace(d))
        results.append([x[-last:].clone() for x in (out, normed, dr, db)] + [bool(x[:-last].any()) for x in (out, normed, dr, db)])
        del res, blk, d_res, d_norm, out, normed, dr, db
    for a, b in zip(results[0][:4], results[1][:4]):
        assert torch.equal(a, b)
    assert not any(results[0][4:])
    del ins
    torch.cuda.empty_cache()
