"""Workloads of the 4-bit expert operators and of the block norms: inputs, plain forms and
64-bit results.

  quantize   rows of bf16 or fp32 to microscaled 4 bits and back (mx4.quantize, mx4.dequantize)
  product    y[r] = A[r] . W[g]^T by ragged group, both operands in microscaled 4 bits; the
             bf16 rows are quantised inside the call (mx4.quantize, mx4.grouped_gemm)
  ffn        the grouped SwiGLU FFN on 4-bit experts (mx4.quantize, mx4.grouped_ffn)
  norm       the norms after one block and before the next, with the block's gate and the
             residual scale (norm.block_norm)
  norm_grad  its gradients (norm.block_norm_backward)

Formats. A row is split into blocks that share a scale; an element is an e2m1 number
(0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), rounded to nearest, ties to even, at most 6.
  mxfp4  blocks of 32, the scale a power of two: 2^(floor(log2(max |x|)) - 2)
  nvfp4  blocks of 16, the scale e4m3(max |x| / (6 t)) * t with a given fp32 factor t
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"mxfp4": 32, "nvfp4": 16}
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


# ---- cases ---------------------------------------------------------------------------------

def listed():
    full = {"H": 6144, "I": 2048}
    return [
        # the activations of a decode batch on their way into 4-bit experts
        {"name": "quantize_decode", "op": "quantize", "fmt": "mxfp4", "dtype": "bf16",
         "rows": 128, "K": 6144},
        # a prefill batch's activations
        {"name": "quantize_prefill", "op": "quantize", "fmt": "nvfp4", "dtype": "bf16",
         "rows": 8192, "K": 6144},
        # one token's picks: one row in each of a few experts, the smallest step of serving
        {"name": "product_one_token", "op": "product", "fmt": "mxfp4", "rows": 8, "groups": 64,
         "N": 4096, "K": 6144, "skew": 0.0},
        # the gate and up products of a decode batch, a few rows in most experts
        {"name": "product_decode", "op": "product", "fmt": "nvfp4", "rows": 863, "groups": 64,
         "N": 4096, "K": 6144, "skew": 1.0},
        # the 768-wide proxy layer's experts, ragged groups and empty ones
        {"name": "product_proxy", "op": "product", "fmt": "nvfp4", "rows": 17081, "groups": 64,
         "N": 512, "K": 768, "skew": 1.5},
        # a prefill batch on the experts of one layer that it loads most
        {"name": "product_prefill", "op": "product", "fmt": "mxfp4", "rows": 32768, "groups": 16,
         "N": 4096, "K": 6144, "skew": 0.5},
        # a decode step's experts, gate, up and down
        {"name": "ffn_decode", "op": "ffn", "fmt": "mxfp4", "rows": 437, "groups": 64, **full,
         "skew": 1.0},
        # a prefill chunk's experts
        {"name": "ffn_prefill", "op": "ffn", "fmt": "nvfp4", "rows": 16384, "groups": 16, **full,
         "skew": 0.5},
        # one token between two blocks of a served model
        {"name": "norm_one_token", "op": "norm", "dtype": "bf16", "T": 1, "H": 6144,
         "gate": "channel"},
        # a prefill or training batch between two blocks
        {"name": "norm_prefill", "op": "norm", "dtype": "bf16", "T": 8192, "H": 6144,
         "gate": "token"},
        # the proxy's training step in fp32, an odd number of tokens
        {"name": "norm_grad_proxy", "op": "norm_grad", "dtype": "fp32", "T": 1021, "H": 768,
         "gate": "token"},
        # a full-width training batch
        {"name": "norm_grad_train", "op": "norm_grad", "dtype": "bf16", "T": 8192, "H": 6144,
         "gate": "channel"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "ffn", "norm", "norm_grad"])
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op == "quantize":
        return {"op": op, "fmt": fmt, "dtype": rng.choice(["bf16", "fp32"]),
                "rows": _spread(rng, 1, 8192), "K": 128 * _spread(rng, 1, 48)}
    if op in ("norm", "norm_grad"):
        return {"op": op, "dtype": rng.choice(["bf16", "fp32"]), "T": _spread(rng, 1, 8192),
                "H": 16 * _spread(rng, 8, 384),
                "gate": rng.choice(["none", "token", "channel"])}
    groups = _spread(rng, 1, 64)
    width = 128 * _spread(rng, 2, 48)
    case = {"op": op, "fmt": fmt, "rows": 0, "groups": groups}
    if op == "product":
        case.update(N=_spread(rng, 128, 4096), K=width)
        most = 32768 * 16 / groups
    else:
        case.update(H=width, I=128 * _spread(rng, 1, 16))
        most = 16384 * 16 / groups
    case["rows"] = _spread(rng, 1, min(most, 16384))
    case["skew"] = round(rng.uniform(0.0, 1.5), 2)
    return case


# ---- the formats in elementary operations ---------------------------------------------------

def _bounds(device):
    """The values half way between two neighbours of the grid. One whose tie goes up to the
    even neighbour is lowered by one step, so that "boundary < value" counts the tie."""
    b = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=device)
    up = torch.tensor([0, 1, 0, 1, 0, 1, 0], dtype=torch.bool, device=device)
    return torch.where(up, torch.nextafter(b, torch.zeros_like(b)), b)


def _scales(x, fmt, t):
    """(scale bytes, scales as fp32) of the blocks of x [..., K] fp32."""
    amax = x.unflatten(-1, (-1, BLOCK[fmt])).abs().amax(-1)
    if fmt == "mxfp4":
        byte = ((amax.view(torch.int32) >> 23) - 2).clamp_(min=0)
        s = torch.where(byte > 0, byte << 23, 1 << 22).view(torch.float32)
        return byte.to(torch.uint8), s
    e = (amax / (6.0 * t)).clamp_(max=448.0).to(torch.float8_e4m3fn)
    return e.view(torch.uint8), e.float() * t


def _codes(x, fmt, t):
    """(4-bit codes one per byte [..., K], scale bytes [..., K / block]) of x fp32."""
    byte, s = _scales(x, fmt, t)
    q = x.unflatten(-1, (-1, BLOCK[fmt])) / s.unsqueeze(-1)
    q = torch.where(s.unsqueeze(-1) > 0, q, 0.0).flatten(-2)
    code = torch.bucketize(q.abs(), _bounds(x.device), out_int32=True).to(torch.uint8)
    return code | (torch.signbit(q).to(torch.uint8) << 3), byte


def _values(codes, byte, fmt, t):
    """fp32 values of packed codes [..., K / 2] (the even element in the low half) with scale
    bytes [..., K / block]."""
    g = torch.tensor(GRID, device=codes.device)
    one = torch.cat([g, -g])
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)
    v = pair[codes.int()].flatten(-2).unflatten(-1, (-1, BLOCK[fmt]))
    if fmt == "mxfp4":
        b = byte.int()
        s = torch.where(b > 0, b << 23, 1 << 22).view(torch.float32)
    else:
        s = byte.view(torch.float8_e4m3fn).float() * t
    return v.mul_(s.unsqueeze(-1)).flatten(-2)


def _round_trip(x, fmt, t):
    code, byte = _codes(x, fmt, t)
    return _values(code[..., 0::2] | (code[..., 1::2] << 4), byte, fmt, t)


def _pad(a, s):
    """The ragged rows a [R, K] as [groups, longest, K], zeros behind each group's rows."""
    p = torch.zeros(s["groups"], s["longest"], a.shape[1], dtype=a.dtype, device=a.device)
    p[s["group"], s["place"]] = a
    return p


def _by_group(a, w, s):
    return torch.bmm(_pad(a, s), w.transpose(1, 2))[s["group"], s["place"]]


# ---- inputs ---------------------------------------------------------------------------------

def _gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(int(seed) * 9176 + 11)


def _weight(gen, groups, n, k, fmt):
    """A 4-bit checkpoint's weight: packed codes [groups, n, k / 2], scale bytes
    [groups, n, k / block] and one fp32 factor per group (nvfp4)."""
    codes = torch.empty(groups, n, k // 2, dtype=torch.uint8, device="cuda")
    byte = torch.empty(groups, n, k // BLOCK[fmt], dtype=torch.uint8, device="cuda")
    t = torch.full((groups,), 2.0 ** -10, device="cuda") if fmt == "nvfp4" else None
    for g in range(groups):
        w = torch.empty(n, k, device="cuda").normal_(0.0, 0.02 / math.sqrt(8.0), generator=gen)
        c, byte[g] = _codes(w, fmt, t[g] if t is not None else 1.0)
        codes[g] = c[:, 0::2] | (c[:, 1::2] << 4)
    return {"codes": codes, "byte": byte, "t": t}


def _ragged(case, seed):
    """The groups' offsets on the device, and each row's group and place in it."""
    g, rows = case["groups"], case["rows"]
    gen = _gen(seed, "cpu")
    load = torch.exp(case["skew"] * torch.randn(g, generator=gen))
    pick = torch.multinomial(load / load.sum(), rows, replacement=True, generator=gen)
    if rows <= g:  # one token: every row in an expert of its own
        pick = torch.randperm(g, generator=gen)[:rows]
    count = torch.bincount(pick, minlength=g)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)])
    group = torch.repeat_interleave(torch.arange(g), count)
    place = torch.arange(rows) - off[group]
    return {"offsets": off.to(torch.int32).cuda(), "group": group.cuda(), "place": place.cuda(),
            "longest": int(count.max()), "groups": g}


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _prepare_norm(case, gen)
    fmt = case["fmt"]
    k = case["H"] if op == "ffn" else case["K"]
    dtype = TYPES[case.get("dtype", "bf16")]
    x = torch.empty(case["rows"], k, dtype=dtype, device="cuda").normal_(0.0, 1.0, generator=gen)
    s = {"case": case, "x": x}
    # the factor of the activations: a calibrated largest value of 8 meets e4m3's largest
    s["tx"] = torch.full((1,), 2.0 ** -8, device="cuda") if fmt == "nvfp4" else None
    if op == "quantize":
        s["out"] = torch.empty_like(x)
        if own:
            from mixture_experts_layer_29_b200 import mx4
            s["a"] = mx4.allocate(fmt, case["rows"], k, tensor_scale=s["tx"])
        return s
    s.update(_ragged(case, seed))
    if op == "product":
        s["w"] = _weight(gen, case["groups"], case["N"], k, fmt)
        n = case["N"]
    else:
        s["w"] = _weight(gen, case["groups"], 2 * case["I"], k, fmt)
        s["wd"] = _weight(gen, case["groups"], k, case["I"], fmt)
        s["th"] = torch.full((1,), 2.0 ** -8, device="cuda") if fmt == "nvfp4" else None
        n = k
    s["out"] = torch.empty(case["rows"], n, dtype=dtype, device="cuda")
    if own:  # the weights laid out once, and the buffers that a serving program keeps
        from mixture_experts_layer_29_b200 import mx4
        s["a"] = mx4.allocate(fmt, case["rows"], k, groups=case["groups"], offsets=s["offsets"],
                              tensor_scale=s["tx"])
        for name in ("w", "wd"):
            if name in s:
                s[name + "4"] = mx4.from_checkpoint(fmt, s[name]["codes"], s[name]["byte"],
                                                    s[name]["t"])
        if op == "product":
            s["ws"] = mx4.gemm_workspace()
        else:
            s["ws"] = mx4.ffn_workspace(s["a"], s["w4"])
    return s


def _prepare_norm(case, gen):
    T, H, dtype = case["T"], case["H"], TYPES[case["dtype"]]

    def rows(std):
        return torch.empty(T, H, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    def fp32(n, mean, std):
        return torch.empty(n, device="cuda").normal_(mean, std, generator=gen)

    s = {"case": case, "residual": rows(2.0), "block": rows(0.5), "w_post": fp32(H, 1.0, 0.1),
         "w_pre": fp32(H, 1.0, 0.1), "scale": 0.5,
         "gate": {"none": None, "token": fp32(T, 0.5, 0.2),
                  "channel": fp32(H, 0.5, 0.2)}[case["gate"]],
         "rstd_block": torch.empty(T, device="cuda"), "rstd_res": torch.empty(T, device="cuda"),
         "res_out": torch.empty(T, H, dtype=dtype, device="cuda"),
         "normed": torch.empty(T, H, dtype=dtype, device="cuda")}
    if case["op"] == "norm_grad":
        # what a training step holds when the gradient comes back: both upstream gradients,
        # the residual stream after the block and the forward's norms
        s["d_res_out"], s["d_normed"] = rows(1.0), rows(1.0)
        n1 = s["block"].float()
        s["rstd_block"] = torch.rsqrt(n1.square().mean(1) + EPS)
        n1 = n1 * s["rstd_block"][:, None] * s["w_post"]
        s["res_out"] = (s["residual"].float() + n1 * _gate(s)).to(dtype)
        s["rstd_res"] = torch.rsqrt(s["res_out"].float().square().mean(1) + EPS)
        s["d_residual"], s["d_block"] = torch.empty_like(s["block"]), torch.empty_like(s["block"])
        s["d_w_post"], s["d_w_pre"] = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        s["d_gate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
    if own:
        from mixture_experts_layer_29_b200 import norm
        s["desc"] = norm.make_desc(T, H, dtype=case["dtype"], gate=case["gate"], eps=EPS,
                                   scale=s["scale"])
        if case["op"] == "norm_grad":
            s["ws"] = norm.workspace(s["desc"])
    return s


def _gate(s, dtype=torch.float32):
    """scale * gate, shaped to multiply [T, H]."""
    if s["gate"] is None:
        return s["scale"]
    g = s["gate"].to(dtype) * s["scale"]
    return g[:, None] if s["case"]["gate"] == "token" else g[None, :]


# ---- one pass -------------------------------------------------------------------------------

def run(s):
    return {"quantize": _quantize, "product": _product, "ffn": _ffn, "norm": _norm,
            "norm_grad": _norm_grad}[s["case"]["op"]](s)


def _tx(t):
    return 1.0 if t is None else t


def _quantize(s):
    if own:
        from mixture_experts_layer_29_b200 import mx4
        mx4.quantize(s["x"], s["a"])
        return mx4.dequantize(s["a"], s["out"])
    return _round_trip(s["x"].float(), s["case"]["fmt"], _tx(s["tx"])).to(s["x"].dtype)


def _product(s):
    if own:
        from mixture_experts_layer_29_b200 import mx4
        mx4.quantize(s["x"], s["a"])
        return mx4.grouped_gemm(s["a"], s["w4"], s["out"], s["ws"])
    fmt, w = s["case"]["fmt"], s["w"]
    a = _round_trip(s["x"].float(), fmt, _tx(s["tx"]))
    return _by_group(a, _values(w["codes"], w["byte"], fmt, _w_factor(w)), s).to(s["x"].dtype)


def _w_factor(w):
    return 1.0 if w["t"] is None else w["t"][:, None, None]


def _ffn(s):
    if own:
        from mixture_experts_layer_29_b200 import mx4
        mx4.quantize(s["x"], s["a"])
        return mx4.grouped_ffn(s["a"], s["w4"], s["wd4"], s["out"], s["ws"], h_scale=s["th"])
    fmt, w, wd, inter = s["case"]["fmt"], s["w"], s["wd"], s["case"]["I"]
    a = _round_trip(s["x"].float(), fmt, _tx(s["tx"]))
    gu = _by_group(a, _values(w["codes"], w["byte"], fmt, _w_factor(w)), s)
    g, u = gu[:, :inter], gu[:, inter:]
    h = _round_trip(g * torch.sigmoid(g) * u, fmt, _tx(s["th"]))
    return _by_group(h, _values(wd["codes"], wd["byte"], fmt, _w_factor(wd)), s).to(s["x"].dtype)


def _norm(s):
    if own:
        from mixture_experts_layer_29_b200 import norm
        norm.block_norm(s["desc"], s["residual"], s["block"], s["w_post"], s["gate"], s["w_pre"],
                        s["res_out"], s["normed"], s["rstd_block"], s["rstd_res"])
        return {"residual": s["res_out"], "normed": s["normed"]}
    dtype = s["block"].dtype
    n1 = s["block"].float()
    n1 = n1 * torch.rsqrt(n1.square().mean(1, keepdim=True) + EPS) * s["w_post"]
    r = (s["residual"].float() + n1 * _gate(s)).to(dtype)
    n2 = r.float()   # the norm reads the residual stream as it is stored
    n2 = n2 * torch.rsqrt(n2.square().mean(1, keepdim=True) + EPS) * s["w_pre"]
    return {"residual": r, "normed": n2.to(dtype)}


def _norm_grad(s):
    if own:
        from mixture_experts_layer_29_b200 import norm
        norm.block_norm_backward(s["desc"], s["d_res_out"], s["d_normed"], s["res_out"],
                                 s["block"], s["w_post"], s["gate"], s["w_pre"],
                                 s["rstd_block"], s["rstd_res"], s["d_residual"], s["d_block"],
                                 s["d_w_post"], s["d_gate"], s["d_w_pre"], s["ws"])
        return {k: s[k] for k in ("d_residual", "d_block", "d_w_post", "d_w_pre", "d_gate")
                if s[k] is not None}
    return _gradients(s, torch.float32, s["block"].dtype)


def _gradients(s, dtype, out):
    """The gradients by the chain rule, in `dtype`."""
    rs_r, rs_b = s["rstd_res"].to(dtype)[:, None], s["rstd_block"].to(dtype)[:, None]
    rhat, bhat = s["res_out"].to(dtype) * rs_r, s["block"].to(dtype) * rs_b
    dn = s["d_normed"].to(dtype)
    c = dn * s["w_pre"].to(dtype)
    g = s["d_res_out"].to(dtype) + rs_r * (c - rhat * (c * rhat).mean(1, keepdim=True))
    d_n1 = g * _gate(s, dtype)
    c = d_n1 * s["w_post"].to(dtype)
    db = rs_b * (c - bhat * (c * bhat).mean(1, keepdim=True))
    got = {"d_residual": g.to(out), "d_block": db.to(out), "d_w_post": (d_n1 * bhat).sum(0),
           "d_w_pre": (dn * rhat).sum(0)}
    if s["gate"] is not None:
        by = 1 if s["case"]["gate"] == "token" else 0
        got["d_gate"] = s["scale"] * (g * bhat * s["w_post"].to(dtype)).sum(by)
    return got


# ---- 64 bits --------------------------------------------------------------------------------

def _nearest(v):
    """The e2m1 number nearest to v (float64), ties to even: a multiple of half the power of
    two below |v|, at least of 0.5."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(1.0, 4.0))) - 1.0)
    return (torch.round(v / step) * step).clamp(-6.0, 6.0)


def _exact_trip(x, fmt, t):
    """Quantised and read back, in float64."""
    v = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK[fmt], BLOCK[fmt])
    top = v.abs().max(-1, keepdim=True).values
    if fmt == "mxfp4":
        scale = torch.exp2((torch.frexp(top).exponent - 3).clamp(min=-127).double())
    else:
        scale = (top / (6.0 * t)).clamp(max=448.0).float().to(torch.float8_e4m3fn).double() * t
    q = torch.where(scale > 0, v / scale, torch.zeros_like(v))
    return (_nearest(q) * scale).reshape(x.shape)


def _exact_weight(w, fmt):
    lo, hi = (w["codes"] & 15).long(), (w["codes"] >> 4).long()
    code = torch.stack([lo, hi], -1).reshape(*w["codes"].shape[:-1], -1)
    mag, exp = (code & 1).double(), (code >> 1) & 3
    v = torch.where(exp > 0, (1.0 + 0.5 * mag) * torch.exp2(exp.double() - 1.0), 0.5 * mag)
    v = torch.where(code > 7, -v, v)
    if fmt == "mxfp4":
        s = torch.exp2(w["byte"].double() - 127.0)
    else:
        s = w["byte"].view(torch.float8_e4m3fn).double() * w["t"].double()[:, None, None]
    return v * s.repeat_interleave(BLOCK[fmt], -1)


def _exact_product(a, w, s, fmt):
    """Group by group, so that one group's weights at a time are held in 64 bits."""
    off = s["offsets"].tolist()
    out = torch.empty(a.shape[0], w["codes"].shape[1], dtype=torch.float64, device=a.device)
    for g in range(s["groups"]):
        if off[g + 1] > off[g]:
            one = {"codes": w["codes"][g:g + 1], "byte": w["byte"][g:g + 1],
                   "t": None if w["t"] is None else w["t"][g:g + 1]}
            out[off[g]:off[g + 1]] = a[off[g]:off[g + 1]] @ _exact_weight(one, fmt)[0].T
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        b = s["block"].double()
        b = b / torch.sqrt((b * b).mean(1, keepdim=True) + EPS) * s["w_post"].double()
        r = s["residual"].double() + _gate(s, torch.float64) * b
        # the norm before the next block reads the residual stream as it is stored
        q = r.to(s["block"].dtype).double()
        n = q / torch.sqrt((q * q).mean(1, keepdim=True) + EPS) * s["w_pre"].double()
        return {"residual": r, "normed": n}
    if op == "norm_grad":
        return _exact_gradients(s)
    fmt = case["fmt"]
    t = 1.0 if s["tx"] is None else s["tx"].double()
    a = _exact_trip(s["x"].double(), fmt, t)
    if op == "quantize":
        return a
    y = _exact_product(a, s["w"], s, fmt)
    if op == "product":
        return y
    g, u = y[:, :case["I"]], y[:, case["I"]:]
    h = _exact_trip(g / (1.0 + torch.exp(-g)) * u, fmt, 1.0 if s["th"] is None else s["th"].double())
    return _exact_product(h, s["wd"], s, fmt)


def _exact_gradients(s):
    """The same gradients from each norm's Jacobian: with n = w x r and r = rstd(x),
    dx = r w dn - x r^3 / H <w dn, x>."""
    H = s["block"].shape[1]
    d = {k: s[k].double() for k in ("res_out", "block", "d_res_out", "d_normed", "w_post",
                                    "w_pre", "rstd_block", "rstd_res")}

    def through(x, r, w, dn):
        r = r.unsqueeze(1)
        return r * w * dn - x * r ** 3 / H * ((w * dn) * x).sum(1, keepdim=True)

    g = d["d_res_out"] + through(d["res_out"], d["rstd_res"], d["w_pre"], d["d_normed"])
    up = g * _gate(s, torch.float64)
    unit = d["block"] * d["rstd_block"].unsqueeze(1)
    got = {"d_residual": g, "d_block": through(d["block"], d["rstd_block"], d["w_post"], up),
           "d_w_post": torch.einsum("th,th->h", up, unit),
           "d_w_pre": torch.einsum("th,th,t->h", d["d_normed"], d["res_out"], d["rstd_res"])}
    if s["gate"] is not None:
        n1 = unit * d["w_post"]
        got["d_gate"] = s["scale"] * torch.einsum(
            "th,th->t" if s["case"]["gate"] == "token" else "th,th->h", g, n1)
    return got


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        size = {"bf16": 2, "fp32": 4}[case["dtype"]] * case["T"] * case["H"]
        arrays, per = (4, 10) if op == "norm" else (6, 22)
        return {"bytes": arrays * size + 12 * case["H"] + 8 * case["T"],
                "flops": per * case["T"] * case["H"]}
    fmt, rows = case["fmt"], case["rows"]
    per = 0.5 + 1.0 / BLOCK[fmt]  # bytes of a 4-bit element with its share of the scale
    if op == "quantize":
        size = {"bf16": 2, "fp32": 4}[case["dtype"]]
        return {"bytes": 2 * size * rows * case["K"], "flops": 4 * rows * case["K"]}
    # the groups without rows need no weights
    hit = min(case["groups"], rows)
    if op == "product":
        n, k = case["N"], case["K"]
        return {"bytes": 2 * rows * (k + n) + hit * n * k * per, "flops": 2.0 * rows * n * k}
    h, i = case["H"], case["I"]
    return {"bytes": 4 * rows * h + hit * 3 * h * i * per, "flops": 6.0 * rows * h * i}
