"""The 4-bit formats and their products in float64, for the tests of mx4 (torch, any device).

Written from the formats' definition (include/moe_mx4.h): elements are rounded by looking for
the nearest grid value, and scales are handled row-major; nothing is shared with the library."""
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def grid_round(q):
    """(code 0..7, value) of |q| (float64): nearest grid value, ties to the even code."""
    g = GRID.to(q.device)
    d = (q.abs().unsqueeze(-1) - g).abs()
    best = d.min(-1).values.unsqueeze(-1)
    tied = d == best
    idx = torch.arange(8, device=q.device)
    # at most two codes tie, and exactly one of the two is even
    odd_penalty = torch.where(tied, idx % 2, 2)
    code = odd_penalty.argmin(-1)
    return code, g[code]


def block_scales(x, fmt, t=1.0):
    """(scale byte, value of the scale) of the blocks of x [..., K] (any float type)."""
    b = x.double().unflatten(-1, (-1, BLOCK[fmt]))
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    top = torch.where(bad, torch.ones_like(top), top)
    if fmt == "mxfp4":
        e = torch.frexp(top).exponent - 3
        byte = torch.where(top > 0, (e + 127).clamp(min=0), torch.zeros_like(e))
        s = torch.ldexp(torch.ones_like(top), byte - 127)
        byte = torch.where(bad, 255, byte)
    else:
        # the definition's fp32 operations
        t32 = torch.as_tensor(t, dtype=torch.float32, device=x.device)
        r = (top.float() / (t32 * 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        byte = r.view(torch.uint8).to(torch.int64)
        s = (r.float() * t32).double()
        byte = torch.where(bad, 0x7F, byte)
    return byte.to(torch.uint8), torch.where(bad, torch.nan, s)


def quantize(x, fmt, t=1.0):
    """(codes one per element, scale bytes, values in float64)."""
    byte, s = block_scales(x, fmt, t)
    s = s.repeat_interleave(BLOCK[fmt], -1)
    q = x.double() / s
    if fmt == "nvfp4":   # one fp32 division
        q = (x.float() / s.float()).double()
    ok = torch.isfinite(s) & (s > 0)
    q = torch.where(ok, q, torch.zeros_like(q))
    code, val = grid_round(q)
    sign = torch.signbit(x) & ok
    value = torch.where(sign, -val, val) * torch.where(torch.isnan(s), s, torch.where(s > 0, s, 0.0))
    return (code + 8 * sign).to(torch.uint8), byte, value


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def scale_index(offsets, K, fmt, device="cpu"):
    """Byte offset of the scale of each (row, block), [rows, K / block]."""
    off = [int(v) for v in offsets]
    nb = K // BLOCK[fmt]
    out = torch.empty(off[-1], nb, dtype=torch.int64)
    b = torch.arange(nb)
    for g in range(len(off) - 1):
        l = torch.arange(off[g + 1] - off[g])[:, None]
        tile = off[g] // 128 + g + l // 128
        out[off[g]:off[g + 1]] = ((tile * (nb // 4) + b // 4) * 512 + (l % 32) * 16
                                  + (l % 128) // 32 * 4 + b % 4)
    return out.to(device)


def grouped(a, w, offsets):
    """(a[r] . w[g]^T, sum of |products|) in float64; a [R, K], w [G, N, K]."""
    off = [int(v) for v in offsets]
    y = torch.zeros(off[-1], w.shape[1], dtype=torch.float64, device=a.device)
    m = torch.zeros_like(y)
    for g in range(len(off) - 1):
        rows = slice(off[g], off[g + 1])
        if off[g + 1] > off[g]:
            y[rows] = a[rows] @ w[g].double().T
            m[rows] = a[rows].abs() @ w[g].double().abs().T
    return y, m
