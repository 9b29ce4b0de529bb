"""The 4-bit operators at the ends of what they take: the largest and smallest finite numbers and
factors. Blocks saturate where the definition does (an element at 6, an NVFP4 scale at 448), and only a
block that holds an infinity or a NaN becomes NaN."""
import pytest
import torch

import mx4_reference as ref
from mixture_experts_layer_29_b200 import mx4

pytestmark = pytest.mark.gpu


def saturating(x, fmt, t):
    """ref.quantize of finite x, with quotients past the float range counted as the largest element."""
    byte, s = ref.block_scales(x, fmt, t)
    wide = s.repeat_interleave(ref.BLOCK[fmt], -1)
    q = (x.float() / wide.float()).double() if fmt == "nvfp4" else x.double() / wide
    q = torch.where(wide > 0, q, 0.0).clamp(-8.0, 8.0)
    code, val = ref.grid_round(q)
    sign = torch.signbit(x) & (wide > 0)
    return (code + 8 * sign).to(torch.uint8), byte, torch.where(sign, -val, val) * wide


def every_binade(rows, K, dtype, seed):
    """Finite numbers of both signs: each block's largest in a binade of its own, from the smallest
    denormal to the largest number of the type, and the others up to 2^40 below it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = rows * K // 16
    top = torch.linspace(-149.0, 127.0, n, device="cuda").round().double().view(rows, K // 16)
    e = top.repeat_interleave(16, 1) - torch.randint(0, 40, (rows, K), device="cuda", generator=g)
    e[:, ::16] = top
    x = torch.exp2(e) * (1.0 + torch.rand(rows, K, device="cuda", generator=g, dtype=torch.float64))
    x *= torch.randint(0, 2, (rows, K), device="cuda", generator=g) * 2.0 - 1.0
    most = torch.finfo(dtype).max
    x = x.clamp(-most, most).to(dtype)
    x[-1, -16:] = torch.tensor([most, -most] * 8, device="cuda", dtype=dtype)
    x[-2, -16:] = -most
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt,exponent", [("mxfp4", 0)] + [("nvfp4", e) for e in (-100, -70, -57, -40, -10, -8, 0, 30, 57, 100)])
def test_finite_blocks_saturate(cuda_device, fmt, exponent, dtype):
    rows, K = 16, 1152
    t = torch.full((1,), 1.25 * 2.0 ** exponent, device="cuda").clamp(max=2.0 ** 100) if fmt == "nvfp4" else None
    x = every_binade(rows, K, dtype, exponent + 200)
    assert torch.isfinite(x).all()
    m = mx4.quantize(x, mx4.allocate(fmt, rows, K, tensor_scale=t))
    code, byte, value = saturating(x, fmt, 1.0 if t is None else t)
    assert torch.equal(m.scales[ref.scale_index([0, rows], K, fmt, "cuda")], byte)
    assert torch.equal(m.codes, ref.pack(code))
    out = mx4.dequantize(m, torch.empty(rows, K, device="cuda"))
    assert torch.equal(out, value.float())
