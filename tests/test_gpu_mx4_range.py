"""The 4-bit operators at the ends of what they take: the largest and smallest finite numbers and
factors. Blocks saturate where the definition does (an element at 6, an NVFP4 scale at 448), and only a
block that holds an infinity or a NaN becomes NaN."""
import pytest
import torch

import mx4_reference as ref
from mixture_experts_layer_29_b200 import abi, mx4

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


def exact_codes(shape, seed):
    """NVFP4 codes and scale bytes 2^-6 to 2^-4, whose products' sums fp32 holds, and their values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    code = torch.randint(0, 16, shape, device="cuda", generator=g).to(torch.uint8)
    e = torch.randint(-6, -3, (*shape[:-1], shape[-1] // 16), device="cuda", generator=g)
    v = ref.GRID.cuda()[(code & 7).long()] * torch.where(code > 7, -1.0, 1.0)
    return code, ((e + 7) << 3).to(torch.uint8), v * torch.exp2(e.double()).repeat_interleave(16, -1)


@pytest.mark.parametrize("ea,ew", [(64, 66), (100, 100), (100, 27), (-64, -64), (-100, -27), (-100, -100), (-63, -60), (100, -100)])
@pytest.mark.parametrize("rows", [40, 200])                     # one CTA per tile, and CTA pairs
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_factors_whose_product_leaves_the_float_range(cuda_device, ea, ew, rows, dtype):
    """y = t_a t_w sum: the sums of zeros stay zero, others are what float64 gives, rounded, infinite
    only where that is."""
    N, K = 136, 256
    code, byte, a = exact_codes((rows, K), 1)
    wc, wb, w = exact_codes((1, N, K), 2)
    code[3], a[3] = 0, 0.0
    ta, tw = (torch.full((1,), m * 2.0 ** e, device="cuda") for m, e in ((1.0, ea), (1.0 if ew == 100 else 1.37, ew)))
    m = mx4.allocate("nvfp4", rows, K, tensor_scale=ta)
    m.codes.copy_(ref.pack(code))
    m.scales[ref.scale_index([0, rows], K, "nvfp4", "cuda")] = byte
    ws = mx4.gemm_workspace()
    y = mx4.grouped_gemm(m, mx4.from_checkpoint("nvfp4", ref.pack(wc), wb, tw), torch.empty(rows, N, device="cuda", dtype=dtype), ws)
    want = (a @ w[0].T) * ta.double() * tw.double()
    assert abi.read_device_status(ws) == 0 and bool((y[3] == 0).all())
    # the factors' product, the multiplication by it, the output's rounding; the smallest denormal's step
    tol = want.abs() * 2.0 ** -23 + 2.0 ** -149
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + want.abs() * 2.0 ** -8 + 2.0 ** -134
    big = want.abs() > torch.finfo(dtype).max * (1 - 2.0 ** -8)
    assert bool((y.double() - want).abs()[~big].le(tol[~big]).all())
    assert torch.equal(y[big].sign().double(), want[big].sign()) and bool((y[big].abs() >= torch.finfo(dtype).max * (1 - 2.0 ** -7)).all())


@pytest.mark.parametrize("rows", [40, 200])
def test_ffn_of_zero_rows_with_the_largest_factors(cuda_device, rows):
    H, inter = 128, 256
    t = torch.full((1,), 2.0 ** 100, device="cuda")
    x = torch.zeros(rows, H, device="cuda")
    a = mx4.quantize(x, mx4.allocate("nvfp4", rows, H, tensor_scale=t))
    w = mx4.quantize_weight(torch.ones(1, 2 * inter, H, device="cuda"), "nvfp4", t)
    d = mx4.quantize_weight(torch.ones(1, H, inter, device="cuda"), "nvfp4", t)
    ws = mx4.ffn_workspace(a, w)
    y = mx4.grouped_ffn(a, w, d, torch.empty(rows, H, device="cuda"), ws, t)
    assert bool((y == 0).all()) and abi.read_device_status(ws) == 0
