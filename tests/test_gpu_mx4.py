"""The 4-bit operators on the GPU against float64: quantisation bit for bit, the ragged product
exactly where every partial sum is a float, within its rounding elsewhere, and the FFN."""
import pytest
import torch

import mx4_reference as ref
from mixture_experts_layer_29_b200 import abi, mx4
from mixture_experts_layer_29_b200 import workloads as wl

pytestmark = pytest.mark.gpu

FORMATS = ["mxfp4", "nvfp4"]
BF16_HALF = 2.0 ** -8            # half a step of bf16, relative
# The tensor cores add the products of one K = 64 step to the accumulator in fp32. Whatever the
# order inside a step, its result is off by no more than a few units in the last place of the
# step's largest partial sum, which sum |a w| bounds: 2^-22 of it per step covers truncation of
# the aligned terms.
STEP = 2.0 ** -22


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def offsets_of(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off


def dev(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def factor(fmt, n=1, v=2.0 ** -6):
    return torch.full((n,), v, device="cuda") * torch.linspace(1.0, 1.5, n, device="cuda") if fmt == "nvfp4" else None


def make_rows(rows, K, dtype, seed):
    x = torch.randn(rows, K, device="cuda", generator=gen(seed))
    # magnitudes over many binades, zero blocks, exact ties and signed zeros
    x *= torch.exp2(torch.randint(-20, 20, (rows, K // 16), device="cuda", generator=gen(seed + 1)).float()
                    ).repeat_interleave(16, 1)
    if rows > 2:
        x[1, :32] = 0.0
        x[2, :16] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] * 2, device="cuda")
        x[2, 16:32] = -x[2, :16]
        x[0, 32:64] = 2.0 ** -130
        x[0, 64:96] = -0.0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,K", [([1], 128), ([33], 256), ([0, 5, 0, 130, 1, 0], 1152), ([64, 64], 2048),
                                      ([257, 3], 384)])
def test_quantize_is_the_definition(cuda_device, fmt, dtype, counts, K):
    off = offsets_of(counts)
    rows = off[-1]
    t = factor(fmt)
    x = make_rows(rows, K, dtype, 3 * rows + K)
    m = mx4.allocate(fmt, rows + 7, K, len(counts), dev(off), t)     # seven rows of no group
    m.codes.fill_(0xA5)
    m.scales.fill_(0x5A)
    out = torch.full((rows + 7, K), 7.0, device="cuda", dtype=dtype)
    mx4.quantize(torch.cat([x, torch.ones(7, K, device="cuda", dtype=dtype)]), m)
    mx4.dequantize(m, out)
    code, byte, value = ref.quantize(x, fmt, 1.0 if t is None else t)
    assert torch.equal(m.codes[:rows], ref.pack(code))
    at = ref.scale_index(off, K, fmt, "cuda")
    assert torch.equal(m.scales[at], byte)
    want = value.to(dtype)
    assert torch.equal(out[:rows], want)
    # rows behind the last group are as they were, and so is every scale byte of none
    assert (m.codes[rows:] == 0xA5).all() and (out[rows:] == 7.0).all()
    left = torch.ones_like(m.scales, dtype=torch.bool)
    left[at.flatten()] = False
    assert (m.scales[left] == 0x5A).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_strided_rows_and_nonfinite_blocks(cuda_device, fmt):
    wide = make_rows(40, 512, torch.bfloat16, 5)
    x = wide[:, 128:384]
    x[3, 5], x[4, 40], x[5, 100] = float("inf"), float("nan"), float("-inf")
    m = mx4.allocate(fmt, 40, 256)
    mx4.quantize(x, m)
    code, byte, value = ref.quantize(x, fmt)
    out = torch.empty(40, 512, device="cuda")[:, :256]
    mx4.dequantize(m, out)
    assert torch.equal(m.codes, ref.pack(code))
    assert torch.equal(torch.isnan(out), torch.isnan(value)) and torch.isnan(out).sum() == 3 * ref.BLOCK[fmt]
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(value.float()))


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_scatters_tokens_to_their_rows(cuda_device, fmt):
    tokens, picks, K, groups = 50, 4, 256, 9
    g = torch.Generator().manual_seed(1)
    expert = torch.stack([torch.randperm(groups + 3, generator=g)[:picks] for _ in range(tokens)])
    counts = [int((expert == e).sum()) for e in range(groups)]
    off = offsets_of(counts)
    row_of = torch.full((tokens, picks), -1, dtype=torch.int32)
    src = torch.empty(off[-1], dtype=torch.long)
    nxt = list(off)
    for t in range(tokens):
        for p in range(picks):
            e = int(expert[t, p])
            if e < groups:
                row_of[t, p], src[nxt[e]] = nxt[e], t
                nxt[e] += 1
    x = make_rows(tokens, K, torch.bfloat16, 11)
    f = factor(fmt)
    a = mx4.allocate(fmt, tokens * picks, K, groups, dev(off), f)
    b = mx4.allocate(fmt, tokens * picks, K, groups, dev(off), f)
    for m in (a, b):
        m.codes.zero_()
        m.scales.zero_()
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    mx4.quantize(x, a, row_of.cuda(), status)
    full = torch.zeros(tokens * picks, K, device="cuda", dtype=torch.bfloat16)
    full[: off[-1]] = x[src.cuda()]
    mx4.quantize(full, b)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert abi.read_device_status(status) == 0
    # an entry past the last group is skipped and reported
    row_of[7, 0] = off[-1] + 3
    mx4.quantize(x, a, row_of.cuda(), status)
    assert abi.read_device_status(status) == -6


@pytest.mark.parametrize("fmt", FORMATS)
def test_checkpoint_scales_and_quantized_weight_agree(cuda_device, fmt):
    groups, N, K = 3, 200, 384
    w = torch.randn(groups, N, K, device="cuda", generator=gen(4)) * 0.02
    t = factor(fmt, groups, 2.0 ** -12)
    per = 1.0 if t is None else t[:, None, None]
    code, byte, value = ref.quantize(w, fmt, per)
    a = mx4.quantize_weight(w, fmt, t)
    b = mx4.from_checkpoint(fmt, ref.pack(code), byte, t)
    assert torch.equal(a.codes, b.codes)
    at = ref.scale_index([g * N for g in range(groups + 1)], K, fmt, "cuda")
    assert torch.equal(a.scales[at], byte.flatten(0, 1)) and torch.equal(b.scales[at], byte.flatten(0, 1))
    out = mx4.dequantize(b, torch.empty(groups * N, K, device="cuda"))
    assert torch.equal(out.view(groups, N, K).double(), value)


def small_checkpoint(shape, fmt, seed):
    """Codes and scale bytes whose products and sums are exact in fp32: scales 1/2, 1 or 2."""
    g = gen(seed)
    code = torch.randint(0, 16, shape, device="cuda", generator=g).to(torch.uint8)
    e = torch.randint(-1, 2, (*shape[:-1], shape[-1] // ref.BLOCK[fmt]), device="cuda", generator=g)
    byte = (e + 127 if fmt == "mxfp4" else (e + 7) << 3).to(torch.uint8)
    v = ref.GRID.cuda()[(code & 7).long()]
    v = torch.where(code > 7, -v, v) * torch.exp2(e.double()).repeat_interleave(ref.BLOCK[fmt], -1)
    return code, byte, v


COUNTS = [[1], [16], [0, 0, 3], [0, 0], [64, 65, 1], [17, 0, 130, 63], [193, 0, 192, 191], [400, 1]]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(1, 128), (128, 128), (256, 256), (200, 384), (515, 640)])
def test_product_of_small_numbers_is_exact(cuda_device, fmt, counts, N, K):
    """|products| <= 144 in steps of 1/16, so sums of 640 are exact in fp32 in any order: a
    wrong scale, row, column or accumulator shows as a difference."""
    groups, off = len(counts), offsets_of(counts)
    rows = off[-1]
    code, byte, a = small_checkpoint((rows, K), fmt, rows + K)
    wc, wb, w = small_checkpoint((groups, N, K), fmt, N)
    m = mx4.allocate(fmt, rows + 5, K, groups, dev(off))
    m.codes.random_(0, 256)                   # rows past the groups hold anything
    m.scales.random_(0, 256)
    m.codes[:rows] = ref.pack(code)
    m.scales[ref.scale_index(off, K, fmt, "cuda")] = byte
    out = torch.full((rows + 5, N), 3.0, device="cuda")
    ws = mx4.gemm_workspace()
    mx4.grouped_gemm(m, mx4.from_checkpoint(fmt, ref.pack(wc), wb), out, ws)
    y, _ = ref.grouped(a, w, off)
    assert abi.read_device_status(ws) == 0
    assert torch.equal(out[:rows].double(), y)
    assert (out[rows:] == 3.0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,N", [([3000, 1, 2500, 190], 2056), ([64, 1, 7, 0, 65, 63] * 10, 4104)])
def test_many_tiles_per_cta_are_exact(cuda_device, fmt, counts, N):
    """More tiles than a persistent CTA (or pair) takes in one turn: 31 and 17 row and channel tiles,
    and 70 x 17; K = 512 in two stages."""
    K, groups, off = 512, len(counts), offsets_of(counts)
    code, byte, a = small_checkpoint((off[-1], K), fmt, 5)
    wc, wb, w = small_checkpoint((groups, N, K), fmt, 6)
    m = mx4.allocate(fmt, off[-1], K, groups, dev(off))
    m.codes.copy_(ref.pack(code))
    m.scales[ref.scale_index(off, K, fmt, "cuda")] = byte
    ws = mx4.gemm_workspace()
    y, _ = ref.grouped(a, w, off)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.empty(off[-1], N, device="cuda", dtype=dtype)
        mx4.grouped_gemm(m, mx4.from_checkpoint(fmt, ref.pack(wc), wb), out, ws)
        assert torch.equal(out, y.to(dtype))
    assert abi.read_device_status(ws) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [[0, 40, 30, 70], [0, 40, 50, 90], [5, 40, 50, 70]])
def test_products_report_offsets_outside_the_matrix(cuda_device, fmt, bad):
    a = mx4.allocate(fmt, 70, 256, 3, dev(bad))
    a.codes.zero_()
    a.scales.zero_()
    w = mx4.quantize_weight(torch.zeros(3, 128, 256, device="cuda"), fmt)
    ws = mx4.gemm_workspace()
    mx4.grouped_gemm(a, w, torch.empty(70, 128, device="cuda"), ws)
    assert abi.read_device_status(ws) == -6 and abi.read_device_status(ws) == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 90, 200], 520, 2048), ([300] * 3, 256, 6144), ([1] * 40, 384, 1024)])
def test_product_of_quantized_rows(cuda_device, fmt, dtype, counts, N, K):
    groups, off = len(counts), offsets_of(counts)
    t, tw = factor(fmt, 1, 2.0 ** -7), factor(fmt, groups, 2.0 ** -12)
    x = torch.randn(off[-1], K, device="cuda", generator=gen(N)).to(torch.bfloat16)
    w = torch.randn(groups, N, K, device="cuda", generator=gen(K)) * 0.02
    a = mx4.quantize(x, mx4.allocate(fmt, off[-1], K, groups, dev(off), t))
    ws = mx4.gemm_workspace()
    out = mx4.grouped_gemm(a, mx4.quantize_weight(w, fmt, tw), torch.empty(off[-1], N, device="cuda", dtype=dtype), ws)
    av = ref.quantize(x, fmt, 1.0 if t is None else t)[2]
    wv = ref.quantize(w, fmt, 1.0 if tw is None else tw[:, None, None])[2]
    y, mag = ref.grouped(av, wv, off)
    # the accumulation, the two factors' product and the multiplication by it, the output's rounding
    tol = mag * (K / 64 + 1) * STEP + y.abs() * 2.0 ** -22
    if dtype == torch.bfloat16:
        tol = tol * (1 + BF16_HALF) + y.abs() * BF16_HALF
    assert abi.read_device_status(ws) == 0
    assert ((out.double() - y).abs() <= tol).all(), ((out.double() - y).abs() / tol).max()


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_keeps_nonfinite_rows_to_themselves(cuda_device, fmt):
    x = torch.randn(70, 256, device="cuda", generator=gen(8))
    clean = x.clone()
    x[5, 17] = float("nan")
    x[69, 200] = float("inf")
    w = mx4.quantize_weight(torch.randn(1, 128, 256, device="cuda", generator=gen(9)), fmt)
    out = []
    for v in (x, clean):
        a = mx4.quantize(v, mx4.allocate(fmt, 70, 256))
        out.append(mx4.grouped_gemm(a, w, torch.empty(70, 128, device="cuda"), mx4.gemm_workspace()))
    bad = torch.zeros(70, dtype=torch.bool, device="cuda")
    bad[[5, 69]] = True
    assert torch.isnan(out[0][bad]).all()
    assert torch.equal(out[0][~bad], out[1][~bad])


def ffn_reference(x, wg, wu, wd, off, fmt, t, th, tw):
    """y in float64, and how far a correct kernel may be from it. h is rounded to 4 bits, so
    an h whose fp32 value lies within its error of the border between two grid values may go
    either way: those are found, and their steps go through |Wd| into the tolerance."""
    av = ref.quantize(x, fmt, 1.0 if t is None else t)[2]
    K, inter = x.shape[1], wg.shape[1]
    G, mg = ref.grouped(av, wg, off)
    U, mu = ref.grouped(av, wu, off)
    sig = torch.sigmoid(G)
    h = G * sig * U
    eg, eu = mg * (K / 64 + 1) * STEP, mu * (K / 64 + 1) * STEP
    # |d silu| <= 1.1; exp and the division of the fp32 silu are good to 2^-20 relative where
    # silu matters (|G| below 20 here)
    eh = 1.1 * eg * U.abs() + (G * sig).abs() * eu + h.abs() * 2.0 ** -19
    thv = 1.0 if th is None else th
    _, byte, hv = ref.quantize(h.float(), fmt, thv)
    s = ref.block_scales(h.float(), fmt, thv)[1].repeat_interleave(ref.BLOCK[fmt], -1)
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device, dtype=torch.float64)
    gap = torch.tensor([0.5, 0.5, 0.5, 0.5, 1.0, 1.0, 2.0], device=x.device, dtype=torch.float64)
    q, eq = (h / s).abs().unsqueeze(-1), (eh / s).unsqueeze(-1)
    near = (q - mid).abs() <= eq
    step = (near * gap).amax(-1) * s
    # a block whose scale itself may go either way: its elements move by at most a step of 2
    blk, ebl = h.unflatten(-1, (-1, ref.BLOCK[fmt])), eh.unflatten(-1, (-1, ref.BLOCK[fmt])).amax(-1)
    top = blk.abs().amax(-1)
    lo = ref.block_scales(((top - ebl).clamp(min=0)).float().repeat_interleave(ref.BLOCK[fmt], -1), fmt, thv)[0]
    hi = ref.block_scales((top + ebl).float().repeat_interleave(ref.BLOCK[fmt], -1), fmt, thv)[0]
    step = torch.maximum(step, ((lo != hi).repeat_interleave(ref.BLOCK[fmt], -1)) * s * 2.0 * 2.0)
    y, my = ref.grouped(hv, wd, off)
    flip, _ = ref.grouped(step, wd.abs(), off)
    return y, my * (inter / 64 + 1) * STEP + flip + y.abs() * 2.0 ** -22, (near.any(-1).float().mean())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts,H,I", [([1], 128, 128), ([5, 0, 70, 130], 256, 384), ([200, 1, 0, 333], 1024, 256),
                                        ([2] * 20, 768, 256)])
def test_ffn_store_and_fused(cuda_device, fmt, counts, H, I):
    groups, off = len(counts), offsets_of(counts)
    rows = off[-1]
    t, th = factor(fmt, 1, 2.0 ** -7), factor(fmt, 1, 2.0 ** -9)
    tw = factor(fmt, groups, 2.0 ** -11)
    per = 1.0 if tw is None else tw[:, None, None]
    x = torch.randn(rows, H, device="cuda", generator=gen(H)).to(torch.bfloat16)
    wgu = torch.randn(groups, 2 * I, H, device="cuda", generator=gen(I)) * H ** -0.5
    wd = torch.randn(groups, H, I, device="cuda", generator=gen(2)) * I ** -0.5
    qg, qd = mx4.quantize_weight(wgu, fmt, tw), mx4.quantize_weight(wd, fmt, tw)
    a = mx4.quantize(x, mx4.allocate(fmt, rows, H, groups, dev(off), t))
    ws = mx4.ffn_workspace(a, qg)
    wv = ref.quantize(wgu, fmt, per)[2]
    y, tol, near = ffn_reference(x, wv[:, :I], wv[:, I:], ref.quantize(wd, fmt, per)[2], off, fmt, t, th, tw)
    out32 = mx4.grouped_ffn(a, qg, qd, torch.empty(rows, H, device="cuda"), ws, th)
    assert abi.read_device_status(ws) == 0
    assert near < 1e-2                      # the borders excuse few elements
    assert ((out32.double() - y).abs() <= tol).all(), ((out32.double() - y).abs() / tol).max()
    out16 = mx4.grouped_ffn(a, qg, qd, torch.empty(rows, H, device="cuda", dtype=torch.bfloat16), ws, th)
    assert torch.equal(out16, out32.to(torch.bfloat16))
    # fused combine: rows of one token are added to it, on top of what is there
    tok = (torch.arange(rows, device="cuda") * 7 % 11).to(torch.int32)
    gate = torch.rand(rows, device="cuda", generator=gen(6))
    acc = torch.ones(11, H, device="cuda")
    mx4.grouped_ffn(a, qg, qd, acc, ws, th, tok, gate, 0.5)
    part = 0.5 * gate.double()[:, None] * out32.double()
    want = torch.ones(11, H, device="cuda", dtype=torch.float64).index_add_(0, tok.long(), part)
    mag = torch.ones(11, H, device="cuda", dtype=torch.float64).index_add_(0, tok.long(), part.abs())
    n = int(torch.bincount(tok.long()).max())
    # at most n additions, each within half a unit of a partial sum <= mag, and two products
    assert ((acc.double() - want).abs() <= mag * (n + 3) * 2.0 ** -24).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows,groups,N,K", [(16384, 8, 4096, 6144), (640, 32, 4096, 6144)])
def test_equal_products_agree_bit_for_bit(cuda_device, fmt, rows, groups, N, K):
    """The same product 200 times, many stages per tile and many tiles per CTA, the rings of both
    kernels full all the time: no launch may differ from the first in a bit."""
    g = torch.Generator(device="cuda").manual_seed(31)
    nb = K // ref.BLOCK[fmt]
    codes = torch.full((groups, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")      # all 1.0
    if fmt == "mxfp4":
        byte = torch.randint(123, 131, (groups, N, nb), dtype=torch.uint8, device="cuda", generator=g)
        scale, factor = torch.exp2(byte.double() - 127), None
    else:
        byte = torch.randint(0x30, 0x48, (groups, N, nb), dtype=torch.uint8, device="cuda", generator=g)
        scale, factor = byte.view(torch.float8_e4m3fn).double(), torch.ones(groups, device="cuda")
    w = mx4.from_checkpoint(fmt, codes, byte, factor)
    off = torch.arange(0, rows + 1, rows // groups, dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda") if fmt == "nvfp4" else None
    a = mx4.allocate(fmt, rows, K, groups, off, tensor_scale=one)
    mx4.quantize(torch.full((rows, K), 6.0, dtype=torch.bfloat16, device="cuda"), a)     # exact: 6, or 1.5 x 4
    want = (scale.sum(-1) * ref.BLOCK[fmt] * 6.0).repeat_interleave(rows // groups, 0)
    ws = mx4.gemm_workspace()
    first, *outs = [torch.empty(rows, N, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
    mx4.grouped_gemm(a, w, first, ws)
    # half a step of bf16, and fp32 sums of terms of one sign: 24 stages of 4 products, each off by 2^-22 at most
    assert bool(((first.double() - want).abs() <= want * (2.0 ** -8 + 96 * 2.0 ** -22)).all())
    differ = 0
    for _ in range(50):
        for out in outs:
            mx4.grouped_gemm(a, w, out, ws)
        differ += sum(int(not torch.equal(out, first)) for out in outs)
    assert differ == 0 and abi.read_device_status(ws) == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K,shift,pad", [(128, 0, 8), (640, 8, 0), (1024, 8, 8), (1664, 0, 8), (1664, 16, 16), (2688, 8, 24)])
def test_rows_aligned_to_16_bytes_only(cuda_device, fmt, dtype, K, shift, pad):
    """Starts and strides of odd multiples of 16 bytes (and of 32), blocks of zeros and rows that end
    inside a warp's step: the bits of the formula."""
    g = torch.Generator(device="cuda").manual_seed(K + shift)
    per = 16 // dtype.itemsize                       # elements of 16 bytes
    shift, pad = shift // 8 * per, pad // 8 * per
    buf = torch.randn(37, shift + K + pad, device="cuda", generator=g).to(dtype)
    x = buf[:, shift:shift + K]
    x[::3, 32:64] = 0.0
    x[5] = 0.0
    t = torch.full((1,), 2.0 ** -6, device="cuda") if fmt == "nvfp4" else None
    m = mx4.allocate(fmt, 37, K, tensor_scale=t)
    mx4.quantize(x, m)
    codes, byte, value = ref.quantize(x, fmt, float(t) if t is not None else 1.0)
    assert torch.equal(m.codes, ref.pack(codes).to(torch.uint8))
    at = ref.scale_index([0, 37], K, fmt, "cuda")
    assert torch.equal(m.scales.flatten()[at].int(), byte.int())
    out = torch.empty(37, K, dtype=torch.float32, device="cuda")
    mx4.dequantize(m, out)
    assert torch.equal(out.double(), value)


@pytest.mark.parametrize("fmt", FORMATS)
def test_offsets_past_32_bits(cuda_device, fmt):
    """More than 2^32 elements in the rows, 2^31 bytes in their codes and 2^31 elements in a product: the
    last rows are what a small matrix of them gives, a weight's last group what that group alone gives."""
    rows, K, N, last = 706_000, 6144, 128, 200
    t = factor(fmt)
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-last:] = torch.randn(last, K, device="cuda", generator=gen(1)).to(torch.bfloat16)
    a, b = mx4.allocate(fmt, rows, K, tensor_scale=t), mx4.allocate(fmt, last, K, tensor_scale=t)
    mx4.quantize(x, a)
    mx4.quantize(x[-last:], b)
    assert torch.equal(a.codes[-last:], b.codes)
    back = torch.empty(last, K, dtype=torch.bfloat16, device="cuda")
    mx4.dequantize(a, x)
    mx4.dequantize(b, back)
    assert torch.equal(x[-last:], back) and not bool(x[:-last].any())
    del x
    w = mx4.quantize_weight(torch.randn(1, N, K, device="cuda", generator=gen(2)).clamp(-6.0, 6.0), fmt)
    ws = mx4.gemm_workspace()
    big, small = (torch.empty(n, N, device="cuda") for n in (rows, last))
    mx4.grouped_gemm(a, w, big, ws)
    mx4.grouped_gemm(b, w, small, ws)
    # the same sums at another place of a tile: each off by 96 steps of sum |a| |w| at most
    mag = back.double().abs().sum(1, keepdim=True) * 6.5          # |w| <= 6, or what its scale rounds that to
    assert bool(((big[-last:] - small).double().abs() <= 2 * mag * 96 * STEP).all())
    assert not bool(big[:-last].any())
    del a, big
    # outputs of more than 2^31 elements
    rows, K, N = 530_000, 128, 4096 + 8
    a, b = mx4.allocate(fmt, rows, K, tensor_scale=t), mx4.allocate(fmt, last, K, tensor_scale=t)
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-last:] = 1.5
    mx4.quantize(x, a)
    mx4.quantize(x[-last:], b)
    w = mx4.quantize_weight(torch.randint(-2, 3, (1, N, K), device="cuda", generator=gen(3)).float(), fmt)
    big, small = (torch.empty(n, N, dtype=torch.bfloat16, device="cuda") for n in (rows, last))
    mx4.grouped_gemm(a, w, big, ws)
    mx4.grouped_gemm(b, w, small, ws)
    assert torch.equal(big[-last:], small) and not bool(big[:-last].any())
    assert abi.read_device_status(ws) == 0
    del a, x, big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("counts", [3, 200])
def test_weights_past_32_bits(cuda_device, fmt, counts):
    """The weights of 400 experts, 5 GB of codes, by both kernels."""
    groups, N, K = 400, 4096, 6144
    codes = torch.randint(0, 256, (groups, N, K // 2), device="cuda", generator=gen(4), dtype=torch.uint8)
    byte = torch.full((groups, N, K // ref.BLOCK[fmt]), 127 if fmt == "mxfp4" else 56, device="cuda", dtype=torch.uint8)
    w = mx4.from_checkpoint(fmt, codes, byte)
    off = [0] * (groups - 1) + [counts, 2 * counts]             # the last two groups have rows
    rows = 2 * counts if counts < 64 else 64 * groups + 1       # as many as there may be: one CTA, or pairs
    m = mx4.allocate(fmt, rows, K, groups, dev(off))
    x = torch.randint(-4, 5, (rows, K), device="cuda", generator=gen(5)).to(torch.bfloat16)
    x[:, ::16] = 4.0                                            # codes are exact: scale 1 (2/3 in NVFP4: rounded)
    mx4.quantize(x, m)
    value = torch.zeros(rows, K, device="cuda")
    mx4.dequantize(m, value)
    out = torch.empty(rows, N, device="cuda")
    ws = mx4.gemm_workspace()
    mx4.grouped_gemm(m, w, out, ws)
    for g in (groups - 2, groups - 1):
        c = torch.stack([codes[g] & 15, codes[g] >> 4], -1).flatten(-2)
        v = ref.GRID.cuda()[(c & 7).long()]
        v = torch.where(c > 7, -v, v)
        r = slice(off[g], off[g + 1])
        y, mag = value[r].double() @ v.T, value[r].double().abs() @ v.abs().T
        assert bool(((out[r].double() - y).abs() <= mag * 96 * STEP).all())
    assert abi.read_device_status(ws) == 0
    del codes, byte, w
    torch.cuda.empty_cache()
