"""The 4-bit operators and the block norms without a GPU: the headers' functions are exported and
bound, sizes come out as documented, and bad arguments are refused on the host."""
import ctypes

import pytest
import torch

import mx4_reference as ref
from mixture_experts_layer_29_b200 import abi, build, mx4, norm

GOOD, BAD = 1 << 20, (1 << 20) + 4
INVALID, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -5


@pytest.fixture(scope="module")
def L():
    build.build()
    norm.lib()
    return mx4.lib()


def test_headers_and_bindings_agree(L):
    assert set(mx4.header_functions()) == set(mx4._SIGS) and len(mx4._SIGS) == 8
    assert set(norm.header_functions()) == set(norm._SIGS) and len(norm._SIGS) == 3
    for n in [*mx4._SIGS, *norm._SIGS]:
        assert hasattr(L, n)
    assert not set(mx4._SIGS) & set(abi._SIGS) and not set(norm._SIGS) & set(abi._SIGS)


def desc(**kw):
    base = dict(format=0, rows=256, K=256, groups=2, group_rows=128, factor_per_group=0,
                offsets=None, factor=None, codes=GOOD, scales=GOOD)
    base.update(kw)
    return mx4.Desc(*[base[f] for f, _ in mx4.Desc._fields_])


MATRIX_ERRORS = [
    (dict(format=2), INVALID), (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(groups=0), INVALID),
    (dict(K=192), UNSUPPORTED), (dict(groups=1025, group_rows=0, offsets=GOOD), UNSUPPORTED),
    (dict(group_rows=127), INVALID), (dict(offsets=GOOD), INVALID),          # both kinds of groups
    (dict(offsets=BAD, group_rows=0), ALIGN), (dict(factor=GOOD), INVALID),  # a factor with mxfp4
    (dict(format=1, factor=(1 << 20) + 2), ALIGN), (dict(factor_per_group=2), INVALID),
    (dict(rows=(1 << 31) - 128, K=1 << 20, group_rows=0, offsets=GOOD), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", MATRIX_ERRORS)
def test_matrix_limits(L, kw, code):
    d = desc(**kw)
    assert L.moe_mx4_quantize(ctypes.byref(d), GOOD, 0, d.K, None, d.rows, 0, None, None) == code
    assert L.moe_mx4_dequantize(ctypes.byref(d), GOOD, 0, d.K, None) == code
    assert L.moe_mx4_pack_scales(ctypes.byref(d), GOOD, None) == code
    w = desc(K=d.K, groups=max(d.groups, 1), rows=128 * max(d.groups, 1))
    assert L.moe_mx4_grouped_gemm(ctypes.byref(d), ctypes.byref(w), GOOD, 0, GOOD, 1024, None) == code


def test_quantize_refusals(L):
    q = L.moe_mx4_quantize
    d = ctypes.byref(desc())
    assert q(None, GOOD, 0, 256, None, 256, 0, None, None) == INVALID
    assert q(d, None, 0, 256, None, 256, 0, None, None) == INVALID
    assert q(d, BAD, 0, 256, None, 256, 0, None, None) == ALIGN
    assert q(d, GOOD, 5, 256, None, 256, 0, None, None) == INVALID
    assert q(d, GOOD, 0, 255, None, 256, 0, None, None) == INVALID           # ld < K
    assert q(d, GOOD, 0, 260, None, 256, 0, None, None) == ALIGN             # rows off 16 bytes
    assert q(d, GOOD, 0, 256, None, 255, 0, None, None) == INVALID           # tokens != rows
    assert q(d, GOOD, 0, 256, GOOD, -1, 2, None, None) == INVALID
    assert q(d, GOOD, 0, 256, GOOD, 4, 0, None, None) == INVALID
    assert q(d, GOOD, 0, 256, GOOD, 4, 33, None, None) == UNSUPPORTED
    assert q(d, GOOD, 0, 256, BAD, 4, 2, None, None) == ALIGN
    per = ctypes.byref(desc(format=1, factor=GOOD, factor_per_group=1))
    assert q(per, GOOD, 0, 256, GOOD, 4, 2, None, None) == INVALID           # one factor per token only
    assert q(ctypes.byref(desc(codes=None)), GOOD, 0, 256, None, 256, 0, None, None) == INVALID
    assert q(ctypes.byref(desc(scales=BAD)), GOOD, 0, 256, None, 256, 0, None, None) == ALIGN
    empty = ctypes.byref(desc(rows=0, group_rows=0, offsets=GOOD, codes=None, scales=None))
    assert q(empty, None, 0, 256, None, 0, 0, None, None) == 0
    assert q(d, None, 0, 256, GOOD, 0, 2, None, None) == 0


def test_product_refusals(L):
    n = ctypes.c_size_t(0)
    assert L.moe_mx4_gemm_workspace_size(ctypes.byref(n)) == 0 and n.value >= 256
    assert L.moe_mx4_gemm_workspace_size(None) == INVALID
    a, ws = desc(group_rows=0, offsets=GOOD), n.value

    def gemm(w=None, a=a, out=GOOD, dtype=0, p=GOOD, size=ws):
        w = desc(rows=400, group_rows=200) if w is None else w
        return L.moe_mx4_grouped_gemm(ctypes.byref(a), ctypes.byref(w), out, dtype, p, size, None)

    assert gemm(w=desc(format=1, rows=400, group_rows=200)) == INVALID       # formats differ
    assert gemm(w=desc(rows=400, group_rows=200, K=384)) == INVALID
    assert gemm(w=desc(rows=600, group_rows=200, groups=3)) == INVALID
    assert gemm(w=desc(rows=400, group_rows=0, offsets=GOOD)) == INVALID     # ragged weights
    assert gemm(a=desc(format=1, factor=GOOD, factor_per_group=1), w=desc(format=1)) == INVALID
    assert gemm(out=None) == INVALID and gemm(out=BAD) == ALIGN
    assert gemm(dtype=3) == INVALID
    assert gemm(size=ws - 1) == WORKSPACE and gemm(p=None) == INVALID and gemm(p=BAD) == ALIGN
    assert gemm(a=desc(rows=0, group_rows=0, offsets=GOOD)) == 0


def test_ffn_refusals(L):
    n = ctypes.c_size_t(0)
    a, g, d = desc(group_rows=0, offsets=GOOD), desc(rows=1024, group_rows=512), desc(rows=512, group_rows=256)

    def size(a=a, g=g):
        return L.moe_mx4_ffn_workspace_size(ctypes.byref(a), ctypes.byref(g), ctypes.byref(n))

    assert size() == 0
    # h of 256 rows x 256 elements: codes and the scales of 256 / 128 + 2 tiles of 2 pieces
    assert n.value >= 256 * 128 + 4 * 2 * 512
    ws = n.value

    def ffn(a=a, g=g, d=d, hf=None, tok=None, gate=None, scale=1.0, out=GOOD, dtype=0, p=GOOD, size=ws):
        return L.moe_mx4_grouped_ffn(ctypes.byref(a), ctypes.byref(g), ctypes.byref(d), hf, tok, gate, scale, out,
                                     dtype, p, size, None)

    assert size(g=desc(rows=1000, group_rows=500)) == UNSUPPORTED and ffn(g=desc(rows=1000, group_rows=500)) == UNSUPPORTED
    assert ffn(g=desc(rows=1002, group_rows=501)) == INVALID                 # an odd number of rows
    assert ffn(d=desc(rows=510, group_rows=255)) == INVALID                  # H rows in w_down
    assert ffn(d=desc(rows=512, group_rows=256, K=128)) == INVALID
    assert ffn(hf=GOOD) == INVALID                                           # a factor with mxfp4
    assert ffn(scale=float("nan")) == INVALID
    assert ffn(size=ws - 1) == WORKSPACE and ffn(p=None) == INVALID
    assert ffn(tok=GOOD, gate=GOOD, dtype=0) == INVALID                      # fused needs fp32
    assert ffn(tok=GOOD, dtype=1) == INVALID and ffn(tok=BAD, gate=GOOD, dtype=1) == ALIGN
    assert ffn(out=BAD) == ALIGN
    assert ffn(a=desc(rows=0, group_rows=0, offsets=GOOD)) == 0


def test_scale_buffer_covers_every_offset_pattern(L):
    """Each row's piece lies inside the buffer and no two (row, block) pairs share a byte."""
    for fmt in ("mxfp4", "nvfp4"):
        for counts in ([1], [0, 0, 1], [128, 1, 127, 129], [1] * 40, [300, 0, 5], [127, 127, 127]):
            off = [0]
            for c in counts:
                off.append(off[-1] + c)
            n = ctypes.c_size_t(0)
            d = desc(format=mx4.FORMATS[fmt], rows=off[-1], K=384, groups=len(counts), group_rows=0, offsets=GOOD)
            assert L.moe_mx4_scale_bytes(ctypes.byref(d), ctypes.byref(n)) == 0
            at = ref.scale_index(off, 384, fmt).flatten()
            assert at.unique().numel() == at.numel() and int(at.max()) < n.value
    assert L.moe_mx4_scale_bytes(None, ctypes.byref(n)) == INVALID
    assert L.moe_mx4_scale_bytes(ctypes.byref(desc(K=100)), ctypes.byref(n)) == UNSUPPORTED


def norm_desc(**kw):
    base = dict(T=4, H=256, dtype="bf16", gate="none", eps=1e-5, scale=1.0)
    base.update(kw)
    return norm.make_desc(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(dtype=4), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(H=250), UNSUPPORTED), (dict(H=16400), UNSUPPORTED), (dict(T=1 << 24), UNSUPPORTED)])
def test_norm_limits(L, kw, code):
    d = norm_desc(**kw)
    n = ctypes.c_size_t(0)
    assert L.moe_block_norm(ctypes.byref(d), *([GOOD] * 10), None) == code
    assert L.moe_block_norm_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code
    assert L.moe_block_norm_backward(ctypes.byref(d), *([GOOD] * 15), 1 << 40, None) == code


def test_norm_parts_have_to_agree(L):
    names = ["residual", "block", "w_post", "gate", "w_pre", "residual_out", "normed", "rstd_block", "rstd_res"]
    full = {k: GOOD for k in names}
    full["gate"] = None

    def fwd(d=None, **kw):
        d = norm_desc() if d is None else d
        return L.moe_block_norm(ctypes.byref(d), *[{**full, **kw}[k] for k in names], None)

    for k in ("residual", "residual_out", "normed", "block", "w_post", "w_pre"):
        assert fwd(**{k: None}) == INVALID, k       # the others still name its part
    assert fwd(gate=GOOD) == INVALID and fwd(norm_desc(gate="token")) == INVALID
    assert fwd(w_post=BAD) == ALIGN and fwd(block=BAD) == ALIGN
    assert fwd(block=None, w_post=None, residual_out=None, rstd_block=None, w_pre=None, normed=None,
               rstd_res=None) == INVALID            # nothing to do
    n = ctypes.c_size_t(0)
    assert L.moe_block_norm_workspace_size(ctypes.byref(norm_desc()), ctypes.byref(n)) == 0
    bn = ["d_residual_out", "d_normed", "residual_out", "block", "w_post", "gate", "w_pre", "rstd_block", "rstd_res",
          "d_residual", "d_block", "d_w_post", "d_gate", "d_w_pre", "ws"]
    fullb = {k: GOOD for k in bn}
    fullb["gate"] = fullb["d_gate"] = None

    def bwd(size=n.value, **kw):
        return L.moe_block_norm_backward(ctypes.byref(norm_desc()), *[{**fullb, **kw}[k] for k in bn], size, None)

    for k in bn[1:]:
        if k not in ("gate", "d_gate"):
            assert bwd(**{k: None}) == INVALID, k
    assert bwd(d_gate=GOOD) == INVALID and bwd(gate=GOOD, d_gate=GOOD) == INVALID
    assert bwd(d_w_pre=BAD) == ALIGN and bwd(size=n.value - 1) == WORKSPACE


def test_python_checks():
    with pytest.raises(ValueError, match="format"):
        mx4.allocate("fp4", 4, 128, device="cpu")
    with pytest.raises(ValueError, match="equal groups"):
        mx4.allocate("mxfp4", 5, 128, groups=2, device="cpu")
    with pytest.raises(ValueError, match="tensor_scale"):
        mx4.allocate("nvfp4", 4, 128, groups=2, tensor_scale=torch.ones(3), device="cpu")
    with pytest.raises(abi.MoEError):
        mx4.allocate("mxfp4", 4, 100, device="cpu")
    with pytest.raises(ValueError, match="gate"):
        norm.make_desc(1, 16, gate="row")
    with pytest.raises(ValueError, match="tensor"):
        mx4._tensor(3, "x", (torch.float32,))
    with pytest.raises(ValueError, match="expected"):
        mx4._tensor(torch.ones(3), "x", (torch.bfloat16,))
    with pytest.raises(ValueError, match="shape"):
        mx4._tensor(torch.ones(3), "x", (torch.float32,), (4,))
    with pytest.raises(ValueError, match="contiguous"):
        mx4._tensor(torch.ones(3, 2).T, "x", (torch.float32,))
