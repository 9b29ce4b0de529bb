"""What the 4-bit binding refuses before it calls the library (no GPU: the device is a stand-in)."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from mixture_experts_layer_29_b200 import abi, build, mx4, norm


@pytest.fixture
def no_calls(monkeypatch):
    """The current device is 0, and a call of the library fails the test."""
    monkeypatch.setattr(mx4, "_device", lambda: 0)
    monkeypatch.setattr(mx4, "_raw_stream", lambda dev: 0)

    def called():
        raise AssertionError("the library was called")

    monkeypatch.setattr(mx4, "lib", called)


def rows_of(n, K=256):
    return SimpleNamespace(rows=n, K=K, groups=1, fmt="mxfp4", desc=lambda dev: None)


@pytest.mark.parametrize("tok,gate,match", [
    (torch.zeros(10, dtype=torch.int32), None, "go together"), (None, torch.zeros(10), "go together"),
    (torch.zeros(9, dtype=torch.int32), torch.zeros(10), "perm_token: 9 elements, 10"),
    (torch.zeros(10, dtype=torch.int32), torch.zeros(3, 3), "row_gate: 9 elements, 10"),
    (torch.zeros(10, dtype=torch.int64), torch.zeros(10), "perm_token: torch.int64"),
    (torch.zeros(10, dtype=torch.int32), torch.zeros(10, dtype=torch.bfloat16), "row_gate: torch.bfloat16")])
def test_fused_combine_needs_a_token_and_a_gate_per_row(no_calls, monkeypatch, tok, gate, match):
    if tok is not None and tok.numel() == 10 and tok.dtype == torch.int32 and gate is not None:
        real = mx4._tensor          # let perm_token, which is right, pass though it is on the CPU
        monkeypatch.setattr(mx4, "_tensor", lambda t, name, *a, **k: 0 if name == "perm_token" else real(t, name, *a, **k))
    with pytest.raises(ValueError, match=match):
        mx4.grouped_ffn(rows_of(10), rows_of(1024), rows_of(256), torch.zeros(4, 256), torch.zeros(8), None, tok, gate)


def test_library_refuses_gates_without_tokens():
    build.build()
    L, good = mx4.lib(), 1 << 20
    a = mx4.Desc(0, 256, 256, 2, 0, 0, good, None, good, good)
    g = mx4.Desc(0, 1024, 256, 2, 512, 0, None, None, good, good)
    d = mx4.Desc(0, 512, 256, 2, 256, 0, None, None, good, good)
    n = ctypes.c_size_t(0)
    assert L.moe_mx4_ffn_workspace_size(ctypes.byref(a), ctypes.byref(g), ctypes.byref(n)) == 0
    args = (ctypes.byref(a), ctypes.byref(g), ctypes.byref(d), None)
    assert L.moe_mx4_grouped_ffn(*args, None, good, 1.0, good, 1, good, n.value, None) == -1


@pytest.mark.parametrize("status,match", [
    (torch.zeros(3, dtype=torch.uint8), "status: 3 elements, 4"), (torch.zeros(0, dtype=torch.int32), "status: 0 elements, 1"),
    (torch.zeros(4, dtype=torch.int64), "status: torch.int64"), (torch.zeros(8, dtype=torch.uint8)[::2], "status: not contiguous"),
    (7, "status: a tensor")])
def test_quantize_needs_a_whole_status_word(no_calls, monkeypatch, status, match):
    monkeypatch.setattr(mx4, "_rows", lambda *a: (0, 0, 256))
    with pytest.raises(ValueError, match=match):
        mx4.quantize(torch.zeros(10, 256), rows_of(10), None, status)


def test_library_refuses_a_status_off_four_bytes():
    build.build()
    good = 1 << 20
    m = mx4.Desc(0, 256, 256, 2, 128, 0, None, None, good, good)
    call = mx4.lib().moe_mx4_quantize
    assert [call(ctypes.byref(m), good, 0, 256, None, 256, 0, good + off, None) for off in (1, 2, 3)] == [-3, -3, -3]


def layer(no_calls, monkeypatch):
    monkeypatch.setattr(abi, "lib", lambda: pytest.fail("the library was called"))
    lay = object.__new__(mx4.Mx4MoELayer)
    lay.shape = abi.make_shape(8, 256, 128, 6, 2, 2, "bf16", "deterministic")
    for name in ("w_router", "bias", "logits", "topk_idx", "topk_gate", "counts", "nffn_hist", "zgate", "scratch"):
        setattr(lay, name, torch.zeros(8))
    return lay


@pytest.mark.parametrize("x,logits,match", [
    (torch.zeros(7, 256, dtype=torch.bfloat16), None, "x: shape"), (torch.zeros(8, 256), None, "x: torch.float32"),
    (torch.zeros(8, 512, dtype=torch.bfloat16)[:, :256], None, "x: not contiguous"),
    (torch.zeros(8, 256, dtype=torch.bfloat16), None, "x: on cpu"), (None, None, "x: a tensor"),
    ("right", torch.zeros(8, 7), "logits_in: shape"), ("right", torch.zeros(8, 8).double(), "logits_in: torch.float64")])
def test_layer_looks_at_its_input_before_the_router_reads_it(no_calls, monkeypatch, x, logits, match):
    lay, real = layer(no_calls, monkeypatch), mx4._tensor
    if isinstance(x, str):
        monkeypatch.setattr(mx4, "_tensor", lambda t, name, *a, **k: 0 if name == "x" else real(t, name, *a, **k))
        x = torch.zeros(8, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=match):
        lay.forward(x, logits)


@pytest.mark.parametrize("kw,match", [
    (dict(fmt="nvfp4"), "w_down: nvfp4"), (dict(router=torch.zeros(8, 255)), "w_router: shape"),
    (dict(bias=torch.zeros(7)), "bias: shape"), (dict(h=torch.zeros(2)), "h_scale: shape")])
def test_layer_looks_at_its_weights(no_calls, monkeypatch, kw, match):
    real = mx4._tensor
    monkeypatch.setattr(mx4, "_tensor", lambda t, name, *a, **k: 0 if t is None else real(t, name, *a, **k) if name in match else 0)
    matrix = lambda n, rows, K, fmt: SimpleNamespace(groups=n, rows=rows, K=K, offsets=None, fmt=fmt)     # noqa: E731
    with pytest.raises(ValueError, match=match):
        mx4.Mx4MoELayer(abi.make_shape(8, 256, 128, 6, 2, 2, "bf16"), kw.get("router", torch.zeros(8, 256)),
                        kw.get("bias", torch.zeros(8)), matrix(6, 6 * 256, 256, "mxfp4"),
                        matrix(6, 6 * 256, 128, kw.get("fmt", "mxfp4")), h_scale=kw.get("h"))


@pytest.mark.parametrize("normed,match", [(torch.zeros(7, 256, dtype=torch.bfloat16), "normed: shape"),
                                          (torch.zeros(8, 256), "normed: torch.float32"),
                                          (torch.zeros(256, 8, dtype=torch.bfloat16).T, "normed: not contiguous")])
def test_block_looks_at_a_norm_that_it_is_given(no_calls, normed, match):
    lay = SimpleNamespace(shape=abi.make_shape(8, 256, 128, 6, 2, 2, "bf16"), out=torch.zeros(8, 256, dtype=torch.bfloat16),
                          forward=lambda *a, **k: pytest.fail("the layer was called"))
    block = norm.MoEBlock(lay, torch.ones(256))
    with pytest.raises(ValueError, match=match):
        block.forward(torch.zeros(8, 256, dtype=torch.bfloat16), normed=normed)


@pytest.mark.parametrize("codes,match", [(torch.zeros(2, 8, 256, dtype=torch.uint8)[:, :, ::2], "codes: not contiguous"),
                                         (torch.zeros(2, 8, 128), "codes: torch.float32"),
                                         (torch.zeros(2, 8, 128, dtype=torch.uint8), "codes: on cpu")])
def test_checkpoint_codes_are_looked_at_first(monkeypatch, codes, match):
    build.build()
    monkeypatch.setattr(mx4, "_device", lambda: 0)
    with pytest.raises(ValueError, match=match):
        mx4.from_checkpoint("mxfp4", codes, torch.zeros(2, 8, 8, dtype=torch.uint8))


def test_matrix_needs_all_of_its_codes(monkeypatch):
    build.build()
    monkeypatch.setattr(mx4, "_device", lambda: 0)
    with pytest.raises(ValueError, match="codes: 384 elements, 512"):
        mx4.Matrix("mxfp4", 4, 256, codes=torch.zeros(3, 128, dtype=torch.uint8), device="cpu")
