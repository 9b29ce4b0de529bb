"""The norms around a block (include/moe_norm.h): the RMS norm after a block, its gate and
residual scale, the residual add and the RMS norm before the next block in one call, and their
gradients.

    d = norm.make_desc(T, H, dtype="bf16", gate="channel", eps=1e-5, scale=0.5)
    norm.block_norm(d, residual, block, w_post, gate, w_pre, residual_out, normed,
                    rstd_block, rstd_res)

Leave a part out with None: block None is the norm before the first block, w_pre None the
residual add after the last one, w_post None a block without a norm after it. The calls marshal
arguments only, like `abi`; tensors are checked for type, shape, device and contiguity
(ValueError), the rest by the library (abi.MoEError).
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

from . import abi
from .mx4 import _U8, _check, _device, _stream, _tensor, _tensors

HEADER = os.path.join(os.path.dirname(abi.HEADER), "moe_norm.h")
GATES = {"none": 0, "token": 1, "channel": 2}


class Desc(ctypes.Structure):
    """moe_norm_t"""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("eps", ctypes.c_float), ("scale", ctypes.c_float)]


_FP32 = torch.float32
_P, _SZ = ctypes.c_void_p, ctypes.c_size_t
_D = ctypes.POINTER(Desc)
_SIGS = {
    "moe_block_norm": [_D] + [_P] * 10,
    "moe_block_norm_workspace_size": [_D, ctypes.POINTER(_SZ)],
    "moe_block_norm_backward": [_D] + [_P] * 15 + [_SZ, _P],
}
_lib = None


def lib() -> ctypes.CDLL:
    """The library (abi.lib()) with this header's signatures set."""
    global _lib
    if _lib is None:
        L = abi.lib()
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.restype, f.argtypes = ctypes.c_int, args
        _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/moe_norm.h declares."""
    return sorted(set(re.findall(r"^int\s+(moe_\w+)\s*\(", open(HEADER).read(), flags=re.M)))


def make_desc(T, H, dtype="bf16", gate="none", eps=1e-5, scale=1.0) -> Desc:
    if gate not in GATES:
        raise ValueError(f"gate {gate!r}: one of {sorted(GATES)}")
    dt = {"bf16": abi.MOE_BF16, "fp32": abi.MOE_FP32}[dtype] if isinstance(dtype, str) else int(dtype)
    return Desc(T, H, dt, GATES[gate], eps, scale)


_ROWS = {abi.MOE_BF16: torch.bfloat16, abi.MOE_FP32: torch.float32}


def _of_gate(d: Desc):
    return (d.T,) if d.gate == GATES["token"] else (d.H,)


def block_norm(d: Desc, residual, block, w_post, gate, w_pre, residual_out, normed, rstd_block=None,
               rstd_res=None, stream=None):
    """moe_block_norm; returns (residual_out, normed)."""
    dev, rows, dt, T, H = _device(), (d.T, d.H), _ROWS.get(d.dtype), (d.T,), (d.H,)
    if residual is None:
        raise ValueError("residual: a tensor is needed")
    _check(lib().moe_block_norm(ctypes.byref(d), *_tensors(
        dev, (residual, "residual", dt, rows), (block, "block", dt, rows), (w_post, "w_post", _FP32, H),
        (gate, "gate", _FP32, _of_gate(d)), (w_pre, "w_pre", _FP32, H), (residual_out, "residual_out", dt, rows),
        (normed, "normed", dt, rows), (rstd_block, "rstd_block", _FP32, T), (rstd_res, "rstd_res", _FP32, T)),
        _stream(stream, dev)), "moe_block_norm")
    return residual_out, normed


def workspace(d: Desc, device="cuda"):
    """Workspace of block_norm_backward (status word, partial sums), zeroed."""
    n = _SZ(0)
    _check(lib().moe_block_norm_workspace_size(ctypes.byref(d), ctypes.byref(n)), "moe_block_norm_workspace_size")
    return torch.zeros(n.value, dtype=torch.uint8, device=device)


def block_norm_backward(d: Desc, d_residual_out, d_normed, residual_out, block, w_post, gate, w_pre,
                        rstd_block, rstd_res, d_residual, d_block, d_w_post, d_gate, d_w_pre, ws,
                        stream=None):
    """moe_block_norm_backward: writes the gradients of the parts that the forward had."""
    dev, rows, dt, T, H = _device(), (d.T, d.H), _ROWS.get(d.dtype), (d.T,), (d.H,)
    G = _of_gate(d)
    if d_residual is None:
        raise ValueError("d_residual: a tensor is needed")
    _check(lib().moe_block_norm_backward(ctypes.byref(d), *_tensors(
        dev, (d_residual_out, "d_residual_out", dt, rows), (d_normed, "d_normed", dt, rows),
        (residual_out, "residual_out", dt, rows), (block, "block", dt, rows), (w_post, "w_post", _FP32, H),
        (gate, "gate", _FP32, G), (w_pre, "w_pre", _FP32, H), (rstd_block, "rstd_block", _FP32, T),
        (rstd_res, "rstd_res", _FP32, T), (d_residual, "d_residual", dt, rows), (d_block, "d_block", dt, rows),
        (d_w_post, "d_w_post", _FP32, H), (d_gate, "d_gate", _FP32, G), (d_w_pre, "d_w_pre", _FP32, H)),
        _tensor(ws, "ws", _U8, dev=dev), ws.numel(), _stream(stream, dev)), "moe_block_norm_backward")


class MoEBlock:
    """A MoE layer on the residual stream: the norm before it, the layer, and the norm after it
    with its gate and residual scale, joined with the norm before the next block.

    layer: abi.MoELayer or mx4.Mx4MoELayer of a [T, H] batch. w_pre [H] fp32; w_post [H] fp32 or
    None; gate fp32 [T] or [H] with its kind, or None. forward(residual, w_next) returns
    (residual_out, normed): the stream after the block and, with w_next [H], its norm before
    the next block (None without). Called with `normed` of a previous block, the norm before
    this one is that block's and is not computed again. Both are the block's own buffers, which its
    next forward writes again.

    Forward only: it keeps no rstd. Training calls block_norm with the rstd_* outputs and
    block_norm_backward around abi.run_steps and abi.backward."""

    def __init__(self, layer, w_pre, w_post=None, gate=None, gate_kind="none", eps=1e-5, scale=1.0):
        s = layer.shape
        if (gate is None) != (gate_kind == "none"):
            raise ValueError("gate and gate_kind go together")
        self.layer, self.w_pre, self.w_post, self.gate = layer, w_pre, w_post, gate
        dt = abi.MOE_BF16 if s.dtype == abi.MOE_BF16 else abi.MOE_FP32
        self.before = make_desc(s.T, s.H, dt, "none", eps, 1.0)
        self.after = make_desc(s.T, s.H, dt, gate_kind, eps, scale)
        self.x = torch.empty_like(layer.out[: s.T])
        self.residual_out, self.normed = torch.empty_like(self.x), torch.empty_like(self.x)

    def forward(self, residual, w_next=None, normed=None, stream=None):
        if normed is None:
            block_norm(self.before, residual, None, None, None, self.w_pre, None, self.x, stream=stream)
            normed = self.x
        else:       # the layer's own call takes it as it is
            _tensor(normed, "normed", (self.x.dtype,), self.x.shape)
        out = self.layer.forward(normed, stream=stream)[0][: self.layer.shape.T]
        return block_norm(self.after, residual, out, self.w_post, self.gate, w_next, self.residual_out,
                          None if w_next is None else self.normed, stream=stream)
