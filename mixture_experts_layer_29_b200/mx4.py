"""The layer's experts in microscaled 4-bit floating point (include/moe_mx4.h).

Two formats: "mxfp4" (blocks of 32 with a power-of-two scale) and "nvfp4" (blocks of 16 with an
e4m3 scale times one fp32 factor per matrix or group). A `Matrix` is a 4-bit matrix on the
device: packed codes, block scales in the tensor cores' layout, and the rows' groups.

    a = mx4.allocate("mxfp4", rows, H, groups=n, offsets=offsets)   # ragged rows
    w = mx4.quantize_weight(w_bf16, "mxfp4")                        # [n, N, H], once
    mx4.quantize(x, a)
    mx4.grouped_gemm(a, w, out, mx4.gemm_workspace())               # out[r] = a[r] . w[g]^T

The calls marshal arguments only, like `abi`: the arithmetic runs in the library's kernels,
there is no fallback, and an error code raises abi.MoEError. Tensors are checked here for type,
device and contiguity (ValueError). Inference only: the 4-bit product has no backward.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re

import torch

from . import abi

HEADER = os.path.join(os.path.dirname(abi.HEADER), "moe_mx4.h")
FORMATS = {"mxfp4": 0, "nvfp4": 1}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
_DTYPES = {torch.bfloat16: abi.MOE_BF16, torch.float32: abi.MOE_FP32}


class Desc(ctypes.Structure):
    """moe_mx4_t"""
    _fields_ = [("format", ctypes.c_int32), ("rows", ctypes.c_int32), ("K", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("group_rows", ctypes.c_int32),
                ("factor_per_group", ctypes.c_int32), ("offsets", ctypes.c_void_p),
                ("factor", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


_P, _SZ, _I32, _I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
_D = ctypes.POINTER(Desc)
_SIGS = {
    "moe_mx4_scale_bytes": [_D, ctypes.POINTER(_SZ)],
    "moe_mx4_quantize": [_D, _P, _I32, _I64, _P, _I32, _I32, _P, _P],
    "moe_mx4_dequantize": [_D, _P, _I32, _I64, _P],
    "moe_mx4_pack_scales": [_D, _P, _P],
    "moe_mx4_gemm_workspace_size": [ctypes.POINTER(_SZ)],
    "moe_mx4_grouped_gemm": [_D, _D, _P, _I32, _P, _SZ, _P],
    "moe_mx4_ffn_workspace_size": [_D, _D, ctypes.POINTER(_SZ)],
    "moe_mx4_grouped_ffn": [_D, _D, _D, _P, _P, _P, ctypes.c_float, _P, _I32, _P, _SZ, _P],
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
    """Names of the functions include/moe_mx4.h declares."""
    return sorted(set(re.findall(r"^int\s+(moe_\w+)\s*\(", open(HEADER).read(), flags=re.M)))


# the current device and its current stream, without the objects around them: a call at a decode
# step takes the GPU a few microseconds, and torch.cuda's own functions as much again
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(stream, dev: int) -> int:
    return _raw_stream(dev) if stream is None else abi._stream(stream)


@contextlib.contextmanager
def _on(stream, dev: int):
    """Makes `stream` (a stream, its handle, or None: the current one) the current stream, so that what a
    call allocates and copies on the way is ordered with its kernels and belongs to their stream."""
    if stream is None:
        yield
        return
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(abi._stream(stream), dev)
    with torch.cuda.stream(stream):
        yield


def _check(rc: int, where: str):
    if rc != 0:
        raise abi.MoEError(rc, where)


def _tensor(t, name, dtypes, shape=None, optional=False, contiguous=True, dev=None, least=0):
    """Checks one tensor argument (of at least `least` elements) and returns its address (None for an
    absent optional one)."""
    if t is None and optional:
        return None
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is needed, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.numel() < least:
        raise ValueError(f"{name}: {t.numel()} elements, {least} are needed")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if t.get_device() != (_device() if dev is None else dev) or not t.is_cuda:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{_device()}")
    return t.data_ptr()


class Matrix:
    """A 4-bit matrix: rows of K elements in groups (see include/moe_mx4.h for the layout).

    codes [rows, K / 2] uint8, scales uint8, offsets int32 [groups + 1] (ragged groups) or None
    (groups of rows / groups rows each), tensor_scale fp32 [1] or [groups] (nvfp4) or None. The
    buffers are checked and kept when the matrix is made; their contents may change."""

    def __init__(self, fmt, rows, K, groups=1, offsets=None, tensor_scale=None, codes=None, device="cuda"):
        if fmt not in FORMATS:
            raise ValueError(f"format {fmt!r}: one of {sorted(FORMATS)}")
        if offsets is None and groups > 0 and rows % groups != 0:
            raise ValueError(f"{rows} rows in {groups} equal groups: give offsets")
        if tensor_scale is not None and tensor_scale.numel() not in (1, groups):
            raise ValueError(f"tensor_scale: {tensor_scale.numel()} values, expected 1 or {groups}")
        self._d = d = Desc(FORMATS[fmt], rows, K, groups, 0 if offsets is not None else rows // max(groups, 1),
                           int(tensor_scale is not None and tensor_scale.numel() > 1), None, None, None, None)
        n = _SZ(0)
        _check(lib().moe_mx4_scale_bytes(ctypes.byref(d), ctypes.byref(n)), "moe_mx4_scale_bytes")
        codes = torch.empty(rows, K // 2, dtype=torch.uint8, device=device) if codes is None else codes
        d.codes = _tensor(codes, "codes", (torch.uint8,), least=rows * (K // 2))
        scales = torch.empty(n.value, dtype=torch.uint8, device=device)
        self._parts = (fmt, rows, K, groups, offsets, tensor_scale, codes.view(rows, K // 2), scales)
        d.offsets = _tensor(offsets, "offsets", (torch.int32,), (groups + 1,), optional=True)
        d.factor = _tensor(tensor_scale, "tensor_scale", (torch.float32,), optional=True)
        d.scales = _tensor(scales, "scales", (torch.uint8,))
        self._dev = codes.get_device()

    fmt = property(lambda self: self._parts[0])
    rows = property(lambda self: self._parts[1])
    K = property(lambda self: self._parts[2])
    groups = property(lambda self: self._parts[3])
    offsets = property(lambda self: self._parts[4])
    tensor_scale = property(lambda self: self._parts[5])
    codes = property(lambda self: self._parts[6])
    scales = property(lambda self: self._parts[7])

    def desc(self, dev: int):
        """The matrix as the C ABI takes it, for a call on device `dev`."""
        if self._dev != dev:
            raise ValueError(f"a 4-bit matrix on cuda:{self._dev}, but the current device is cuda:{dev}")
        return ctypes.byref(self._d)


def allocate(fmt, rows, K, groups=1, offsets=None, tensor_scale=None, device="cuda") -> Matrix:
    """A Matrix with room for `rows` rows; quantize() fills it. offsets: device int32
    [groups + 1], read by every call (they may change between calls)."""
    return Matrix(fmt, rows, K, groups, offsets, tensor_scale, device=device)


def from_checkpoint(fmt, codes, scales, tensor_scale=None, stream=None) -> Matrix:
    """A weight from a 4-bit checkpoint: codes [groups, N, K / 2] uint8 (used as they are) and
    row-major block scales [groups, N, K / B] uint8, laid out for the tensor cores here, once.

    Here and in quantize_weight, with a stream given, all of the work is queued on it, the matrix's memory
    is that stream's, and the inputs have to be ready on it."""
    groups, N, half = codes.shape
    dev = _device()
    with _on(stream, dev):
        m = Matrix(fmt, groups * N, 2 * half, groups, None, tensor_scale, codes=codes, device=codes.device)
        p = _tensor(scales, "scales", (torch.uint8,), (groups, N, m.K // BLOCK[fmt]))
        _check(lib().moe_mx4_pack_scales(m.desc(dev), p, _raw_stream(dev)), "moe_mx4_pack_scales")
    return m


def quantize_weight(w, fmt, tensor_scale=None, stream=None) -> Matrix:
    """A weight [groups, N, K] bf16 or fp32, of any strides, in 4 bits, once, at load time."""
    groups, N, K = w.shape
    with _on(stream, _device()):
        m = Matrix(fmt, groups * N, K, groups, None, tensor_scale, device=w.device)
        return quantize(w.reshape(groups * N, K), m)


_FLOATS = (torch.bfloat16, torch.float32)
_F32, _I32T, _U8 = (torch.float32,), (torch.int32,), (torch.uint8,)
_STATUS = (torch.uint8, torch.int32)


def _tensors(dev, *args):
    """The addresses of several contiguous arguments (tensor or None, name, dtype, shape), None for absent
    ones. One loop without a call per tensor: the gradients of a small block norm, 15 of them, take
    14.4 us on the host instead of 15.7."""
    out = []
    for t, name, dtype, shape in args:
        if t is None:
            out.append(None)
            continue
        try:
            ok = t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()
        except AttributeError:
            ok = False
        out.append(t.data_ptr() if ok else _tensor(t, name, (dtype,), shape, dev=dev))
    return out


def _rows(t, name, K, rows, dev):
    """(address, dtype code, row stride) of a [rows, K] operand whose rows may be strided."""
    p = _tensor(t, name, _FLOATS, (rows, K), contiguous=False, dev=dev)
    if rows and t.stride(1) != 1:
        raise ValueError(f"{name}: elements of a row are not adjacent")
    return p, _DTYPES[t.dtype], t.stride(0) if rows > 1 else K


def quantize(x, m: Matrix, row_of=None, status=None, stream=None) -> Matrix:
    """Rounds x into m. Without row_of, row r of m is row r of x [rows, K]. With row_of int32
    [tokens, picks] (abi.permute's), row t of x [tokens, K] goes to each row row_of[t, p] >= 0
    of m. status: a device int32 that receives a device-side check's failure (or a workspace, in whose
    first word abi.read_device_status looks for it)."""
    dev = _device()
    tokens, picks = m.rows, 0
    if row_of is not None:
        if row_of.dim() != 2:
            raise ValueError("row_of: [tokens, picks]")
        tokens, picks = row_of.shape
        row_of = _tensor(row_of, "row_of", _I32T, dev=dev)
    p, dt, ld = _rows(x, "x", m.K, tokens, dev)
    if status is not None:
        status = _tensor(status, "status", _STATUS, dev=dev, least=1 if getattr(status, "dtype", None) is torch.int32 else 4)
    _check(lib().moe_mx4_quantize(m.desc(dev), p, dt, ld, row_of, tokens, picks, status, _stream(stream, dev)),
           "moe_mx4_quantize")
    return m


def dequantize(m: Matrix, out, stream=None):
    """The values of m into out [rows, K] bf16 or fp32 (rows of no group are left alone)."""
    dev = _device()
    p, dt, ld = _rows(out, "out", m.K, m.rows, dev)
    _check(lib().moe_mx4_dequantize(m.desc(dev), p, dt, ld, _stream(stream, dev)), "moe_mx4_dequantize")
    return out


def gemm_workspace(device="cuda"):
    """Workspace of grouped_gemm (status word), zeroed."""
    n = _SZ(0)
    _check(lib().moe_mx4_gemm_workspace_size(ctypes.byref(n)), "moe_mx4_gemm_workspace_size")
    return torch.zeros(n.value, dtype=torch.uint8, device=device)


def grouped_gemm(a: Matrix, w: Matrix, out, ws, stream=None):
    """out[r] = a[r] . w[g]^T for the rows r of each group g; out [a.rows, N] bf16 or fp32."""
    dev = _device()
    p = _tensor(out, "out", _FLOATS, (a.rows, w.rows // max(w.groups, 1)), dev=dev)
    _check(lib().moe_mx4_grouped_gemm(a.desc(dev), w.desc(dev), p, _DTYPES[out.dtype],
                                      _tensor(ws, "ws", _U8, dev=dev), ws.numel(), _stream(stream, dev)),
           "moe_mx4_grouped_gemm")
    return out


def ffn_workspace(a: Matrix, w_gate_up: Matrix, device="cuda"):
    """Workspace of grouped_ffn (status word and h), zeroed."""
    n = _SZ(0)
    _check(lib().moe_mx4_ffn_workspace_size(ctypes.byref(a._d), ctypes.byref(w_gate_up._d), ctypes.byref(n)),
           "moe_mx4_ffn_workspace_size")
    return torch.zeros(n.value, dtype=torch.uint8, device=device)


def grouped_ffn(a: Matrix, w_gate_up: Matrix, w_down: Matrix, out, ws, h_scale=None, perm_token=None,
                row_gate=None, scale=1.0, stream=None):
    """The grouped SwiGLU FFN on 4-bit experts. Without perm_token: out [a.rows, H] bf16 or
    fp32, one row each. With it (fused combine): out fp32 [tokens, H], to which
    scale * row_gate[r] * y[r] is added at perm_token[r] (int32, from 0 to tokens - 1; perm_token and
    row_gate have an element for each of a's rows, those of no group are not looked at)."""
    dev = _device()
    if (perm_token is None) != (row_gate is None):
        raise ValueError("perm_token and row_gate go together")
    perm_token = _tensor(perm_token, "perm_token", _I32T, None, True, dev=dev, least=a.rows)
    row_gate = _tensor(row_gate, "row_gate", _F32, None, True, dev=dev, least=a.rows)
    p = _tensor(out, "out", _FLOATS, (a.rows if perm_token is None else out.shape[0], a.K), dev=dev)
    _check(lib().moe_mx4_grouped_ffn(
        a.desc(dev), w_gate_up.desc(dev), w_down.desc(dev), _tensor(h_scale, "h_scale", _F32, (1,), True, dev=dev),
        perm_token, row_gate, scale, p, _DTYPES[out.dtype],
        _tensor(ws, "ws", _U8, dev=dev), ws.numel(), _stream(stream, dev)), "moe_mx4_grouped_ffn")
    return out


class Mx4MoELayer:
    """One LongCat-Flash MoE layer whose FFN experts are 4-bit: the router, the permutation, the
    combine and the PID bias of abi.MoELayer around mx4.grouped_ffn. Each token's activations
    are rounded once and written to its picks' rows.

    w_gate_up, w_down: Matrix (quantize_weight or from_checkpoint). x_scale, h_scale: the
    activations' nvfp4 factors, fp32 [1], or None. forward(x), x [T, H] bf16, returns what
    abi.MoELayer.forward returns."""

    def __init__(self, shape: abi.Shape, w_router, bias, w_gate_up: Matrix, w_down: Matrix,
                 pid: abi.Pid | None = None, x_scale=None, h_scale=None):
        if shape.dtype != abi.MOE_BF16:
            raise ValueError("4-bit experts need a bf16 layer")
        N = shape.n_ffn
        for name, m, want in (("w_gate_up", w_gate_up, (N, N * 2 * shape.I, shape.H)),
                              ("w_down", w_down, (N, N * shape.H, shape.I))):
            if (m.groups, m.rows, m.K) != want or m.offsets is not None:
                raise ValueError(f"{name}: {m.groups} groups of {m.rows} x {m.K} in all, expected {want}")
        if w_down.fmt != w_gate_up.fmt:
            raise ValueError(f"w_down: {w_down.fmt}, but w_gate_up is {w_gate_up.fmt}")
        _tensor(w_router, "w_router", _F32, (shape.E, shape.H))
        _tensor(bias, "bias", _F32, (shape.E,))
        _tensor(h_scale, "h_scale", _F32, (1,), optional=True)
        self.shape, self.w_router, self.bias = shape, w_router, bias
        self.w_gate_up, self.w_down, self.h_scale, self.pid = w_gate_up, w_down, h_scale, pid
        dev = w_gate_up.codes.device
        T, H, K, rows = shape.T, shape.H, shape.K, shape.T * shape.K
        i32, f32 = torch.int32, torch.float32
        fused = shape.combine == abi.MOE_COMBINE_FUSED
        self.scratch = torch.zeros(max(abi.scratch_size(shape), 256), dtype=torch.uint8, device=dev)
        self.logits = torch.empty(T, shape.E, dtype=f32, device=dev)
        self.topk_idx = torch.empty(T, K, dtype=i32, device=dev)
        self.topk_gate = torch.empty(T, K, dtype=f32, device=dev)
        self.counts = torch.empty(shape.E, dtype=i32, device=dev)
        self.nffn_hist = torch.empty(K + 1, dtype=i32, device=dev)
        self.zgate = torch.empty(T, dtype=f32, device=dev)
        self.offsets = torch.zeros(N + 1, dtype=i32, device=dev)
        self.perm_token = torch.empty(rows, dtype=i32, device=dev)
        self.row_of = torch.empty(T, K, dtype=i32, device=dev)
        self.row_gate = torch.empty(rows, dtype=f32, device=dev)
        self.out_acc = torch.empty(T, H, dtype=f32, device=dev) if fused else None
        self.y = None if fused else torch.empty(rows, H, dtype=torch.bfloat16, device=dev)
        self.out = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        self.a = allocate(w_gate_up.fmt, rows, H, N, self.offsets, x_scale, device=dev)
        self.ws = ffn_workspace(self.a, w_gate_up, device=dev)
        self.pid_state = torch.empty(3 * N, dtype=f32, device=dev)
        self.stats = torch.zeros(8, dtype=f32, device=dev)
        abi.pid_init(shape, bias, self.pid_state)

    def forward(self, x, logits_in=None, stream=None):
        s, dev = self.shape, _device()
        _tensor(x, "x", (torch.bfloat16,), (s.T, s.H), dev=dev)
        _tensor(logits_in, "logits_in", _F32, (s.T, s.E), optional=True, dev=dev)
        abi.route(s, x, self.w_router, logits_in, self.bias, None if logits_in is not None else self.logits,
                  self.topk_idx, self.topk_gate, self.counts, self.nffn_hist, self.zgate, self.scratch, stream)
        abi.permute(s, self.topk_idx, self.topk_gate, self.zgate, x, self.offsets, self.perm_token,
                    self.row_of, self.row_gate, None, self.out_acc, self.scratch, stream)
        quantize(x, self.a, self.row_of, self.ws, stream)
        if self.out_acc is not None:
            grouped_ffn(self.a, self.w_gate_up, self.w_down, self.out_acc, self.ws, self.h_scale,
                        self.perm_token, self.row_gate, s.ffn_out_scale, stream)
        else:
            grouped_ffn(self.a, self.w_gate_up, self.w_down, self.y, self.ws, self.h_scale, stream=stream)
        abi.combine(s, x, self.y, self.out_acc, self.topk_gate, self.row_of, self.zgate, self.out, stream)
        return self.out, self.topk_idx, self.topk_gate, self.counts, self.nffn_hist

    def update_bias(self, stream=None):
        if self.pid is None:
            raise ValueError("no PID gains given")
        abi.pid_bias_update(self.pid, self.shape, self.counts, self.nffn_hist, self.bias, self.pid_state,
                            self.stats, stream)
        return self.stats
