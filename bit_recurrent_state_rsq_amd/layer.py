"""Operators of the layer around the decode step: the short causal convolution,
the selective state-space scan of prompts and its single-token step, the RMS
norm with an 8-bit output, and products with 4-bit weights.

Argument marshalling for the C ABI (include/rsq.h, which documents every
argument); the arithmetic runs in the HIP kernels. Activations are fp32 or
bf16 tensors on one device, parameters fp32. Calls go to `stream` (default: the
device's current stream) and can be captured in a graph; a tensor argument's
rows may be strided, its elements within a row are contiguous. A tensor that a
call makes belongs to the stream the call ran on.

    y = causal_conv(xbc, weight, bias, state=conv_state, activation="silu")
    y, S = ssm_scan(x, dt, A, B, C, D=D, dt_bias=dt_bias, softplus=True)     # a prompt
    y = ssm_step(S, x, dt, A, B, C, D=D, dt_bias=dt_bias, softplus=True)     # the next token

A token's kernels take a few microseconds, so the checks here are laid out for
the call that passes them: one comparison a property, messages made only on
failure, the argument struct packed in one go.
"""
import ctypes
import struct

import torch
from torch import Tensor

from . import _abi
from ._abi import check, lib

__all__ = ["causal_conv", "causal_conv_step", "ssm_scan", "ssm_step", "rms_norm", "W4Weight", "w4_linear"]

_F32, _BF16 = torch.float32, torch.bfloat16
_DTYPE = {_F32: _abi.F32, _BF16: _abi.BF16}
_OUT = {"f32": (_abi.F32, _F32), "bf16": (_abi.BF16, _BF16), "int8": (_abi.INT8, torch.int8),
        "e4m3": (_abi.E4M3, torch.float8_e4m3fn)}
_W4_X = {_F32: _abi.F32, _BF16: _abi.BF16, torch.int8: _abi.INT8, torch.float8_e4m3fn: _abi.E4M3}
_ACTIVATIONS = {None: _abi.ACT_NONE, "none": _abi.ACT_NONE, "silu": _abi.ACT_SILU}

# the structs of include/rsq.h in their C layout
_CONV = struct.Struct("@5i2q2PqPPPPq")
_SSM = struct.Struct("@8i2q2PqPqPqPqPPPPPqPN")
_NORM = struct.Struct("@4ifqPqPqPPqP")
_W4 = struct.Struct("@8iPqPPNPq")
for _s, _t in ((_CONV, _abi.Conv), (_SSM, _abi.Ssm), (_NORM, _abi.Norm), (_W4, _abi.W4)):
    assert _s.size == ctypes.sizeof(_t)

_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Same:
    """The context of a call on the current device's current stream: nothing to change."""

    def __init__(self, ptr):
        self.ptr = ptr

    def __enter__(self):
        return self.ptr

    def __exit__(self, *exc):
        return False


class _Other:
    """The context of a call on another device or stream: the tensors made inside belong to both."""

    def __init__(self, index, stream):
        self.device = torch.cuda.device(index)
        self.stream = stream

    def __enter__(self):
        self.device.__enter__()
        if self.stream is None:
            self.ctx = None
            return _raw_stream(self.device.idx)
        self.ctx = torch.cuda.stream(self.stream)
        self.ctx.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        return self.device.__exit__(*exc)


def on(index, stream):
    """Context of a call on GPU `index`; its value is the hipStream_t."""
    if index < 0:
        raise ValueError("the tensors must be on a GPU")
    if stream is None:
        if torch._C._cuda_getDevice() == index:
            return _Same(_raw_stream(index))
    elif stream.device.index != index:
        raise ValueError("stream is on %s, the tensors on GPU %d" % (stream.device, index))
    return _Other(index, stream)


def _need(cond, fmt, *args):
    if not cond:
        raise ValueError(fmt % args)


def _param(t, index, shape, name, dtype=_F32):
    """Address of a contiguous tensor of `shape` and `dtype` on GPU `index`; 0 for None."""
    if t is None:
        return 0
    if isinstance(t, Tensor) and t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    raise ValueError("%s must be a contiguous %s tensor of shape %s on the device of the others, got %s" % (
        name, dtype, tuple(shape), "%s %s %s on %s" % ("strided" if not t.is_contiguous() else "contiguous", t.dtype,
                                                      tuple(t.shape), t.device) if isinstance(t, Tensor) else type(t)))


def _stride(t, index, dtype, shape, inner, name):
    """Step between the rows of a tensor [*lead, *inner] = shape with contiguous rows; `inner` is how many
    dimensions a row has, lead one or two dimensions of one common step."""
    if not (isinstance(t, Tensor) and t.get_device() == index and t.dtype is dtype and t.shape == shape):
        raise ValueError("%s must be a %s tensor of shape %s on the device of the others, got %s" % (
            name, dtype, tuple(shape), "%s %s on %s" % (t.dtype, tuple(t.shape), t.device) if isinstance(t, Tensor) else type(t)))
    st = t.stride()
    lead = len(shape) - inner
    if st[-1] != 1 and shape[-1] != 1 or inner == 2 and st[-2] != shape[-1] and shape[-2] != 1:
        raise ValueError("%s must have contiguous rows" % name)
    if lead == 1:
        rows, step = shape[0], st[0]
    else:
        rows, step = shape[0] * shape[1], st[1] if shape[1] > 1 else st[0]
        if shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
            raise ValueError("%s must have rows at one common step" % name)
    if rows <= 1:
        # no row follows: any step will do, in the 16 bytes that the library asks of strides
        width = shape[-1] * (shape[-2] if inner == 2 else 1)
        step = -(-width // 8) * 8
    return step


def _sequences(x, inner, offsets, max_len):
    """(seqs, tokens, max_len, offsets address) of x [seqs, T, ...], or packed [tokens, ...] with offsets."""
    lead = x.dim() - inner
    shape = x.shape
    if offsets is None:
        _need(lead == 2, "x must have shape [sequences, tokens, ...] without offsets, got %s", tuple(shape))
        _need(max_len is None or max_len == shape[1], "max_len is %s, x has %d tokens a sequence", max_len, shape[1])
        return shape[0], shape[0] * shape[1], shape[1], 0
    _need(lead == 1, "x must have shape [tokens, ...] with offsets, got %s", tuple(shape))
    if not (offsets.get_device() == x.get_device() and offsets.dtype is torch.int32 and offsets.dim() == 1
            and offsets.shape[0] > 1 and offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous int32 tensor [sequences + 1] on %s" % x.device)
    if max_len is None or not 0 <= max_len <= shape[0]:
        raise ValueError("max_len, the longest sequence, must be given with offsets, at most %d; got %s" % (shape[0], max_len))
    return offsets.shape[0] - 1, shape[0], int(max_len), offsets.data_ptr()


def _act(x):
    """The C type of an activation tensor."""
    d = _DTYPE.get(x.dtype)
    if d is None:
        raise ValueError("x must be float32 or bfloat16, got %s" % x.dtype)
    return d


def _conv(x, seqs, tokens, max_len, offsets, weight, bias, state, activation, out, stream):
    dtype, index, shape = x.dtype, x.get_device(), x.shape
    d = _act(x)
    _need(weight.dim() == 2, "weight must have shape [channels, width], got %s", tuple(weight.shape))
    C, W = weight.shape
    act = _ACTIVATIONS.get(activation)
    _need(act is not None, "activation must be None or 'silu', got %r", activation)
    _need(shape[-1] == C, "x must have %d channels, got %s", C, tuple(shape))
    xs = _stride(x, index, dtype, shape, 1, "x")
    w, b = _param(weight, index, (C, W), "weight"), _param(bias, index, (C,), "bias")
    st = _param(state, index, (seqs, C, W - 1), "state", dtype)
    with on(index, stream) as s:
        if out is None:
            out = x.new_empty(shape)
        ys = _stride(out, index, dtype, shape, 1, "out")
        check(lib.rsq_causal_conv(_CONV.pack(d, seqs, C, W, act, tokens, max_len, offsets, x.data_ptr(), xs, w, b, st,
                                             out.data_ptr(), ys), s))
    return out


def causal_conv(x, weight, bias=None, state=None, offsets=None, max_len=None, activation=None, out=None, stream=None):
    """Short causal convolution of each channel of prompts (rsq_causal_conv).

    x: [sequences, tokens, channels], or packed [tokens, channels] with offsets
    (int32 device tensor [sequences + 1]) and max_len (the longest sequence).
    weight: [channels, width], width 2..4, the last tap on the current token.
    state: [sequences, channels, width - 1] of x's type, the inputs before each
    sequence; replaced by its last ones. Returns y of x's shape; with packed
    sequences, rows that belong to none are left as they were.
    """
    seqs, tokens, longest, off = _sequences(x, 1, offsets, max_len)
    return _conv(x, seqs, tokens, longest, off, weight, bias, state, activation, out, stream)


def causal_conv_step(x, weight, bias=None, state=None, activation=None, out=None, stream=None):
    """causal_conv of one token of every sequence: x [sequences, channels]."""
    _need(x.dim() == 2, "x must have shape [sequences, channels], got %s", tuple(x.shape))
    n = x.shape[0]
    return _conv(x, n, n, 1, 0, weight, bias, state, activation, out, stream)


class _Ssm:
    """Checked arguments of a selective scan or step, packed for the library once y and state are known."""
    __slots__ = ("index", "dtype", "shape", "d", "H", "G", "dk", "dv", "head", "tail")

    def __init__(self, x, dt, A, B, C, D, dt_bias):
        self.dtype, self.index, self.shape = x.dtype, x.get_device(), x.shape
        self.d = _act(x)
        index, dtype = self.index, self.dtype
        *lead, H, dv = self.shape
        G, dk = B.shape[-2:]
        lead = tuple(lead)
        self.H, self.G, self.dk, self.dv = H, G, dk, dv
        _need(A is not None, "A is required")
        keys = lead + (G, dk)
        self.head = (x.data_ptr(), _stride(x, index, dtype, self.shape, 2, "x"),
                     B.data_ptr(), _stride(B, index, dtype, keys, 2, "B"),
                     C.data_ptr(), _stride(C, index, dtype, keys, 2, "C"),
                     dt.data_ptr(), _stride(dt, index, dtype, lead + (H,), 1, "dt"),
                     _param(A, index, (H,), "A"), _param(D, index, (H,), "D"), _param(dt_bias, index, (H,), "dt_bias"))

    def pack(self, seqs, tokens, max_len, offsets, softplus, state_in, state, out, work, work_bytes):
        return _SSM.pack(self.d, seqs, self.H, self.G, self.dk, self.dv, 1 if softplus else 0, state_in, tokens, max_len,
                         offsets, *self.head, state, out.data_ptr(),
                         _stride(out, self.index, self.dtype, self.shape, 2, "out"), work, work_bytes)


def ssm_scan(x, dt, A, B, C, D=None, dt_bias=None, softplus=False, state=None, offsets=None, max_len=None,
             out=None, stream=None):
    """Selective state-space scan of prompts (rsq_ssm_scan); returns (y, state).

    x: [sequences, tokens, heads, d_v] (or packed [tokens, ...] with offsets and
    max_len, as causal_conv); B, C: [..., groups, d_k]; dt: [..., heads]; A, D,
    dt_bias: fp32 [heads]. state: fp32 [sequences, heads, d_k, d_v] to start
    from, updated in place; None starts from zero and makes one.
    """
    _need(x.dim() in (3, 4) and B.dim() == x.dim(),
          "x and B must have shape [..., heads, d_v] and [..., groups, d_k], got %s and %s", tuple(x.shape), tuple(B.shape))
    seqs, tokens, longest, off = _sequences(x, 2, offsets, max_len)
    p = _Ssm(x, dt, A, B, C, D, dt_bias)
    shape = (seqs, p.H, p.dk, p.dv)
    with on(p.index, stream) as s:
        state_in = 0 if state is None else 1
        if state is None:
            state = x.new_empty(shape, dtype=_F32)
        if out is None:
            out = x.new_empty(x.shape)
        args = (seqs, tokens, longest, off, softplus, state_in, _param(state, p.index, shape, "state"), out)
        need = ctypes.c_size_t()
        packed = p.pack(*args, 0, 0)
        check(lib.rsq_ssm_scan_workspace(packed, ctypes.byref(need)))
        if need.value:
            # the call's stream owns it: it is reused there only
            work = x.new_empty(need.value, dtype=torch.uint8)
            packed = p.pack(*args, work.data_ptr(), need.value)
        check(lib.rsq_ssm_scan(packed, s))
    return out, state


def ssm_step(state, x, dt, A, B, C, D=None, dt_bias=None, softplus=False, out=None, stream=None):
    """One token of every sequence on a dense fp32 state [sequences, heads, d_k, d_v],
    updated in place (rsq_ssm_step): x [sequences, heads, d_v], B, C [sequences,
    groups, d_k], dt [sequences, heads]. Returns y of x's shape."""
    _need(x.dim() == 3 and B.dim() == 3, "x and B must have shape [sequences, heads, d_v] and [sequences, groups, d_k]")
    _need(state is not None, "state is required")
    n = x.shape[0]
    p = _Ssm(x, dt, A, B, C, D, dt_bias)
    st = _param(state, p.index, (n, p.H, p.dk, p.dv), "state")
    with on(p.index, stream) as s:
        if out is None:
            out = x.new_empty(p.shape)
        check(lib.rsq_ssm_step(p.pack(n, n, 1, 0, softplus, 1, st, out, 0, 0), s))
    return out


def state_ssm_step(st, x, dt, A, B, C, D, dt_bias, softplus, out, stream):
    """State.ssm_step."""
    _need(x.dim() == 3 and B.dim() == 3, "x and B must have shape [batch, heads, d_v] and [batch, groups, d_k]")
    _need(x.device == st.device, "x must be on %s", st.device)
    n = x.shape[0]
    p = _Ssm(x, dt, A, B, C, D, dt_bias)
    need = ctypes.c_size_t()
    check(lib.rsq_decode_ssm_workspace(st.h, ctypes.byref(need)))
    with on(p.index, stream) as s:
        if out is None:
            out = x.new_empty(p.shape)
        # torch's allocations are 512-byte aligned; the call's stream owns this one
        work = x.new_empty(need.value, dtype=torch.uint8)
        check(lib.rsq_decode_ssm_step(st.h, p.pack(n, n, 1, 0, softplus, 1, 0, out, work.data_ptr(), need.value), s))
    return out


def rms_norm(x, weight, eps=1e-5, residual=None, out_dtype=None, group=0, out=None, scales=None, stream=None):
    """RMS norm of the rows of x [..., cols] (rsq_rms_norm), after x + residual,
    which replaces the residual where one is given.

    out_dtype: 'f32' or 'bf16' (default: x's type) returns y; 'int8' or 'e4m3'
    returns (codes, scales), one fp32 scale a row, or per `group` columns."""
    dtype, index, shape = x.dtype, x.get_device(), x.shape
    d = _act(x)
    _need(len(shape) in (2, 3), "x must have shape [rows, cols] or [sequences, tokens, cols], got %s", tuple(shape))
    cols = shape[-1]
    if out_dtype is None:
        out_dtype = "bf16" if dtype is _BF16 else "f32"
    _need(out_dtype in _OUT, "out_dtype must be one of %s, got %r", sorted(_OUT), out_dtype)
    od, torch_out = _OUT[out_dtype]
    codes = od == _abi.INT8 or od == _abi.E4M3
    rows = shape[0] if len(shape) == 2 else shape[0] * shape[1]
    xs = _stride(x, index, dtype, shape, 1, "x")
    w = _param(weight, index, (cols,), "weight")
    _need(w or cols == 0, "weight is required")
    rp = rs = 0
    if residual is not None:
        rp, rs = residual.data_ptr(), _stride(residual, index, dtype, shape, 1, "residual")
    with on(index, stream) as s:
        if out is None:
            out = x.new_empty(shape, dtype=torch_out)
        ys = _stride(out, index, torch_out, shape, 1, "out")
        sp = 0
        if codes:
            sshape = shape[:-1] + (cols // group if group > 0 else 1,)
            if scales is None:
                scales = x.new_empty(sshape, dtype=_F32)
            sp = _param(scales, index, sshape, "scales")
        else:
            _need(scales is None, "scales go with an 8-bit output")
        check(lib.rsq_rms_norm(_NORM.pack(d, od, cols, group, eps, rows, x.data_ptr(), xs, rp, rs, w, out.data_ptr(), ys,
                                          sp), s))
    return (out, scales) if codes else out


class W4Weight:
    """A weight matrix [n, k] of 4-bit codes with group scales, laid out once for w4_linear.

    codes: int8 [n, k], values -8..7; scales: fp32 or fp16 [n, k / group], group
    32, 64 or 128. The packed copy (`packed`, uint8) is all that is kept."""

    def __init__(self, codes, scales, stream=None):
        _need(codes.dim() == 2 and codes.dtype is torch.int8 and codes.is_contiguous(),
              "codes must be a contiguous int8 tensor [n, k], got %s %s", codes.dtype, tuple(codes.shape))
        self.n, self.k = codes.shape
        _need(scales.dim() == 2 and scales.shape[0] == self.n and scales.is_contiguous()
              and scales.device == codes.device and scales.dtype in (_F32, torch.float16),
              "scales must be a contiguous float32 or float16 tensor [%d, k / group] on %s", self.n, codes.device)
        _need(scales.shape[1] > 0 and self.k % scales.shape[1] == 0, "%d scales a row for %d columns", scales.shape[1], self.k)
        self.group = self.k // scales.shape[1]
        self.scale_dtype = _abi.F16 if scales.dtype is torch.float16 else _abi.F32
        self.device = codes.device
        need = ctypes.c_size_t()
        check(lib.rsq_w4_bytes(self.n, self.k, self.group, self.scale_dtype, ctypes.byref(need)))
        self.packed_bytes = need.value
        with on(codes.get_device(), stream) as s:
            self.packed = codes.new_empty(need.value, dtype=torch.uint8)
            check(lib.rsq_w4_pack(codes.data_ptr(), scales.data_ptr(), self.n, self.k, self.group, self.scale_dtype,
                                  self.packed.data_ptr(), need.value, s))


def w4_linear(x, weight, x_scale=None, out_dtype=None, out=None, stream=None):
    """x [..., k] times a W4Weight [n, k]: y [..., n] (rsq_w4_linear).

    x: float32 or bfloat16, or int8 / float8_e4m3fn codes with x_scale (fp32, one
    a row, or [..., k / group] with the weight's group), as rms_norm returns
    them. out_dtype: 'f32' or 'bf16' (default: x's type; bf16 with codes)."""
    dtype, index, shape = x.dtype, x.get_device(), x.shape
    xd = _W4_X.get(dtype)
    _need(xd is not None, "x must be float32, bfloat16, int8 or float8_e4m3fn, got %s", dtype)
    _need(len(shape) in (2, 3), "x must have shape [rows, k] or [sequences, tokens, k], got %s", tuple(shape))
    n, k = weight.n, weight.k
    _need(shape[-1] == k, "x must have %d columns, got %s", k, tuple(shape))
    packed = weight.packed
    _need(packed.get_device() == index, "weight and x must be on one device, got %s and %s", weight.device, x.device)
    lead = shape[:-1]
    m = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    xs = _stride(x, index, dtype, shape, 1, "x")
    sp = xgroup = 0
    if x_scale is not None:
        groups = k // weight.group
        ss = x_scale.shape
        if groups > 1 and ss == lead + (groups,):
            xgroup = weight.group
        else:
            _need(ss == lead or ss == lead + (1,), "x_scale must have shape %s or %s, got %s", tuple(lead),
                  tuple(lead) + (groups,), tuple(ss))
        sp = _param(x_scale, index, ss, "x_scale")
    if out_dtype is None:
        out_dtype = "f32" if dtype is _F32 else "bf16"
    _need(out_dtype in ("f32", "bf16"), "out_dtype must be 'f32' or 'bf16', got %r", out_dtype)
    od, torch_out = _OUT[out_dtype]
    yshape = lead + (n,)
    with on(index, stream) as s:
        if out is None:
            out = x.new_empty(yshape, dtype=torch_out)
        ys = _stride(out, index, torch_out, yshape, 1, "out")
        check(lib.rsq_w4_linear(_W4.pack(xd, od, m, n, k, weight.group, weight.scale_dtype, xgroup, x.data_ptr(), xs, sp,
                                         packed.data_ptr(), weight.packed_bytes, out.data_ptr(), ys), s))
    return out
