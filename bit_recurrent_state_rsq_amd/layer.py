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
"""
import ctypes
from contextlib import nullcontext

from . import _abi
from ._abi import check, lib

__all__ = ["causal_conv", "causal_conv_step", "ssm_scan", "ssm_step", "rms_norm", "W4Weight", "w4_linear"]

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
        _DTYPE.update({torch.float32: _abi.F32, torch.bfloat16: _abi.BF16})
    return _torch_module


_DTYPE = {}   # activation types, filled with torch


class On:
    """The device and stream of a call: tensors made inside belong to both."""

    def __init__(self, device, stream):
        torch = _torch()
        if device.type != "cuda":
            raise ValueError("x must be on a GPU, got %s" % device)
        if stream is not None and stream.device != device:
            raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
        self.stream = stream if stream is not None else torch.cuda.current_stream(device)
        self.ptr = ctypes.c_void_p(self.stream.cuda_stream)
        # entering them costs a few microseconds: only where they differ from the current ones
        self.ctx = [nullcontext()] * 2
        if device.index != torch.cuda.current_device():
            self.ctx[0] = torch.cuda.device(device)
        if stream is not None:
            self.ctx[1] = torch.cuda.stream(stream)

    def __enter__(self):
        self.ctx[0].__enter__()
        self.ctx[1].__enter__()
        return self

    def __exit__(self, *exc):
        self.ctx[1].__exit__(*exc)
        self.ctx[0].__exit__(*exc)


def _need(cond, fmt, *args):
    if not cond:
        raise ValueError(fmt % args)


def _param(t, device, shape, name):
    """Address of a contiguous fp32 tensor of `shape`, or None."""
    if t is None:
        return None
    torch = _torch()
    _need(t.device == device, "%s must be on %s", name, device)
    _need(t.dtype == torch.float32, "%s must be %s, got %s", name, torch.float32, t.dtype)
    _need(tuple(t.shape) == tuple(shape), "%s must have shape %s, got %s", name, tuple(shape), tuple(t.shape))
    _need(t.is_contiguous(), "%s must be contiguous", name)
    return t.data_ptr()


def _rows(t, like, inner, name, lead=None):
    """(rows, row stride) of a tensor [..., *inner] of like's device and type whose leading dimensions
    (one, or two of equal step) index rows of contiguous elements."""
    n = len(inner)
    _need(t.device == like.device, "%s must be on %s", name, like.device)
    _need(t.dtype == like.dtype, "%s must be %s, got %s", name, like.dtype, t.dtype)
    _need(t.dim() in (n + 1, n + 2) and tuple(t.shape[t.dim() - n:]) == tuple(inner),
          "%s must have shape [..., %s], got %s", name, ", ".join(map(str, inner)), tuple(t.shape))
    if lead is not None:
        _need(tuple(t.shape[: t.dim() - n]) == tuple(lead), "%s must have leading dimensions %s, got %s", name,
              tuple(lead), tuple(t.shape))
    step, width = 1, 1
    for size, stride in zip(reversed(t.shape[t.dim() - n:]), reversed(t.stride()[t.dim() - n:])):
        _need(size == 1 or stride == step, "%s must have contiguous rows", name)
        step *= size
        width *= size
    size, stride = t.shape[: t.dim() - n], t.stride()[: t.dim() - n]
    if len(size) == 1:
        rows, row = size[0], stride[0]
    else:
        rows, row = size[0] * size[1], stride[1] if size[1] > 1 else stride[0]
        _need(size[0] <= 1 or size[1] <= 1 or stride[0] == size[1] * stride[1],
              "%s must have rows at one common step", name)
    if rows <= 1:
        row = max(row, width)   # a stride that no row follows
        # keep 16-byte granularity, which the library asks of strides
        row = -(-row // 8) * 8
    return rows, row


def _sequences(x, inner_dims, offsets, max_len):
    """(seqs, tokens, max_len, offsets address) of x [seqs, T, ...], or packed [tokens, ...] with offsets."""
    torch = _torch()
    lead = x.shape[: x.dim() - inner_dims]
    if offsets is None:
        _need(len(lead) == 2, "x must have shape [sequences, tokens, ...] without offsets, got %s", tuple(x.shape))
        _need(max_len is None or max_len == lead[1], "max_len is %s, x has %d tokens a sequence", max_len, lead[1])
        return lead[0], lead[0] * lead[1], lead[1], None
    _need(len(lead) == 1, "x must have shape [tokens, ...] with offsets, got %s", tuple(x.shape))
    _need(offsets.device == x.device and offsets.dtype == torch.int32 and offsets.dim() == 1 and offsets.numel() > 1
          and offsets.is_contiguous(), "offsets must be a contiguous int32 tensor [sequences + 1] on %s", x.device)
    _need(max_len is not None and 0 <= max_len <= lead[0],
          "max_len, the longest sequence, must be given with offsets, at most %d; got %s", lead[0], max_len)
    return offsets.numel() - 1, lead[0], int(max_len), offsets.data_ptr()


def _act_dtype(x, name="x"):
    _torch()
    d = _DTYPE.get(x.dtype)
    _need(d is not None, "%s must be float32 or bfloat16, got %s", name, x.dtype)
    return d


_ACTIVATIONS = {None: _abi.ACT_NONE, "none": _abi.ACT_NONE, "silu": _abi.ACT_SILU}


def _conv(x, seqs, tokens, max_len, offsets, weight, bias, state, activation, out, stream):
    torch = _torch()
    c = _abi.Conv()
    c.dtype = _act_dtype(x)
    _need(weight.dim() == 2, "weight must have shape [channels, width], got %s", tuple(weight.shape))
    C, W = weight.shape
    _need(activation in _ACTIVATIONS, "activation must be None or 'silu', got %r", activation)
    c.seqs, c.channels, c.width, c.activation = seqs, C, W, _ACTIVATIONS[activation]
    c.tokens, c.max_len, c.offsets = tokens, max_len, offsets
    _, c.x_stride = _rows(x, x, (C,), "x")
    c.weight = _param(weight, x.device, (C, W), "weight")
    c.bias = _param(bias, x.device, (C,), "bias")
    if state is not None:
        _need(state.device == x.device and state.dtype == x.dtype and state.is_contiguous()
              and tuple(state.shape) == (seqs, C, W - 1), "state must be a contiguous %s tensor of shape %s on %s, got %s %s",
              x.dtype, (seqs, C, W - 1), x.device, state.dtype, tuple(state.shape))
        c.state = state.data_ptr()
    with On(x.device, stream) as on:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _, c.y_stride = _rows(out, x, (C,), "out", x.shape[:-1])
        c.x, c.y = x.data_ptr(), out.data_ptr()
        check(lib.rsq_causal_conv(ctypes.byref(c), on.ptr))
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
    return _conv(x, n, n, 1, None, weight, bias, state, activation, out, stream)


def _ssm(x, dt, A, B, C, D, dt_bias, softplus, seqs, tokens, max_len, offsets):
    """The rsq_ssm of a call but for state, y and workspace, and its checks."""
    p = _abi.Ssm()
    p.dtype = _act_dtype(x)
    H, dv = x.shape[-2:]
    G, dk = B.shape[-2:]
    lead = x.shape[:-2]
    p.seqs, p.heads, p.groups, p.d_k, p.d_v = seqs, H, G, dk, dv
    p.softplus, p.tokens, p.max_len, p.offsets = int(bool(softplus)), tokens, max_len, offsets
    _, p.x_stride = _rows(x, x, (H, dv), "x")
    _, p.b_stride = _rows(B, x, (G, dk), "B", lead)
    _, p.c_stride = _rows(C, x, (G, dk), "C", lead)
    _, p.dt_stride = _rows(dt, x, (H,), "dt", lead)
    p.A = _param(A, x.device, (H,), "A")
    _need(A is not None, "A is required")
    p.D = _param(D, x.device, (H,), "D")
    p.dt_bias = _param(dt_bias, x.device, (H,), "dt_bias")
    p.x, p.B, p.C, p.dt = x.data_ptr(), B.data_ptr(), C.data_ptr(), dt.data_ptr()
    return p


def ssm_scan(x, dt, A, B, C, D=None, dt_bias=None, softplus=False, state=None, offsets=None, max_len=None,
             out=None, stream=None):
    """Selective state-space scan of prompts (rsq_ssm_scan); returns (y, state).

    x: [sequences, tokens, heads, d_v] (or packed [tokens, ...] with offsets and
    max_len, as causal_conv); B, C: [..., groups, d_k]; dt: [..., heads]; A, D,
    dt_bias: fp32 [heads]. state: fp32 [sequences, heads, d_k, d_v] to start
    from, updated in place; None starts from zero and makes one.
    """
    torch = _torch()
    _need(x.dim() in (3, 4) and B.dim() >= 2, "x and B must have shape [..., heads, d_v] and [..., groups, d_k]")
    seqs, tokens, longest, off = _sequences(x, 2, offsets, max_len)
    p = _ssm(x, dt, A, B, C, D, dt_bias, softplus, seqs, tokens, longest, off)
    shape = (seqs, p.heads, p.d_k, p.d_v)
    need = ctypes.c_size_t()
    p.y_stride = p.x_stride
    p.state_in = int(state is not None)
    with On(x.device, stream) as on:
        if state is None:
            state = torch.empty(shape, dtype=torch.float32, device=x.device)
        p.state = _param(state, x.device, shape, "state")
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _, p.y_stride = _rows(out, x, (p.heads, p.d_v), "out", x.shape[:-2])
        p.y = out.data_ptr()
        check(lib.rsq_ssm_scan_workspace(ctypes.byref(p), ctypes.byref(need)))
        if need.value:
            # the call's stream owns it: it is reused there only
            work = torch.empty(need.value, dtype=torch.uint8, device=x.device)
            p.workspace, p.workspace_bytes = work.data_ptr(), need.value
        check(lib.rsq_ssm_scan(ctypes.byref(p), on.ptr))
    return out, state


def ssm_step(state, x, dt, A, B, C, D=None, dt_bias=None, softplus=False, out=None, stream=None):
    """One token of every sequence on a dense fp32 state [sequences, heads, d_k, d_v],
    updated in place (rsq_ssm_step): x [sequences, heads, d_v], B, C [sequences,
    groups, d_k], dt [sequences, heads]. Returns y of x's shape."""
    torch = _torch()
    _need(x.dim() == 3 and B.dim() == 3, "x and B must have shape [sequences, heads, d_v] and [sequences, groups, d_k]")
    n = x.shape[0]
    p = _ssm(x, dt, A, B, C, D, dt_bias, softplus, n, n, 1, None)
    _need(state is not None, "state is required")
    p.state = _param(state, x.device, (n, p.heads, p.d_k, p.d_v), "state")
    p.state_in = 1
    with On(x.device, stream) as on:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _, p.y_stride = _rows(out, x, (p.heads, p.d_v), "out", x.shape[:-2])
        p.y = out.data_ptr()
        check(lib.rsq_ssm_step(ctypes.byref(p), on.ptr))
    return out


def state_ssm_step(st, x, dt, A, B, C, D, dt_bias, softplus, out, stream):
    """State.ssm_step."""
    torch = _torch()
    _need(x.dim() == 3 and B.dim() == 3, "x and B must have shape [batch, heads, d_v] and [batch, groups, d_k]")
    _need(x.device == st.device, "x must be on %s", st.device)
    n = x.shape[0]
    p = _ssm(x, dt, A, B, C, D, dt_bias, softplus, n, n, 1, None)
    need = ctypes.c_size_t()
    check(lib.rsq_decode_ssm_workspace(st.h, ctypes.byref(need)))
    with On(x.device, stream) as on:
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _, p.y_stride = _rows(out, x, (p.heads, p.d_v), "out", x.shape[:-2])
        p.y = out.data_ptr()
        # torch's allocations are 512-byte aligned; the call's stream owns this one
        work = torch.empty(need.value, dtype=torch.uint8, device=x.device)
        p.workspace, p.workspace_bytes = work.data_ptr(), need.value
        check(lib.rsq_decode_ssm_step(st.h, ctypes.byref(p), on.ptr))
    return out


def _out_dtypes():
    torch = _torch()
    return {"f32": (_abi.F32, torch.float32), "bf16": (_abi.BF16, torch.bfloat16), "int8": (_abi.INT8, torch.int8),
            "e4m3": (_abi.E4M3, torch.float8_e4m3fn)}


def rms_norm(x, weight, eps=1e-5, residual=None, out_dtype=None, group=0, out=None, scales=None, stream=None):
    """RMS norm of the rows of x [..., cols] (rsq_rms_norm), after x + residual,
    which replaces the residual where one is given.

    out_dtype: 'f32' or 'bf16' (default: x's type) returns y; 'int8' or 'e4m3'
    returns (codes, scales), one fp32 scale a row, or per `group` columns."""
    torch = _torch()
    p = _abi.Norm()
    p.dtype = _act_dtype(x)
    _need(x.dim() in (2, 3), "x must have shape [rows, cols] or [sequences, tokens, cols], got %s", tuple(x.shape))
    cols = x.shape[-1]
    types = _out_dtypes()
    if out_dtype is None:
        out_dtype = "bf16" if p.dtype == _abi.BF16 else "f32"
    _need(out_dtype in types, "out_dtype must be one of %s, got %r", sorted(types), out_dtype)
    p.out_dtype, torch_out = types[out_dtype]
    codes = out_dtype in ("int8", "e4m3")
    p.cols, p.group, p.eps = cols, int(group), float(eps)
    p.rows, p.x_stride = _rows(x, x, (cols,), "x")
    p.weight = _param(weight, x.device, (cols,), "weight")
    _need(weight is not None, "weight is required")
    if residual is not None:
        _, p.residual_stride = _rows(residual, x, (cols,), "residual", x.shape[:-1])
        p.residual = residual.data_ptr()
    groups = cols // p.group if p.group > 0 else 1
    with On(x.device, stream) as on:
        if out is None:
            out = torch.empty(x.shape, dtype=torch_out, device=x.device)
        _need(out.dtype == torch_out, "out must be %s, got %s", torch_out, out.dtype)
        like = out if out.device == x.device else x
        _, p.y_stride = _rows(out, like, (cols,), "out", x.shape[:-1])
        if codes:
            if scales is None:
                scales = torch.empty(x.shape[:-1] + (groups,), dtype=torch.float32, device=x.device)
            p.scales = _param(scales, x.device, x.shape[:-1] + (groups,), "scales")
        else:
            _need(scales is None, "scales go with an 8-bit output")
        p.x, p.y = x.data_ptr(), out.data_ptr()
        check(lib.rsq_rms_norm(ctypes.byref(p), on.ptr))
    return (out, scales) if codes else out


class W4Weight:
    """A weight matrix [n, k] of 4-bit codes with group scales, laid out once for w4_linear.

    codes: int8 [n, k], values -8..7; scales: fp32 or fp16 [n, k / group], group
    32, 64 or 128. The packed copy (`packed`, uint8) is all that is kept."""

    def __init__(self, codes, scales, stream=None):
        torch = _torch()
        _need(codes.dim() == 2 and codes.dtype == torch.int8 and codes.is_contiguous(),
              "codes must be a contiguous int8 tensor [n, k], got %s %s", codes.dtype, tuple(codes.shape))
        self.n, self.k = codes.shape
        _need(scales.dim() == 2 and scales.shape[0] == self.n and scales.is_contiguous()
              and scales.device == codes.device and scales.dtype in (torch.float32, torch.float16),
              "scales must be a contiguous float32 or float16 tensor [%d, k / group] on %s", self.n, codes.device)
        _need(scales.shape[1] > 0 and self.k % scales.shape[1] == 0, "%d scales a row for %d columns", scales.shape[1], self.k)
        self.group = self.k // scales.shape[1]
        self.scale_dtype = _abi.F16 if scales.dtype == torch.float16 else _abi.F32
        self.device = codes.device
        need = ctypes.c_size_t()
        check(lib.rsq_w4_bytes(self.n, self.k, self.group, self.scale_dtype, ctypes.byref(need)))
        with On(codes.device, stream) as on:
            self.packed = torch.empty(need.value, dtype=torch.uint8, device=codes.device)
            check(lib.rsq_w4_pack(codes.data_ptr(), scales.data_ptr(), self.n, self.k, self.group, self.scale_dtype,
                                  self.packed.data_ptr(), need.value, on.ptr))


def w4_linear(x, weight, x_scale=None, out_dtype=None, out=None, stream=None):
    """x [..., k] times a W4Weight [n, k]: y [..., n] (rsq_w4_linear).

    x: float32 or bfloat16, or int8 / float8_e4m3fn codes with x_scale (fp32, one
    a row, or [..., k / group] with the weight's group), as rms_norm returns
    them. out_dtype: 'f32' or 'bf16' (default: x's type; bf16 with codes)."""
    torch = _torch()
    p = _abi.W4()
    types = {torch.float32: _abi.F32, torch.bfloat16: _abi.BF16, torch.int8: _abi.INT8,
             torch.float8_e4m3fn: _abi.E4M3}
    _need(x.dtype in types, "x must be float32, bfloat16, int8 or float8_e4m3fn, got %s", x.dtype)
    _need(x.dim() in (2, 3), "x must have shape [rows, k] or [sequences, tokens, k], got %s", tuple(x.shape))
    _need(weight.device == x.device, "weight must be on %s", x.device)
    p.x_dtype = types[x.dtype]
    p.n, p.k, p.group, p.scale_dtype = weight.n, weight.k, weight.group, weight.scale_dtype
    p.m, p.x_stride = _rows(x, x, (weight.k,), "x")
    lead = tuple(x.shape[:-1])
    if x_scale is not None:
        _need(x_scale.device == x.device and x_scale.dtype == torch.float32 and x_scale.is_contiguous(),
              "x_scale must be a contiguous float32 tensor on %s", x.device)
        groups = weight.k // weight.group
        _need(tuple(x_scale.shape) in (lead, lead + (1,), lead + (groups,)),
              "x_scale must have shape %s or %s, got %s", lead, lead + (groups,), tuple(x_scale.shape))
        p.x_group = weight.group if tuple(x_scale.shape) == lead + (groups,) else 0
        p.x_scale = x_scale.data_ptr()
    outs = {"f32": (_abi.F32, torch.float32), "bf16": (_abi.BF16, torch.bfloat16)}
    if out_dtype is None:
        out_dtype = "f32" if x.dtype == torch.float32 else "bf16"
    _need(out_dtype in outs, "out_dtype must be 'f32' or 'bf16', got %r", out_dtype)
    p.out_dtype, torch_out = outs[out_dtype]
    with On(x.device, stream) as on:
        if out is None:
            out = torch.empty(lead + (weight.n,), dtype=torch_out, device=x.device)
        _need(out.dtype == torch_out and out.device == x.device, "out must be %s on %s", torch_out, x.device)
        _, p.y_stride = _rows(out, out, (weight.n,), "out", lead)
        p.x, p.y = x.data_ptr(), out.data_ptr()
        p.packed, p.packed_bytes = weight.packed.data_ptr(), weight.packed.numel()
        check(lib.rsq_w4_linear(ctypes.byref(p), on.ptr))
    return out
