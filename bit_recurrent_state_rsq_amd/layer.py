"""Operators of the layer around the decode step: the short causal convolution,
the selective state-space scan of prompts and its single-token step, the RMS
norm with an 8-bit output, and products with 4-bit weights.

Argument marshalling for the C ABI (include/rsq.h, which documents every
argument); the arithmetic runs in the HIP kernels. Activations are fp32 or
bf16 tensors on one device, parameters fp32. Calls go to `stream` (default: the
device's current stream) and can be captured in a graph; a tensor argument's
rows may be strided, its elements within a row are contiguous. A tensor that a
call makes belongs to the stream the call ran on. With `stream` given, the caller
makes it wait for what the operands' own stream still does to them; they are
recorded on it, so that they may be dropped once the call has returned.

    y = causal_conv(xbc, weight, bias, state=conv_state, activation="silu")
    y, S = ssm_scan(x, dt, A, B, C, D=D, dt_bias=dt_bias, softplus=True)     # a prompt
    y = ssm_step(S, x, dt, A, B, C, D=D, dt_bias=dt_bias, softplus=True)     # the next token
"""
import ctypes

import torch

from . import _abi, _binding
from ._abi import check, lib

__all__ = ["causal_conv", "causal_conv_step", "ssm_scan", "ssm_step", "rms_norm", "W4Weight", "w4_linear"]

# _binding checks the operands, makes the outputs and calls the library
_binding.bind(check, *[ctypes.cast(getattr(lib, "rsq_" + name), ctypes.c_void_p).value for name in (
    "causal_conv", "ssm_scan_workspace", "ssm_scan", "ssm_step", "decode_ssm_workspace", "decode_ssm_step", "rms_norm",
    "w4_linear")])

_ACTIVATIONS = {None: _abi.ACT_NONE, "none": _abi.ACT_NONE, "silu": _abi.ACT_SILU}
_OUT = {None: -1, "f32": _abi.F32, "bf16": _abi.BF16, "int8": _abi.INT8, "e4m3": _abi.E4M3}

_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


class on:
    """Context of a call on GPU `index`, on `stream` or its current one, where the tensors made inside
    belong to both; its value is the hipStream_t."""

    def __init__(self, index, stream):
        if index < 0:
            raise ValueError("the tensors must be on a GPU")
        if stream is not None and stream.device.index != index:
            raise ValueError("stream is on %s, the tensors on GPU %d" % (stream.device, index))
        self.index, self.stream = index, stream

    def __enter__(self):
        self.device = torch.cuda.device(self.index)
        self.device.__enter__()
        if self.stream is None:
            self.ctx = None
            return _raw_stream(self.index)
        self.ctx = torch.cuda.stream(self.stream)
        self.ctx.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        return self.device.__exit__(*exc)


def _run(call, x, stream, *args):
    """call(stream, *args) on x's device. Entering a context costs a few microseconds: only where device
    or stream differ from the current ones."""
    index = x.get_device()
    if stream is None and index >= 0 and _current_device() == index:
        return call(_raw_stream(index), *args)
    with on(index, stream) as s:
        made = call(s, *args)
    record(stream, *args)
    return made


def record(stream, *operands):
    """The tensors among the operands are in use on `stream` (where one is given) until its work so far is done."""
    if stream is not None:
        for t in operands:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)


def _choice(table, key, name):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError("%s must be one of %s, got %r" % (name, sorted(k for k in table if k), key)) from None


def causal_conv(x, weight, bias=None, state=None, offsets=None, max_len=None, activation=None, out=None, stream=None):
    """Short causal convolution of each channel of prompts (rsq_causal_conv).

    x: [sequences, tokens, channels], or packed [tokens, channels] with offsets
    (int32 device tensor [sequences + 1]) and max_len (the longest sequence).
    weight: [channels, width], width 2..4, the last tap on the current token.
    state: [sequences, channels, width - 1] of x's type, the inputs before each
    sequence; replaced by its last ones. Returns y of x's shape; with packed
    sequences, rows that belong to none are left as they were.
    """
    return _run(_binding.conv, x, stream, x, weight, bias, state, offsets, max_len,
                _choice(_ACTIVATIONS, activation, "activation"), False, out)


def causal_conv_step(x, weight, bias=None, state=None, activation=None, out=None, stream=None):
    """causal_conv of one token of every sequence: x [sequences, channels]."""
    return _run(_binding.conv, x, stream, x, weight, bias, state, None, None,
                _choice(_ACTIVATIONS, activation, "activation"), True, out)


def ssm_scan(x, dt, A, B, C, D=None, dt_bias=None, softplus=False, state=None, offsets=None, max_len=None,
             out=None, stream=None):
    """Selective state-space scan of prompts (rsq_ssm_scan); returns (y, state).

    x: [sequences, tokens, heads, d_v] (or packed [tokens, ...] with offsets and
    max_len, as causal_conv); B, C: [..., groups, d_k]; dt: [..., heads]; A, D,
    dt_bias: fp32 [heads]. state: fp32 [sequences, heads, d_k, d_v] to start
    from, updated in place; None starts from zero and makes one.
    """
    return _run(_binding.scan, x, stream, x, dt, A, B, C, D, dt_bias, softplus, state, offsets, max_len, out)


def ssm_step(state, x, dt, A, B, C, D=None, dt_bias=None, softplus=False, out=None, stream=None):
    """One token of every sequence on a dense fp32 state [sequences, heads, d_k, d_v],
    updated in place (rsq_ssm_step): x [sequences, heads, d_v], B, C [sequences,
    groups, d_k], dt [sequences, heads]. Returns y of x's shape."""
    return _run(_binding.step, x, stream, state, x, dt, A, B, C, D, dt_bias, softplus, out)


def state_ssm_step(st, x, dt, A, B, C, D, dt_bias, softplus, out, stream):
    """State.ssm_step."""
    if x.device != st.device:
        raise ValueError("x must be on %s, got %s" % (st.device, x.device))
    y = _run(_binding.state_step, x, stream, st.h.value, x, dt, A, B, C, D, dt_bias, softplus, out)
    record(stream, st.buf)
    return y


def rms_norm(x, weight, eps=1e-5, residual=None, out_dtype=None, group=0, out=None, scales=None, stream=None):
    """RMS norm of the rows of x, [rows, cols] or [sequences, tokens, cols]
    (rsq_rms_norm), after x + residual, which replaces the residual where one is given.

    out_dtype: 'f32' or 'bf16' (default: x's type) returns y; 'int8' or 'e4m3'
    returns (codes, scales), one fp32 scale a row, or per `group` columns."""
    return _run(_binding.norm, x, stream, x, weight, eps, residual, _choice(_OUT, out_dtype, "out_dtype"), group, out, scales)


def _need(cond, fmt, *args):
    if not cond:
        raise ValueError(fmt % args)


class W4Weight:
    """A weight matrix [n, k] of 4-bit codes with group scales, laid out once for w4_linear.

    codes: int8 [n, k], values -8..7; scales: fp32 or fp16 [n, k / group], group
    32, 64 or 128. The packed copy (`packed`, uint8) is all that is kept."""

    def __init__(self, codes, scales, stream=None):
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
        with on(codes.get_device(), stream) as s:
            self.packed = codes.new_empty(need.value, dtype=torch.uint8)
            check(lib.rsq_w4_pack(codes.data_ptr(), scales.data_ptr(), self.n, self.k, self.group, self.scale_dtype,
                                  self.packed.data_ptr(), need.value, s))
        record(stream, codes, scales)


def w4_linear(x, weight, x_scale=None, out_dtype=None, out=None, stream=None):
    """x, [rows, k] or [sequences, tokens, k], times a W4Weight [n, k]: y [..., n]
    (rsq_w4_linear).

    x: float32 or bfloat16, or int8 / float8_e4m3fn codes with x_scale (fp32, one
    a row, or [..., k / group] with the weight's group), as rms_norm returns
    them. out_dtype: 'f32' or 'bf16' (default: x's type; bf16 with codes)."""
    return _run(_binding.w4, x, stream, x, weight.packed, weight.n, weight.k, weight.group, weight.scale_dtype, x_scale,
                _choice(_OUT, out_dtype, "out_dtype"), out)
