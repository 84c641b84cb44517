"""Argument checks of the layer operators. No GPU is used: every call here
returns before the library touches a device (addresses are made up)."""
import ctypes

import pytest
import torch

rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
from bit_recurrent_state_rsq_amd import _abi  # noqa: E402
from bit_recurrent_state_rsq_amd._abi import lib  # noqa: E402

BASE = 0x10000000
INVALID, UNSUPPORTED, BUFFER = _abi.RSQ_E_INVALID, _abi.RSQ_E_UNSUPPORTED, _abi.RSQ_E_BUFFER


def addr(i):
    """Made-up addresses 16 MB apart."""
    return BASE + i * (16 << 20)


def fill(struct, kw):
    s = struct()
    for k, v in kw.items():
        setattr(s, k, v)
    return s


CONV = dict(dtype=_abi.BF16, seqs=2, channels=64, width=4, activation=_abi.ACT_SILU, tokens=20, max_len=10,
            offsets=None, x=addr(0), x_stride=64, weight=addr(1), bias=addr(2), state=addr(3), y=addr(4), y_stride=64)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=_abi.F16), INVALID),
    (dict(width=1), UNSUPPORTED),
    (dict(width=5), UNSUPPORTED),
    (dict(seqs=0), INVALID),
    (dict(channels=0), INVALID),
    (dict(activation=2), INVALID),
    (dict(tokens=-1), INVALID),
    (dict(tokens=1 << 40, offsets=addr(5)), INVALID),
    (dict(max_len=21), INVALID),
    (dict(max_len=9), INVALID),                        # 2 x 9 rows are not 20
    (dict(x=None), INVALID),
    (dict(weight=None), INVALID),
    (dict(y=None), INVALID),
    (dict(x_stride=63), INVALID),
    (dict(y_stride=63), INVALID),
    (dict(x=addr(0) + 1), INVALID),
    (dict(state=addr(3) + 1), INVALID),
    (dict(y=addr(0)), INVALID),                        # in place
    (dict(y=addr(0) + 20 * 128 - 2), INVALID),         # the last element of x
    (dict(state=addr(0)), INVALID),
    (dict(state=addr(4)), INVALID),                    # two outputs
    (dict(y=addr(1) - 64), INVALID),                   # runs into the weights
])
def test_conv_refusals(change, code):
    c = fill(_abi.Conv, {**CONV, **change})
    assert lib.rsq_causal_conv(ctypes.byref(c), None) == code
    assert lib.rsq_last_error().decode() != "no error"


def test_calls_without_rows_do_nothing():
    c = fill(_abi.Conv, {**CONV, "tokens": 0, "max_len": 0, "x": None, "y": None})
    assert lib.rsq_causal_conv(ctypes.byref(c), None) == 0
    n = fill(_abi.Norm, {**NORM, "rows": 0, "x": None, "y": None})
    assert lib.rsq_rms_norm(ctypes.byref(n), None) == 0
    w = fill(_abi.W4, {**W4, "m": 0, "x": None, "y": None})
    assert lib.rsq_w4_linear(ctypes.byref(w), None) == 0


SSM = dict(dtype=_abi.BF16, seqs=2, heads=8, groups=2, d_k=128, d_v=64, softplus=1, state_in=1, tokens=20, max_len=10,
           offsets=None, x=addr(0), x_stride=512, B=addr(1), b_stride=256, C=addr(2), c_stride=256, dt=addr(3),
           dt_stride=8, A=addr(4), D=addr(5), dt_bias=addr(6), state=addr(7), y=addr(8), y_stride=512,
           workspace=None, workspace_bytes=0)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=_abi.F16), INVALID),
    (dict(groups=3), INVALID),
    (dict(groups=0), INVALID),
    (dict(heads=0), INVALID),
    (dict(d_k=12), INVALID),
    (dict(d_v=4), INVALID),
    (dict(d_k=264), UNSUPPORTED),
    (dict(dtype=_abi.F32, d_k=136, b_stride=272, c_stride=272), UNSUPPORTED),
    (dict(d_v=4104), UNSUPPORTED),
    (dict(tokens=-1), INVALID),
    (dict(max_len=21), INVALID),
    (dict(max_len=9), INVALID),
    (dict(x_stride=504), INVALID),
    (dict(x_stride=516), INVALID),                     # not a multiple of 16 bytes
    (dict(x_stride=(1 << 23) + 8), UNSUPPORTED),       # rows above 2^24 bytes apart
    (dict(y_stride=(1 << 62) + 8), UNSUPPORTED),
    (dict(dt_stride=(1 << 23) + 1), UNSUPPORTED),
    (dict(tokens=0x7FFFFFFF, max_len=0x7FFFF001, offsets=addr(9)), UNSUPPORTED),
    (dict(b_stride=260), INVALID),
    (dict(y_stride=514), INVALID),
    (dict(dt_stride=7), INVALID),
    (dict(x=addr(0) + 8), INVALID),
    (dict(dt=addr(3) + 1), INVALID),
    (dict(A=None), INVALID),
    (dict(dt=None), INVALID),
    (dict(state=None), INVALID),
    (dict(y=addr(0)), INVALID),
    (dict(y=addr(7)), INVALID),
    (dict(state=addr(1)), INVALID),
])
def test_scan_refusals(change, code):
    p = fill(_abi.Ssm, {**SSM, **change})
    assert lib.rsq_ssm_scan(ctypes.byref(p), None) == code


def test_scan_workspace_is_checked():
    long = {**SSM, "seqs": 1, "tokens": 8192, "max_len": 8192, "heads": 2, "groups": 1, "x_stride": 128,
            "b_stride": 128, "c_stride": 128, "dt_stride": 2, "y_stride": 128}
    p, n = fill(_abi.Ssm, long), ctypes.c_size_t()
    assert lib.rsq_ssm_scan_workspace(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value > 0
    assert lib.rsq_ssm_scan(ctypes.byref(p), None) == INVALID                      # none given
    p = fill(_abi.Ssm, {**long, "workspace": addr(9) + 8, "workspace_bytes": n.value})
    assert lib.rsq_ssm_scan(ctypes.byref(p), None) == INVALID                      # not aligned
    p = fill(_abi.Ssm, {**long, "workspace": addr(9), "workspace_bytes": n.value - 1})
    assert lib.rsq_ssm_scan(ctypes.byref(p), None) == BUFFER
    p = fill(_abi.Ssm, {**long, "workspace": addr(0), "workspace_bytes": n.value})
    assert lib.rsq_ssm_scan(ctypes.byref(p), None) == INVALID                      # over x
    # short prompts need none
    p = fill(_abi.Ssm, SSM)
    assert lib.rsq_ssm_scan_workspace(ctypes.byref(p), ctypes.byref(n)) == 0 and n.value == 0


@pytest.mark.parametrize("change,code", [
    (dict(offsets=addr(9)), INVALID),
    (dict(tokens=4, max_len=2), INVALID),
    (dict(d_v=1032, x_stride=8 * 1032, y_stride=8 * 1032), UNSUPPORTED),
    (dict(d_k=4104, b_stride=2 * 4104, c_stride=2 * 4104), UNSUPPORTED),
    (dict(state=None), INVALID),
    (dict(y=addr(7)), INVALID),
])
def test_step_refusals(change, code):
    p = fill(_abi.Ssm, {**SSM, "tokens": 2, "max_len": 1, **change})
    assert lib.rsq_ssm_step(ctypes.byref(p), None) == code


def test_step_and_load_on_a_null_state():
    p = fill(_abi.Ssm, {**SSM, "tokens": 2, "max_len": 1, "state": None})
    n = ctypes.c_size_t()
    assert lib.rsq_decode_ssm_step(None, ctypes.byref(p), None) == INVALID
    assert lib.rsq_decode_ssm_workspace(None, ctypes.byref(n)) == INVALID
    assert lib.rsq_state_load(None, ctypes.c_void_p(16), None) == INVALID


NORM = dict(dtype=_abi.BF16, out_dtype=_abi.INT8, cols=256, group=0, eps=1e-5, rows=4, x=addr(0), x_stride=256,
            residual=addr(1), residual_stride=256, weight=addr(2), y=addr(3), y_stride=256, scales=addr(4))


@pytest.mark.parametrize("change,code", [
    (dict(dtype=_abi.F16), INVALID),
    (dict(out_dtype=_abi.F16), INVALID),
    (dict(cols=0), INVALID),
    (dict(rows=-1), INVALID),
    (dict(cols=32776, x_stride=32776, residual_stride=32776, y_stride=32776), UNSUPPORTED),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(group=16), INVALID),
    (dict(group=128, cols=192), INVALID),
    (dict(group=64, out_dtype=_abi.BF16, scales=None), INVALID),
    (dict(scales=None), INVALID),
    (dict(out_dtype=_abi.F32), INVALID),               # scales without codes
    (dict(x_stride=255), INVALID),
    (dict(residual_stride=255), INVALID),
    (dict(weight=None), INVALID),
    (dict(x=addr(0) + 1), INVALID),
    (dict(y=addr(0)), INVALID),
    (dict(residual=addr(0)), INVALID),
    (dict(scales=addr(3)), INVALID),
])
def test_norm_refusals(change, code):
    p = fill(_abi.Norm, {**NORM, **change})
    assert lib.rsq_rms_norm(ctypes.byref(p), None) == code


def w4_bytes(n, k, group, scale_dtype=_abi.F16):
    b = ctypes.c_size_t()
    return lib.rsq_w4_bytes(n, k, group, scale_dtype, ctypes.byref(b)), b.value


@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (17, 160, 32), (16, 128, 128), (100, 192, 64)])
def test_w4_bytes(n, k, group):
    code, got = w4_bytes(n, k, group)
    rows, blocks = -(-n // 16) * 16, -(-k // 128)
    assert code == 0 and got == rows * blocks * 64 + rows * blocks * (128 // group) * 2


@pytest.mark.parametrize("n,k,group", [(0, 128, 128), (16, 0, 32), (16, 100, 32), (16, 128, 16), (16, 128, 256)])
def test_w4_bytes_refusals(n, k, group):
    assert w4_bytes(n, k, group)[0] == INVALID


@pytest.mark.parametrize("n,k,group", [((1 << 26) + 1, 32, 32), (16, (1 << 22) + 32, 32), (1 << 26, 256, 32),
                                       (1 << 25, 512 + 32, 32), (0x7FFFFFFF, 32, 32)])
def test_w4_bytes_limits(n, k, group):
    assert w4_bytes(n, k, group)[0] == UNSUPPORTED
    assert w4_bytes(1 << 26, 96, group)[0] == 0 and w4_bytes(16, 1 << 22, group)[0] == 0


W4 = dict(x_dtype=_abi.INT8, out_dtype=_abi.BF16, m=4, n=64, k=256, group=64, scale_dtype=_abi.F16, x_group=0,
          x=addr(0), x_stride=256, x_scale=addr(1), packed=addr(2), packed_bytes=1 << 20, y=addr(3), y_stride=64)


@pytest.mark.parametrize("change,code", [
    (dict(x_dtype=_abi.F16), INVALID),
    (dict(out_dtype=_abi.INT8), INVALID),
    (dict(scale_dtype=_abi.BF16), INVALID),
    (dict(k=250), INVALID),
    (dict(x_scale=None), INVALID),
    (dict(x_dtype=_abi.BF16), INVALID),                # a scale without 8-bit x
    (dict(x_group=32), INVALID),
    (dict(m=-1), INVALID),
    (dict(x=None), INVALID),
    (dict(packed=None), INVALID),
    (dict(packed=addr(2) + 4), INVALID),
    (dict(packed_bytes=64), BUFFER),
    (dict(x_stride=255), INVALID),
    (dict(y_stride=63), INVALID),
    (dict(x_stride=(1 << 24) + 1), UNSUPPORTED),
    (dict(x_stride=1 << 63 - 1), UNSUPPORTED),
    (dict(m=65535 * 16 + 1), INVALID),
    (dict(y=addr(0)), INVALID),
    (dict(y=addr(2)), INVALID),
])
def test_w4_refusals(change, code):
    p = fill(_abi.W4, {**W4, **change})
    assert lib.rsq_w4_linear(ctypes.byref(p), None) == code


def test_w4_pack_refusals():
    P = ctypes.c_void_p
    _, need = w4_bytes(64, 256, 64)
    args = lambda **kw: [kw.get(k, v) for k, v in dict(codes=P(addr(0)), scales=P(addr(1)), n=64, k=256, group=64,  # noqa: E731
                                                       sd=_abi.F16, packed=P(addr(2)), size=need, stream=None).items()]
    assert lib.rsq_w4_pack(*args(codes=None)) == INVALID
    assert lib.rsq_w4_pack(*args(scales=P(addr(1) + 1))) == INVALID
    assert lib.rsq_w4_pack(*args(packed=P(addr(2) + 8))) == INVALID
    assert lib.rsq_w4_pack(*args(size=need - 1)) == BUFFER
    assert lib.rsq_w4_pack(*args(packed=P(addr(0)))) == INVALID
    assert lib.rsq_w4_pack(*args(k=250)) == INVALID


# ------------------------------------------------------------------ the Python functions' own checks

def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: rsq.causal_conv(z(2, 5, 8), z(8, 4)),                                           # not on a GPU
    lambda: rsq.causal_conv(z(10, 8), z(8, 4)),                                             # packed without offsets
    lambda: rsq.causal_conv(z(10, 8), z(8, 4), offsets=torch.zeros(3, dtype=torch.int32)),  # without max_len
    lambda: rsq.causal_conv(z(10, 8), z(8, 4), offsets=torch.zeros(3), max_len=5),          # float offsets
    lambda: rsq.causal_conv(z(10, 8), z(8, 4), offsets=torch.zeros(3, dtype=torch.int32), max_len=11),
    lambda: rsq.causal_conv(z(2, 5, 8), z(7, 4)),                                           # channels differ
    lambda: rsq.causal_conv(z(2, 5, 8), z(8, 4), activation="gelu"),
    lambda: rsq.causal_conv(z(2, 5, 8), z(8, 4, dtype=torch.bfloat16)),                     # parameters are fp32
    lambda: rsq.causal_conv(z(2, 5, 8, dtype=torch.float16), z(8, 4)),
    lambda: rsq.causal_conv(z(2, 5, 8), z(8, 4), state=z(2, 8, 4)),
    lambda: rsq.causal_conv(z(2, 8, 5).transpose(1, 2), z(8, 4)),                           # strided channels
    lambda: rsq.causal_conv(z(2, 6, 8)[:, :5], z(8, 4)),                                    # rows at two steps
    lambda: rsq.causal_conv_step(z(2, 5, 8), z(8, 4)),
    lambda: rsq.ssm_scan(z(2, 5, 4, 8), z(2, 5, 4), z(4), z(2, 5, 1, 8), z(2, 4, 1, 8)),    # C's tokens differ
    lambda: rsq.ssm_scan(z(2, 5, 4, 8), z(2, 5, 3), z(4), z(2, 5, 1, 8), z(2, 5, 1, 8)),
    lambda: rsq.ssm_scan(z(2, 5, 4, 8), z(2, 5, 4), z(3), z(2, 5, 1, 8), z(2, 5, 1, 8)),
    lambda: rsq.ssm_step(z(2, 4, 8, 16), z(2, 4, 16), z(2, 4), z(4), z(2, 1, 8), z(2, 1, 16)),
    lambda: rsq.ssm_step(None, z(2, 4, 16), z(2, 4), z(4), z(2, 1, 8), z(2, 1, 8)),
    lambda: rsq.rms_norm(z(8), z(8)),
    lambda: rsq.rms_norm(z(2, 8), z(8), out_dtype="fp4"),
    lambda: rsq.rms_norm(z(2, 8), None),
    lambda: rsq.rms_norm(z(2, 64), z(64), out_dtype="int8", group=(1 << 32) + 64),
    lambda: rsq.rms_norm(z(2, 8), z(8), residual=z(2, 7)),
    lambda: rsq.W4Weight(z(16, 128), z(16, 1)),
    lambda: rsq.W4Weight(z(16, 128, dtype=torch.int8), z(15, 1)),
    lambda: rsq.W4Weight(z(16, 128, dtype=torch.int8), z(16, 3)),
])
def test_python_checks(call):
    with pytest.raises(ValueError):
        call()
