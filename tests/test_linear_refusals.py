"""Argument checks of linear attention, block norms and 8-bit products. No GPU is used: every call here returns before
the library touches a device (addresses are made up)."""
import ctypes

import pytest
import torch

rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
from bit_recurrent_state_rsq_amd import _abi  # noqa: E402
from bit_recurrent_state_rsq_amd._abi import lib  # noqa: E402

INVALID, UNSUPPORTED, BUFFER = _abi.RSQ_E_INVALID, _abi.RSQ_E_UNSUPPORTED, _abi.RSQ_E_BUFFER


def addr(i):
    """Made-up addresses 16 MB apart."""
    return 0x10000000 + i * (16 << 20)


def fill(struct, kw):
    s = struct()
    for k, v in kw.items():
        setattr(s, k, v)
    return s


# ---------------------------------------------------------------- attention

ATTN = dict(dtype=_abi.BF16, seqs=2, heads=8, key_heads=2, d_k=128, d_v=64, state_in=1, tokens=20, max_len=10, offsets=None,
            q=addr(0), q_stride=256, k=addr(1), k_stride=256, v=addr(2), v_stride=512, alpha=addr(3), alpha_stride=8,
            beta=addr(4), beta_stride=8, state=addr(5), o=addr(6), o_stride=512, workspace=addr(8), workspace_bytes=32 << 20)


def attention(**change):
    p = fill(_abi.LinearAttn, {**ATTN, **change})
    return lib.rsq_linear_attention(ctypes.byref(p), None)


SHARED = [
    (dict(dtype=_abi.F16), INVALID),
    (dict(seqs=0), INVALID),
    (dict(heads=0), INVALID),
    (dict(key_heads=3), INVALID),
    (dict(key_heads=0), INVALID),
    (dict(d_k=12), INVALID),
    (dict(d_v=4), INVALID),
    (dict(d_k=264, q_stride=528, k_stride=528), UNSUPPORTED),
    (dict(d_v=4104, v_stride=8 * 4104, o_stride=8 * 4104), UNSUPPORTED),
    (dict(tokens=-1), INVALID),
    (dict(max_len=21), INVALID),
    (dict(q_stride=248), INVALID),
    (dict(k_stride=252), INVALID),
    (dict(v_stride=504), INVALID),
    (dict(o_stride=516), INVALID),
    (dict(alpha_stride=7), INVALID),
    (dict(beta_stride=7), INVALID),
    (dict(q=None), INVALID),
    (dict(o=None), INVALID),
    (dict(state=None), INVALID),
    (dict(k=addr(1) + 8), INVALID),
    (dict(alpha=addr(3) + 2), INVALID),
    (dict(beta=addr(4) + 1), INVALID),
    (dict(o=addr(2)), INVALID),                       # over v
    (dict(o=addr(3) - 64), INVALID),                  # runs into alpha
    (dict(state=addr(0)), INVALID),
    (dict(state=addr(6)), INVALID),                   # two outputs
]


@pytest.mark.parametrize("beta", [True, False])
@pytest.mark.parametrize("change,code", SHARED + [
    (dict(max_len=9), INVALID),                       # 2 x 9 rows are not 20
    (dict(dtype=_abi.F32, d_k=136, q_stride=272, k_stride=272), UNSUPPORTED),
    (dict(v_stride=(1 << 23) + 8), UNSUPPORTED),      # rows above 2^24 bytes apart
    (dict(o_stride=(1 << 62) + 8), UNSUPPORTED),
    (dict(alpha_stride=(1 << 22) + 1), UNSUPPORTED),
    (dict(tokens=0x7FFFFFFF, max_len=0x7FFFF001, offsets=addr(9)), UNSUPPORTED),
])
def test_attention_refusals(change, code, beta):
    if not beta and "beta_stride" in change or change.get("beta"):
        if not beta:
            pytest.skip("no beta")
    assert attention(**{**({} if beta else dict(beta=None)), **change}) == code
    assert lib.rsq_last_error().decode() != "no error"


@pytest.mark.parametrize("change,code", SHARED + [
    (dict(offsets=addr(9)), INVALID),
    (dict(tokens=4, max_len=2), INVALID),
])
def test_attention_step_refusals(change, code):
    p = fill(_abi.LinearAttn, {**ATTN, "tokens": 2, "max_len": 1, "workspace": None, "workspace_bytes": 0, **change})
    assert lib.rsq_linear_attention_step(ctypes.byref(p), None) == code


def test_attention_on_null():
    n = ctypes.c_size_t()
    assert lib.rsq_linear_attention(None, None) == INVALID
    assert lib.rsq_linear_attention_step(None, None) == INVALID
    assert lib.rsq_linear_attention_workspace(None, ctypes.byref(n)) == INVALID
    p = fill(_abi.LinearAttn, ATTN)
    assert lib.rsq_linear_attention_workspace(ctypes.byref(p), None) == INVALID


def workspace(**change):
    p, n = fill(_abi.LinearAttn, {**ATTN, **change}), ctypes.c_size_t()
    assert lib.rsq_linear_attention_workspace(ctypes.byref(p), ctypes.byref(n)) == 0
    return n.value


def test_attention_workspace():
    need = workspace()
    assert need > 0
    assert attention(workspace=None) == INVALID
    assert attention(workspace=addr(8) + 8) == INVALID
    assert attention(workspace_bytes=need - 1) == BUFFER
    assert attention(workspace=addr(0)) == INVALID                                  # over q
    # without the delta rule short prompts need none, without rows nothing does
    assert workspace(beta=None) == 0
    assert workspace(tokens=0, max_len=0) == 0
    # up to 8 tokens are taken one by one
    assert workspace(seqs=1, tokens=8, max_len=8) == 0 and workspace(seqs=1, tokens=9, max_len=9) > 0
    # the documented size, and a size that follows the tokens rather than sequences x the longest one
    heads, tokens = 32, 1 << 20
    wide = dict(heads=heads, key_heads=16, d_v=128, q_stride=2048, k_stride=2048, v_stride=4096, o_stride=4096, alpha_stride=32,
                beta_stride=32, offsets=addr(9), tokens=tokens)
    assert workspace(**wide, seqs=1, max_len=tokens) <= 400 * heads * (tokens + 64)
    assert workspace(**wide, seqs=1000, max_len=tokens - 999) <= 400 * heads * (tokens + 64 * 1000)
    f32 = {**wide, "dtype": _abi.F32}
    assert workspace(**f32, seqs=1, max_len=tokens) <= (496 * heads + 1536 * 16) * (tokens + 64)


@pytest.mark.parametrize("change", [dict(seqs=1 << 24, tokens=1 << 25, max_len=2, offsets=addr(9)),
                                    dict(seqs=1 << 20, heads=64, key_heads=2, v_stride=4096, o_stride=4096, alpha_stride=64, beta_stride=64,
                                         tokens=1 << 20, max_len=1, state=1 << 45)])
def test_attention_launch_limits(change):
    """2^32 threads and more are refused."""
    p, n = fill(_abi.LinearAttn, {**ATTN, **change}), ctypes.c_size_t()
    assert lib.rsq_linear_attention_workspace(ctypes.byref(p), ctypes.byref(n)) == UNSUPPORTED
    p = fill(_abi.LinearAttn, {**ATTN, "q": 1 << 40, "k": 1 << 41, "v": 1 << 42, "o": 1 << 43, "alpha": 1 << 44, "beta": 1 << 46, **change,
                               "state": 1 << 47, "workspace": None, "workspace_bytes": 0})
    assert lib.rsq_linear_attention(ctypes.byref(p), None) == UNSUPPORTED


# ---------------------------------------------------------------- block norm

BLOCK = dict(dtype=_abi.BF16, out_dtype=_abi.INT8, cols=256, group=64, weight_cols=64, scale_group=0, activation=_abi.ACT_SILU,
             gate_first=0, eps=1e-5, residual_scale=0.5, rows=4, x=addr(0), x_stride=256, gate=addr(1), gate_stride=256, residual=addr(2),
             residual_stride=256, weight=addr(3), next_weight=addr(4), y=addr(5), y_stride=256, scales=addr(6))


@pytest.mark.parametrize("change,code", [
    (dict(dtype=_abi.F16), INVALID),
    (dict(out_dtype=_abi.F16), INVALID),
    (dict(cols=0), INVALID),
    (dict(rows=-1), INVALID),
    (dict(cols=32832, x_stride=32832, gate_stride=32832, residual_stride=32832, y_stride=32832), UNSUPPORTED),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(residual_scale=float("inf")), INVALID),
    (dict(residual_scale=float("nan")), INVALID),
    (dict(residual=None), INVALID),                    # a residual_scale without a residual
    (dict(activation=3), INVALID),
    (dict(activation=-1), INVALID),
    (dict(group=-64), INVALID),
    (dict(group=60, weight_cols=60), INVALID),
    (dict(group=96, weight_cols=96), INVALID),         # does not divide 256
    (dict(weight_cols=128), INVALID),
    (dict(group=0), INVALID),                          # weight_cols is then cols
    (dict(weight=None), INVALID),                      # a group without weight
    (dict(scale_group=16), INVALID),
    (dict(scale_group=64, out_dtype=_abi.BF16, scales=None), INVALID),
    (dict(scales=None), INVALID),
    (dict(out_dtype=_abi.F32), INVALID),               # scales without codes
    (dict(x=None), INVALID),
    (dict(y=None), INVALID),
    (dict(y=None, out_dtype=_abi.BF16, scales=None), INVALID),                                 # there is a second norm
    (dict(y=None, out_dtype=_abi.BF16, scales=None, next_weight=None, residual=None, residual_scale=1.0), INVALID),
    (dict(x_stride=255), INVALID),
    (dict(gate_stride=255), INVALID),
    (dict(residual_stride=255), INVALID),
    (dict(y_stride=255), INVALID),
    (dict(x=addr(0) + 1), INVALID),
    (dict(gate=addr(1) + 1), INVALID),
    (dict(weight=addr(3) + 2), INVALID),
    (dict(y=addr(0)), INVALID),
    (dict(y=addr(1)), INVALID),
    (dict(residual=addr(0)), INVALID),
    (dict(residual=addr(4)), INVALID),
    (dict(scales=addr(5)), INVALID),
])
def test_block_norm_refusals(change, code):
    p = fill(_abi.Block, {**BLOCK, **change})
    assert lib.rsq_block_norm(ctypes.byref(p), None) == code


def test_calls_without_rows_do_nothing():
    p = fill(_abi.Block, {**BLOCK, "rows": 0, "x": None, "y": None, "residual": None, "gate": None, "scales": None})
    assert lib.rsq_block_norm(ctypes.byref(p), None) == 0
    assert lib.rsq_block_norm(None, None) == INVALID
    p = fill(_abi.W8, {**W8, "m": 0, "x": None, "y": None, "x_scale": None})
    assert lib.rsq_w8_linear(ctypes.byref(p), None) == 0


# ---------------------------------------------------------------- 8-bit products

W8 = dict(out_dtype=_abi.BF16, m=4, n=64, k=256, x=addr(0), x_stride=256, x_scale=addr(1), bias=addr(2), packed=addr(3),
          packed_bytes=1 << 20, y=addr(4), y_stride=64, workspace=None, workspace_bytes=0)


def w8_bytes(n, k):
    b = ctypes.c_size_t()
    return lib.rsq_w8_bytes(n, k, ctypes.byref(b)), b.value


@pytest.mark.parametrize("n,k", [(1, 1), (16, 64), (17, 65), (100, 1000)])
def test_w8_bytes(n, k):
    code, got = w8_bytes(n, k)
    assert code == 0 and got == -(-n // 16) * -(-k // 64) * 1024 + 4 * n


@pytest.mark.parametrize("n,k,code", [(0, 64, INVALID), (16, 0, INVALID), (-1, 64, INVALID), (16, 1 << 17, UNSUPPORTED),
                                      ((1 << 26) + 1, 64, UNSUPPORTED)])
def test_w8_bytes_refusals(n, k, code):
    assert w8_bytes(n, k)[0] == code
    assert w8_bytes(1 << 26, 64)[0] == 0 and w8_bytes(16, (1 << 17) - 1)[0] == 0
    assert lib.rsq_w8_bytes(16, 64, None) == INVALID


@pytest.mark.parametrize("change,code", [
    (dict(out_dtype=_abi.INT8), INVALID),
    (dict(m=-1), INVALID),
    (dict(n=0), INVALID),
    (dict(k=1 << 17, x_stride=1 << 17), UNSUPPORTED),
    (dict(x=None), INVALID),
    (dict(x_scale=None), INVALID),
    (dict(packed=None), INVALID),
    (dict(y=None), INVALID),
    (dict(packed=addr(3) + 8), INVALID),
    (dict(packed_bytes=64), BUFFER),
    (dict(x_stride=255), INVALID),
    (dict(y_stride=63), INVALID),
    (dict(y=addr(4) + 1), INVALID),
    (dict(x_scale=addr(1) + 2), INVALID),
    (dict(bias=addr(2) + 1), INVALID),
    (dict(y=addr(0)), INVALID),
    (dict(y=addr(3)), INVALID),
    (dict(y=addr(2) - 64), INVALID),                   # runs into the bias
    (dict(m=0x7FFFFFFF, n=1 << 26, y_stride=1 << 26, packed_bytes=1 << 40, packed=1 << 44, y=1 << 60, x=1 << 45, x_scale=1 << 50,
          bias=1 << 52), UNSUPPORTED),                 # 2^32 threads and more
])
def test_w8_refusals(change, code):
    p = fill(_abi.W8, {**W8, **change})
    assert lib.rsq_w8_linear(ctypes.byref(p), None) == code


def test_w8_workspace():
    """Only where many rows do not begin at multiples of 16 bytes."""
    n = ctypes.c_size_t()
    need = lambda **kw: (lib.rsq_w8_workspace(ctypes.byref(fill(_abi.W8, {**W8, **kw})), ctypes.byref(n)), n.value)[1]  # noqa: E731
    many = dict(m=1000, n=1024, y_stride=1024)
    assert need() == 0 and need(**many) == 0 and need(m=4, x_stride=257) == 0
    for kw in (dict(x_stride=257), dict(x=addr(0) + 1), dict(k=250), dict(x_stride=1 << 23)):
        assert need(**many, **kw) == 1000 * 256
        p = lambda **w: lib.rsq_w8_linear(ctypes.byref(fill(_abi.W8, {**W8, **many, **kw, **w})), None)  # noqa: E731
        far = dict(y=1 << 40, packed=1 << 41, x_scale=1 << 42, bias=1 << 43)
        assert p(**far) == INVALID
        assert p(**far, workspace=(1 << 44) + 4, workspace_bytes=1 << 20) == INVALID
        assert p(**far, workspace=1 << 44, workspace_bytes=1000 * 256 - 1) == BUFFER
        assert p(**far, workspace=addr(0), workspace_bytes=1 << 20) == INVALID
    assert lib.rsq_w8_workspace(None, ctypes.byref(n)) == INVALID


def test_w8_pack_refusals():
    P = ctypes.c_void_p
    _, need = w8_bytes(64, 256)
    args = lambda **kw: [kw.get(k, v) for k, v in dict(codes=P(addr(0)), scales=P(addr(1)), n=64, k=256, packed=P(addr(2)),  # noqa: E731
                                                       size=need, stream=None).items()]
    assert lib.rsq_w8_pack(*args(codes=None)) == INVALID
    assert lib.rsq_w8_pack(*args(scales=P(addr(1) + 1))) == INVALID
    assert lib.rsq_w8_pack(*args(packed=P(addr(2) + 8))) == INVALID
    assert lib.rsq_w8_pack(*args(size=need - 1)) == BUFFER
    assert lib.rsq_w8_pack(*args(packed=P(addr(0)))) == INVALID
    assert lib.rsq_w8_pack(*args(k=0)) == INVALID


# ---------------------------------------------------------------- the Python functions' own checks

def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


I8 = torch.int8


@pytest.mark.parametrize("call", [
    lambda: rsq.linear_attention(z(2, 5, 1, 8), z(2, 5, 1, 8), z(2, 5, 4, 8)),                       # not on a GPU
    lambda: rsq.linear_attention(z(10, 1, 8), z(10, 1, 8), z(10, 4, 8)),                             # packed without offsets
    lambda: rsq.linear_attention(z(2, 5, 1, 8), z(2, 4, 1, 8), z(2, 5, 4, 8)),                       # k's tokens differ
    lambda: rsq.linear_attention(z(2, 5, 1, 8), z(2, 5, 1, 16), z(2, 5, 4, 8)),                      # q's and k's widths differ
    lambda: rsq.linear_attention(z(2, 5, 1, 8), z(2, 5, 1, 8), z(2, 5, 4, 8), alpha=z(2, 5, 3)),
    lambda: rsq.linear_attention(z(2, 5, 1, 8), z(2, 5, 1, 8), z(2, 5, 4, 8), beta=z(4)),            # one beta for all tokens
    lambda: rsq.linear_attention(z(2, 5, 1, 8), z(2, 5, 1, 8), z(2, 5, 4, 8), state=z(2, 4, 8, 16)),
    lambda: rsq.linear_attention(z(2, 5, 1, 8), z(2, 5, 1, 8), z(2, 5, 4, 8), max_len=6),
    lambda: rsq.linear_attention(None, z(2, 5, 1, 8), z(2, 5, 4, 8)),
    lambda: rsq.linear_attention(z(5, 8), z(5, 8), z(5, 8)),
    lambda: rsq.linear_attention_step(None, z(2, 1, 8), z(2, 1, 8), z(2, 4, 8)),
    lambda: rsq.linear_attention_step(z(2, 4, 8, 8), z(2, 5, 1, 8), z(2, 5, 1, 8), z(2, 5, 4, 8)),
    lambda: rsq.block_norm(z(8), z(8)),
    lambda: rsq.block_norm(z(2, 8), z(8), activation="gelu"),
    lambda: rsq.block_norm(z(2, 8), z(8), out_dtype="fp4"),
    lambda: rsq.block_norm(z(2, 8), z(8), gate=z(2, 7)),
    lambda: rsq.block_norm(z(2, 16), z(4), group=8),
    lambda: rsq.block_norm(z(2, 64), z(64), group=(1 << 32) + 64),
    lambda: rsq.W8Weight(z(16, 128), z(16)),
    lambda: rsq.W8Weight(z(16, 128, dtype=I8), z(15)),
    lambda: rsq.W8Weight(z(16, 128, dtype=I8), z(16, 1)),
    lambda: rsq.W8Weight(z(16, 128, dtype=I8), z(16, dtype=torch.float16)),
    lambda: rsq.W8Weight(z(128, 16, dtype=I8).t(), z(16)),
])
def test_python_checks(call):
    with pytest.raises(ValueError):
        call()
