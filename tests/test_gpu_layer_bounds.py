"""Layer operators where the bounds of their plain comparison leave room: results held to what their arithmetic leaves."""
import numpy as np
import numpy as np
import pytest
import torch

import layer_reference as ref
from layer_bounds import w4_norm_limit
from layer_reference import H, U, check
from test_gpu_layer import BF16, F32, gen, offsets_of, same, ssm_case, w4_case

pytestmark = pytest.mark.gpu

rsq = None


@pytest.fixture(scope="module", autouse=True)
def _package():
    global rsq
    rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
    assert torch.cuda.is_available()


# ---------------------------------------------------------------- selective scan

@pytest.mark.parametrize("heads,groups,dk,dv", [(2, 1, 128, 64), (4, 2, 64, 72), (1, 1, 256, 64), (2, 2, 16, 136)])
def test_scan_bf16_factors_keep_sixteen_bits(heads, groups, dk, dv):
    """y of bf16 inputs, without D x: S and the token weights enter it to 2^-8 of 2^-8, so that little but its own
    rounding is left.

    The reference's bound for bf16 is 1.01 (fp32 + 1.01 H t + 1.01 H |y|) + 1e-37 with t the magnitudes of those terms,
    and the one for fp32 has U |y| and no t: t follows from the two.
    """
    lengths = [130, 1, 70]
    x, dt, A, B, C, _, bias = ssm_case(sum(lengths), heads, groups, dk, dv, BF16, seed=dk)
    state = gen(1)(len(lengths), heads, dk, dv)
    off, _ = offsets_of(lengths)
    seqs = [(int(a), n) for a, n in zip(off[:-1].tolist(), lengths)]
    want, S, wide, bS = ref.scan(x, dt, A, B, C, None, bias, True, state, seqs, BF16)
    _, _, narrow, _ = ref.scan(x, dt, A, B, C, None, bias, True, state, seqs, F32)
    terms = (wide - narrow - 1.01 * 1.01 * (H - U) * want.abs()).clamp(min=0)      # 1.01 1.01 H t
    bound = narrow + 1.01 * 1.01 * H * want.abs() + terms * H
    y, got = rsq.ssm_scan(x, dt, A, B, C, dt_bias=bias, softplus=True, state=state, offsets=off, max_len=max(lengths))
    check(y, want, bound, "y")
    check(got, S, bS, "state")


# ---------------------------------------------------------------- more rows than one launch has threads for

@pytest.mark.parametrize("out", ["bf16", "int8"])
def test_norm_rows_of_two_launches(out):
    """Four rows of 8 columns a workgroup of 256 threads: 2^26 - 4 rows a launch."""
    edge = (1 << 26) - 4
    rows = edge + 4099
    x = torch.zeros(rows, 8, dtype=BF16, device="cuda")
    res = torch.zeros(rows, 8, dtype=BF16, device="cuda")
    r = gen(3)
    w = r(8)
    some = torch.cat([torch.arange(0, 70), torch.arange(edge - 70, edge + 70), torch.arange(rows - 70, rows)]).cuda()
    x[some], res[some] = r(len(some), 8, dtype=BF16), r(len(some), 8, dtype=BF16)
    few = res[some]
    want = rsq.rms_norm(x[some], w, residual=few, out_dtype=out)
    got = rsq.rms_norm(x, w, residual=res, out_dtype=out)
    assert torch.equal(res[some], few)
    for a, b in zip(got if out == "int8" else [got], want if out == "int8" else [want]):
        assert torch.equal(a[some], b)


def test_conv_tokens_of_two_launches():
    """An element a lane (an odd number of channels): 2^32 - 256 of them a launch."""
    C = 4353
    per = ((1 << 32) - 256) // C
    n = per + 2000
    x = torch.zeros(n, C, dtype=BF16, device="cuda")
    st = torch.zeros(n, C, 1, dtype=BF16, device="cuda")
    r = gen(4)
    w, b = r(C, 2), r(C)
    some = torch.cat([torch.arange(0, 5), torch.arange(per - 5, per + 5), torch.arange(n - 5, n)]).cuda()
    x[some], st[some] = r(len(some), C, dtype=BF16), r(len(some), C, 1, dtype=BF16)
    few = st[some]
    want = rsq.causal_conv_step(x[some], w, b, state=few, activation="silu")
    y = rsq.causal_conv_step(x, w, b, state=st, activation="silu")
    assert torch.equal(y[some], want) and torch.equal(st[some], few)


# ---------------------------------------------------------------- ragged batches

def scan_bounded(case, off, seqs, state, longest):
    """ssm_scan within the reference's bounds, rows of no sequence untouched."""
    x, dt, A, B, C, D, bias = case
    want, S, by, bS = ref.scan(x, dt, A, B, C, D, bias, True, state, seqs, x.dtype)
    out = torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
    y, got = rsq.ssm_scan(x, dt, A, B, C, D=D, dt_bias=bias, softplus=True, state=state, offsets=off, max_len=longest, out=out)
    inside = torch.zeros(x.shape[0], dtype=torch.bool)
    for a, m in seqs:
        inside[a: a + m] = True
    check(y[inside.cuda()], want[inside], by[inside], "y")
    check(got, S, bS, "state")
    assert (y[~inside.cuda()] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("given", [True, False])
def test_scan_long_prompts_among_hundreds(dtype, given):
    """Cut prompts at the front, in the middle and at the end of 200 sequences of a few tokens or none."""
    lengths = [n % 4 for n in range(200)]
    lengths[1], lengths[70], lengths[130], lengths[199] = 900, 400, 321, 700
    case = ssm_case(sum(lengths) + 5, 2, 1, 16, 16, dtype, seed=2)
    off, _ = offsets_of(lengths, 2, 3)
    seqs = [(int(a), n) for a, n in zip(off[:-1].tolist(), lengths)]
    scan_bounded(case, off, seqs, gen(5)(200, 2, 16, 16) if given else None, 900)


def test_scan_falling_offsets_of_long_sequences():
    """Sequences over the same rows have more segments than rows allow for: those that do not fit run whole."""
    n = 700
    case = ssm_case(n, 2, 1, 16, 16, F32, seed=3)
    off = torch.tensor([0, n] * 6 + [300, n], dtype=torch.int32).cuda()
    o = off.tolist()
    seqs = [(a, max(0, b - a)) for a, b in zip(o[:-1], o[1:])]
    x, dt, A, B, C, D, bias = case
    want, S, by, bS = ref.scan(x, dt, A, B, C, D, bias, True, None, seqs, F32)
    y, got = rsq.ssm_scan(x, dt, A, B, C, D=D, dt_bias=bias, softplus=True, offsets=off, max_len=n)
    check(got, S, bS, "state")
    assert torch.isfinite(y).all()


def conv_bounded(C, width, lengths_or_offsets, n, longest, dtype, given):
    """causal_conv within the reference's bounds, rows of no sequence untouched, states as they follow."""
    off = torch.tensor(lengths_or_offsets, dtype=torch.int32).cuda()
    o = off.tolist()
    seqs = [(a, max(0, b - a)) for a, b in zip(o[:-1], o[1:])]
    r = gen(C)
    x, w, b = r(n, C, dtype=dtype), r(C, width) * 0.5, r(C)
    st = r(len(seqs), C, width - 1, dtype=dtype) if given else None
    want, new, bound = ref.conv(x, w, b, st, seqs, True, dtype)
    out = torch.full(x.shape, 7.0, dtype=dtype, device="cuda")
    y = rsq.causal_conv(x, w, b, state=st, offsets=off, max_len=longest, activation="silu", out=out)
    inside = torch.zeros(n, dtype=torch.bool)
    for a, m in seqs:
        inside[a: a + m] = True
    check(y[inside.cuda()], want[inside], bound[inside], "y")
    assert (y[~inside.cuda()] == 7.0).all()
    if given:
        assert torch.equal(st.cpu().double(), new)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C,width", [(520, 4), (37, 3)])
@pytest.mark.parametrize("count", [40, 300, 1500])
def test_conv_long_prompts_among_many(dtype, C, width, count):
    """Long prompts at the front, in the middle and at the end of sequences of a few tokens or none."""
    lengths = [n % 3 for n in range(count)]
    lengths[0], lengths[count // 2], lengths[-1] = 900, 333, 700
    o = 3 + np.concatenate([[0], np.cumsum(lengths)])
    conv_bounded(C, width, o.tolist(), int(o[-1]) + 2, 900, dtype, count == 300)


def test_conv_falling_offsets_of_long_sequences():
    """Sequences over the same rows have more blocks than rows allow for; no state, so that all give the same rows."""
    n = 3000
    conv_bounded(64, 4, [0, n] * 40, n, n, F32, False)


def test_conv_more_equal_sequences_than_workgroups():
    """2^24 - 1 workgroups of 256 threads a launch: two tokens each, an element a lane."""
    n = (1 << 24) + 3
    x = torch.zeros(n, 2, 5, dtype=BF16, device="cuda")
    r = gen(6)
    w, b = r(5, 3), r(5)
    some = torch.cat([torch.arange(0, 9), torch.arange((1 << 23) - 5, (1 << 23) + 5), torch.arange(n - 9, n)]).cuda()
    x[some] = r(len(some), 2, 5, dtype=BF16)
    y = rsq.causal_conv(x, w, b)
    assert torch.equal(y[some], rsq.causal_conv(x[some], w, b))


# ---------------------------------------------------------------- the scan's range

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk", [16, 128])
def test_scan_large_products_of_b_and_c(dtype, dk):
    """C . B of about 2^95 and x of 2^-80 under decays of 2^-76 a chunk: weights and outputs are in range throughout."""
    n = 130
    r = gen(dk)
    x, B, C = r(n, 2, 16) * 2.0 ** -80, r(n, 1, dk) * 2.0 ** 55, r(n, 1, dk) * 2.0 ** 38
    x, B, C = x.to(dtype), B.to(dtype), C.to(dtype)
    dt = torch.full((n, 2), 0.825, device="cuda").to(dtype)
    A = -torch.ones(2, device="cuda")
    want, S, by, bS = ref.scan(x, dt, A, B, C, None, None, False, None, [(0, n)], dtype)
    y, got = rsq.ssm_scan(x[None], dt[None], A, B[None], C[None])
    check(y[0], want, by, "y")
    check(got, S, bS, "state")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 64, 100, 700])
def test_scan_heads_that_keep_nothing(dtype, n):
    """A of -inf: e^(delta A) is 0, so y is (C . B) delta x and the state what the last token adds, also where a chunk
    is not full. 16 products and their sum, delta, the weight and its parts: at most 16 + 8 roundings of fp32."""
    r = gen(n)
    x, B, C = r(1, n, 2, 16, dtype=dtype), r(1, n, 1, 16, dtype=dtype), r(1, n, 1, 16, dtype=dtype)
    dt = (r(1, n, 2).abs() + 0.1).to(dtype)
    A = torch.tensor([-float("inf"), -1.0], device="cuda")
    y, S = rsq.ssm_scan(x, dt, A, B, C)
    xd, Bd, Cd, d = (t[0].cpu().double() for t in (x, B, C, dt))
    want = (Cd * Bd).sum(2) * d[:, :1] * xd[:, 0]
    mag = (Cd * Bd).abs().sum(2) * d[:, :1] * xd[:, 0].abs()
    check(y[0, :, 0], want, mag * (24 * U + (2.0 ** -15 if dtype == BF16 else 0)) + 1.01 * ref.half_step(dtype) * want.abs())
    last = Bd[-1, 0][:, None] * d[-1, 0] * xd[-1, 0][None]
    check(S[0, 0], last, last.abs() * 8 * U)
    assert torch.isfinite(y).all() and torch.isfinite(S).all()


# ---------------------------------------------------------------- the step on a quantized state

def test_state_step_refuses_operands_in_the_states_buffer():
    st = rsq.State(model="mamba2", batch=2, heads=4, d_k=128, d_v=64, group=64, bits=8, in_dtype="bf16")
    x, dt, A, B, C, D, bias = ssm_case(2, 4, 2, 128, 64, BF16, slices=False)
    st.load_dense(gen(1)(2, 4, 128, 64))
    before = st.buf.clone()
    part = lambda t: st.buf[8192: 8192 + t.numel() * t.element_size()].view(t.dtype).view(t.shape)  # noqa: E731
    for i in range(8):
        args = [x, dt, A, B, C, D, bias, torch.empty_like(x)]
        args[i] = part(args[i])
        with pytest.raises(rsq.Error) as e:
            st.ssm_step(*args[:5], D=args[5], dt_bias=args[6], softplus=True, out=args[7])
        assert e.value.code == rsq._abi.RSQ_E_INVALID
    assert torch.equal(st.buf, before) and st.counters() == (0, 0)


# ---------------------------------------------------------------- streams

def test_operands_dropped_while_another_stream_has_yet_to_read_them():
    """stream=: the operands' memory is not given to the current stream's next tensors before the call has run."""
    side = torch.cuda.Stream()
    x, dt, A, B, C, D, bias = ssm_case(512, 2, 1, 64, 64, BF16, slices=False)
    r = gen(9)
    w, nw, cols = r(128, 4), r(128), r(512, 128, dtype=BF16)
    codes, scales, _, _ = w4_case(1, 64, 128, 64, BF16, torch.float16)
    given = r(1, 2, 64, 64)
    opt = dict(D=D, dt_bias=bias, softplus=True)
    w4 = rsq.W4Weight(codes, scales)
    token = [t[:1].clone() for t in (x, dt, B, C)]

    def quantized(dense, stream):
        st = rsq.State(model="mamba2", batch=1, heads=2, d_k=128, d_v=64, group=64, bits=8, in_dtype="bf16")
        torch.cuda.current_stream().synchronize()
        st.load_dense(dense, stream=stream)
        return st.buf

    calls = [
        (lambda v, s: rsq.causal_conv(v[0], w, stream=s), [cols[None]]),
        (lambda v, s: rsq.causal_conv_step(v[0], w, stream=s), [cols]),
        (lambda v, s: rsq.ssm_scan(v[0], v[1], A, v[2], v[3], stream=s, **opt)[0], [x[None], dt[None], B[None], C[None]]),
        (lambda v, s: rsq.ssm_step(v[4], v[0], v[1], A, v[2], v[3], stream=s, **opt), token + [given]),
        (lambda v, s: rsq.rms_norm(v[0], nw, stream=s), [cols]),
        (lambda v, s: rsq.w4_linear(v[0], w4, stream=s), [cols]),
        (lambda v, s: rsq.W4Weight(v[0], v[1], stream=s).packed, [codes, scales]),
        (lambda v, s: quantized(v[0], s), [r(1, 2, 128, 64)]),
    ]
    for call, operands in calls:
        want = call([t.clone() for t in operands], None)
        mine = [t.clone() for t in operands]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(mine, side)
        sizes = [(t.shape, t.dtype) for t in mine]
        del mine
        over = [torch.full(s, 3, dtype=d, device="cuda") for s, d in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del over


# ---------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("xt", [F32, BF16, "e4m3", "int8"])
@pytest.mark.parametrize("mean", [0.0, 1.0])
@pytest.mark.parametrize("m,n,k,group", [(16, 512, 4736, 128), (3, 100, 1280, 32), (59, 705, 3712, 64), (70, 5500, 512, 128),
                                         (40, 6100, 1024, 32)])
def test_w4_norm_of_the_error(xt, mean, m, n, k, group):
    """The error's norm within what the sums' roundings leave (layer_bounds), where the elementwise bound has room for
    a lost piece of x."""
    codes, s, x, xs = w4_case(m, n, k, group, xt, F32, seed=k)
    if mean:
        if xs is None:
            x = (x.float() + mean).to(x.dtype)
        else:
            v = (x.float() * xs + mean)
            xs = (v.abs().amax(1, keepdim=True) / (127 if xt == "int8" else 448)).contiguous()
            x = torch.round(v / xs).to(torch.int8) if xt == "int8" else (v / xs).to(torch.float8_e4m3fn)
    y = rsq.w4_linear(x, rsq.W4Weight(codes, s), x_scale=xs, out_dtype="f32").cpu().double().numpy()
    c, sd, xd = codes.cpu().double().numpy(), s.cpu().double().numpy(), x.float().cpu().double().numpy()
    if xs is not None:
        xd = xd * xs.cpu().double().numpy()
    want = xd @ (c * sd.repeat(group, 1)).T
    if xt == "int8":      # exact inside a group: only y's own roundings are left
        limit = 2 * U * np.sqrt((k // group / 4 + 8 + 3) / 3) * np.linalg.norm(want)
    else:
        limit = w4_norm_limit(c, sd, xd, group, xt is F32, xs is not None)
    assert np.linalg.norm(y - want) <= limit


@pytest.mark.parametrize("xt", [F32, BF16, "e4m3", "int8"])
@pytest.mark.parametrize("m,n,k,group", [(16, 8512, 2048, 128), (64, 4096, 1024, 32), (1, 28672, 1024, 64)])
def test_w4_is_repeatable(xt, m, n, k, group):
    codes, s, x, xs = w4_case(m, n, k, group, xt, F32, seed=1)
    w = rsq.W4Weight(codes, s)
    first = rsq.w4_linear(x, w, x_scale=xs, out_dtype="f32")
    for _ in range(8):
        assert torch.equal(rsq.w4_linear(x, w, x_scale=xs, out_dtype="f32"), first)


# ---------------------------------------------------------------- the scan cut into segments

def workspace_of(tokens, seqs, longest, heads, groups, dk, dv, dtype):
    """Bytes that ssm_scan asks for."""
    import ctypes
    abi = rsq._abi
    p = abi.Ssm()
    kw = dict(dtype=abi.BF16 if dtype == BF16 else abi.F32, seqs=seqs, heads=heads, groups=groups, d_k=dk, d_v=dv,
              tokens=tokens, max_len=longest, offsets=16, x_stride=heads * dv, y_stride=heads * dv, b_stride=groups * dk,
              c_stride=groups * dk, dt_stride=heads)
    for k, v in kw.items():
        setattr(p, k, v)
    n = ctypes.c_size_t()
    rsq._abi.check(rsq._abi.lib.rsq_ssm_scan_workspace(ctypes.byref(p), ctypes.byref(n)))
    return n.value


@pytest.mark.parametrize("heads,groups,dk,dv,dtype", [(3, 1, 128, 72, BF16), (2, 2, 256, 136, BF16), (4, 2, 64, 200, BF16),
                                                      (3, 1, 128, 136, F32), (4, 4, 64, 72, F32), (5, 1, 72, 8, F32)])
@pytest.mark.parametrize("given", [True, False])
def test_scan_segments_of_every_head_and_column_block(heads, groups, dk, dv, dtype, given):
    lengths = [700, 5, 0, 300, 256]
    n = sum(lengths)
    assert workspace_of(n, 5, 700, heads, groups, dk, dv, dtype) > 0
    case = ssm_case(n, heads, groups, dk, dv, dtype, seed=dk + dv)
    off, _ = offsets_of(lengths)
    seqs = [(int(a), m) for a, m in zip(off[:-1].tolist(), lengths)]
    scan_bounded(case, off, seqs, gen(2)(5, heads, dk, dv) if given else None, 700)


@pytest.mark.parametrize("heads,dk,dtype", [(64, 64, F32), (16, 128, F32), (64, 128, BF16), (16, 256, BF16)])
def test_scan_repeats_to_the_bit(heads, dk, dtype):
    """Kernels of every type and width, with the chip full: a result read before its product is done would differ."""
    n = 2500
    case = ssm_case(n, heads, 1, dk, 64, dtype, seed=5)
    off, _ = offsets_of([1500, 7, 993])
    args = (*case[:5], case[5], case[6], True, None, off, 1500)
    y0, S0 = rsq.ssm_scan(*args)
    assert torch.isfinite(y0).all()
    for _ in range(10):
        y, S = rsq.ssm_scan(*args)
        assert torch.equal(y, y0) and torch.equal(S, S0)


# ---------------------------------------------------------------- the step on a quantized state, to the bit

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kw", [dict(bits=4), dict(bits=6), dict(bits=8), dict(bits=32), dict(head_bits=[8, 6, 4, 8]),
                                dict(bits=4, hadamard=True), dict(bits=8, scale_mode="yoked"), dict(bits=4, lrb_k=2, lrb_m=6)])
def test_state_step_is_the_gates_and_a_decode_step(kw, dtype):
    """State.ssm_step gives what decode_step does with q = C, k = B, v = delta x rounded to the inputs' type and alpha =
    e^(delta A), and D x on its output. The dense step shows the same alpha (on a state of ones, without inputs) and
    delta x (on a zero state, with B = 1)."""
    n, heads, groups, dk, dv = 2, 4, 2, 128, 64
    full = dict(model="mamba2", batch=n, heads=heads, d_k=dk, d_v=dv, group=64, in_dtype="bf16" if dtype == BF16 else "f32", **kw)
    a, b = rsq.State(**full), rsq.State(**full)
    S = gen(6)(n, heads, dk, dv)
    a.load_dense(S)
    b.load_dense(S)
    for t in range(3):
        x, dt, A, B, C, D, bias = ssm_case(n, heads, groups, dk, dv, dtype, seed=t)
        opt = dict(dt_bias=bias, softplus=True)
        y = a.ssm_step(x, dt, A, B, C, D=D, **opt)
        none, one = torch.zeros_like(B[..., :8]), torch.ones_like(B[..., :8])
        decay = torch.ones(n, heads, 8, 8, device="cuda")
        rsq.ssm_step(decay, torch.zeros_like(x[..., :8]).contiguous(), dt, A, none, none, **opt)
        added = torch.zeros(n, heads, 8, dv, device="cuda")
        rsq.ssm_step(added, x.contiguous(), dt, A, one, none, **opt)
        per = heads // groups
        o = b.decode_step(C.repeat_interleave(per, 1).contiguous(), B.repeat_interleave(per, 1).contiguous(),
                          added[:, :, 0].to(dtype).contiguous(), alpha=decay[..., 0, 0].contiguous())
        assert torch.equal(a.buf, b.buf)
        # (the sum's 53 bits rounded to fp32 as one operation would)
        want = (o.double() + D.double()[:, None] * x.double()).float().to(dtype)
        assert torch.equal(y, want)


def test_stream_given_inside_a_capture():
    """stream= of the capturing stream, operands dropped while the capture runs: replays give the eager result."""
    x, dt, A, B, C, D, bias = ssm_case(700, 2, 1, 64, 64, BF16, slices=False)
    w = gen(2)(64, 4)
    want = rsq.ssm_scan(x[None], dt[None], A, B[None], C[None], D=D)[0].clone()
    rows = rsq.causal_conv(want[:, :, 0].contiguous(), w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = torch.cuda.current_stream()
        y, _ = rsq.ssm_scan(x[None], dt[None], A, B[None], C[None], D=D, stream=s)
        part = y[:, :, 0].contiguous()
        z = rsq.causal_conv(part, w, stream=s)
        del part
    for _ in range(4):
        y.zero_(), z.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same(y, want) and same(z, rows)      # (the state grows until it overflows)
        torch.randn(1000, device="cuda").sum().item()
