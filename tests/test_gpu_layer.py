"""Layer operators around the decode step against their fp64 definitions."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from layer_reference import H, U, check

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
rsq = None


@pytest.fixture(scope="module", autouse=True)
def _package():
    global rsq
    rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
    assert torch.cuda.is_available()


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s, dtype=F32: torch.randn(*s, generator=g).to(dtype).cuda()


def offsets_of(lengths, first=0, gap=0):
    """Packed offsets; the rows before `first` and `gap` rows at the end belong to no sequence."""
    o = first + np.concatenate([[0], np.cumsum(lengths)])
    return torch.tensor(o, dtype=torch.int32).cuda(), int(o[-1]) + gap


# ---------------------------------------------------------------- convolution

def conv_case(C, width, dtype, lengths, bias=True, state=True, silu=True, wide_rows=0, shift=0, first=0, gap=0, seed=0):
    r = gen(seed)
    off, n = offsets_of(lengths, first, gap)
    buf = r(n * (C + wide_rows) + shift + 8, dtype=dtype)
    x = buf[shift: shift + n * (C + wide_rows)].view(n, C + wide_rows)[:, :C]
    w, b = r(C, width) * 0.5, r(C) if bias else None
    st = r(len(lengths), C, width - 1, dtype=dtype) if state else None
    return x, w, b, st, off


def run_conv(x, w, b, st, off, lengths, silu, packed=True):
    seqs = [(int(a), n) for a, n in zip(off[:-1].tolist(), lengths)]
    want, new, bound = ref.conv(x, w, b, st, seqs, silu, x.dtype)
    out = torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
    y = rsq.causal_conv(x, w, b, state=st, offsets=off, max_len=max(lengths), activation="silu" if silu else None, out=out)
    assert y is out
    inside = torch.zeros(x.shape[0], dtype=torch.bool)
    for a, n in seqs:
        inside[a: a + n] = True
    check(y[inside.cuda()], want[inside], bound[inside], "y")
    assert (y[~inside.cuda()] == 7.0).all(), "rows of no sequence are left as they were"
    if st is not None:
        assert torch.equal(st.cpu().double(), new), "state"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("C", [8, 520, 37])
def test_conv_prompt(dtype, width, C):
    lengths = [0, 1, 2, 3, 33, 129, 300]
    x, w, b, st, off = conv_case(C, width, dtype, lengths, first=2, gap=3, seed=C + width)
    run_conv(x, w, b, st, off, lengths, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bias,state,silu", [(False, True, True), (True, False, True), (False, False, False), (True, True, False)])
def test_conv_options(dtype, bias, state, silu):
    lengths = [40, 1, 0, 7]
    x, w, b, st, off = conv_case(64, 4, dtype, lengths, bias, state, silu)
    run_conv(x, w, b, st, off, lengths, silu)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("wide_rows,shift", [(64, 0), (3, 0), (0, 1), (64, 4)])
def test_conv_strides_and_alignment(dtype, wide_rows, shift):
    lengths = [70, 5]
    x, w, b, st, off = conv_case(96, 4, dtype, lengths, wide_rows=wide_rows, shift=shift)
    run_conv(x, w, b, st, off, lengths, True)


def test_conv_batch_form_and_step_continue_a_prompt():
    """[B, T, C] equals the packed form; a prompt in two parts, then token by token, equals the whole."""
    r = gen(5)
    x, w, b = r(3, 50, 72, dtype=BF16), r(72, 4), r(72)
    off = torch.arange(4, dtype=torch.int32).cuda() * 50
    whole = rsq.causal_conv(x, w, b, activation="silu")
    packed = rsq.causal_conv(x.view(150, 72), w, b, offsets=off, max_len=50, activation="silu").view(3, 50, 72)
    assert torch.equal(whole, packed)
    st = torch.zeros(3, 72, 3, dtype=BF16, device="cuda")
    got = [rsq.causal_conv(x[:, :2].contiguous(), w, b, state=st, activation="silu"),
           rsq.causal_conv(x[:, 2:37].contiguous(), w, b, state=st, activation="silu")]
    got += [rsq.causal_conv_step(x[:, t], w, b, state=st, activation="silu")[:, None] for t in range(37, 50)]
    assert torch.equal(torch.cat(got, 1), whole)
    assert torch.equal(st, x[:, -3:].transpose(1, 2))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width,C,batch", [(2, 8, 1), (3, 37, 5), (4, 4352, 3), (4, 64, 129)])
def test_conv_step(dtype, width, C, batch):
    r = gen(C)
    x, w, b, st = r(batch, C + 8, dtype=dtype)[:, :C], r(C, width), r(C), r(batch, C, width - 1, dtype=dtype)
    want, new, bound = ref.conv(x, w, b, st, [(i, 1) for i in range(batch)], True, dtype)
    check(rsq.causal_conv_step(x, w, b, state=st, activation="silu"), want, bound, "y")
    assert torch.equal(st.cpu().double(), new)


def test_conv_extremes_stay_in_their_channel_and_time():
    """Infinities and NaN reach only the width - 1 following tokens of their channel; rows behind the sequences
    do not matter; silu of large negative values is zero."""
    lengths = [40]
    x, w, b, st, off = conv_case(16, 4, F32, lengths, gap=4)
    x[40:] = float("nan")
    x[10, 3], x[20, 5], x[30, 7] = float("nan"), float("inf"), -1e30
    w[7] = 1.0
    b[:] = 0
    clean = x.clone()
    clean[10, 3], clean[20, 5], clean[30, 7] = 0, 0, 0
    y = rsq.causal_conv(x, w, b, offsets=off, max_len=40, activation="silu")
    z = rsq.causal_conv(clean, w, b, offsets=off, max_len=40, activation="silu")
    touched = torch.zeros(44, 16, dtype=torch.bool)
    touched[10:14, 3], touched[20:24, 5], touched[30:34, 7] = True, True, True
    touched[40:] = True
    assert torch.equal(y[~touched.cuda()], z[~touched.cuda()])
    assert torch.isnan(y[10:14, 3]).all() and not torch.isfinite(y[20:24, 5]).any() and (y[30:34, 7] == 0).all()


def test_conv_offsets_out_of_range_are_clamped():
    """Offsets are device data: ends past the rows and falling offsets cannot leave the tensors."""
    x, w, b, _, _ = conv_case(64, 4, BF16, [30])
    off = torch.tensor([-5, 10, 4, 1000], dtype=torch.int32).cuda()
    y = rsq.causal_conv(x, w, b, offsets=off, max_len=30)
    want, _, bound = ref.conv(x, w, b, None, [(0, 10)], False, BF16)
    check(y[:4], want[:4], bound[:4])      # rows 4.. belong to two of these sequences


# ---------------------------------------------------------------- selective scan

def ssm_case(n, heads, groups, dk, dv, dtype, seed=0, slices=True):
    r = gen(seed)
    if slices:   # x, B, C as slices of one row, dt of a wider one
        row = r(n, heads * dv + 2 * groups * dk, dtype=dtype)
        x = row[:, : heads * dv].view(n, heads, dv)
        B = row[:, heads * dv: heads * dv + groups * dk].view(n, groups, dk)
        C = row[:, heads * dv + groups * dk:].view(n, groups, dk)
        dt = r(n, heads + 5, dtype=dtype)[:, 3: 3 + heads]
    else:
        x, B, C, dt = r(n, heads, dv, dtype=dtype), r(n, groups, dk, dtype=dtype), r(n, groups, dk, dtype=dtype), r(n, heads, dtype=dtype)
    A, D, bias = -torch.exp(r(heads)), r(heads), r(heads) - 3.0
    return x, dt, A, B, C, D, bias


def run_scan(case, lengths, state=None, softplus=True, D=True, bias=True, first=0, gap=0):
    x, dt, A, B, C, Dv, bv = case
    Dv, bv = Dv if D else None, bv if bias else None
    off, n = offsets_of(lengths, first, gap)
    assert n == x.shape[0]
    seqs = [(int(a), m) for a, m in zip(off[:-1].tolist(), lengths)]
    want, S, by, bS = ref.scan(x, dt, A, B, C, Dv, bv, softplus, state, seqs, x.dtype)
    out = torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
    y, got = rsq.ssm_scan(x, dt, A, B, C, D=Dv, dt_bias=bv, softplus=softplus, state=state, offsets=off,
                          max_len=max(lengths), out=out)
    inside = torch.zeros(n, dtype=torch.bool)
    for a, m in seqs:
        inside[a: a + m] = True
    check(y[inside.cuda()], want[inside], by[inside], "y")
    check(got, S, bS, "state")
    assert (y[~inside.cuda()] == 7.0).all()
    return y, got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,groups,dk,dv", [(1, 1, 8, 8), (4, 2, 64, 64), (2, 1, 128, 64), (3, 3, 72, 72), (2, 2, 16, 136)])
def test_scan_shapes(dtype, heads, groups, dk, dv):
    lengths = [0, 1, 17, 63, 64, 65, 130]
    case = ssm_case(sum(lengths) + 4, heads, groups, dk, dv, dtype, seed=dk + dv)
    run_scan(case, lengths, state=gen(1)(len(lengths), heads, dk, dv), first=1, gap=3)


def test_scan_wide_keys():
    lengths = [100, 3]
    case = ssm_case(103, 2, 1, 256, 64, BF16)
    run_scan(case, lengths, state=gen(1)(2, 2, 256, 64))
    case = ssm_case(103, 2, 1, 200, 32, BF16)
    run_scan(case, lengths)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("softplus,D,bias,state", [(True, False, True, False), (True, True, False, True), (False, False, True, True)])
def test_scan_options(dtype, softplus, D, bias, state):
    lengths = [70, 0, 20]
    case = list(ssm_case(90, 4, 2, 64, 64, dtype, slices=False))
    if not softplus:
        case[1] = case[1].abs() * 0.1
        case[6] = case[6].abs() * 0.01
    run_scan(tuple(case), lengths, gen(3)(3, 4, 64, 64) if state else None, softplus, D, bias)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_in_segments(dtype):
    """One head's long prompts run in several segments side by side, next to short and empty ones."""
    lengths = [700, 5, 0, 300, 256]
    case = ssm_case(sum(lengths), 1, 1, 64, 64, dtype, seed=9)
    run_scan(case, lengths, state=gen(2)(5, 1, 64, 64))
    run_scan(case, lengths)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_decays_strong_weak_and_none(dtype):
    """Decays of e^-60 a token between tokens that keep everything: differences of large running sums."""
    r = gen(4)
    x, dt, A, B, C, D, _ = ssm_case(150, 4, 1, 64, 64, dtype, slices=False)
    A = torch.tensor([-60.0, -1.0, 0.0, -1e-6]).cuda()
    dt = (torch.rand(150, 4, generator=torch.Generator().manual_seed(1)) < 0.3).to(dtype).cuda()   # 0 or 1
    want, S, by, bS = ref.scan(x, dt, A, B, C, D, None, False, None, [(0, 150)], dtype)
    y, got = rsq.ssm_scan(x[None], dt[None], A, B[None], C[None], D=D)
    check(y[0], want, by, "y")
    check(got, S, bS, "state")


def test_scan_growing_state():
    """A > 0 grows: the weights of later tokens, which overflow, stay out."""
    x, dt, A, B, C, D, _ = ssm_case(64, 2, 1, 16, 16, F32, slices=False)
    A = torch.tensor([3.0, 0.5]).cuda()
    dt = torch.full((64, 2), 1.0).cuda()
    want, S, by, bS = ref.scan(x, dt, A, B, C, D, None, False, None, [(0, 25), (25, 39)], F32)
    off = torch.tensor([0, 25, 64], dtype=torch.int32).cuda()
    y, got = rsq.ssm_scan(x, dt, A, B, C, D=D, offsets=off, max_len=39)
    fine = want.abs() < 1e30
    check(torch.where(fine, y.cpu().double(), 0.0), torch.where(fine, want, 0.0), by, "y")


def test_scan_parts_and_steps_continue_a_prompt():
    """A prompt in parts, then token by token on the same state, follows the definition throughout."""
    x, dt, A, B, C, D, bias = ssm_case(100, 4, 2, 64, 64, F32, seed=11)
    want, S, by, bS = ref.scan(x, dt, A, B, C, D, bias, True, None, [(0, 100)], F32)
    y1, st = rsq.ssm_scan(x[None, :70], dt[None, :70], A, B[None, :70], C[None, :70], D=D, dt_bias=bias, softplus=True)
    y2, st2 = rsq.ssm_scan(x[None, 70:90], dt[None, 70:90], A, B[None, 70:90], C[None, 70:90], D=D, dt_bias=bias,
                           softplus=True, state=st)
    assert st2 is st
    ys = [y1[0], y2[0]]
    for t in range(90, 100):
        ys.append(rsq.ssm_step(st, x[t: t + 1], dt[t: t + 1], A, B[t: t + 1], C[t: t + 1], D=D, dt_bias=bias, softplus=True))
    check(torch.cat(ys), want, by, "y")
    check(st, S, bS, "state")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_bad_values_do_not_reach_earlier_tokens(bad, where, dtype):
    case = list(ssm_case(260, 4, 2, 64, 64, dtype, slices=False))
    x, dt, A, B, C, D, bias = [t.clone() for t in case]
    run = lambda: rsq.ssm_scan(x[None], dt[None], A, B[None], C[None], D=D, dt_bias=bias, softplus=True)  # noqa: E731
    y0, S0 = run()
    t = 90
    if where == "x":
        x[t, 1, 5] = bad
    elif where == "B":
        B[t, 0, 3] = bad
    elif where == "C":
        C[t, 0, 3] = bad
    else:
        dt[t, 1] = bad
    y, S = run()
    assert torch.equal(y[:, :t], y0[:, :t])
    assert torch.equal(y[:, :, 2:], y0[:, :, 2:]) and torch.equal(S[:, 2:], S0[:, 2:])     # the other group
    if where == "x":      # one column of one head, for good
        assert torch.isnan(y[0, t:, 1, 5]).all() and torch.isnan(S[0, 1, :, 5]).all()
        y[0, :, 1, 5], y0[0, :, 1, 5], S[0, 1, :, 5], S0[0, 1, :, 5] = 0, 0, 0, 0
        assert torch.equal(y, y0) and torch.equal(S, S0)
    elif where == "C":    # this token only
        assert not torch.isfinite(y[0, t, :2]).any()
        assert torch.equal(y[:, t + 1:], y0[:, t + 1:]) and torch.equal(S, S0)
    elif where == "B":
        assert not torch.isfinite(y[0, t, :2]).any() and not torch.isfinite(S[0, :2, 3]).any()
    elif bad == bad and bad < 0:
        assert torch.isfinite(y).all()    # softplus(-inf) = 0: the token neither decays nor adds
    else:
        assert not torch.isfinite(y[0, t, 1]).any()


def test_scan_rows_behind_the_sequences_do_not_matter():
    lengths = [70, 33]
    case = ssm_case(110, 2, 1, 64, 64, BF16)
    y0, S0 = run_scan(case, lengths, gap=7)
    for t in (case[0], case[1], case[3], case[4]):
        t[103:] = float("nan")
    off, _ = offsets_of(lengths)
    y, S = rsq.ssm_scan(case[0], case[1], case[2], case[3], case[4], D=case[5], dt_bias=case[6], softplus=True,
                        offsets=off, max_len=70)
    assert torch.equal(y[:103], y0[:103]) and torch.equal(S, S0)


def test_scan_is_repeatable():
    lengths = [700, 300]
    case = ssm_case(1000, 2, 1, 128, 64, BF16)
    off, _ = offsets_of(lengths)
    args = (*case[:5], case[5], case[6], True, None, off, 700)
    y0, S0 = rsq.ssm_scan(*args)
    for _ in range(5):
        y, S = rsq.ssm_scan(*args)
        assert torch.equal(y, y0) and torch.equal(S, S0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_far_apart(dtype):
    """Rows 2^24 bytes apart, the most the scan takes: 150 of them pass 2^31 bytes (two chunks, several bases)."""
    n, cols = 150, (1 << 24) // torch.finfo(dtype).bits * 8
    case = ssm_case(n, 2, 1, 64, 64, dtype, slices=False)
    far = torch.empty(n, cols, dtype=dtype, device="cuda")
    far[:, :128], far[:, 256: 320], far[:, 512: 576] = case[0].view(n, 128), case[3][:, 0], case[4][:, 0]
    x, B, C = far[:, :128].view(n, 2, 64), far[:, 256: 320].view(n, 1, 64), far[:, 512: 576].view(n, 1, 64)
    off = torch.tensor([0, 3, n], dtype=torch.int32).cuda()
    want = rsq.ssm_scan(*case[:5], offsets=off, max_len=n - 3)
    out = torch.empty(n, cols, dtype=dtype, device="cuda")[:, :128].view(n, 2, 64)
    y, S = rsq.ssm_scan(x, case[1], case[2], B, C, offsets=off, max_len=n - 3, out=out)
    assert torch.equal(y, want[0]) and torch.equal(S, want[1])
    w = gen(4)(128, 4)
    z = rsq.causal_conv(far[:, :128], w, offsets=off, max_len=n - 3, out=out.view(n, 128))
    assert torch.equal(z, rsq.causal_conv(case[0].reshape(n, 128), w, offsets=off, max_len=n - 3))


def test_nothing_to_do():
    """No tokens, no rows: outputs are empty, states as they were, a new scan state zero."""
    e = lambda *s: torch.zeros(*s, dtype=BF16, device="cuda")   # noqa: E731
    A, w = -torch.ones(2, device="cuda"), torch.ones(8, 4, device="cuda")
    cs = gen(1)(3, 8, 3, dtype=BF16)
    for x, off in ((e(3, 0, 8), None), (e(0, 8), torch.zeros(4, dtype=torch.int32, device="cuda")),
                   (e(5, 8), torch.full((4,), 2, dtype=torch.int32, device="cuda"))):
        st = cs.clone()
        y = rsq.causal_conv(x, w, state=st, offsets=off, max_len=0 if off is not None else None)
        assert y.shape == x.shape and torch.equal(st, cs)
    given = gen(2)(3, 2, 8, 16)
    for lead, off in (((3, 0), None), ((0,), torch.zeros(4, dtype=torch.int32, device="cuda")),
                      ((5,), torch.full((4,), 2, dtype=torch.int32, device="cuda"))):
        args = e(*lead, 2, 16), e(*lead, 2), A, e(*lead, 1, 8), e(*lead, 1, 8)
        kw = dict(offsets=off, max_len=0 if off is not None else None)
        y, S = rsq.ssm_scan(*args, **kw)
        assert y.shape == args[0].shape and S.shape == (3, 2, 8, 16) and (S == 0).all()
        st = given.clone()
        y, S = rsq.ssm_scan(*args, state=st, **kw)
        assert S is st and torch.equal(st, given)
    assert rsq.rms_norm(e(0, 64), torch.ones(64, device="cuda")).shape == (0, 64)
    q, sc = rsq.rms_norm(e(2, 0, 64), torch.ones(64, device="cuda"), out_dtype="int8", group=32)
    assert q.shape == (2, 0, 64) and sc.shape == (2, 0, 2)
    w4 = rsq.W4Weight(torch.ones(16, 64, dtype=torch.int8, device="cuda"), torch.ones(16, 2, device="cuda"))
    assert rsq.w4_linear(e(0, 64), w4).shape == (0, 16) and rsq.w4_linear(e(2, 0, 64), w4).shape == (2, 0, 16)
    assert rsq.w4_linear(q, w4, x_scale=sc).shape == (2, 0, 16)


def test_scan_offsets_out_of_range_are_clamped():
    case = ssm_case(60, 2, 1, 64, 64, BF16)
    off = torch.tensor([0, 20, 15, 1000], dtype=torch.int32).cuda()
    y, S = rsq.ssm_scan(*case[:5], offsets=off, max_len=60)
    want, Sw, by, bS = ref.scan(*case[:5], None, None, False, None, [(0, 20), (20, 0), (15, 45)], BF16)
    check(S, Sw, bS, "state")


# ---------------------------------------------------------------- single tokens

def step_bounds(state, x, dt, A, B, C, D, bias, softplus):
    n = x.shape[0]
    return ref.scan(x, dt, A, B, C, D, bias, softplus, state, [(i, 1) for i in range(n)], F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,heads,groups,dk,dv", [(1, 1, 1, 8, 8), (2, 64, 1, 128, 64), (5, 3, 3, 72, 24), (3, 2, 1, 264, 1000), (2, 4, 2, 16, 1024)])
def test_step(dtype, batch, heads, groups, dk, dv):
    x, dt, A, B, C, D, bias = ssm_case(batch, heads, groups, dk, dv, dtype, seed=dv)
    st = gen(2)(batch, heads, dk, dv)
    want, S, by, bS = step_bounds(st, x, dt, A, B, C, D, bias, True)
    if dtype == BF16:
        by = by + H * 1.01 * want.abs()
    check(rsq.ssm_step(st, x, dt, A, B, C, D=D, dt_bias=bias, softplus=True), want, by, "y")
    check(st, S, bS, "state")


def test_step_without_options():
    x, dt, A, B, C, D, bias = ssm_case(2, 4, 2, 64, 64, F32, slices=False)
    dt = dt.abs()
    st = gen(2)(2, 4, 64, 64)
    want, S, by, bS = step_bounds(st, x, dt, A, B, C, None, None, False)
    check(rsq.ssm_step(st, x, dt, A, B, C), want, by, "y")
    check(st, S, bS, "state")


def test_step_large_state_offsets():
    """A state of more than 2^31 elements: the last sequences' tiles are right."""
    n, heads, dk, dv = 264, 64, 256, 512
    r = gen(3)
    st = torch.zeros(n, heads, dk, dv, device="cuda")
    assert st.numel() > 2 ** 31
    x, B, C = r(n, heads, dv, dtype=BF16), r(n, 1, dk, dtype=BF16), r(n, 1, dk, dtype=BF16)
    dt, A = r(n, heads, dtype=BF16).abs(), -torch.ones(heads, device="cuda")
    st[-1] = 1.0
    y = rsq.ssm_step(st, x, dt, A, B, C)
    one = torch.ones(1, heads, dk, dv, device="cuda")
    z = rsq.ssm_step(one, x[-1:], dt[-1:], A, B[-1:], C[-1:])
    assert torch.equal(y[-1:], z) and torch.equal(st[-1:], one)


# ---------------------------------------------------------------- norm

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 8), (5, 37), (4, 512), (2, 1000), (7, 1024), (3, 2048), (2, 4100), (1, 8192), (2, 16384), (1, 32768)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_norm(dtype, rows, cols, out):
    r = gen(cols)
    x, res, w = r(rows, cols, dtype=dtype), r(rows, cols, dtype=dtype) * 3, r(cols)
    want, h, rel = ref.norm(x, w, 1e-5, res)
    y = rsq.rms_norm(x, w, eps=1e-5, residual=res, out_dtype=out)
    check(y, want, want.abs() * (rel + (H * 1.01 if out == "bf16" else U)) + 1e-37, "y")
    check(res, h, h.abs() * (1.01 * ref.half_step(dtype) + U) + 1e-37, "residual")
    want, _, rel = ref.norm(x, w, 1e-5, None)
    check(rsq.rms_norm(x, w, out_dtype=out), want, want.abs() * (rel + (H * 1.01 if out == "bf16" else U)) + 1e-37, "y")


def check_codes(codes, scales, want, rel, group, out):
    """codes * scale within half a step (of the code, for e4m3 2^-4 of the value or 2^-10 below 2^-6), and the scale
    absmax / qmax."""
    rows, cols = want.shape
    g = group or cols
    qmax = 448.0 if out == "e4m3" else 127.0
    w = want.view(rows, cols // g, g)
    s = w.abs().amax(2) / qmax
    check(scales.view(rows, -1), s, s * (rel + 2 * U), "scales")
    got = codes.float().cpu().double().view_as(w) * scales.cpu().double().view(rows, -1, 1)
    if out == "e4m3":
        half = torch.maximum(w.abs() * 2.0 ** -4, s[..., None] * 2.0 ** -10)
    else:
        half = 0.5 * s[..., None].expand_as(w)
        assert (codes.int().abs() <= 127).all()
    check(got, w, half * 1.0001 + w.abs() * (2 * rel + 4 * U), "codes")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("out", ["int8", "e4m3"])
@pytest.mark.parametrize("rows,cols,group", [(1, 8, 0), (3, 37, 0), (5, 1024, 0), (2, 2048, 64), (3, 4096, 32), (2, 96, 32), (4, 640, 128), (1, 16384, 128), (2, 5000, 0)])
def test_norm_codes(dtype, out, rows, cols, group):
    r = gen(cols + group)
    x, res, w = r(rows, cols, dtype=dtype), r(rows, cols, dtype=dtype), r(cols)
    want, _, rel = ref.norm(x, w, 1e-5, res)
    codes, scales = rsq.rms_norm(x, w, residual=res, out_dtype=out, group=group)
    assert scales.shape == (rows, cols // group if group else 1)
    check_codes(codes, scales, want, rel, group, out)


def test_norm_strides_alignment_and_leading_dimensions():
    r = gen(1)
    buf = r(2 * 5 * 130 + 1)
    x = buf[1:].view(2, 5, 130)[:, :, :100]
    res = r(2, 5, 104)[:, :, :100]
    res0 = res.clone()
    w = r(101)[1:].contiguous()
    out = torch.full((2, 5, 120), 9, dtype=torch.int8, device="cuda")[:, :, :100]
    want, _, rel = ref.norm(x, w, 1e-3, res0)
    codes, scales = rsq.rms_norm(x, w, eps=1e-3, residual=res, out_dtype="int8", out=out)
    assert scales.shape == (2, 5, 1)
    check_codes(codes.reshape(10, 100), scales.reshape(10, 1), want.reshape(10, 100), rel, 0, "int8")


@pytest.mark.parametrize("out", ["int8", "e4m3", "f32"])
def test_norm_extremes(out):
    """Zero rows give zero codes and steps; a NaN or an infinity spoils its row (or group) visibly and no other."""
    x = gen(2)(6, 256)
    w = torch.ones(256, device="cuda")
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 9] = float("inf")
    x[4] = 1e-30
    x[5, :128] = 0
    y = rsq.rms_norm(x, w, eps=0.0 if out == "f32" else 1e-12, out_dtype=out, group=0 if out == "f32" else 128)
    if out == "f32":
        assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()       # 0 / 0 without eps
        assert torch.isfinite(y[0]).all()
        return
    codes, scales = y
    val = codes.float().view(6, 2, 128) * scales[..., None]
    assert (codes[1].float() == 0).all() and (scales[1] == 0).all()
    assert torch.isnan(scales[2]).all() and torch.isnan(val[2]).any()      # the whole row: its mean is one
    assert torch.isfinite(val[0]).all() and torch.isfinite(val[4]).all() and torch.isfinite(val[5]).all()
    assert (scales[5, 0] == 0) and (codes[5, :128].float() == 0).all()
    assert not torch.isfinite(val[3]).all()


# ---------------------------------------------------------------- 4-bit weights

def w4_case(m, n, k, group, xt, scales, seed=0):
    r = gen(seed)
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-8, 8, (n, k), generator=g, dtype=torch.int8).cuda()
    s = (r(n, k // group).abs() + 0.1).to(scales)
    x, xs = r(m, k), None
    if xt in ("int8", "e4m3", "int8g", "e4m3g"):
        grp = group if xt.endswith("g") else k
        q = 127.0 if xt.startswith("int8") else 448.0
        xv = x.view(m, k // grp, grp)
        xs = (xv.abs().amax(2) / q).contiguous()
        v = (xv / xs[..., None]).view(m, k)
        x = torch.round(v).to(torch.int8) if xt.startswith("int8") else v.to(torch.float8_e4m3fn)
    else:
        x = x.to(xt)
    return codes, s, x, xs


def w4_reference(codes, s, x, xs, group, out):
    n, k = codes.shape
    w = codes.cpu().double() * s.cpu().double().repeat_interleave(group, 1)
    xv = x.float().cpu().double()
    if xs is not None:
        xv = xv * xs.cpu().double().repeat_interleave(k // xs.shape[1], 1)
    want = xv @ w.t()
    # fp32 sums of 24 + c: at most (31 + 24) / 1 times |x| a code; k + k additions, three pieces of fp32 x, the scales' products
    smax = s.cpu().double().repeat_interleave(group, 1)
    mag = xv.abs() @ (smax * 55.0 if x.dtype != torch.int8 else w.abs()).t()
    pieces = 3 if x.dtype == torch.float32 else 1
    bound = mag * (2.0 * k / 8 * pieces + 2.0 * k / group + 24) * U
    return want, bound * 1.01 + (H * 1.01 if out == "bf16" else U) * want.abs() + 1e-37


@pytest.mark.parametrize("xt", [BF16, F32, "int8", "e4m3", "int8g", "e4m3g"])
@pytest.mark.parametrize("m,n,k,group", [(1, 1, 32, 32), (1, 16, 128, 128), (3, 17, 160, 32), (16, 50, 192, 64), (17, 100, 1280, 128), (40, 33, 320, 64), (65, 20, 96, 32), (130, 6200, 256, 128), (2, 17000, 384, 64)])
def test_w4(xt, m, n, k, group):
    scales = torch.float16 if (m + n) % 2 else F32
    codes, s, x, xs = w4_case(m, n, k, group, xt, scales, seed=n)
    w = rsq.W4Weight(codes, s)
    for out in ("f32", "bf16"):
        want, bound = w4_reference(codes, s, x, xs, group, out)
        check(rsq.w4_linear(x, w, x_scale=xs, out_dtype=out), want, bound, out)


@pytest.mark.parametrize("xt", [BF16, F32, "int8g", "e4m3"])
@pytest.mark.parametrize("m,n,k,group", [(60, 1990, 384, 64), (30, 6100, 160, 32), (40, 6100, 256, 128), (33, 8003, 96, 32),
                                         (17, 12820, 160, 32), (5, 20500, 192, 64), (70, 5500, 192, 64), (90, 5500, 96, 32)])
def test_w4_more_rows(xt, m, n, k, group):
    """Several tiles of weight rows and of x a workgroup, the last ones cut."""
    codes, s, x, xs = w4_case(m, n, k, group, xt, torch.float16, seed=m)
    w = rsq.W4Weight(codes, s)
    want, bound = w4_reference(codes, s, x, xs, group, "f32")
    out = torch.full((m + 1, n + 1), 3.0, device="cuda")
    check(rsq.w4_linear(x, w, x_scale=xs, out_dtype="f32", out=out[:m, :n]), want, bound)
    assert (out[m] == 3).all() and (out[:, n] == 3).all()


@pytest.mark.parametrize("scales", [F32, torch.float16])
def test_w4_large_weights(scales):
    """Packed codes of more than 2^32 bytes: the last rows are right, and the first."""
    n, k, group = (1 << 18) + 3, 1 << 15, 32
    codes = torch.zeros(n, k, dtype=torch.int8, device="cuda")
    s = torch.zeros(n, k // group, dtype=scales, device="cuda")
    some = torch.tensor([0, 1, 17, n // 2, n - 20, n - 1], device="cuda")
    c0, s0, x, _ = w4_case(3, 6, k, group, BF16, scales)
    codes[some], s[some] = c0, s0
    y = rsq.w4_linear(x, rsq.W4Weight(codes, s), out_dtype="f32")
    want, bound = w4_reference(c0, s0, x, None, group, "f32")
    check(y[:, some], want, bound)
    y[:, some] = 0
    assert (y == 0).all()


def test_w4_rows_far_apart():
    """Rows of x 2^24 bytes apart, the most there is."""
    codes, s, x, _ = w4_case(40, 40, 192, 64, BF16, torch.float16)
    far = torch.empty(40, 1 << 23, dtype=BF16, device="cuda")
    far[:, 5:197] = x
    w = rsq.W4Weight(codes, s)
    assert torch.equal(rsq.w4_linear(far[:, 5:197], w), rsq.w4_linear(x, w))


@pytest.mark.parametrize("xt", [BF16, F32, "int8", "e4m3"])
def test_w4_strides_and_alignment(xt):
    codes, s, x, xs = w4_case(5, 40, 192, 64, xt, torch.float16)
    w = rsq.W4Weight(codes, s)
    want, bound = w4_reference(codes, s, x, xs, 64, "f32")
    wide = torch.zeros(5, 211, device="cuda").to(x.dtype)
    wide[:, 3:195] = x
    out = torch.full((5, 45), 3.0, device="cuda")
    y = rsq.w4_linear(wide[:, 3:195], w, x_scale=xs, out_dtype="f32", out=out[:, 1:41])
    check(y, want, bound)
    assert (out[:, 0] == 3).all() and (out[:, 41:] == 3).all()


def test_w4_bad_rows_stay_alone():
    codes, s, x, xs = w4_case(6, 40, 256, 64, BF16, torch.float16)
    w = rsq.W4Weight(codes, s)
    y0 = rsq.w4_linear(x, w, out_dtype="f32")
    x[2, 100], x[4, 3] = float("nan"), float("inf")
    y = rsq.w4_linear(x, w, out_dtype="f32")
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], y0[keep])
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[4]).any()


def test_w4_takes_the_norms_codes():
    """int8 and e4m3 codes with row or group scales go from the norm into the product."""
    r = gen(8)
    x, nw = r(3, 4, 256, dtype=BF16), r(256)
    codes, s, _, _ = w4_case(1, 100, 256, 64, BF16, torch.float16)
    w = rsq.W4Weight(codes, s)
    for out in ("int8", "e4m3"):
        for group in (0, 64):
            q, qs = rsq.rms_norm(x, nw, out_dtype=out, group=group)
            y = rsq.w4_linear(q, w, x_scale=qs, out_dtype="f32")
            assert y.shape == (3, 4, 100)
            want, bound = w4_reference(codes, s, q.view(12, 256), qs.view(12, -1), 64, "f32")
            check(y.view(12, 100), want, bound, out)


# ---------------------------------------------------------------- from a prompt to the quantized state

def dense_states(dk, dv, batch=2, heads=3):
    S = gen(dk + dv)(batch, heads, dk, dv)
    S[0, 0, :8] = 0
    S[0, 1, 3] *= 1e-6
    S[1, 2] *= 1e3
    return S


@pytest.mark.parametrize("scale_dtype", ["f32", "f16"])
@pytest.mark.parametrize("kw", [dict(bits=4), dict(bits=8), dict(head_bits=[8, 6, 4]), dict(bits=4, hadamard=True),
                                dict(bits=6, scale_mode="persistent"), dict(bits=4, scale_mode="yoked"),
                                dict(bits=4, lrb_k=2, lrb_m=6)])
@pytest.mark.parametrize("dk,dv,group", [(128, 128, 32), (128, 64, 64)])
def test_load_dense_quantizes_as_the_step_does(scale_dtype, kw, dk, dv, group):
    """Codes, steps and reference against the oracle's quantizer on the same values."""
    import oracle
    from oracle import recurrence, hadamard
    from rsq_workloads import Workload
    S = dense_states(dk, dv)
    full = dict(model="mamba2", batch=2, heads=3, d_k=dk, d_v=dv, group=group, scale_dtype=scale_dtype, **kw)
    st = rsq.State(**full)
    st.load_dense(S)
    got = st.read_tiles()
    bits = np.array([st.head_bits()[t % 3] for t in range(6)])
    x = S.cpu().numpy().reshape(6, dk, dv)
    if kw.get("hadamard"):
        x = hadamard.fwht(x, group, oracle.F32)
    w = Workload(name="t", model="mamba2", batch=2, heads=3, d_k=dk, d_v=dv, steps=1, in_dtype="f32", bits=4,
                 group=group, scale_mode=kw.get("scale_mode", "dynamic"), scale_dtype=scale_dtype)
    zero = oracle.OState(codes=np.zeros((6, dk, dv), np.int32), scales=np.zeros((6, dk, dv // group), np.float32), bits=bits)
    codes, scales, _, diag = recurrence._requantize(zero, w, x.astype(np.float32), None, None, oracle.F32)
    assert np.array_equal(got["scales"], scales)
    assert np.array_equal(got["codes"], codes)
    assert st.counters() == (0, 0) and st.get_status() & rsq._abi.F_NONFINITE == 0
    if "ref" in got:
        assert np.array_equal(got["ref"], S.cpu().numpy().reshape(6, dk, dv))
    if kw.get("lrb_m"):
        assert not got["U"].any() and not got["W"].any()


def test_load_dense_fp32_state_window_and_flags():
    S = dense_states(128, 64)
    st = rsq.State(model="mamba2", batch=2, heads=3, d_k=128, d_v=64, group=64, bits=32)
    st.load_dense(S)
    assert np.array_equal(st.read_tiles()["S32"].reshape(2, 3, 128, 64), S.cpu().numpy())
    st = rsq.State(model="gdn", batch=1, heads=2, d_k=128, d_v=128, group=32, bits=4, pw_window=4)
    r = gen(1)
    S = r(1, 2, 128, 128)
    q, k, v = r(1, 2, 128), r(1, 2, 128) * 0.05, r(1, 2, 128)
    gates = dict(alpha=torch.full((1, 2), 0.9).cuda(), beta=torch.full((1, 2), 0.5).cuda())
    st.load_dense(S)
    first = [st.decode_step(q, k, v, **gates) for _ in range(6)]
    st.load_dense(S)      # a used window is empty again
    again = [st.decode_step(q, k, v, **gates) for _ in range(6)]
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    S[0, 1, 5, 5] = float("nan")
    st.load_dense(S)
    assert st.get_status() & rsq._abi.F_NONFINITE
    with pytest.raises(ValueError):
        st.load_dense(S[:, :1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_state_step_matches_the_dense_step(dtype):
    """On an fp32 state (bits = 32) the quantized path's step is the dense one, but for v = delta x rounded to
    the inputs' type: |B| |delta x| H a token."""
    n, heads, dk, dv = 2, 4, 128, 64
    x, dt, A, B, C, D, bias = ssm_case(n, heads, 2, dk, dv, dtype, seed=3)
    S = gen(6)(n, heads, dk, dv)
    want, Sw, by, bS = step_bounds(S, x, dt, A, B, C, D, bias, True)
    st = rsq.State(model="mamba2", batch=n, heads=heads, d_k=dk, d_v=dv, group=64, bits=32,
                   in_dtype="bf16" if dtype == BF16 else "f32")
    st.load_dense(S)
    y = st.ssm_step(x, dt, A, B, C, D=D, dt_bias=bias, softplus=True)
    d = torch.nn.functional.softplus(dt.float() + bias).cpu().double()
    rep = lambda t: t.cpu().double().repeat_interleave(2, 1)  # noqa: E731
    v = (d[..., None] * x.cpu().double()).abs() * ref.half_step(dtype) * 1.01
    extra = rep(B).abs()[..., :, None] * v[..., None, :]
    check(torch.from_numpy(st.read_tiles()["S32"]).view(n, heads, dk, dv), Sw, bS + extra, "state")
    ey = torch.matmul(rep(C).abs()[..., None, :], extra).squeeze(-2)
    check(y, want, by + ey + ref.half_step(dtype) * 1.01 * want.abs(), "y")


def test_state_step_refusals():
    x, dt, A, B, C, D, bias = ssm_case(2, 4, 2, 128, 64, F32)
    st = rsq.State(model="gla", batch=2, heads=4, d_k=128, d_v=64, group=64, bits=8)
    with pytest.raises(rsq.Error):
        st.ssm_step(x, dt, A, B, C)
    st = rsq.State(model="mamba2", batch=2, heads=4, d_k=128, d_v=64, group=64, bits=8, in_dtype="bf16")
    with pytest.raises(rsq.Error):
        st.ssm_step(x, dt, A, B, C)          # fp32 inputs for a bf16 state
    st = rsq.State(model="mamba2", batch=2, heads=4, d_k=128, d_v=64, group=64, bits=8, lrb_k=0, lrb_m=2)
    for _ in range(2):
        st.ssm_step(x, dt, A, B, C)
    with pytest.raises(rsq.Error) as e:
        st.ssm_step(x, dt, A, B, C)
    assert e.value.code == rsq._abi.RSQ_E_BYPASS_FULL and st.counters() == (2, 2)


# ---------------------------------------------------------------- the layer, streams and graphs

class Layer:
    """A Mamba2 block from the operators: norm -> 4-bit projection -> convolution -> scan or step -> norm -> projection."""

    def __init__(self, d=256, heads=4, dk=128, dv=64, groups=1, seed=0):
        r = gen(seed)
        self.d, self.H, self.dk, self.dv, self.G = d, heads, dk, dv, groups
        self.inner, self.conv = heads * dv, heads * dv + 2 * groups * dk
        self.w_in = self.weight(self.conv + heads, d, seed)
        self.w_out = self.weight(d, self.inner, seed + 1)
        self.n1, self.n2 = 1 + 0.1 * r(d), 1 + 0.1 * r(self.inner)
        self.cw, self.cb = 0.5 * r(self.conv, 4), 0.1 * r(self.conv)
        self.A, self.D, self.bias = -torch.exp(r(heads)), r(heads), r(heads) - 3

    @staticmethod
    def weight(n, k, seed):
        g = torch.Generator().manual_seed(seed)
        codes = torch.randint(-8, 8, (n, k), generator=g, dtype=torch.int8).cuda()
        return rsq.W4Weight(codes, torch.full((n, k // 64), 1.0 / (4.6 * k ** 0.5), device="cuda").half())

    def __call__(self, h, conv_state, mix, offsets=None, max_len=None):
        """h: residual rows [n, d] (replaced); mix(x, dt, B, C) -> y [n, H, dv]."""
        zero = torch.zeros_like(h)
        q, qs = rsq.rms_norm(zero, self.n1, residual=h, out_dtype="int8")
        p = rsq.w4_linear(q, self.w_in, x_scale=qs)
        n = h.shape[0]
        xbc = p[:, : self.conv]
        if offsets is None:
            xbc = rsq.causal_conv_step(xbc, self.cw, self.cb, state=conv_state, activation="silu")
        else:
            xbc = rsq.causal_conv(xbc, self.cw, self.cb, state=conv_state, offsets=offsets, max_len=max_len, activation="silu")
        x = xbc[:, : self.inner].view(n, self.H, self.dv)
        B = xbc[:, self.inner: self.inner + self.G * self.dk].view(n, self.G, self.dk)
        C = xbc[:, self.inner + self.G * self.dk:].view(n, self.G, self.dk)
        y = mix(x, p[:, self.conv:], B, C)
        q, qs = rsq.rms_norm(y.reshape(n, self.inner), self.n2, out_dtype="int8", group=64)
        return rsq.w4_linear(q, self.w_out, x_scale=qs)


def test_a_layers_prompt_and_tokens():
    """Prompts through the layer, then tokens one by one on the dense state and on an INT8 one: the dense tokens
    follow a prompt that holds them all, the quantized ones the dense ones."""
    torch.manual_seed(0)
    L = Layer()
    lengths, more = [40, 25], 6
    hs = [torch.randn(n + more, L.d).cuda().to(BF16) for n in lengths]
    opt = dict(D=L.D, dt_bias=L.bias, softplus=True)

    def prompt(parts):
        off, n = offsets_of([len(p) for p in parts])
        cs = torch.zeros(2, L.conv, 3, dtype=BF16, device="cuda")
        box = {}

        def mix(x, dt, B, C):
            y, box["S"] = rsq.ssm_scan(x, dt, L.A, B, C, offsets=off, max_len=max(map(len, parts)), **opt)
            return y
        out = L(torch.cat(parts).clone(), cs, mix, off, max(map(len, parts)))
        return out, box["S"], cs

    whole, S_all, _ = prompt(hs)
    _, S, cs = prompt([h[:n] for h, n in zip(hs, lengths)])
    st = rsq.State(model="mamba2", batch=2, heads=L.H, d_k=L.dk, d_v=L.dv, group=64, bits=8, in_dtype="bf16")
    st.load_dense(S)
    cs8 = cs.clone()
    for t in range(more):
        tok = torch.stack([h[n + t] for h, n in zip(hs, lengths)])
        dense = L(tok.clone(), cs, lambda x, dt, B, C: rsq.ssm_step(S, x, dt, L.A, B, C, **opt))
        quant = L(tok.clone(), cs8, lambda x, dt, B, C: st.ssm_step(x, dt, L.A, B, C, **opt))
        row = torch.tensor([lengths[0] + t, lengths[0] + more + lengths[1] + t]).cuda()
        want = whole[row].double()
        # int8 codes of two norms flip where bf16 roundings differ (2^-8 a value, steps of 2^-6 of it): a few percent at most
        assert (dense.double() - want).norm() <= 0.03 * want.norm()
        assert (quant.double() - dense.double()).norm() <= 0.05 * want.norm()
    assert (S.double() - S_all.double()).norm() <= 0.01 * S_all.double().norm()


def graph_check(call, outs, restore):
    """Capture call, replay it several times with eager work between, compare every replay with the eager result."""
    restore()
    call()
    want = [o.clone() for o in outs()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        restore()
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    restore()
    with torch.cuda.graph(g):
        call()
    for _ in range(4):
        restore()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs(), want):
            assert torch.equal(a, b)
        torch.randn(1000, device="cuda").sum().item()


def test_captured_calls_replay():
    r = gen(0)
    box = {}
    outs = lambda: box["o"]  # noqa: E731
    # convolution, prompt and token
    x, w, b, s0, off = conv_case(72, 4, BF16, [70, 9])
    st = s0.clone()

    def conv():
        box["o"] = [rsq.causal_conv(x, w, b, state=st, offsets=off, max_len=70, activation="silu"), st]
    graph_check(conv, outs, lambda: st.copy_(s0))

    def step():
        box["o"] = [rsq.causal_conv_step(x[:2], w, b, state=st, activation="silu"), st]
    graph_check(step, outs, lambda: st.copy_(s0))
    # scan in several segments (workspace from the graph's pool), twice in one graph, and step
    case = ssm_case(1100, 2, 1, 64, 64, BF16)
    S0 = r(1, 2, 64, 64)
    S = S0.clone()
    opt = dict(D=case[5], dt_bias=case[6], softplus=True)
    lead = [t[None] for t in (case[0], case[1])], [t[None] for t in (case[3], case[4])]

    def scan():
        y1, _ = rsq.ssm_scan(*lead[0], case[2], *lead[1], state=S, **opt)
        y2, _ = rsq.ssm_scan(*lead[0], case[2], *lead[1], state=S, **opt)
        box["o"] = [y1, y2, S]
    graph_check(scan, outs, lambda: S.copy_(S0))

    def ssm():
        box["o"] = [rsq.ssm_step(S, case[0][:1], case[1][:1], case[2], case[3][:1], case[4][:1], **opt), S]
    graph_check(ssm, outs, lambda: S.copy_(S0))
    # norm and product
    res0 = r(5, 256, dtype=BF16)
    res, nx, nw = res0.clone(), r(5, 256, dtype=BF16), r(256)
    codes, sc, _, _ = w4_case(1, 100, 256, 64, BF16, torch.float16)
    W = rsq.W4Weight(codes, sc)

    def norm():
        q, qs = rsq.rms_norm(nx, nw, residual=res, out_dtype="int8", group=64)
        box["o"] = [q, qs, res, rsq.w4_linear(q, W, x_scale=qs)]
    graph_check(norm, outs, lambda: res.copy_(res0))
    # a token on a quantized state
    q8 = rsq.State(model="mamba2", batch=1, heads=2, d_k=128, d_v=64, group=64, bits=8, in_dtype="bf16")
    c2 = ssm_case(1, 2, 1, 128, 64, BF16)
    q8.load_dense(r(1, 2, 128, 64))
    saved = q8.buf.clone()

    def qstep():
        box["o"] = [q8.ssm_step(c2[0], c2[1], c2[2], c2[3], c2[4], D=c2[5], dt_bias=c2[6], softplus=True)]
    graph_check(qstep, outs, lambda: q8.buf.copy_(saved))
    with pytest.raises(rsq.Error):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q8.load_dense(S0.new_zeros(1, 2, 128, 64))


def same(a, b):
    """Equal, with NaNs (of a state that grows without bound) in the same places."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)])


def test_two_captured_scans_share_no_workspace():
    """Graphs of two different scans replayed in turn on two streams."""
    graphs, outs, wants = [], [], []
    for seed in (1, 2):
        case = ssm_case(1100, 2, 1, 64, 64, BF16, seed=seed)
        args = [t[None] for t in case[:2]] + [case[2]] + [t[None] for t in case[3:5]]
        wants.append([t.clone() for t in rsq.ssm_scan(*args, D=case[5])])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(rsq.ssm_scan(*args, D=case[5]))
        graphs.append((g, args, case))
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for i in (0, 1):
            with torch.cuda.stream(s[i]):
                graphs[i][0].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            assert same(outs[i][0], wants[i][0]) and same(outs[i][1], wants[i][1])


def test_calls_on_a_stream_of_their_own():
    """stream=: the call, its workspace and its outputs belong to that stream."""
    side = torch.cuda.Stream()
    case = ssm_case(1100, 2, 1, 64, 64, BF16)
    args = [t[None] for t in case[:2]] + [case[2]] + [t[None] for t in case[3:5]]
    want = rsq.ssm_scan(*args, D=case[5])
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got.append(rsq.ssm_scan(*args, D=case[5], stream=side))
        torch.randn(1 << 20, device="cuda")       # the current stream's allocations do not take the workspace
    x, w, b, _, _ = conv_case(64, 4, BF16, [30])
    c = rsq.causal_conv(x[None], w, b, stream=side)
    side.synchronize()
    for y, S in got:
        assert same(y, want[0]) and same(S, want[1])
    assert torch.equal(c, rsq.causal_conv(x[None], w, b))


def test_calls_on_two_streams_at_once():
    """Calls that run side by side, from two threads: workspaces, staging and errors are each call's own."""
    import threading

    r = gen(12)
    x, w = r(32, 1024, dtype=BF16), torch.ones(1024, device="cuda")
    codes, s, _, _ = w4_case(1, 2048, 1024, 64, BF16, torch.float16)
    w4 = rsq.W4Weight(codes, s)
    cases = [ssm_case(2100, 2, 1, 64, 64, BF16, seed=i) for i in range(2)]
    args = [[t[None] for t in c[:2]] + [c[2]] + [t[None] for t in c[3:5]] for c in cases]

    def calls(i, stream=None):
        q, sc = rsq.rms_norm(x, w, out_dtype="int8", stream=stream)
        return [rsq.w4_linear(q, w4, x_scale=sc, stream=stream), *rsq.ssm_scan(*args[i], stream=stream)]

    want = [calls(i) for i in range(2)]
    torch.cuda.synchronize()
    streams, got, wrong = [torch.cuda.Stream() for _ in range(2)], [None, None], []

    def work(i):
        try:
            for _ in range(20):
                got[i] = calls(i, streams[i])
                with pytest.raises(ValueError):
                    rsq.rms_norm(x, w[:-1], stream=streams[i])
            streams[i].synchronize()
        except Exception as e:  # a failure of a thread is the test's
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    for i in range(2):
        assert all(same(a, b) for a, b in zip(got[i], want[i]))
