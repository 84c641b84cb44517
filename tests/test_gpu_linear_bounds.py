"""Attention with the delta rule where the bounds of its plain comparison leave room: operands chosen so that little but
the arithmetic under test is left in o. Terms that cancel make o small, so that its own rounding to bf16 hides nothing."""
import pytest
import torch

from layer_reference import H, U, check, f64
from test_gpu_linear import compare, compare_step, expected, make

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
rsq = None


@pytest.fixture(scope="module", autouse=True)
def _package():
    global rsq
    import test_gpu_linear
    rsq = test_gpu_linear.rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
    assert torch.cuda.is_available()


def zeros(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("heads,dk,dv", [(1, 8, 16), (2, 128, 40), (1, 256, 24), (300, 128, 104)])
def test_a_state_enters_bf16_prompts_to_sixteen_bits(heads, dk, dv):
    """o = S_a - S_b of two rows of the state, with nothing written. S_b is a bf16 value. Of S_a, whose last 16 bits are all
    ones, two pieces may leave 2^-16 (two cut ones leave twice that); four terms are added, in fp32."""
    T = 20
    q, k, v = zeros(1, T, 1, dk, dtype=BF16), zeros(1, T, 1, dk, dtype=BF16), zeros(1, T, heads, dv, dtype=BF16)
    k[..., 0] = 1.0
    q[..., 2], q[..., 5] = 1.0, -1.0
    S = zeros(1, heads, dk, dv)
    scale = torch.exp2(torch.arange(dv, device="cuda") % 9 - 4.0)
    S[:, :, 2], S[:, :, 5] = (1 + 2.0 ** -7 - 2.0 ** -23) * scale, (1 + 2.0 ** -7) * scale
    before = S.clone()
    o, S = rsq.linear_attention(q, k, v, beta=zeros(1, T, heads), state=S)
    assert torch.equal(S, before)
    want = (f64(S[:, None, :, 2]) - f64(S[:, None, :, 5])).expand(1, T, heads, dv)
    bound = f64(S[:, None, :, 2]) * (2.0 ** -16 + 2 * 4 * 1.01 * U) + H * want.abs()
    check(o, want, bound.expand_as(want), "o")


@pytest.mark.parametrize("heads,dk,dv", [(1, 8, 16), (2, 128, 40), (1, 256, 24), (300, 128, 104)])
def test_values_and_token_weights_enter_bf16_prompts_to_sixteen_bits(heads, dk, dv):
    """o = P u_0 - u_1 with P = u_0 = 1 + x, whose two pieces hold all of them, so that the product of the second pieces, x^2,
    is to be there. P's decay: its fraction's rounding and two powers of two (1 U and 2 U each), two products; u: the sum
    of six products of pieces, and the strength; o: eight terms of fp32 sums."""
    T, x = 24, 2.0 ** -8 - 2.0 ** -12
    q, k, v = zeros(1, T, 1, dk, dtype=BF16), zeros(1, T, 1, dk, dtype=BF16), zeros(1, T, heads, dv, dtype=BF16)
    k[:, 3, :, 1], k[:, 4, :, 6] = 1.0, 1.0
    q[..., 1], q[..., 6] = 2.0, 1.0
    v[:, 3], v[:, 4] = 1.0, -(1 + 2.0 ** -7)
    alpha, beta = torch.ones(1, T, heads, device="cuda"), zeros(1, T, heads)
    alpha[:, 4] = (1 + x) / 2
    beta[:, 3], beta[:, 4] = 1 + x, 1.0
    o, _ = rsq.linear_attention(q, k, v, alpha=alpha, beta=beta)
    want = torch.zeros(1, T, heads, dv, dtype=torch.float64)
    want[:, 3] = 2 * (1 + x)
    want[:, 4:] = (1 + x) ** 2 - (1 + 2.0 ** -7)
    terms = torch.zeros_like(want)
    terms[:, 3], terms[:, 4:] = 2 * (1 + x), (1 + x) ** 2 + 1 + 2.0 ** -7
    check(o, want, 1.01 * (7 + 7 + 8) * U * terms + H * want.abs(), "o")


def test_products_of_pieces_leave_out_either_sign():
    """o = q S of one row, fp32: three pieces of both, without the products below 2^-22. What is left out is of either sign,
    as are the roundings of five additions (U each at most, 1.5 U in the mean square with it): in the mean of 16384 of
    them nothing is left, where pieces that are all cut miss 1.1 U."""
    heads, T, dv = 4, 64, 64
    g = torch.Generator().manual_seed(1)
    q, k, v = zeros(1, T, 1, 8), zeros(1, T, 1, 8), zeros(1, T, heads, dv)
    q[..., 3] = (1 + torch.rand(1, T, 1, generator=g)).cuda()
    S = zeros(1, heads, 8, dv)
    S[:, :, 3] = (1 + torch.rand(1, heads, dv, generator=g)).cuda()
    o, S = rsq.linear_attention(q, k, v, beta=zeros(1, T, heads), state=S)
    want = f64(q[..., 3])[..., None] * f64(S[:, None, :, 3])
    off = (f64(o) - want) / want
    assert off.abs().max() < 12 * U
    assert off.mean().abs() < 0.3 * U, off.mean() / U


# ---------------------------------------------------------------- kernels of their own

def framed(t, value):
    """A copy of t with a row of `value` before and behind it, and the frame."""
    buf = torch.full((t.shape[0] + 2,) + tuple(t.shape[1:]), value, dtype=t.dtype, device="cuda")
    buf[1:-1] = t
    return buf[1:-1], buf


@pytest.mark.parametrize("dtype,dk,dv", [
    (BF16, 64, 72), (BF16, 40, 72), (BF16, 128, 72), (BF16, 120, 72), (BF16, 256, 72), (BF16, 200, 104),   # two column tiles a workgroup
    (F32, 64, 72), (F32, 40, 104), (F32, 128, 72), (F32, 120, 104),
    (BF16, 64, 104), (BF16, 24, 104), (BF16, 128, 104), (BF16, 72, 104)])                                  # four
@pytest.mark.parametrize("state", [True, False])
def test_workgroups_of_several_column_tiles(dtype, dk, dv, state):
    """Many heads: two or four column tiles a workgroup, the last of which have no columns, or eight of them. Sums are added
    in another order than by one tile a workgroup: each is held to the definition, and what surrounds the outputs stays."""
    heads, keys, lengths = 300, 3, [100, 40]
    c = make(lengths, heads, keys, dk, dv, dtype, seed=dk + dv, first=2, gap=3, pad=8, state=state)
    wide = torch.full((c["v"].shape[0], heads * dv + 16), 7.0, dtype=dtype, device="cuda")
    out = wide[:, 8: 8 + heads * dv].view(-1, heads, dv)
    S, frame = framed(c["state"], 5.0) if state else (None, None)
    o, S = rsq.linear_attention(c["q"], c["k"], c["v"], alpha=c["alpha"], beta=c["beta"], state=S, offsets=c["offsets"],
                                max_len=c["max_len"], out=out)
    for h in (0, 157, 299):
        g = h // (heads // keys)
        one = {**c, "q": c["q"][:, g: g + 1], "k": c["k"][:, g: g + 1], "v": c["v"][:, h: h + 1], "alpha": c["alpha"][:, h: h + 1],
               "beta": c["beta"][:, h: h + 1], "state": c["state"][:, h: h + 1] if state else None}
        compare(one, o[:, h: h + 1], S[:, h: h + 1], expected(one))
    assert (wide[:, :8] == 7.0).all() and (wide[:, -8:] == 7.0).all() and (o[:2] == 7.0).all() and (o[-3:] == 7.0).all()
    if state:
        assert (frame[0] == 5.0).all() and (frame[-1] == 5.0).all()
    assert torch.isfinite(S).all() and torch.isfinite(o).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("dk,dv", [(64, 40), (24, 136), (72, 104), (128, 72), (200, 40), (256, 200)])
def test_steps_on_states_past_the_caches(dtype, delta, dk, dv):
    """States of 16 MB and more, which are read and written past the caches."""
    heads = 16
    seqs = -(-(1 << 24) // (heads * dk * dv * 4))
    c = make([1] * seqs, heads, 4, dk, dv, dtype, seed=dk + dv, pad=8, delta=delta)
    S, frame = framed(c["state"], 5.0)
    o = rsq.linear_attention_step(S, c["q"], c["k"], c["v"], alpha=c["alpha"], beta=c["beta"])
    compare_step(c, o, S)
    assert (frame[0] == 5.0).all() and (frame[-1] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens", [1, 5, 20, 150])
@pytest.mark.parametrize("delta", [True, False])
def test_states_that_are_not_finite(dtype, tokens, delta):
    """A state's column that is not finite gives no finite o, also where a decay of zero clears what is finite (0 times an
    infinity is a NaN); other columns keep their bits. A state that is to be dropped is left out."""
    c = make([tokens] * 2, 2, 1, 64, 40, dtype, seed=tokens, delta=delta)
    c["alpha"][0] = 0.0
    k = c["k"]
    k[k == 0] = 1.0
    args = dict(alpha=c["alpha"], beta=c["beta"], offsets=c["offsets"], max_len=c["max_len"])
    o0, S0 = rsq.linear_attention(c["q"], k, c["v"], state=c["state"].clone(), **args)
    bad = c["state"].clone()
    bad[0, 1, 7, 3], bad[1, 0, 9, 39] = float("inf"), float("nan")
    o, S = rsq.linear_attention(c["q"], k, c["v"], state=bad, **args)
    mask = torch.zeros_like(o0, dtype=torch.bool)
    mask[:tokens, 1, 3] = mask[tokens:, 0, 39] = True
    state = torch.zeros_like(S0, dtype=torch.bool)
    state[0, 1, :, 3] = state[1, 0, :, 39] = True
    assert not torch.isfinite(o[mask]).any() and torch.equal(o[~mask], o0[~mask]) and torch.equal(S[~state], S0[~state])
    assert not torch.isfinite(S[0, 1, 7, 3]) and torch.isnan(S[1, 0, 9, 39])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", ["k", "alpha"])
@pytest.mark.parametrize("lengths", [[150, 90], [1500, 300]])
def test_keys_and_decays_that_are_not_finite_without_the_delta_rule(dtype, what, lengths):
    """Earlier tokens, other heads and other sequences keep their bits; from the token on the head's state is not finite."""
    c = make(lengths, 2, 2, 64, 32, dtype, seed=7, delta=False)
    args = lambda **kw: {"alpha": c["alpha"], "state": c["state"].clone(), "offsets": c["offsets"], "max_len": c["max_len"], **kw}  # noqa: E731
    o0, S0 = rsq.linear_attention(c["q"], c["k"], c["v"], **args())
    t = c[what].clone()
    t[(100, 1, 3) if what == "k" else (100, 1)] = float("nan")
    o, S = rsq.linear_attention(c["q"], t if what == "k" else c["k"], c["v"], **args(**({"alpha": t} if what == "alpha" else {})))
    n = lengths[0]
    assert torch.equal(o[:100], o0[:100]) and torch.equal(o[:, 0], o0[:, 0]) and torch.equal(o[n:], o0[n:])
    assert torch.isnan(o[100:n, 1]).all()
    assert torch.equal(S[0, 0], S0[0, 0]) and torch.equal(S[1], S0[1])
    assert torch.isnan(S[0, 1] if what == "alpha" else S[0, 1, 3]).all()
