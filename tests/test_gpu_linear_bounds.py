"""Attention with the delta rule where the bounds of its plain comparison leave room: operands chosen so that little but
the arithmetic under test is left in o. Terms that cancel make o small, so that its own rounding to bf16 hides nothing."""
import pytest
import torch

from layer_reference import H, U, check, f64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
rsq = None


@pytest.fixture(scope="module", autouse=True)
def _package():
    global rsq
    rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
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
