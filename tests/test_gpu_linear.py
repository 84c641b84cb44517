"""Attention with a decay for each head against its fp64 definition: prompts with and without the delta rule, the
token step, and a layer made of the operators around it."""
import numpy as np
import pytest
import torch

import linear_reference as ref
from layer_reference import H, U, check, f64
from linear_reference import check_columns

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
rsq = None


@pytest.fixture(scope="module", autouse=True)
def _package():
    global rsq
    rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
    assert torch.cuda.is_available()


def make(lengths, heads, keys, dk, dv, dtype, seed=0, first=0, gap=0, pad=0, alpha="token", delta=True, state=True):
    """Operands as a layer has them: q, k (of unit length) and v slices of one buffer's rows."""
    g = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    off = first + np.concatenate([[0], np.cumsum(lengths)])
    n = int(off[-1]) + gap
    qkv = randn(n, 2 * keys * dk + heads * dv + pad)
    keyed = qkv[:, : 2 * keys * dk].reshape(n, 2 * keys, dk)
    qkv[:, : 2 * keys * dk] = (keyed / keyed.norm(dim=2, keepdim=True)).reshape(n, 2 * keys * dk)
    qkv = qkv.to(dtype).cuda()
    c = dict(q=qkv[:, : keys * dk].view(n, keys, dk), k=qkv[:, keys * dk: 2 * keys * dk].view(n, keys, dk),
             v=qkv[:, 2 * keys * dk: 2 * keys * dk + heads * dv].view(n, heads, dv))
    if alpha == "token":
        c["alpha"] = torch.exp(-torch.rand(n, heads, generator=g) ** 4 * 3.0).cuda()
    elif alpha == "head":
        c["alpha"] = (1 - 2.0 ** -(3 + 4 * torch.rand(heads, generator=g))).cuda()
    else:
        c["alpha"] = None
    c["beta"] = torch.rand(n, heads, generator=g).cuda() if delta else None
    c["state"] = (0.5 * randn(len(lengths), heads, dk, dv)).cuda() if state else None
    c["offsets"], c["max_len"] = torch.tensor(off, dtype=torch.int32).cuda(), max(lengths)
    c["seqs"] = [(int(a), n) for a, n in zip(off[:-1], lengths)]
    return c


def expected(c):
    return ref.attention(c["q"], c["k"], c["v"], c["alpha"], c["beta"], c["state"], c["seqs"], c["q"].dtype)


def call(c, **kw):
    state = None if c["state"] is None else c["state"].clone()
    if "stream" in kw:
        kw["stream"].wait_stream(torch.cuda.current_stream())   # for the operands, that copy among them
    return rsq.linear_attention(c["q"], c["k"], c["v"], alpha=c["alpha"], beta=c["beta"], state=state, offsets=c["offsets"],
                                max_len=c["max_len"], **kw)


def compare(c, o, S, want):
    wo, wS, bo, bS = want
    inside = torch.zeros(wo.shape[0], dtype=torch.bool)
    for a, n in c["seqs"]:
        inside[a: a + n] = True
    check(o[inside.cuda()], wo[inside], bo[inside], "o")
    if c["beta"] is None:
        check(S, wS, bS, "S")
    else:
        check_columns(S, wS, bS, "S")
    return inside


SHAPES = [(1, 1, 8, 8), (4, 2, 64, 64), (3, 1, 24, 40), (2, 2, 128, 128), (2, 1, 72, 200), (2, 2, 256, 24)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("heads,keys,dk,dv", SHAPES)
def test_prompts(dtype, delta, heads, keys, dk, dv):
    if dtype == F32 and dk > 128:
        pytest.skip("d_k up to 128 in fp32")
    c = make([0, 1, 63, 64, 65, 200], heads, keys, dk, dv, dtype, seed=dk + dv, first=3, gap=5, pad=8, delta=delta)
    want = expected(c)
    out = torch.full(c["v"].shape, 7.0, dtype=dtype, device="cuda")
    o, S = call(c, out=out)
    assert o is out
    inside = compare(c, o, S, want)
    assert (o[~inside.cuda()] == 7.0).all(), "rows of no sequence are left as they were"
    assert torch.equal(S[0], c["state"][0]), "an empty sequence keeps its state"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("alpha", ["head", None])
@pytest.mark.parametrize("state", [True, False])
def test_decays_and_first_states(dtype, delta, alpha, state):
    c = make([70, 0, 130], 4, 4, 64, 48, dtype, alpha=alpha, delta=delta, state=state)
    o, S = call(c)
    compare(c, o, S, expected(c))
    if not state:
        assert not S[1].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("delta", [True, False])
def test_batch_form_and_a_decay_row_for_all(dtype, delta):
    c = make([150, 150, 150], 4, 2, 64, 64, dtype, alpha="head", delta=delta)
    o, S = call(c)
    batch = lambda t: None if t is None else t.reshape(3, 150, *t.shape[1:])  # noqa: E731
    o3, S3 = rsq.linear_attention(batch(c["q"].contiguous()), batch(c["k"].contiguous()), batch(c["v"].contiguous()),
                                  alpha=c["alpha"].expand(3, 150, 4), beta=batch(c["beta"]), state=c["state"].clone())
    assert torch.equal(o3.reshape(450, 4, 64), o) and torch.equal(S3, S)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("delta", [True, False])
def test_gates_at_their_ends(dtype, delta):
    """Decays of zero clear the state, write strengths of zero write nothing, tiny decays are as good as zero."""
    c = make([180, 100], 2, 2, 64, 32, dtype, seed=3, delta=delta)
    c["alpha"][::37] = 0.0
    c["alpha"][5::41] = 1e-30
    c["alpha"][7::13] = 1.0
    if delta:
        c["beta"][3::5] = 0.0
        c["beta"][4::5] = 1.0
    o, S = call(c)
    compare(c, o, S, expected(c))
    # a cleared state is the same as none
    c["alpha"][0] = c["alpha"][180] = 0.0
    first = call(c)
    again = call({**c, "state": torch.zeros_like(c["state"])})
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_equal_keys():
    """The same key over and over: the hardest system of a chunk, each token takes the last one's value back."""
    c = make([140], 2, 2, 64, 32, F32, seed=4)
    c["k"][:] = c["k"][:1].clone()
    c["beta"][:] = 1.0
    c["alpha"][:] = 1.0
    o, S = call(c)
    compare(c, o, S, expected(c))
    # all writes but the last are gone: reading along the key gives its value
    got = torch.einsum("hk,hkv->hv", f64(c["k"][0]), f64(S[0]))
    kk = (f64(c["k"][0]) ** 2).sum(1, keepdim=True)
    # k.k misses 1 by 64 half steps of fp32 at most, and so much stays of the value before (4 at most here); the sums of
    # 140 tokens' differences, of magnitude 8, are off by some 3 * 64 half steps each at most, and each token takes all
    # but 64 half steps of the errors before it back
    assert (got - kk * f64(c["v"][139])).abs().max() < (64 * 4 + 2 * 3 * 64 * 8) * U


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("delta", [True, False])
def test_error_norm(dtype, delta):
    """States keep all of fp32: a lost third piece of a factor (2^-17 / sqrt(3) of it in the mean square, 4e-6) would
    be seen. A state's element passes about 54 roundings a chunk (12 + 12 + 6 products of 32 terms, 20 of the inverse,
    4 of X and the weights), each U / sqrt(3) in the mean square of terms about its own size, and the decays' own
    relative errors, up to 10 U; twice their joint size is the limit."""
    c = make([320, 64], 4, 4, 128, 64, dtype, seed=9, delta=delta)
    _, S = call(c)
    want = expected(c)[1]
    for s, chunks in ((0, 5), (1, 1)):
        off = float((f64(S[s]) - want[s]).norm() / want[s].norm())
        assert off < 2 * (54 * chunks / 3) ** 0.5 * U + 10 * U, off


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("delta", [True, False])
def test_values_that_are_not_finite(dtype, delta):
    """A v that is not finite makes its own column NaN from its token on, and nothing else differs."""
    c = make([150, 90], 2, 1, 64, 48, dtype, seed=6, delta=delta)
    o0, S0 = call(c)
    bad = {**c, "v": c["v"].clone()}
    bad["v"][70, 1, 5], bad["v"][100, 0, 47], bad["v"][150, 0, 0] = float("nan"), float("inf"), -float("inf")
    o, S = call(bad)
    mask = torch.zeros_like(o0, dtype=torch.bool)
    mask[70:150, 1, 5] = mask[100:150, 0, 47] = mask[150:, 0, 0] = True
    assert torch.isnan(o[mask]).all() and torch.equal(o[~mask], o0[~mask])
    state = torch.zeros_like(S0, dtype=torch.bool)
    state[0, 1, :, 5] = state[0, 0, :, 47] = state[1, 0, :, 0] = True
    assert torch.isnan(S[state]).all() and torch.equal(S[~state], S0[~state])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("what", ["k", "alpha", "beta"])
def test_keys_and_gates_that_are_not_finite(dtype, what):
    """They make their head NaN from their token on; other heads, tokens and sequences keep their bits."""
    c = make([150, 90], 2, 2, 64, 32, dtype, seed=7)
    o0, S0 = call(c)
    t = c[what].clone()
    t[(70, 1, 3) if what == "k" else (70, 1)] = float("nan")
    o, S = call({**c, what: t})
    mask = torch.zeros_like(o0, dtype=torch.bool)
    mask[70:150, 1] = True
    assert torch.isnan(o[mask]).all() and torch.equal(o[~mask], o0[~mask])
    assert torch.isnan(S[0, 1]).all() and torch.equal(S[0, 0], S0[0, 0]) and torch.equal(S[1], S0[1])


@pytest.mark.parametrize("delta", [True, False])
def test_queries_that_are_not_finite(delta):
    c = make([150], 2, 2, 64, 32, BF16, seed=8, delta=delta)
    o0, S0 = call(c)
    q = c["q"].clone()
    q[70, 1, 3] = float("inf")
    o, S = call({**c, "q": q})
    mask = torch.zeros_like(o0, dtype=torch.bool)
    mask[70, 1] = True
    assert not torch.isfinite(o[mask]).any() and torch.equal(o[~mask], o0[~mask]) and torch.equal(S, S0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("delta", [True, False])
def test_parts_and_tokens_go_on_from_a_prompt(dtype, delta):
    c = make([170], 3, 3, 64, 40, dtype, seed=10, delta=delta)
    want = expected(c)
    part = lambda t, a, b: None if t is None else t[a:b].unsqueeze(0).contiguous()  # noqa: E731
    S, got = c["state"].clone(), []
    for a, b in ((0, 64), (64, 101), (101, 160)):
        o, S2 = rsq.linear_attention(*(part(c[n], a, b) for n in "qkv"), alpha=part(c["alpha"], a, b),
                                     beta=part(c["beta"], a, b), state=S)
        assert S2 is S
        got.append(o[0])
    for t in range(160, 170):
        got.append(rsq.linear_attention_step(S, *(c[n][t: t + 1] for n in "qkv"), alpha=c["alpha"][t: t + 1],
                                             beta=None if c["beta"] is None else c["beta"][t: t + 1]))
    # (other cuts into chunks: twice the bounds' own roundings at most)
    wo, wS, bo, bS = want
    check(torch.cat(got), wo, 2 * bo + half(dtype) * wo.abs(), "o")
    if delta:
        check_columns(S, wS, 2 * bS, "S")
    else:
        check(S, wS, 2 * bS, "S")


def half(dtype):
    return H if dtype == BF16 else U


def compare_step(c, o, S):
    """o and S of one token of every sequence: sums of up to 256 terms, the update's three roundings and o's two
    products, in fp32."""
    dtype, dk, per = c["v"].dtype, c["k"].shape[2], c["v"].shape[1] // c["k"].shape[1]
    k, q = f64(c["k"]).repeat_interleave(per, 1), f64(c["q"]).repeat_interleave(per, 1)
    a, S0, u = f64(c["alpha"])[..., None], f64(c["state"]), f64(c["v"])
    aS = a[..., None] * S0
    eu = torch.zeros_like(u)
    if c["beta"] is not None:
        b = f64(c["beta"])[..., None]
        ks, ksm = (k[..., None] * aS).sum(2), (k.abs()[..., None] * aS.abs()).sum(2)
        eu = b * U * ((dk + 4) * ksm + u.abs() + ksm) + 2 * U * (b * (u - ks)).abs()
        u = b * (u - ks)
    want = aS + k[..., None] * u[..., None, :]
    bound = 2 * U * aS.abs() + k.abs()[..., None] * eu[..., None, :] + U * (k[..., None] * u[..., None, :]).abs() + U * want.abs()
    check(S, want, 1.05 * bound + 1e-37, "S")
    qk, qkm = (q * k).sum(2)[..., None], (q * k).abs().sum(2)[..., None]
    qs, qsm = (q[..., None] * aS).sum(2), (q.abs()[..., None] * aS.abs()).sum(2)
    wo = qs + qk * u
    bo = U * ((dk + 4) * qsm + (dk + 4) * qkm * u.abs() + wo.abs()) + qk.abs() * eu + half(dtype) * wo.abs()
    check(o, wo, 1.05 * bo + 1e-37, "o")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("heads,keys,dk,dv", SHAPES + [(1, 1, 200, 1032)])
def test_step(dtype, delta, heads, keys, dk, dv):
    c = make([1] * 5, heads, keys, dk, dv, dtype, seed=dk, pad=8, delta=delta)
    S = c["state"].clone()
    o = rsq.linear_attention_step(S, c["q"], c["k"], c["v"], alpha=c["alpha"], beta=c["beta"])
    compare_step(c, o, S)


@pytest.mark.parametrize("dv", [64, 128, 200])
def test_step_of_many_heads(dv):
    """64 and 128 columns a workgroup."""
    c = make([1] * 130, 8, 2, 128, dv, BF16, seed=dv)
    S = c["state"].clone()
    o = rsq.linear_attention_step(S, c["q"], c["k"], c["v"], alpha=c["alpha"], beta=c["beta"])
    compare_step(c, o, S)


def test_step_of_decay_rows_strides_and_no_decay():
    c = make([1] * 6, 4, 2, 64, 64, BF16, alpha="head")
    S0 = c["state"]
    args = lambda: (S0.clone(), c["q"], c["k"], c["v"])  # noqa: E731
    ones = torch.ones(6, 4, device="cuda")
    a, b = args(), args()
    oa = rsq.linear_attention_step(*a, alpha=c["alpha"], beta=c["beta"])
    wide = torch.zeros(6, 12, device="cuda")
    wide[:, 4:8] = c["alpha"]
    ob = rsq.linear_attention_step(*b, alpha=wide[:, 4:8], beta=c["beta"])
    assert torch.equal(oa, ob) and torch.equal(a[0], b[0])
    a, b = args(), args()
    oa, ob = rsq.linear_attention_step(*a), rsq.linear_attention_step(*b, alpha=ones)
    assert torch.equal(oa, ob) and torch.equal(a[0], b[0])


def test_a_state_past_32_bits():
    """States, and rows of prompts, whose bytes pass 2^32."""
    heads, seqs = 32, 2100                                   # 64 KB a head: 4.4 GB
    S = torch.zeros(seqs, heads, 128, 128, device="cuda")
    c = make([1] * 2, heads, heads, 128, 128, BF16)
    big = {n: c[n][:1].expand(seqs, *c[n].shape[1:]).contiguous() for n in "qkv"}
    gates = {n: c[n][:1].expand(seqs, heads).contiguous() for n in ("alpha", "beta")}
    S[:] = c["state"][0]
    o = rsq.linear_attention_step(S, big["q"], big["k"], big["v"], **gates)
    one = {**{n: c[n][:1] for n in ("q", "k", "v", "alpha", "beta", "state")}}
    compare_step(one, o[-1:], S[-1:])
    assert torch.equal(o[-1], o[0]) and torch.equal(S[-1], S[0])


@pytest.mark.parametrize("delta", [True, False])
def test_rows_past_32_bits(delta):
    n, last = 280000, 130                                    # rows of 16 KB: 4.6 GB
    rows = torch.zeros(n, 8192, dtype=BF16, device="cuda")
    c = make([last], 2, 2, 128, 128, BF16, seed=12, delta=delta)
    view = lambda a, d: rows[:, a: a + 256].view(n, 2, d)  # noqa: E731
    q, k, v = view(0, 128), view(256, 128), view(512, 128)
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        t[n - last:] = c[name]
    gate = lambda t: None if t is None else torch.cat([torch.ones(n - last, 2, device="cuda"), t])  # noqa: E731
    off = torch.tensor([0, 5, n - last, n], dtype=torch.int32, device="cuda")
    off[2] = n - last
    S = torch.cat([torch.zeros(2, 2, 128, 128, device="cuda"), c["state"]])
    o, S = rsq.linear_attention(q, k, v, alpha=gate(c["alpha"]), beta=gate(c["beta"]), state=S, offsets=off, max_len=n)
    o1, S1 = call(c)
    assert not o[: n - last].any() and not S[:2].any()
    # (a sequence cut into segments takes other sums than a whole one)
    want = expected(c)
    check(o[n - last:], want[0], want[2], "o")
    if delta:
        assert torch.equal(o[n - last:], o1) and torch.equal(S[2:], S1)


@pytest.mark.parametrize("delta", [True, False])
@pytest.mark.parametrize("seqs", [63, 64, 65, 300])
def test_many_sequences(delta, seqs):
    """Sequences are looked for 64 at a time, and up to 64 sorted by length; each gets what it gets alone."""
    g = torch.Generator().manual_seed(seqs)
    lengths = torch.randint(0, 90, (seqs,), generator=g).tolist()
    lengths[0], lengths[-1] = 0, 70
    c = make(lengths, 2, 1, 64, 32, BF16, seed=seqs, delta=delta)
    o, S = call(c)
    for s in (1, seqs // 2, seqs - 1):
        a, n = c["seqs"][s]
        if n == 0:
            assert torch.equal(S[s], c["state"][s])
            continue
        one = {**{name: c[name][a: a + n] for name in "qkv"}, "alpha": c["alpha"][a: a + n],
               "beta": None if c["beta"] is None else c["beta"][a: a + n], "state": c["state"][s: s + 1], "seqs": [(0, n)],
               "offsets": torch.tensor([0, n], dtype=torch.int32).cuda(), "max_len": n}
        want = expected(one)
        compare(one, o[a: a + n], S[s: s + 1], want)


@pytest.mark.parametrize("heads,dv", [(2, 128), (40, 128), (300, 64), (70, 24)])
def test_column_shapes(heads, dv):
    """One, two and four column tiles a workgroup give the same bits: sums do not cross columns."""
    c = make([100, 40], heads, 1, 128, dv, BF16, seed=heads)
    o, S = call(c)
    for h in (0, heads - 1):
        one = {**c, "v": c["v"][:, h: h + 1].contiguous(), "alpha": c["alpha"][:, h: h + 1].contiguous(),
               "beta": c["beta"][:, h: h + 1].contiguous(), "state": c["state"][:, h: h + 1].contiguous()}
        compare(one, o[:, h: h + 1], S[:, h: h + 1], expected(one))


def few(c, o, S, want):
    """Sequences of a few tokens, which round the state twice for every token: with decays and write strengths up to
    one and keys of unit length it stays below its first norm and those of the values written."""
    wo, wS, bo, bS = want
    most = (0 if c["state"] is None else f64(c["state"]).norm(dim=2)) + torch.stack(
        [f64(c["v"][a: a + n]).abs().sum(0) for a, n in c["seqs"]])
    n = torch.tensor([n for _, n in c["seqs"]], dtype=torch.float64)[:, None, None]
    extra = 2 * n * U * most
    check_columns(S, wS, bS + extra, "S")
    per = c["v"].shape[1] // c["q"].shape[1]
    norm = f64(c["q"]).norm(dim=2).repeat_interleave(per, 1)[..., None]
    for i, (a, n) in enumerate(c["seqs"]):
        check(o[a: a + n], wo[a: a + n], bo[a: a + n] + norm[a: a + n] * extra[i], "o")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("heads,keys,dk,dv", SHAPES)
def test_few_tokens(dtype, state, heads, keys, dk, dv):
    """Alone, and beside sequences of one and of several chunks: the same bits."""
    if dtype == F32 and dk > 128:
        pytest.skip("d_k up to 128 in fp32")
    c = make([1, 0, 8, 3, 7, 0, 5], heads, keys, dk, dv, dtype, seed=dk, first=2, gap=3, pad=8, state=state)
    out = torch.full(c["v"].shape, 7.0, dtype=dtype, device="cuda")
    o, S = call(c, out=out)
    few(c, o, S, expected(c))
    assert (o[:2] == 7.0).all() and (o[-3:] == 7.0).all(), "rows of no sequence are left as they were"
    for i in (1, 5):
        assert torch.equal(S[i], c["state"][i]) if state else not S[i].any()
    d = make([1, 0, 8, 3, 7, 0, 5, 9, 64, 130], heads, keys, dk, dv, dtype, seed=dk + 1, state=state)
    for name in ("q", "k", "v", "alpha", "beta"):
        d[name] = d[name].clone()
        d[name][:24] = c[name][2:26]
    if state:
        d["state"][:7] = c["state"]
    o2, S2 = call(d)
    assert torch.equal(o2[:24], o[2:26]) and torch.equal(S2[:7], S)
    few(d, o2, S2, expected(d))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_tokens_of_a_batch(dtype):
    """Without offsets: as with them, and as the token step after it goes on."""
    c = make([4] * 5, 6, 3, 64, 72, dtype, seed=30, alpha="head")
    o, S = call(c)
    batch = lambda t: t.reshape(5, 4, *t.shape[1:]).contiguous()  # noqa: E731
    o3, S3 = rsq.linear_attention(*(batch(c[n]) for n in "qkv"), alpha=c["alpha"], beta=batch(c["beta"]), state=c["state"].clone())
    assert torch.equal(o3.reshape(20, 6, 72), o) and torch.equal(S3, S)
    T, got = c["state"].clone(), []
    for t in range(4):
        got.append(rsq.linear_attention_step(T, *(batch(c[n])[:, t].contiguous() for n in "qkv"),
                                             alpha=c["alpha"].expand(5, 6).contiguous(), beta=batch(c["beta"])[:, t].contiguous()))
    few(c, torch.stack(got, 1).reshape(20, 6, 72), T, expected(c))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_tokens_that_are_not_finite(dtype):
    """As in longer sequences: a v takes its column from its token on, a k, alpha or beta the head, a q its row."""
    c = make([8, 6], 4, 2, 64, 40, dtype, seed=31)
    o0, S0 = call(c)
    bad = {**c, **{name: c[name].clone() for name in ("q", "k", "v", "alpha", "beta")}}
    bad["v"][3, 0, 5], bad["v"][8, 1, 39] = float("inf"), float("nan")
    bad["beta"][8, 1] = 0.0
    c["beta"][8, 1] = 0.0
    o0, S0 = call(c)
    bad["k"][5, 1, 7] = float("inf")           # heads 2 and 3
    bad["alpha"][10, 2], bad["beta"][12, 3] = -0.5, float("inf")
    bad["q"][1, 0, 0] = float("nan")           # heads 0 and 1
    o, S = call(bad)
    mask = torch.zeros_like(o0, dtype=torch.bool)
    mask[3:8, 0, 5] = mask[8:, 1, 39] = mask[5:8, 2:] = mask[10:, 2] = mask[12:, 3] = mask[1, :2] = True
    assert torch.isnan(o[mask]).all() and torch.equal(o[~mask], o0[~mask])
    state = torch.zeros_like(S0, dtype=torch.bool)
    state[0, 0, :, 5] = state[1, 1, :, 39] = state[0, 2:] = state[1, 2:] = True
    assert torch.isnan(S[state]).all() and torch.equal(S[~state], S0[~state])


@pytest.mark.parametrize("delta", [True, False])
def test_repeated_calls_give_the_same_bits(delta):
    c = make([700, 3, 250], 4, 2, 128, 128, BF16, seed=20, delta=delta)
    first = call(c)
    for _ in range(5):
        again = call(c)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_offsets_that_run_out_of_the_rows():
    """Offsets are clamped to the rows, a sequence past max_len is cut, one whose end is before its begin is empty."""
    c = make([100, 60], 2, 2, 64, 32, BF16, seed=21)
    c["offsets"] = torch.tensor([-5, 80, 70, 1000], dtype=torch.int32).cuda()
    c["state"] = torch.randn(3, 2, 64, 32, generator=torch.Generator().manual_seed(1)).cuda()
    for delta in (True, False):
        d = {**c, "beta": c["beta"] if delta else None}
        o, S = call({**d, "max_len": 75})
        assert torch.equal(S[1], d["state"][1])
        one = {**d, "seqs": [(0, 75)], "state": d["state"][:1]}
        want = expected(one)
        # rows 70 to 74 belong to the last sequence too
        check(o[:70], want[0][:70], want[2][:70], "o")


@pytest.mark.parametrize("delta", [True, False])
def test_captured_and_replayed(delta):
    c = make([200, 90], 4, 2, 64, 64, BF16, seed=22, delta=delta)
    S = c["state"].clone()
    out = torch.empty_like(c["v"])
    run = lambda: rsq.linear_attention(c["q"], c["k"], c["v"], alpha=c["alpha"], beta=c["beta"], state=S,  # noqa: E731
                                       offsets=c["offsets"], max_len=c["max_len"], out=out)
    step = lambda: rsq.linear_attention_step(S, c["q"][:2], c["k"][:2], c["v"][:2], alpha=c["alpha"][:2],  # noqa: E731
                                             beta=None if c["beta"] is None else c["beta"][:2])
    run(), step()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    made = []
    for g in graphs:
        with torch.cuda.graph(g):
            run()
            made.append(step())
    for i in range(3):
        S.copy_(c["state"])
        run()
        want_o, want_y, want_S = out.clone(), step(), S.clone()
        torch.cuda.synchronize()
        for g, y in zip(graphs, made):
            S.copy_(c["state"])
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want_o) and torch.equal(y, want_y) and torch.equal(S, want_S), i


def test_on_another_stream():
    c = make([300], 4, 4, 128, 128, BF16, seed=23)
    want = call(c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, S = call(c, stream=side)
    y = rsq.linear_attention_step(S, c["q"][:1], c["k"][:1], c["v"][:1], alpha=c["alpha"][:1], beta=c["beta"][:1], stream=side)
    side.synchronize()
    S1 = want[1].clone()
    y1 = rsq.linear_attention_step(S1, c["q"][:1], c["k"][:1], c["v"][:1], alpha=c["alpha"][:1], beta=c["beta"][:1])
    assert torch.equal(o, want[0]) and torch.equal(S, S1) and torch.equal(y, y1)


def test_two_streams_at_once():
    """Calls on two streams have workspaces of their own."""
    cases = [make([900], 8, 8, 128, 128, BF16, seed=s) for s in (1, 2)]
    want = [call(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cases, streams)):
            got[i] = call(c, stream=s)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_no_rows():
    c = make([0, 0], 2, 2, 64, 32, BF16)
    o, S = call({**c, "state": None})
    assert o.shape == (0, 2, 32) and not S.any()
    o, S = call(c)
    assert torch.equal(S, c["state"])


def test_prompt_into_a_quantized_state():
    """A prompt's state goes into the decode step's: dequantized it is within half a step of the scan's, and the next
    token's o is what the dense step gives, up to the state's quantization."""
    B, Hd, dk, dv, T = 3, 4, 128, 128, 150
    c = make([T] * B, Hd, Hd, dk, dv, BF16, seed=30, state=False)
    _, S = call(c)
    for model, beta in (("gdn", c["beta"]), ("mamba2", None)):
        S = call({**c, "beta": beta})[1]
        st = rsq.State(model=model, batch=B, heads=Hd, d_k=dk, d_v=dv, group=32, bits=8, in_dtype="bf16")
        st.load_dense(S)
        nxt = make([1] * B, Hd, Hd, dk, dv, BF16, seed=31)
        kw = dict(alpha=nxt["alpha"], beta=nxt["beta"] if beta is not None else None)
        o8 = st.decode_step(nxt["q"].contiguous(), nxt["k"].contiguous(), nxt["v"].contiguous(), **kw)
        o = rsq.linear_attention_step(S.clone(), nxt["q"], nxt["k"], nxt["v"], **kw)
        # half an 8-bit step of a group's largest, 1 / 254, for each of the state's elements: by the norms
        off = (f64(o8) - f64(o)).norm() / f64(S).abs().amax()
        limit = (f64(nxt["q"]).norm() + f64(nxt["k"]).norm()) * dv ** 0.5 / 254 + H * f64(o).norm() / f64(S).abs().amax()
        assert off <= limit, (model, off, limit)


def test_a_layer_of_prompts_and_tokens():
    """A Gated DeltaNet layer from its operators: 8-bit norm, 8-bit projection, convolution, keys of unit length,
    attention with the delta rule, gated norm into 8 bits, projection, the sum into the residual; then the next token
    on the state. Against the same layer in fp64 on the same weights, at what 8-bit activations (1 / 254 of a row's
    largest) and bf16 values between the operators leave: tested for running together, each operator's own bounds hold
    it elsewhere."""
    D, Hk, Hv, d, T, B = 256, 2, 4, 64, 96, 2
    g = torch.Generator().manual_seed(40)
    randn = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    qkv_cols = 2 * Hk * d + Hv * d

    def weight(n, k):
        w = randn(n, k) / k ** 0.5
        s = w.abs().amax(1) / 127
        codes = torch.round(w / s[:, None]).to(torch.int8)
        return rsq.W8Weight(codes, s), f64(codes) * f64(s)[:, None]

    (w_qkv, m_qkv), (w_gate, m_gate), (w_ab, m_ab), (w_out, m_out) = (weight(n, D if n != D else Hv * d)
                                                                      for n in (qkv_cols, Hv * d, 2 * Hv, D))
    w_norm, w_head = 1 + 0.1 * randn(D), 1 + 0.1 * randn(d)
    w_conv, b_conv = 0.5 * randn(qkv_cols, 4), 0.1 * randn(qkv_cols)
    unit = torch.full((d,), d ** -0.5, device="cuda")

    def layer(x, conv_state, state, step):
        res = x.clone()
        h, hs = rsq.rms_norm(x, w_norm, out_dtype="int8")
        lin = lambda w, **kw: rsq.w8_linear(h, w, hs, **kw)  # noqa: E731
        qkv = lin(w_qkv)
        qkv = rsq.causal_conv_step(qkv, w_conv, b_conv, state=conv_state, activation="silu") if step else \
            rsq.causal_conv(qkv, w_conv, b_conv, state=conv_state, activation="silu")
        ab = lin(w_ab, out_dtype="f32")
        alpha, beta = torch.sigmoid(ab[..., :Hv] + 3.0).contiguous(), torch.sigmoid(ab[..., Hv:]).contiguous()
        qk = rsq.block_norm(qkv[..., : 2 * Hk * d], unit, group=d, eps=1e-6)
        qk = qk.view(*qk.shape[:-1], 2, Hk, d)
        q, k = qk[..., 0, :, :], qk[..., 1, :, :]
        v = qkv[..., 2 * Hk * d:].unflatten(-1, (Hv, d))
        if step:
            o = rsq.linear_attention_step(state, q, k, v, alpha=alpha, beta=beta)
        else:
            o, state = rsq.linear_attention(q, k, v, alpha=alpha, beta=beta)
        y, ys = rsq.block_norm(o.flatten(-2), w_head, gate=lin(w_gate), group=d, out_dtype="int8")
        return rsq.block_norm(rsq.w8_linear(y, w_out, ys), residual=res), state

    def exact(x):
        x = f64(x)
        rms = lambda t, eps: t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)  # noqa: E731
        h = rms(x, 1e-5) * f64(w_norm)
        qkv = h @ m_qkv.t()
        pad = torch.cat([torch.zeros(B, 3, qkv_cols, dtype=torch.float64), qkv], 1)
        z = sum(f64(w_conv)[:, j] * pad[:, j: j + x.shape[1]] for j in range(4)) + f64(b_conv)
        qkv = z * torch.sigmoid(z)
        ab = h @ m_ab.t()
        a, b = torch.sigmoid(ab[..., :Hv] + 3.0), torch.sigmoid(ab[..., Hv:])
        qk = rms(qkv[..., : 2 * Hk * d].reshape(B, -1, 2, Hk, d), 1e-6) * d ** -0.5
        q, k = (qk[:, :, i].repeat_interleave(Hv // Hk, 2) for i in (0, 1))
        v = qkv[..., 2 * Hk * d:].reshape(B, -1, Hv, d)
        S, o = torch.zeros(B, Hv, d, d, dtype=torch.float64), []
        for t in range(x.shape[1]):
            S = a[:, t, :, None, None] * S
            u = b[:, t, :, None] * (v[:, t] - torch.matmul(k[:, t, :, None, :], S)[..., 0, :])
            S = S + k[:, t, :, :, None] * u[..., None, :]
            o.append(torch.matmul(q[:, t, :, None, :], S)[..., 0, :])
        gate = h @ m_gate.t()
        y = (rms(torch.stack(o, 1), 1e-5) * f64(w_head)).flatten(-2) * gate * torch.sigmoid(gate)
        return x + y @ m_out.t()

    x = randn(B, T + 2, D).to(BF16)
    conv_state = torch.zeros(B, qkv_cols, 3, dtype=BF16, device="cuda")
    y, state = layer(x[:, :T].contiguous(), conv_state, None, False)
    ys = [y]
    for t in (T, T + 1):
        yt, state = layer(x[:, t].contiguous(), conv_state, state, True)
        ys.append(yt[:, None])
    got, want = f64(torch.cat(ys, 1)) - f64(x), exact(x) - f64(x)
    # 8-bit codes leave at most 1 / 254 of a row's largest, about 4 of its mean square's root: 1.6% at the most of
    # each of two products, and the norms between them double that at most; bf16 roundings are small beside it
    assert (got - want).norm() <= 2 * 2 * 4 / 254 * want.norm()
