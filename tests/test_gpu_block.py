"""Norms around a block and products of 8-bit integers against their fp64 definitions."""
import pytest
import torch

import linear_reference as ref
from layer_reference import H, U, check, f64

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


def half(dtype):
    return H if dtype == BF16 else U


# ---------------------------------------------------------------- norms

def norm_case(rows, cols, dtype, group=0, gate="after", residual=True, nxt=True, weight=True, shared=True, wide=0, seed=0):
    r = gen(seed)
    rowed = lambda: r(rows, cols + wide, dtype=dtype)[:, :cols]  # noqa: E731
    return dict(x=rowed(), weight=1 + 0.3 * r(group if shared and group else cols) if weight else None,
                gate=rowed() if gate else None, gate_first=gate == "before", group=group if weight else 0,
                residual=rowed() if residual else None, residual_scale=0.375 if residual else 1.0,
                next_weight=1 + 0.3 * r(cols) if nxt else None)


def run_norm(c, activation="silu", eps=1e-5, out_dtype="f32", **kw):
    c = dict(c)
    res = c.pop("residual")
    res = None if res is None else res.clone()
    y = rsq.block_norm(c.pop("x"), c.pop("weight"), residual=res, activation=activation, eps=eps, out_dtype=out_dtype, **c, **kw)
    return y, res


def compare(c, activation="silu", eps=1e-5, out_dtype="f32"):
    y, res = run_norm(c, activation, eps, out_dtype)
    want, h, by, bh = ref.block_norm(c["x"], c["weight"], c["gate"], c["gate_first"], activation, c["group"], eps, c["residual"],
                                     c["residual_scale"], c["next_weight"])
    dt = {"f32": F32, "bf16": BF16}[out_dtype]
    assert y.dtype == dt
    check(y, want, by + half(dt) * want.abs(), "y")
    if res is not None:
        check(res, h, bh + half(res.dtype) * h.abs(), "residual")


@pytest.mark.parametrize("dtype,out", [(BF16, "bf16"), (F32, "f32"), (BF16, "f32"), (F32, "bf16")])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 37), (5, 512), (2, 1000), (4, 1024), (3, 2048), (2, 2056), (2, 4096), (2, 8192),
                                       (2, 16384), (2, 20000), (1, 32768), (700, 64)])
def test_norm_sizes(dtype, out, rows, cols):
    compare(norm_case(rows, cols, dtype, seed=cols), out_dtype=out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gate", [None, "before", "after"])
@pytest.mark.parametrize("residual,nxt,weight", [(True, True, True), (True, False, True), (False, True, True), (False, False, True),
                                                 (True, True, False), (False, True, False), (True, False, False)])
def test_norm_parts(dtype, gate, residual, nxt, weight):
    for cols in (96, 3080):
        compare(norm_case(4, cols, dtype, gate=gate, residual=residual, nxt=nxt, weight=weight, seed=cols))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("group,parts", [(8, 5), (16, 3), (24, 7), (64, 1), (64, 32), (96, 20), (128, 32), (256, 3), (512, 5), (704, 4),
                                         (1000, 2), (1024, 9), (4096, 2), (16384, 2), (8, 4096)])
def test_norm_groups(dtype, shared, group, parts):
    compare(norm_case(3, group * parts, dtype, group=group, shared=shared, seed=group))


@pytest.mark.parametrize("activation", ["silu", "sigmoid", None])
def test_norm_activations(activation):
    c = norm_case(4, 200, F32)
    c["gate"][0] *= 30.0
    c["gate"][1, :4] = torch.tensor([-200.0, 200.0, -88.0, 0.0])
    compare(c, activation=activation)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("wide,cols", [(8, 256), (3, 256), (1, 96), (4, 100)])
def test_norm_strides_and_alignment(dtype, wide, cols):
    compare(norm_case(6, cols, dtype, wide=wide))


def test_norm_results():
    """What comes back: y, codes with scales, or the residual itself."""
    c = norm_case(5, 256, BF16)
    y, res = run_norm(c, out_dtype=None)
    assert y.dtype == BF16 and y is not res
    c["next_weight"] = None
    y, res = run_norm(c, out_dtype=None)
    assert y is res
    y2, res2 = run_norm(c, out_dtype="f32")
    assert y2.dtype == F32 and torch.equal(res2, res) and torch.equal(y2.to(BF16), res)
    c["x"], c["gate"], c["residual"] = (c[n].view(1, 5, 256) for n in ("x", "gate", "residual"))
    assert torch.equal(run_norm(c, out_dtype=None)[0], res.view(1, 5, 256))
    out = torch.empty(1, 5, 256, dtype=BF16, device="cuda")
    y, _ = run_norm(c, out_dtype=None, out=out)
    assert y is out and torch.equal(out.view(5, 256), res)


@pytest.mark.parametrize("out,qmax", [("int8", 127.0), ("e4m3", 448.0)])
@pytest.mark.parametrize("cols,scale_group", [(256, 0), (256, 32), (4096, 128), (37, 0), (20480, 64)])
def test_norm_codes(out, qmax, cols, scale_group):
    c = norm_case(4, cols, BF16, seed=cols)
    c["x"][2] = 0
    c["residual"][2] = 0
    (codes, scales), _ = run_norm(c, out_dtype=out, scale_group=scale_group)
    want, _, by, _ = ref.block_norm(c["x"], c["weight"], c["gate"], False, "silu", 0, 1e-5, c["residual"], c["residual_scale"], c["next_weight"])
    g = scale_group or cols
    assert scales.shape == (4, cols // g)
    s = f64(scales).repeat_interleave(g, 1)
    largest = want.abs().view(4, -1, g).amax(2)
    # absmax over qmax: y's own bound there, a quotient
    check(scales, largest / qmax, by.view(4, -1, g).amax(2) / qmax + 2 * U * largest / qmax, "scales")
    # half a step of the code at most (e4m3: 2^-4 of the value, 2^-10 below the smallest normal), y's bound, a quotient
    step = 0.5 * s if out == "int8" else torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10)
    check(f64(codes) * s, want, step * (1 + 8 * U) + by * (1 + 2.0 ** -3) + 4 * U * want.abs() + (2.0 ** -4 * by if out == "e4m3" else 0), "codes")
    assert not f64(codes)[2].any() and not scales[2].any()


def test_norm_not_finite_stays_in_its_row():
    c = norm_case(4, 512, F32, group=64)
    y0, r0 = run_norm(c)
    c["x"][1, 70], c["gate"][2, 3], c["residual"][3, 400] = float("nan"), float("nan"), float("inf")
    y, r = run_norm(c)
    assert torch.equal(y[0], y0[0]) and torch.equal(r[0], r0[0])
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all() and torch.isnan(y[3, 400])
    # before the second norm only the group, and the column, are met
    assert torch.isnan(r[1, 64:128]).all() and torch.equal(r[1, :64], r0[1, :64]) and torch.equal(r[1, 128:], r0[1, 128:])
    assert torch.isnan(r[2, 3]) and torch.equal(r[2, 4:], r0[2, 4:])
    (codes, scales), _ = run_norm(c, out_dtype="int8")
    assert torch.isnan(scales[1]).all() and not codes[1].any()


def test_norm_captured_and_replayed():
    c = norm_case(40, 2048, BF16)
    res = c["residual"].clone()
    args = {k: v for k, v in c.items() if k not in ("x", "residual")}
    run = lambda: rsq.block_norm(c["x"], residual=res, out_dtype="int8", **args)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        codes, scales = run()
    for _ in range(3):
        res.copy_(c["residual"])
        a, b = run()
        want = [t.clone() for t in (a, b, res)]
        res.copy_(c["residual"])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((codes, scales, res), want))


def test_norm_of_rows_past_32_bits():
    n = 66000                                                     # rows of 64 KB: 4.3 GB
    x = torch.ones(n, 32768, dtype=BF16, device="cuda")
    r = gen(3)
    x[-1] = r(32768, dtype=BF16)
    w = 1 + 0.2 * r(32768)
    codes, scales = rsq.block_norm(x, w, group=0, out_dtype="int8")
    one = rsq.block_norm(x[-1:].contiguous(), w, out_dtype="int8")
    assert torch.equal(codes[-1], one[0][0]) and torch.equal(scales[-1], one[1][0])


# ---------------------------------------------------------------- 8-bit products

def w8_case(m, n, k, bias=True, lead=None, seed=0, stride=None, shift=0):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-128, 128, (n, k), generator=g).to(torch.int8).cuda()
    stride = stride or k
    buf = torch.randint(-128, 128, (m * stride + shift + 16,), generator=g).to(torch.int8).cuda()
    x = buf[shift: shift + m * stride].view(m, stride)[:, :k]
    scales, xs = (0.01 + torch.rand(n, generator=g)).cuda(), (0.01 + torch.rand(m, generator=g)).cuda()
    return x, codes, scales, xs, torch.randn(n, generator=g).cuda() * 100 if bias else None


def compare_w8(x, codes, scales, xs, bias, out_dtype):
    y = rsq.w8_linear(x, rsq.W8Weight(codes, scales), xs, bias=bias, out_dtype=out_dtype)
    want, bound = ref.w8(x, codes, scales, xs, bias)
    dt = {"f32": F32, "bf16": BF16}[out_dtype]
    assert y.dtype == dt
    check(y, want, bound + half(dt) * want.abs(), "y")
    return y


# each shape of the kernels: few rows (16 and 32 at a time), blocks of 64 x 64, 64 x 128 and 256 x 256
SIZES = [(1, 1, 1), (1, 16, 64), (3, 17, 63), (16, 128, 65), (5, 33, 4096), (16, 12352, 100), (33, 1031, 705), (48, 1040, 128), (100, 130, 1000),
         (64, 4096, 192), (130, 2000, 257), (200, 16500, 130), (257, 513, 320), (2560, 4096, 64), (2570, 4100, 144), (4100, 2500, 72)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("out_dtype,bias", [("bf16", False), ("f32", True)])
def test_w8(m, n, k, out_dtype, bias):
    compare_w8(*w8_case(m, n, k, bias, seed=m + n), out_dtype)


@pytest.mark.parametrize("m,n,k", [(7, 100, 96), (300, 600, 96), (2600, 4096, 96)])
@pytest.mark.parametrize("stride,shift", [(112, 0), (97, 0), (96, 1), (112, 8), (128, 16)])
def test_w8_strides_and_alignment(m, n, k, stride, shift):
    compare_w8(*w8_case(m, n, k, stride=stride, shift=shift), "f32")


@pytest.mark.parametrize("m,n,k", [(1500, 4100, 1104), (1500, 4100, 1101), (3300, 4090, 6208), (3300, 4090, 6201)])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_w8_of_large_blocks(m, n, k, out_dtype):
    """Blocks of 128 x 256, and of 256 x 256 with long rows; the sums are whole numbers, exact in fp64 on the GPU."""
    x, codes, scales, xs, bias = w8_case(m, n, k, seed=k)
    y = rsq.w8_linear(x, rsq.W8Weight(codes, scales), xs, bias=bias, out_dtype=out_dtype)
    want = (x.double() @ codes.double().t().contiguous()) * xs.double()[:, None] * scales.double()
    bound = 3.05 * U * want.abs()
    want = want + bias.double()
    bound += 1.05 * U * want.abs() + 1e-37 + half(BF16 if out_dtype == "bf16" else F32) * want.abs()
    assert bool(((y.double() - want).abs() <= bound).all())


def test_w8_largest_sums():
    """The longest row of -128 by -128 that int32 holds."""
    k = (1 << 17) - 1
    for m in (1, 70):
        x = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
        codes = torch.full((65 if m == 1 else 1000, k), -128, dtype=torch.int8, device="cuda")
        one = torch.ones(codes.shape[0], device="cuda")
        y = rsq.w8_linear(x, rsq.W8Weight(codes, one), torch.ones(m, device="cuda"), out_dtype="f32")
        assert (y.double() == torch.tensor(float(k * 16384), dtype=F32).double().item()).all()


def test_w8_shapes_scales_and_outputs():
    x, codes, scales, xs, bias = w8_case(12, 40, 64)
    w = rsq.W8Weight(codes, scales)
    y = rsq.w8_linear(x, w, xs, bias=bias)
    assert y.dtype == BF16
    y3 = rsq.w8_linear(x.view(3, 4, 64), w, xs.view(3, 4, 1), bias=bias)
    assert y3.shape == (3, 4, 40) and torch.equal(y3.view(12, 40), y)
    wide = torch.full((12, 56), 7.0, dtype=BF16, device="cuda")
    got = rsq.w8_linear(x, w, xs[:, None], bias=bias, out=wide[:, 3:43])
    assert torch.equal(got, y) and (wide[:, :3] == 7.0).all() and (wide[:, 43:] == 7.0).all()
    assert rsq.w8_linear(x[:0], w, xs[:0]).shape == (0, 40)


@pytest.mark.parametrize("m,n,k", [(300, 777, 130), (3000, 4100, 64)])
def test_w8_writes_its_rows_and_columns_only(m, n, k):
    x, codes, scales, xs, bias = w8_case(m, n, k)
    for dt in (BF16, F32):
        out = torch.full((m + 2, n + 9), 7.0, dtype=dt, device="cuda")
        y = rsq.w8_linear(x, rsq.W8Weight(codes, scales), xs, bias=bias, out=out[1: m + 1, 4: n + 4],
                          out_dtype="bf16" if dt == BF16 else "f32")
        want, bound = ref.w8(x, codes, scales, xs, bias)
        check(y, want, bound + half(dt) * want.abs(), "y")
        assert (out[0] == 7.0).all() and (out[-1] == 7.0).all() and (out[:, :4] == 7.0).all() and (out[:, n + 4:] == 7.0).all()


def test_w8_of_normed_rows():
    """As a layer calls them: a norm's codes and scales go straight in."""
    r = gen(4)
    x, w = r(50, 256, dtype=BF16), 1 + 0.1 * r(256)
    codes, scales = rsq.block_norm(x, w, out_dtype="int8")
    _, wc, ws, _, _ = w8_case(1, 96, 256)
    y = rsq.w8_linear(codes, rsq.W8Weight(wc, ws), scales, out_dtype="f32")
    want, bound = ref.w8(codes, wc, ws, scales, None)
    check(y, want, bound + U * want.abs(), "y")


def test_w8_rows_past_32_bits():
    """y past 2^32 bytes, and rows of x far apart."""
    m, n, k = 70000, 16500, 64
    x, codes, scales, xs, _ = w8_case(m, n, k, seed=5)
    w = rsq.W8Weight(codes, scales)
    y = rsq.w8_linear(x, w, xs, out_dtype="f32")
    for a in (0, m - 300):
        want, bound = ref.w8(x[a: a + 300], codes, scales, xs[a: a + 300], None)
        check(y[a: a + 300], want, bound + U * want.abs(), "y")
    far = torch.zeros(600, 1 << 23, dtype=torch.int8, device="cuda")
    far[:, :64] = x[:600]
    assert torch.equal(rsq.w8_linear(far[:, :64], w, xs[:600], out_dtype="f32"), y[:600])


def test_w8_captured_and_replayed():
    """With the workspace for rows that are laid out again: two graphs, replayed in turn."""
    cases = [w8_case(300, 1200, 65, seed=s) for s in (1, 2)]
    ws = [rsq.W8Weight(c[1], c[2]) for c in cases]
    run = lambda i: rsq.w8_linear(cases[i][0], ws[i], cases[i][3], bias=cases[i][4])  # noqa: E731
    want = [run(i).clone() for i in (0, 1)]
    torch.cuda.synchronize()
    graphs, made = [torch.cuda.CUDAGraph() for _ in (0, 1)], [None, None]
    for i in (0, 1):
        with torch.cuda.graph(graphs[i]):
            made[i] = run(i)
    for _ in range(3):
        for m in made:
            m.zero_()
        for g in graphs:
            g.replay()
        eager = [run(i) for i in (0, 1)]
        torch.cuda.synchronize()
        assert all(torch.equal(made[i], want[i]) and torch.equal(eager[i], want[i]) for i in (0, 1))


def test_w8_on_another_stream():
    x, codes, scales, xs, bias = w8_case(500, 1000, 300)
    want = rsq.w8_linear(x, rsq.W8Weight(codes, scales), xs, bias=bias)
    xb = x.to(BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())   # for all that the operands' own stream does to them
    w = rsq.W8Weight(codes, scales, stream=side)
    y = rsq.w8_linear(x, w, xs, bias=bias, stream=side)
    z = rsq.block_norm(xb, stream=side, out_dtype="f32")
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(z, x.float())
