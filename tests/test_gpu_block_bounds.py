"""Norms around a block and products of 8-bit integers at the sizes and arguments where a kernel of their own, or threads
without columns, take part."""
import ctypes

import pytest
import torch

import linear_reference as ref
from layer_reference import U, check, f64
from test_gpu_block import BF16, F32, compare, compare_w8, half, norm_case, run_norm, w8_case

pytestmark = pytest.mark.gpu

rsq = _abi = None


@pytest.fixture(scope="module", autouse=True)
def _package():
    global rsq, _abi
    import test_gpu_block
    rsq = test_gpu_block.rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
    from bit_recurrent_state_rsq_amd import _abi
    assert torch.cuda.is_available()


def definition(c, eps):
    return ref.block_norm(c["x"], c["weight"], c["gate"], c["gate_first"], "silu", c["group"], eps, c["residual"], c["residual_scale"],
                          c["next_weight"])


# ---------------------------------------------------------------- norms

# columns that leave threads of a row without any: of a wavefront, of 256, 512 and 1024 threads; groups of a power of two
# of threads and of others
@pytest.mark.parametrize("cols,group", [(384, 128), (168, 24), (2000, 1000), (896, 128), (1152, 128), (4608, 512), (9216, 1024), (17408, 1024),
                                        (384, 0), (1500, 0)])
@pytest.mark.parametrize("out", ["f32", "int8", "e4m3"])
def test_norm_without_eps(cols, group, out):
    """eps = 0: a sum of no columns is zero, and its root's reciprocal an infinity that nothing may take in."""
    for residual, nxt in ((True, True), (False, True), (False, False)):
        c = norm_case(5, cols, BF16, group=group, residual=residual, nxt=nxt, seed=cols)
        y, res = run_norm(c, eps=0.0, out_dtype=out)
        want, h, by, bh = definition(c, 0.0)
        if res is not None:
            check(res, h, bh + half(BF16) * h.abs(), "residual")
        if out == "f32":
            check(y, want, by + U * want.abs(), "y")
            continue
        codes, scales = y
        qmax = 127.0 if out == "int8" else 448.0
        largest = want.abs().amax(1, keepdim=True)
        check(scales, largest / qmax, by.amax(1, keepdim=True) / qmax + 2 * U * largest / qmax, "scales")
        # half a step of the code, y's bound (a code of e4m3 moves with it by a sixteenth more), a quotient
        s = f64(scales)
        step = 0.5 * s if out == "int8" else torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10)
        check(f64(codes) * s, want, step * (1 + 8 * U) + by * (1 + 2.0 ** -3) + 4 * U * want.abs(), "codes")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols,group,gate", [(600, 16384, 0, "after"), (513, 8200, 0, "before"), (513, 8200, 1640, "after"),
                                                  (520, 9216, 1152, "before"), (515, 16384, 4096, None), (514, 12288, 128, "after"),
                                                  (257, 16384, 512, "after"), (256, 16384, 512, "after"), (300, 9000, 1800, "before")])
def test_norm_of_many_long_rows(dtype, rows, cols, group, gate):
    """More rows than compute units, of 8193 to 16384 columns: 32 columns a thread, gate and residual read where they are
    used; and as many."""
    compare(norm_case(rows, cols, dtype, group=group, gate=gate, seed=rows), out_dtype="f32")


def test_norm_of_many_long_rows_to_codes():
    c = norm_case(515, 8200, BF16, group=1640, seed=2)
    (codes, scales), res = run_norm(c, out_dtype="int8")
    want, h, by, bh = definition(c, 1e-5)
    check(res, h, bh + half(BF16) * h.abs(), "residual")
    largest, s = want.abs().amax(1, keepdim=True), f64(scales)
    check(scales, largest / 127, by.amax(1, keepdim=True) / 127 + 2 * U * largest / 127, "scales")
    check(f64(codes) * s, want, 0.5 * s * (1 + 8 * U) + by * (1 + 2.0 ** -3) + 4 * U * want.abs(), "codes")


# ---------------------------------------------------------------- 8-bit products

# rows x n x k that take 32 rows and four tiles a workgroup, and blocks of 64 x 64
FEW = [(333, 1031, 705), (256, 2048, 2100), (270, 1500, 96), (100, 3700, 1000), (257, 2001, 2049)]
BLOCKS = [(130, 4100, 200), (128, 12352, 100), (100, 4500, 333), (40, 12352, 1000), (520, 4096, 96), (1000, 1024, 256), (300, 2400, 65)]


@pytest.mark.parametrize("m,n,k", FEW + BLOCKS)
@pytest.mark.parametrize("out_dtype,bias", [("bf16", True), ("f32", False)])
def test_w8_of_a_few_hundred_rows(m, n, k, out_dtype, bias):
    compare_w8(*w8_case(m, n, k, bias, seed=m + n), out_dtype)


@pytest.mark.parametrize("m,n,k", [(270, 1500, 96), (300, 2400, 96)])
@pytest.mark.parametrize("stride,shift", [(112, 0), (97, 0), (96, 1), (112, 8), (128, 16)])
def test_w8_of_a_few_hundred_rows_strides_and_alignment(m, n, k, stride, shift):
    x, codes, scales, xs, bias = w8_case(m, n, k, stride=stride, shift=shift)
    out = torch.full((m + 2, n + 9), 7.0, device="cuda")
    y = rsq.w8_linear(x, rsq.W8Weight(codes, scales), xs, bias=bias, out=out[1: m + 1, 4: n + 4], out_dtype="f32")
    want, bound = ref.w8(x, codes, scales, xs, bias)
    check(y, want, bound + U * want.abs(), "y")
    assert (out[0] == 7.0).all() and (out[-1] == 7.0).all() and (out[:, :4] == 7.0).all() and (out[:, n + 4:] == 7.0).all()


@pytest.mark.parametrize("m,n,k", [(300, 2400, 65), (1500, 4100, 1101), (2600, 4096, 90)])
def test_w8_with_a_workspace_captured_and_replayed(m, n, k):
    """Rows that do not begin at multiples of 16 bytes and are laid out again, in blocks of 64 x 64, 128 x 256 and 64 x 128: two
    graphs, replayed in turn with eager calls between them, each against the definition."""
    cases = [w8_case(m, n, k, seed=s) for s in (1, 2)]
    need = ctypes.c_size_t()
    p = _abi.W8(out_dtype=_abi.BF16, m=m, n=n, k=k, x=cases[0][0].data_ptr(), x_stride=k, y_stride=n)
    assert _abi.lib.rsq_w8_workspace(ctypes.byref(p), ctypes.byref(need)) == 0 and need.value > 0
    ws = [rsq.W8Weight(c[1], c[2]) for c in cases]
    run = lambda i: rsq.w8_linear(cases[i][0], ws[i], cases[i][3], bias=cases[i][4])  # noqa: E731
    want = [run(i).clone() for i in (0, 1)]
    for c, y in zip(cases, want):
        # (whole numbers, of which fp64 holds every sum)
        exact = (c[0].double() @ c[1].double().t().contiguous()) * c[3].double()[:, None] * c[2].double()
        bound = 3.05 * U * exact.abs()
        exact = exact + c[4].double()
        assert bool(((y.double() - exact).abs() <= bound + (1.05 * U + half(BF16)) * exact.abs() + 1e-37).all())
    graphs, made = [torch.cuda.CUDAGraph() for _ in (0, 1)], [None, None]
    for i in (0, 1):
        with torch.cuda.graph(graphs[i]):
            made[i] = run(i)
    for _ in range(3):
        for y in made:
            y.zero_()
        for g in graphs:
            g.replay()
        eager = [run(i) for i in (0, 1)]
        torch.cuda.synchronize()
        assert all(torch.equal(made[i], want[i]) and torch.equal(eager[i], want[i]) for i in (0, 1))
