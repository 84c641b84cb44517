"""Norms around a block and products of 8-bit integers at the sizes and arguments where a kernel of their own, or threads
without columns, take part."""
import pytest
import torch

import linear_reference as ref
from layer_reference import U, check, f64
from test_gpu_block import BF16, F32, compare, half, norm_case, run_norm

pytestmark = pytest.mark.gpu

rsq = None


@pytest.fixture(scope="module", autouse=True)
def _package():
    global rsq
    import test_gpu_block
    rsq = test_gpu_block.rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
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
                                                  (520, 9216, 1152, "before"), (515, 16384, 4096, None), (514, 12288, 128, "after")])
def test_norm_of_many_long_rows(dtype, rows, cols, group, gate):
    """More than 512 rows of 8193 to 16384 columns: 32 columns a thread, gate and residual read where they are used."""
    compare(norm_case(rows, cols, dtype, group=group, gate=gate, seed=rows), out_dtype="f32")


def test_norm_of_many_long_rows_to_codes():
    c = norm_case(515, 8200, BF16, group=1640, seed=2)
    (codes, scales), res = run_norm(c, out_dtype="int8")
    want, h, by, bh = definition(c, 1e-5)
    check(res, h, bh + half(BF16) * h.abs(), "residual")
    largest, s = want.abs().amax(1, keepdim=True), f64(scales)
    check(scales, largest / 127, by.amax(1, keepdim=True) / 127 + 2 * U * largest / 127, "scales")
    check(f64(codes) * s, want, 0.5 * s * (1 + 8 * U) + by * (1 + 2.0 ** -3) + 4 * U * want.abs(), "codes")
