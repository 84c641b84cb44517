"""Layer operators where the bounds of their plain comparison leave room: results held to what their arithmetic leaves."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from layer_reference import H, U, check
from test_gpu_layer import BF16, F32, gen, offsets_of, ssm_case, w4_case

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
