"""Sizes of the layer operators at the edge of what one launch may have (2^32 threads along x). No GPU is used:
every call here is a query, or is refused before the library touches a device."""
import ctypes

import pytest

rsq = pytest.importorskip("bit_recurrent_state_rsq_amd")
from bit_recurrent_state_rsq_amd import _abi  # noqa: E402
from bit_recurrent_state_rsq_amd._abi import lib  # noqa: E402
from test_layer_refusals import CONV, INVALID, SSM, UNSUPPORTED, addr, fill  # noqa: E402


def ssm(seqs, heads, max_len=1, d_v=8, **kw):
    """Equal sequences of 8 x d_v states in memory wide enough for all of them."""
    far = 1 << 40
    return fill(_abi.Ssm, {**SSM, "seqs": seqs, "heads": heads, "groups": 1, "d_k": 8, "d_v": d_v,
                           "tokens": seqs * max_len, "max_len": max_len, "x": far, "x_stride": heads * d_v, "B": 2 * far,
                           "b_stride": 8, "C": 3 * far, "c_stride": 8, "dt": 4 * far, "dt_stride": heads, "state": 5 * far,
                           "y": 6 * far, "y_stride": heads * d_v, "D": None, "dt_bias": None, "A": 7 * far, **kw})


@pytest.mark.parametrize("seqs,heads,d_v,fits", [((1 << 24) - 1, 1, 8, True), (1 << 24, 1, 8, False), (1 << 20, 16, 64, False),
                                                (1 << 20, 8, 72, False), ((1 << 20) - 1, 8, 128, True)])
def test_scan_workgroups(seqs, heads, d_v, fits):
    """256 threads a workgroup, one per sequence, head and 64 columns."""
    p, n = ssm(seqs, heads, d_v=d_v), ctypes.c_size_t()
    code = lib.rsq_ssm_scan_workspace(ctypes.byref(p), ctypes.byref(n))
    assert code == (0 if fits else UNSUPPORTED)
    if not fits:
        assert lib.rsq_ssm_scan(ctypes.byref(p), None) == UNSUPPORTED


@pytest.mark.parametrize("seqs,heads", [(1 << 24, 1), (1 << 18, 64)])
def test_step_workgroups(seqs, heads):
    p = ssm(seqs, heads)
    assert lib.rsq_ssm_step(ctypes.byref(p), None) == UNSUPPORTED


@pytest.mark.parametrize("seqs,tokens,max_len", [(256, 16384 + 255, 16384), (1024, 65536, 60000), (2000, 1 << 20, 1 << 19)])
def test_scan_workspace_goes_by_the_segments_that_exist(seqs, tokens, max_len):
    """One long prompt beside many short ones: the slots of at most every 64 per rows and of as many sequences, at the
    head's 128 x 64 fp32 state and its decay each. More than three segments for each of 768 workgroups are never wanted."""
    p = fill(_abi.Ssm, {**SSM, "seqs": seqs, "heads": 64, "groups": 1, "tokens": tokens, "max_len": max_len,
                        "offsets": addr(9), "x_stride": 4096, "b_stride": 128, "c_stride": 128, "dt_stride": 64,
                        "y_stride": 4096})
    n = ctypes.c_size_t()
    assert lib.rsq_ssm_scan_workspace(ctypes.byref(p), ctypes.byref(n)) == 0
    assert 0 < n.value <= 3 * 768 * (128 * 64 * 4 + 4)


def test_outputs_over_the_offsets_of_the_most_sequences():
    """2^31 - 1 sequences have 2^31 offsets: their bytes do not pass for none."""
    most, far = 0x7FFFFFFF, 1 << 44
    c = fill(_abi.Conv, {**CONV, "seqs": most, "state": None, "offsets": addr(4), "y": addr(4)})
    assert lib.rsq_causal_conv(ctypes.byref(c), None) == INVALID
    p = ssm(most, 1, max_len=10, tokens=20, offsets=addr(4), state=far, y=addr(4))
    assert lib.rsq_ssm_scan(ctypes.byref(p), None) == INVALID
