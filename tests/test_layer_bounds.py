"""The limit that products with 4-bit weights are held to: the sums as they are made keep it, lesser ones do not."""
import numpy as np
import pytest

from layer_bounds import w4_norm_limit, w4_sums


def case(m, n, k, group, mean=0.0):
    r = np.random.RandomState(k)
    codes = r.randint(-8, 8, (n, k)).astype(np.float64)
    scales = (np.abs(r.randn(n, k // group)) + 0.1).astype(np.float32).astype(np.float64)
    x = (r.randn(m, k) + mean).astype(np.float32)
    want = x.astype(np.float64) @ (codes * scales.repeat(group, 1)).T
    return codes, scales, x, want


@pytest.mark.parametrize("group", [32, 64, 128])
def test_fp32_rows_need_their_pieces_and_their_sums(group):
    codes, scales, x, want = case(4, 64, 4736, group)
    limit = w4_norm_limit(codes, scales, x.astype(np.float64), group, True, False)
    off = lambda *a: np.linalg.norm(w4_sums(codes, scales, x, group, *a) - want)  # noqa: E731
    assert off(3, True) < 0.5 * limit
    assert off(2, True) > 4 * limit and off(1, True) > 100 * limit
    assert off(3, False) > 1.7 * off(3, True)       # 24 sum(x) in the sums of whole groups


@pytest.mark.parametrize("mean", [0.0, 1.0])
def test_bf16_rows_keep_the_limit(mean):
    codes, scales, x, _ = case(4, 64, 1280, 128, mean)
    x = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
    want = x.astype(np.float64) @ (codes * scales.repeat(128, 1)).T
    limit = w4_norm_limit(codes, scales, x.astype(np.float64), 128, False, False)
    assert np.linalg.norm(w4_sums(codes, scales, x, 128, 1, False) - want) < 0.7 * limit
    seven = (x.view(np.uint32) & np.uint32(0xFFFE0000)).view(np.float32)
    assert np.linalg.norm(w4_sums(codes, scales, seven, 128, 1, False) - want) > 100 * limit
