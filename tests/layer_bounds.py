"""What fp32 sums leave of a product with 4-bit weights, as a norm, and the sums step by step (test infrastructure).

The kernels add up products of x with 24 + c and take 24 sum(x) off, 32 columns a product: each product's result is
rounded to fp32 at its own size. Sums of fp32 rows' leading pieces start anew every 32 columns, those of other rows
every `group` columns. A rounding is off by at most U of its size, evenly spread: by U / sqrt(3) in the mean square,
and roundings are independent. Twice their joint size is the limit.
"""
import numpy as np

U = 2.0 ** -24


def w4_norm_limit(codes, scales, x, group, fp32_rows, scaled):
    """Limit of the error's 2-norm over all outputs, fp64 arrays: codes [n, k], scales [n, k / group], x [m, k] (with its
    own scales, `scaled`, in it)."""
    m, k = x.shape
    steps = x.reshape(m, k // group, group // 32, 32).sum(3)                # of 32 columns each
    if fp32_rows:
        size2 = (24 * steps) ** 2                                           # start's; the rest is small against it
    else:
        upto = np.cumsum(steps, 2)
        left = upto[:, :, -1:] - upto                                       # what the code products have yet to cancel
        size2 = (24 * upto) ** 2 + (24 * left) ** 2
    offset = size2.sum(2) @ (scales ** 2).T                                 # [m, n]
    y = x @ (codes * scales.repeat(group, 1)).T
    # y itself: a running sum's steps are at half its final square in the mean, and no wavefront has more than half
    # of the groups; a join of up to 16; x's scales
    own = (k // group / 4 + 8 + 3 * scaled) * y ** 2
    return 2 * U * np.sqrt((offset + own).sum() / 3)


def pieces(x, n):
    """fp32 values as n bf16 pieces of the leading 8 bits of what is left."""
    out, x = [], x.astype(np.float32)
    for _ in range(n):
        p = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        out.append(p.astype(np.float64))
        x = x - p
    return out


def w4_sums(codes, scales, x, group, n_pieces, own_sums):
    """The product with every step's sum rounded to fp32; own_sums: the leading pieces' sums of 32 columns apart."""
    m, k = x.shape
    r = lambda v: v.astype(np.float32).astype(np.float64)  # noqa: E731
    xp = pieces(x, n_pieces)
    y = np.zeros((m, codes.shape[0]))
    for g in range(k // group):
        acc, low = np.zeros_like(y), np.zeros_like(y)
        cols = [slice(g * group + 32 * j, g * group + 32 * j + 32) for j in range(group // 32)]
        if own_sums:
            for c in cols:
                for p in range(n_pieces - 1, 0, -1):
                    low = r(low - 24 * xp[p][:, c].sum(1, keepdims=True))
            for c in cols:
                one = r(np.zeros_like(y) - 24 * xp[0][:, c].sum(1, keepdims=True))
                acc = r(acc + r(one + xp[0][:, c] @ (24 + codes[:, c]).T))
                for p in range(n_pieces - 1, 0, -1):
                    low = r(low + xp[p][:, c] @ (24 + codes[:, c]).T)
            acc = r(acc + low)
        else:
            for c in cols:
                for p in range(n_pieces - 1, -1, -1):
                    acc = r(acc - 24 * xp[p][:, c].sum(1, keepdims=True))
            for c in cols:
                for p in range(n_pieces - 1, -1, -1):
                    acc = r(acc + xp[p][:, c] @ (24 + codes[:, c]).T)
        y = r(y + acc * scales[:, g])
    return y
