"""Definitions of the layer operators in fp64 on the CPU, token by token, with
bounds on what the kernels' fp32 arithmetic and their roundings may add (test
infrastructure).

A bound is elementwise: U = 2^-24 is half a step of fp32 and H = 2^-8 half a
step of bf16, both relative to the value rounded; a sum of n terms in any order
is off by at most n U times the sum of their magnitudes (to first order; the
bounds carry a factor for the rest).
"""
import torch

U = 2.0 ** -24
H = 2.0 ** -8


def half_step(dtype):
    return {torch.float32: U, torch.bfloat16: H}[dtype]


def f64(t):
    return None if t is None else t.detach().cpu().double()


def check(got, want, bound, what=""):
    """got within bound of want, elementwise; NaNs and infinities in the same places."""
    got, want = f64(got), f64(want)
    assert got.shape == want.shape, what
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaNs differ"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    off = torch.where(fine, (got - want).abs() - bound, torch.full_like(want, -1.0))
    worst = off.max() if off.numel() else torch.tensor(-1.0)
    assert worst <= 0, "%s: %g over the bound, at %s" % (what, worst, (off == worst).nonzero()[0].tolist())


def spans(x, seqs, offsets, inner):
    """[(first row, rows)] of every sequence, and x as packed rows."""
    if offsets is None:
        T = x.shape[1]
        return [(s * T, T) for s in range(seqs)]
    o = offsets.cpu().tolist()
    return [(a, b - a) for a, b in zip(o[:-1], o[1:])]


def conv(x, weight, bias, state, sequences, silu, dtype):
    """Packed rows x [n, C] -> (y, new state, bound of y); rows of no sequence are NaN in y."""
    x, w = f64(x), f64(weight)
    b = torch.zeros(w.shape[0], dtype=torch.float64) if bias is None else f64(bias)
    W = w.shape[1]
    y = torch.full_like(x, float("nan"))
    bound = torch.zeros_like(x)
    new = None if state is None else f64(state).clone()
    for s, (a, n) in enumerate(sequences):
        hist = torch.zeros(W - 1, x.shape[1], dtype=torch.float64) if state is None else f64(state)[s].t()
        seq = torch.cat([hist, x[a: a + n]])
        z, mag = b.expand(n, -1).clone(), b.abs().expand(n, -1).clone()
        for j in range(W):
            z += w[:, j] * seq[j: j + n]
            mag += (w[:, j] * seq[j: j + n]).abs()
        # W + 1 additions; silu' <= 1.1; e^-z to 2^-22 plus the rounding of its argument (U |z| log2 e, twice),
        # then an addition, a reciprocal and a product to 2^-23 each
        err = (W + 1) * U * mag
        if silu:
            out = z * torch.sigmoid(z)
            err = 1.1 * err + out.abs() * (10 + 4 * z.abs()) * U
        else:
            out = z
        y[a: a + n] = out
        bound[a: a + n] = 1.01 * err + half_step(dtype) * out.abs() * 1.01 + 1e-38
        if new is not None and n > 0:
            new[s] = seq[n:].t()
    return y, new, bound


def scan(x, dt, A, B, C, D, dt_bias, softplus, state, sequences, dtype, chunk=64):
    """Packed rows x [n, H, dv], dt [n, H], B, C [n, G, dk] -> (y, S, bounds of both).

    Roundings to bf16 (half a step H each) that the bound allows for, with bf16
    inputs: S at the start of a chunk of 64 tokens and the weight P_ts of x_s
    within the chunk, where they enter y; y itself. fp32 inputs have none.
    """
    x, dt, A, B, C = f64(x), f64(dt), f64(A), f64(B), f64(C)
    n, heads, dv = x.shape
    dk, per = B.shape[2], heads // B.shape[1]
    B, C = B.repeat_interleave(per, 1), C.repeat_interleave(per, 1)
    z = dt + (0 if dt_bias is None else f64(dt_bias))
    d = torch.logaddexp(z, torch.zeros((), dtype=torch.float64)) if softplus else z
    # an infinite z is its own softplus (logaddexp agrees); NaN stays NaN
    a = torch.exp(d * A)
    lam = (d * A).abs()
    lossy = dtype == torch.bfloat16
    y = torch.full_like(x, float("nan"))
    by = torch.zeros_like(x)
    N = len(sequences)
    S = torch.zeros(N, heads, dk, dv, dtype=torch.float64) if state is None else f64(state).clone()
    bS = torch.zeros_like(S)
    for s, (r0, length) in enumerate(sequences):
        st, mag = S[s], S[s].abs()          # the state, and the same sums of magnitudes
        local = torch.zeros_like(st)        # what the chunk's own tokens added
        chunks = 0
        drift = torch.zeros(heads, dtype=torch.float64)
        for t in range(length):
            r = r0 + t
            if t % chunk == 0:
                start, local, decay, ps = st.clone(), torch.zeros_like(st), torch.ones(heads, dtype=torch.float64), []
                chunks += 1
            add = B[r][:, :, None] * (d[r][:, None] * x[r])[:, None, :]
            st = a[r][:, None, None] * st + add
            mag = a[r][:, None, None] * mag + add.abs()
            decay = decay * a[r]
            drift = torch.maximum(drift, lam[r])
            y[r] = torch.matmul(C[r][:, None, :], st).squeeze(1) + (0 if D is None else f64(D)[:, None] * x[r])
            # magnitudes: |C| |S|
            m = torch.matmul(C[r].abs()[:, None, :], mag).squeeze(1)
            ps = [(a[r][:, None] * p, q, v) for p, q, v in ps] + [(d[r][:, None], B[r], x[r])]
            by[r] = m * _fp32_terms(t + 1, dk, lam[r0: r + 1].sum(0)[:, None])
            by[r] += 0 if D is None else (f64(D)[:, None] * x[r]).abs() * 2 * U
            if lossy:
                rounded = decay[:, None] * torch.matmul(C[r].abs()[:, None, :], start.abs()).squeeze(1)
                for p, q, v in ps:
                    rounded = rounded + ((C[r] * q).sum(1, keepdim=True) * p).abs() * v.abs()
                by[r] += 1.01 * H * rounded
            by[r] += half_step(dtype) * 1.01 * y[r].abs()
        S[s] = st
        bS[s] = mag * _fp32_terms(length, 0, lam[r0: r0 + length].sum(0)[:, None, None] if length else 0.0)
    return y, S, by * 1.01 + 1e-37, bS * 1.01 + 1e-37


def _fp32_terms(tokens, dk, lam):
    """Half steps of fp32 that a sum over `tokens` terms of three pieces (and d_k products) gathers: each
    addition, the weight's exponential (2^-22), its argument (lam half steps twice), delta (2^-21: log1p of exp)."""
    return (3.0 * tokens + 3.0 * dk + 2.0 * tokens / 64 + 40.0 + 4.0 * lam) * U


def norm(x, weight, eps, residual):
    """(y, h, relative error of y before its own rounding)."""
    h = f64(x) if residual is None else f64(x) + f64(residual)
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * f64(weight)
    # h, its square and the sums over at most 32 columns a thread, 6 + 16 joins, mean, root, reciprocal, two products
    return y, h, 70 * U
