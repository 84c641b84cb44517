"""Attention with a decay for each head, norms around a block and 8-bit products: their definitions in fp64 on the
CPU, with bounds on what fp32 sums and the kernels' roundings may add (test infrastructure; the bounds' terms are
those of layer_reference).

With the delta rule an error of the state goes through a chunk by the chunk's own linear map, of which the 2-norm is
taken; a column's error is held in that norm. What a chunk adds to it is bounded element by element.
"""
import torch

from layer_reference import U, _fp32_terms, f64, half_step

CHUNK = 64
PIECES = 2.0 ** -16     # what two bf16 pieces of a factor leave of it, at most


def attention(q, k, v, alpha, beta, state, sequences, dtype):
    """Packed rows q, k [n, keys, dk], v [n, heads, dv], alpha, beta [n, heads] (alpha also [heads]) or None ->
    (o, S, bound of o, bound of S: element by element, or of each column's 2-norm [sequences, heads, dv] with beta).
    Rows of no sequence are NaN in o."""
    n, heads, dv = v.shape
    per = heads // k.shape[1]
    q, k, v = f64(q).repeat_interleave(per, 1), f64(k).repeat_interleave(per, 1), f64(v)
    dk = k.shape[2]
    a = torch.ones(n, heads, dtype=torch.float64) if alpha is None else f64(alpha).expand(n, heads)
    b = None if beta is None else f64(beta)
    lossy = dtype == torch.bfloat16
    N = len(sequences)
    S = torch.zeros(N, heads, dk, dv, dtype=torch.float64) if state is None else f64(state).clone()
    o, bo = torch.full_like(v, float("nan")), torch.zeros_like(v)
    bS = torch.zeros(N, heads, dv, dtype=torch.float64) if b is not None else torch.zeros_like(S)
    for s, (r0, length) in enumerate(sequences):
        for h in range(heads):
            rows = slice(r0, r0 + length)
            f = _plain if b is None else _delta
            args = (q[rows, h], k[rows, h], v[rows, h], a[rows, h], None if b is None else b[rows, h], S[s, h], lossy)
            o[rows, h], bo[rows, h], S[s, h], bS[s, h] = f(*args)
    bo += half_step(dtype) * o.abs()
    return o, S, 1.05 * bo + 1e-37, 1.05 * bS + 1e-37


def _logs(a):
    """Decays may be zero, which the kernels take as 2^-2000."""
    return torch.log(a.clamp(min=0)).clamp(min=-1386.0)


def _plain(q, k, v, a, b, S, lossy):
    o, bo = torch.zeros_like(v), torch.zeros_like(v)
    mag, lam = S.abs(), 0.0
    for t in range(v.shape[0]):
        if t % CHUNK == 0:
            start, since = S.clone(), 1.0
        lam = min(lam + float(-_logs(a[t])), 40.0)     # (of what is decayed by e^-40 nothing is left to be off)
        add = k[t][:, None] * v[t][None, :]
        S = a[t] * S + add
        mag = a[t] * mag + add.abs()
        since = since * a[t]
        o[t] = q[t] @ S
        m = q[t].abs() @ mag
        bo[t] = m * _fp32_terms(t + 1, q.shape[1], lam)
        if lossy:
            bo[t] += 2 * PIECES * (m + since * (q[t].abs() @ start.abs()))
    return o, bo, S, mag * _fp32_terms(v.shape[0], 0, lam)


def _delta(q, k, v, a, b, S, lossy):
    o, bo = torch.zeros_like(v), torch.zeros_like(v)
    dk = k.shape[1]
    carried = torch.zeros(v.shape[1], dtype=torch.float64)
    for t0 in range(0, v.shape[0], CHUNK):
        K, Q, V, B = (x[t0: t0 + CHUNK] for x in (k, q, v, b))
        n = K.shape[0]
        c = torch.cumsum(_logs(a[t0: t0 + CHUNK]), 0)
        lower = torch.ones(n, n, dtype=torch.bool).tril()
        diff = torch.where(lower, c[:, None] - c[None, :], torch.full((n, n), -float("inf"), dtype=torch.float64))
        D, ec, w, dec = torch.exp(diff), torch.exp(c)[:, None], torch.exp(c[-1] - c)[:, None], torch.exp(c[-1])
        lam = float((-c[-1]).clamp(max=40.0))
        eye = torch.eye(n, dtype=torch.float64)
        A = (B[:, None] * D * (K @ K.t())).tril(-1)
        inv = torch.linalg.solve_triangular(eye + A, eye, upper=False, unitriangular=True)
        T = inv * B[None, :]
        X = V - ec * (K @ S)
        W = T @ X
        P = D * (Q @ K.t())
        o[t0: t0 + n] = ec * (Q @ S) + P @ W
        # ---- what fp32 adds, each operation's terms by their magnitudes
        KS, QS = ec * (K.abs() @ S.abs()), ec * (Q.abs() @ S.abs())
        eX = U * ((3 * dk + 12 + 2 * lam) * KS + V.abs() + X.abs())
        dA = U * (3 * dk + 16 + 2 * lam) * (B.abs()[:, None] * D * (K.abs() @ K.abs().t())).tril(-1)
        dT = (inv.abs() @ (dA + 4 * CHUNK * U * A.abs()) @ inv.abs() + 4 * U * inv.abs()) * B.abs()[None, :]
        eW = T.abs() @ eX + dT @ X.abs() + U * (3 * CHUNK + 12) * (T.abs() @ X.abs())
        Pm = D * (Q.abs() @ K.abs().t())
        eo = U * (3 * dk + 16 + 2 * lam) * QS + P.abs() @ eW + U * (3 * CHUNK + 3 * dk + 24 + 2 * lam) * (Pm @ W.abs())
        if lossy:
            eo += PIECES * QS + 2 * PIECES * (P.abs() @ W.abs())
        # ---- and the state's own error
        R = ec * Q - P @ (T @ (ec * K))
        bo[t0: t0 + n] = eo + R.norm(dim=1)[:, None] * carried[None, :]
        local = K.abs().t() @ (w * eW) + U * (3 * CHUNK + 16 + 2 * lam) * (K.abs().t() @ (w * W.abs())) + U * (8 + lam) * dec * S.abs()
        Phi = dec * torch.eye(dk, dtype=torch.float64) - K.t() @ (w * (T @ (ec * K)))
        carried = torch.linalg.matrix_norm(Phi, 2) * carried + local.norm(dim=0)
        S = dec * S + K.t() @ (w * W)
    return o, bo, S, carried


def check_columns(got, want, bound, what=""):
    """Columns of a state within the bound of their 2-norm."""
    off = (f64(got) - want).norm(dim=-2) - bound
    assert bool((off <= 0).all()), "%s: %g over the bound" % (what, float(off.max()))


def block_norm(x, weight, gate, gate_first, activation, group, eps, residual, residual_scale, next_weight):
    """(y, h, bounds of both before their own rounding): h is what replaces the residual."""
    rows, cols = x.shape
    u = f64(x)
    err = torch.zeros_like(u)
    act = None
    if gate is not None:
        g = f64(gate)
        # e^-g to 2^-22 and its argument's rounding, an addition, a quotient
        act = {"silu": g * torch.sigmoid(g), "sigmoid": torch.sigmoid(g), None: g}[activation]
        act_err = act.abs() * (10 + 2 * g.abs()) * U if activation else torch.zeros_like(g)

    def gated(u, err):
        return u * act, err * act.abs() + u.abs() * act_err + (u * act).abs() * U

    def normed(u, err, w):
        rms = torch.sqrt((u * u).mean(-1, keepdim=True) + eps)
        y = u / rms * w
        # the mean's relative error: its terms', 70 half steps of the sums, root, reciprocal and products
        rel = 2 * (u.abs() * err).sum(-1, keepdim=True) / (u * u).sum(-1, keepdim=True).clamp(min=1e-300)
        return y, (err / rms) * w.abs() + y.abs() * (rel + 70 * U)

    if gate is not None and gate_first:
        u, err = gated(u, err)
    if weight is not None:
        parts = cols // group if group else 1
        w = f64(weight).view(-1, cols // parts) if weight.numel() == cols else f64(weight)
        u, err = normed(u.view(rows, parts, -1), err.view(rows, parts, -1), w)
        u, err = u.reshape(rows, cols), err.reshape(rows, cols)
    if gate is not None and not gate_first:
        u, err = gated(u, err)
    h, eh = u, err
    if residual is not None:
        h = f64(residual) + residual_scale * u
        eh = abs(residual_scale) * err + U * ((residual_scale * u).abs() + h.abs())
    y, ey = (h, eh) if next_weight is None else normed(h, eh, f64(next_weight))
    return y, h, 1.05 * ey + 1e-37, 1.05 * eh + 1e-37


def w8(x, codes, scales, x_scale, bias):
    """(y, bound before its own rounding): whole sums, then the sum to fp32, a product and a fused one."""
    y = (f64(x) @ f64(codes).t()) * f64(x_scale).view(-1, 1) * f64(scales)
    bound = 3.05 * U * y.abs()
    if bias is not None:
        y = y + f64(bias)
    return y, bound + 1.05 * U * y.abs() + 1e-37
