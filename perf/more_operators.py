"""Cases of the operators of a linear-attention layer: attention with a decay for
each head (with or without the delta rule) over prompts and for single tokens,
the norms before and after a block with its gate and residual, and products of
8-bit integers with scales for each token and channel.

With own = False run() computes a pass from elementary torch operations in
fp32 (decay sums in fp64); with own = True it makes the package's calls.
exact() evaluates the definitions in fp64, token by token.

Sizes: the Gated DeltaNet workloads of rsq_workloads (16 and 32 heads of 128 x
128), with half as many key heads where key heads are shared, a model width of
2048 and so an input projection of 2*16*128 + 2*32*128 + 64 = 12352 rows (q, k,
v, the output's gate, decays and write strengths); the largest product has
generic feed-forward sizes.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


# ---------------------------------------------------------------- the cases
def listed():
    gdn = dict(dk=128, dv=128, dtype="bf16", delta=True, gamma=False)
    return [
        # one long prompt: as few sequences as there can be, every chunk waits for the last one
        dict(name="delta_long", op="attention", seqs=1, tokens=16384, heads=32, keys=16, **gdn),
        # a prefill batch of eight ragged prompts, packed, continuing from their states
        dict(name="delta_ragged", op="attention", seqs=8, tokens=8192, heads=32, keys=32, **gdn),
        # a short fp32 prompt with shared keys and narrow heads
        dict(name="delta_short_f32", op="attention", seqs=2, tokens=333, heads=8, keys=2, dk=64, dv=64, dtype="f32",
             delta=True, gamma=False),
        # retention: one decay a head for all tokens
        dict(name="retention_ragged", op="attention", seqs=8, tokens=8192, heads=16, keys=16, dk=128, dv=128, dtype="bf16",
             delta=False, gamma=True),
        # a decay for each token and head, without the delta rule, fp32
        dict(name="decay_short_f32", op="attention", seqs=3, tokens=517, heads=8, keys=8, dk=64, dv=128, dtype="f32",
             delta=False, gamma=False),
        # one sequence's token: latency
        dict(name="delta_step_b1", op="step", batch=1, heads=32, keys=16, **gdn),
        # a decode batch's token: the state's bandwidth
        dict(name="delta_step_b64", op="step", batch=64, heads=32, keys=32, **gdn),
        # a few tokens' heads, normed one by one and gated, into 8 bits for the output projection
        dict(name="norm_heads_e4m3", op="norm", rows=16, cols=4096, dtype="bf16", group=128, gate="after", residual=False,
             next=False, out="e4m3"),
        # between two blocks of a prefill batch: the block's output normed and added, the next block's input normed
        dict(name="norm_between_blocks", op="norm", rows=16384, cols=2048, dtype="bf16", group=0, gate="none", residual=True,
             next=True, out="bf16"),
        # the input projection of sixteen sequences' tokens
        dict(name="w8_m16", op="w8", m=16, n=12352, k=2048, bias=False, out="bf16"),
        # odd sizes, with a bias
        dict(name="w8_odd", op="w8", m=333, n=1031, k=705, bias=True, out="f32"),
        # a feed-forward product of a prefill batch
        dict(name="w8_prompt", op="w8", m=4096, n=28672, k=8192, bias=False, out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "step", "norm", "norm", "w8", "w8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("attention", "step"):
        keys = _log(rng, 1, 16)
        delta = rng.random() < 0.6
        size = dict(heads=keys * rng.choice([1, 1, 2, 4]), keys=keys, dk=8 * _log(rng, 2, 16), dv=8 * _log(rng, 1, 16),
                    dtype=dtype, delta=delta, gamma=not delta and rng.random() < 0.5)
        if op == "step":
            return dict(op=op, batch=_log(rng, 1, 64), **size)
        seqs = _log(rng, 1, 8)
        return dict(op=op, seqs=seqs, tokens=_log(rng, seqs, 4096), **size)
    if op == "norm":
        group = rng.choice([0, 0, 32, 64, 96, 128, 256])
        cols = group * _log(rng, 1, 8192 // group) if group else _log(rng, 8, 8192)
        return dict(op=op, rows=_log(rng, 1, 8192), cols=cols, dtype=dtype, group=group,
                    gate=rng.choice(["none", "before", "after"]), residual=rng.random() < 0.5, next=rng.random() < 0.5,
                    out=rng.choice(["bf16", "f32", "e4m3"]))
    return dict(op=op, m=_log(rng, 1, 4096), n=_log(rng, 1, 16384), k=_log(rng, 1, 8192), bias=rng.random() < 0.5,
                out=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------- the inputs
def _lengths(case, seed):
    """seqs lengths that add up to tokens: random cuts, so some are short or zero."""
    cuts = np.random.RandomState(seed % (1 << 31)).randint(0, case["tokens"] + 1, case["seqs"] - 1)
    return np.diff(np.concatenate([[0], np.sort(cuts), [case["tokens"]]])).tolist()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    op, dt = case["op"], TYPES.get(case.get("dtype"))
    s = {"case": case}
    if op in ("attention", "step"):
        H, G, dk, dv = case["heads"], case["keys"], case["dk"], case["dv"]
        n = case["tokens"] if op == "attention" else case["batch"]
        if op == "attention":
            lens = _lengths(case, seed)
            s["max_len"] = max(lens)
            s["offsets"] = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")
        # q, k and v are slices of the convolution's output; q and k have unit length, q scaled for the products
        qkv = randn(n, 2 * G * dk + H * dv)
        keyed = qkv[:, : 2 * G * dk].view(n, 2 * G, dk)
        keyed /= keyed.norm(dim=2, keepdim=True)
        qkv[:, : G * dk] /= math.sqrt(dk)
        qkv = qkv.to(dt)
        s["q"] = qkv[:, : G * dk].view(n, G, dk)
        s["k"] = qkv[:, G * dk: 2 * G * dk].view(n, G, dk)
        s["v"] = qkv[:, 2 * G * dk:].view(n, H, dv)
        if case["gamma"]:
            s["alpha"] = 1.0 - torch.exp2(-5.0 - 3.0 * rand(H))                  # retention's: 1 - 2^-5 .. 1 - 2^-8
        else:
            # e^{-A d}: rates A of 1 to 16, steps d of 0.001 to 0.1
            s["alpha"] = torch.exp(-torch.exp(2.77 * rand(H)) * torch.exp(math.log(0.001) + 4.6 * rand(n, H)))
        s["beta"] = torch.sigmoid(randn(n, H)) if case["delta"] else None
        s["state"] = 0.3 * randn(case.get("seqs", case.get("batch")), H, dk, dv)
    elif op == "norm":
        rows, cols = case["rows"], case["cols"]
        s["x"] = randn(rows, cols).to(dt)
        s["weight"] = 1.0 + 0.2 * randn(case["group"] or cols)                   # of a head, shared by all of them
        s["gate"] = (1.5 * randn(rows, cols)).to(dt) if case["gate"] != "none" else None
        s["residual"] = (2.0 * randn(rows, cols)).to(dt) if case["residual"] else None
        s["next_weight"] = 1.0 + 0.2 * randn(cols) if case["next"] else None
    else:
        M, N, K = case["m"], case["n"], case["k"]
        w = randn(N, K)
        s["w_scale"] = w.abs().amax(1) / 127
        s["codes"] = torch.round(w / s["w_scale"][:, None]).to(torch.int8)
        s["w_scale"] /= math.sqrt(K)
        del w
        x = randn(M, K)
        s["x_scale"] = x.abs().amax(1, keepdim=True) / 127
        s["x"] = torch.round(x / s["x_scale"]).to(torch.int8)
        s["bias"] = 0.1 * randn(N) if case["bias"] else None
        if own:
            import bit_recurrent_state_rsq_amd as rsq
            s["w"] = rsq.W8Weight(s["codes"], s["w_scale"])                      # laid out once, as a program keeps it
    return s


RESIDUAL_SCALE = 0.5


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _own(case, s)
    return _PLAIN[case["op"]](case, s)


def _own(case, s):
    import bit_recurrent_state_rsq_amd as rsq
    op = case["op"]
    if op == "attention":
        return rsq.linear_attention(s["q"], s["k"], s["v"], alpha=s["alpha"], beta=s["beta"], state=s["state"],
                                    offsets=s["offsets"], max_len=s["max_len"])
    if op == "step":
        return rsq.linear_attention_step(s["state"], s["q"], s["k"], s["v"], alpha=s["alpha"], beta=s["beta"]), s["state"]
    if op == "norm":
        y = rsq.block_norm(s["x"], s["weight"], gate=s["gate"], gate_first=case["gate"] == "before", activation="silu",
                           group=case["group"], eps=EPS, residual=s["residual"],
                           residual_scale=RESIDUAL_SCALE if case["residual"] else 1.0, next_weight=s["next_weight"],
                           out_dtype=case["out"])
        return (y, s["residual"]) if case["residual"] else y
    return rsq.w8_linear(s["x"], s["w"], s["x_scale"], bias=s["bias"], out_dtype=case["out"])


CHUNK = 64


def _plain_attention(case, s):
    N, H, G, dk, dv = case["seqs"], case["heads"], case["keys"], case["dk"], case["dv"]
    dev = s["q"].device
    nc = max(1, -(-s["max_len"] // CHUNK))
    at = s["offsets"][:-1, None].long() + torch.arange(nc * CHUNK, device=dev)
    inside = at < s["offsets"][1:, None].long()
    at = torch.where(inside, at, 0)

    def chunks(v, heads):     # rows [n, h, d] -> [N, nc, heads, CHUNK, d], zeros past a sequence's end
        v = torch.where(inside[..., None, None], v.float()[at], 0.0).view(N, nc, CHUNK, v.shape[1], v.shape[2])
        v = v.permute(0, 1, 3, 2, 4)
        return v[:, :, :, None].expand(-1, -1, -1, heads // v.shape[2], -1, -1).reshape(N, nc, heads, CHUNK, v.shape[4])

    gates = lambda v: torch.where(inside[..., None], v[at], 0.0).view(N, nc, CHUNK, H).permute(0, 1, 3, 2)  # noqa: E731
    Q, K, V = chunks(s["q"], H), chunks(s["k"], H), chunks(s["v"], H)
    cum = gates(torch.log(s["alpha"].double()).expand(s["q"].shape[0], H)).cumsum(3)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    D = torch.exp(torch.where(lower, cum[..., :, None] - cum[..., None, :], -math.inf)).float()
    ec, last = torch.exp(cum).float()[..., None], torch.exp(cum[..., -1]).float()[..., None, None]
    w = torch.exp(cum[..., -1:] - cum).float()[..., None]
    KT = K.transpose(-1, -2).contiguous()
    P = torch.matmul(Q, KT) * D
    U, W = V, None
    if case["delta"]:
        beta = gates(s["beta"])[..., None]
        A = (beta * torch.matmul(K, KT) * D).tril(-1)
        T = torch.eye(CHUNK, device=dev).expand(N, nc, H, CHUNK, CHUNK).contiguous()
        for i in range(1, CHUNK):          # (1 + A)^-1, row by row
            T[..., i: i + 1, :i] = -torch.matmul(A[..., i: i + 1, :i], T[..., :i, :i].contiguous())
        del A
        U, W = torch.matmul(T, beta * V), torch.matmul(T, beta * ec * K)
        del T
    del D, V
    S, out = s["state"], []
    for c in range(nc):
        u = U[:, c] if W is None else U[:, c] - torch.matmul(W[:, c], S)
        out.append(torch.matmul(ec[:, c] * Q[:, c], S) + torch.matmul(P[:, c], u))
        S = last[:, c] * S + torch.matmul(KT[:, c], w[:, c] * u)
    o = torch.stack(out, 1).permute(0, 1, 3, 2, 4).reshape(N, nc * CHUNK, H, dv)[inside].to(s["v"].dtype)
    s["state"].copy_(S)
    return o, s["state"]


def _plain_step(case, s):
    S, per = s["state"], case["heads"] // case["keys"]
    k, q = (s[n].float().repeat_interleave(per, 1)[..., None] for n in ("k", "q"))
    a = s["alpha"].expand(S.shape[0], -1)
    u = s["v"].float()
    S.mul_(a[..., None, None])
    if case["delta"]:
        u = s["beta"][..., None] * (u - (S * k).sum(2))
    S.add_(k * u[..., None, :])
    return (S * q).sum(2).to(s["v"].dtype), S


def _plain_norm(case, s):
    rows, cols, group = case["rows"], case["cols"], case["group"] or case["cols"]
    rms = lambda v: torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)  # noqa: E731
    h = s["x"].float()
    act = None
    if s["gate"] is not None:
        act = s["gate"].float()
        act = act / (1.0 + torch.exp(-act))
    if case["gate"] == "before":
        h = h * act
    h = h.view(rows, cols // group, group)
    h = (h * rms(h) * s["weight"]).view(rows, cols)
    if case["gate"] == "after":
        h = h * act
    rest = ()
    if s["residual"] is not None:
        h = s["residual"].float() + RESIDUAL_SCALE * h
        s["residual"].copy_(h)
        rest = (s["residual"],)
    y = h * rms(h) * s["next_weight"] if case["next"] else h
    if case["out"] == "e4m3":
        scale = y.abs().amax(1, keepdim=True) / 448
        y = (torch.where(scale > 0, y / scale, 0.0).clamp(-448, 448).to(torch.float8_e4m3fn), scale)
    else:
        y = y.to(TYPES[case["out"]])
    return (y,) + rest if rest else y


def _plain_w8(case, s):
    y = torch.matmul(s["x"].float(), s["codes"].float().t()) * s["x_scale"] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(TYPES[case["out"]])


_PLAIN = {"attention": _plain_attention, "step": _plain_step, "norm": _plain_norm, "w8": _plain_w8}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("attention", "step"):
        H, G, dk, dv, e = case["heads"], case["keys"], case["dk"], case["dv"], SIZE[case["dtype"]]
        n = case["tokens"] if op == "attention" else case["batch"]
        seqs = case.get("seqs", case.get("batch"))
        gates = (H if case["gamma"] else n * H) + (n * H if case["delta"] else 0)
        return {"bytes": n * e * (2 * H * dv + 2 * G * dk) + 4 * gates + seqs * H * dk * dv * 8,
                "flops": (7 if case["delta"] else 5) * n * H * dk * dv}
    if op == "norm":
        n, e = case["rows"] * case["cols"], SIZE[case["dtype"]]
        reads = 1 + (case["gate"] != "none") + 2 * case["residual"]
        weights = 4 * ((case["group"] or case["cols"]) + (case["cols"] if case["next"] else 0))
        return {"bytes": n * (reads * e + SIZE[case["out"]]) + weights + (4 * case["rows"] if case["out"] == "e4m3" else 0),
                "flops": n * (5 + 4 * (case["gate"] != "none") + 2 * case["residual"] + 4 * case["next"])}
    M, N, K = case["m"], case["n"], case["k"]
    return {"bytes": N * K + M * K + M * N * SIZE[case["out"]] + 4 * (M + N) + (4 * N if case["bias"] else 0),
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False
    try:
        s = prepare(case, seed)
    finally:
        globals()["own"] = was
    op = case["op"]
    f = lambda v: v.double()  # noqa: E731
    if op in ("attention", "step"):
        per = case["heads"] // case["keys"]
        q, k = f(s["q"]).repeat_interleave(per, 1), f(s["k"]).repeat_interleave(per, 1)
        v, n = f(s["v"]), s["v"].shape[0]
        a = f(s["alpha"]).expand(n, -1)
        b = f(s["beta"]) if case["delta"] else None
        off = (s["offsets"] if op == "attention" else torch.arange(n + 1, device="cuda")).long()
        lens = (off[1:] - off[:-1]).tolist()
        order = sorted(range(len(lens)), key=lambda i: -lens[i])      # live sequences first
        S, o = f(s["state"])[order], torch.empty_like(v)
        start = off[:-1][order]
        for t in range(max(lens)):
            live = sum(m > t for m in lens)
            r = start[:live] + t
            kt = k[r][..., :, None]
            Sd = a[r][..., None, None] * S[:live]
            u = v[r]
            if b is not None:
                u = b[r][..., None] * (u - (Sd * kt).sum(2))
            S[:live] = Sd + kt * u[..., None, :]
            o[r] = (S[:live] * q[r][..., :, None]).sum(2)
        out = torch.empty_like(S)
        out[order] = S
        return o, out
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        parts = cols // (case["group"] or cols)
        norm = lambda v: v / torch.sqrt((v ** 2).sum(-1, keepdim=True) / v.shape[-1] + EPS)  # noqa: E731
        h = f(s["x"])
        act = None if s["gate"] is None else f(s["gate"]) * torch.sigmoid(f(s["gate"]))
        if case["gate"] == "before":
            h = h * act
        h = (norm(h.reshape(rows, parts, -1)) * f(s["weight"])).reshape(rows, cols)
        if case["gate"] == "after":
            h = h * act
        if case["residual"]:
            h = f(s["residual"]) + RESIDUAL_SCALE * h
        y = norm(h) * f(s["next_weight"]) if case["next"] else h
        if case["out"] == "e4m3":
            scale = y.abs().amax(1, keepdim=True) / 448
            v = torch.where(scale > 0, y / scale, torch.zeros_like(y))
            # e4m3: three mantissa bits, exponents from -6
            step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -12))), min=-6.0) - 3)
            y = (torch.round(v / step) * step, scale)
        return (y, h) if case["residual"] else y
    if case["m"] * case["n"] * case["k"] > 1 << 38:      # whole numbers, products and sums of which 64 bits hold exactly
        return torch.cat([_exact_w8(s, slice(i, i + 512)) for i in range(0, case["m"], 512)])
    return _exact_w8(s, slice(None))


def _exact_w8(s, rows):
    y = torch.matmul(s["x"][rows].double(), s["codes"].double().t())
    y *= s["x_scale"][rows].double()
    y *= s["w_scale"].double()
    if s["bias"] is not None:
        y += s["bias"].double()
    return y
