"""Cases that measure the gated delta rule (whole sequences forward and backward, and one token at a time) and layer
normalisation (forward, and backward with the sums over rows that its weight and bias get).

``run`` computes a case with elementary torch operations in float32, or, where ``own`` is true, with the calls of
``cnn_convolution_forward_amd.binding``.  ``exact`` is the definition in float64: the delta rule token by token.
"""
import math
import random

import torch

own = False

BLOCK = 64          # tokens between two saved states
UNIT_EPS = 1e-6     # added to a row's sum of squares where q and k are brought to unit length
NORM_EPS = 1e-5


# ---- the cases ---------------------------------------------------------------

def listed():
    return [
        # training on whole batches: 8 sequences of 2048 tokens through 16 heads of 128, a block of width 2048; states saved
        {"name": "delta fwd train", "op": "delta_fwd", "dtype": "bf16", "B": 8, "T": 2048, "Hk": 16, "Hv": 16, "Dk": 128, "Dv": 128,
         "unit": True, "states": True},
        {"name": "delta bwd train", "op": "delta_bwd", "dtype": "bf16", "B": 8, "T": 2048, "Hk": 16, "Hv": 16, "Dk": 128, "Dv": 128, "unit": True},
        # one long prompt read before answering: a single sequence, so few heads' chains of blocks
        {"name": "delta fwd long", "op": "delta_fwd", "dtype": "bf16", "B": 1, "T": 32768, "Hk": 8, "Hv": 8, "Dk": 128, "Dv": 128,
         "unit": True, "states": False},
        # documents of odd lengths (an empty one and one of a single token among them) packed into one row of tokens; two value
        # heads share a query and key head; odd widths
        {"name": "delta fwd packed f32", "op": "delta_fwd", "dtype": "f32", "B": 9, "T": 0, "tokens": 5003, "Hk": 3, "Hv": 6, "Dk": 72, "Dv": 99,
         "unit": False, "states": False},
        {"name": "delta bwd packed", "op": "delta_bwd", "dtype": "bf16", "B": 9, "T": 0, "tokens": 5003, "Hk": 4, "Hv": 8, "Dk": 64, "Dv": 96, "unit": True},
        # one new token for each of 64 sequences that are being answered, and for a single one
        {"name": "delta step", "op": "delta_step", "dtype": "bf16", "B": 64, "Hk": 16, "Hv": 16, "Dk": 128, "Dv": 128, "unit": True},
        {"name": "delta step one", "op": "delta_step", "dtype": "bf16", "B": 1, "Hk": 16, "Hv": 16, "Dk": 128, "Dv": 128, "unit": True},
        # the norm in front of such a block, in training
        {"name": "norm fwd train", "op": "norm_fwd", "dtype": "bf16", "rows": 16384, "C": 2048},
        {"name": "norm bwd train", "op": "norm_bwd", "dtype": "bf16", "rows": 16384, "C": 2048},
        # a norm over each head of 128 channels
        {"name": "norm bwd heads", "op": "norm_bwd", "dtype": "bf16", "rows": 131072, "C": 128},
        # tokens being answered, and packed documents in float32 of odd width
        {"name": "norm fwd few", "op": "norm_fwd", "dtype": "bf16", "rows": 64, "C": 2048},
        {"name": "norm bwd odd f32", "op": "norm_bwd", "dtype": "f32", "rows": 5003, "C": 999},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "delta_step", "norm_fwd", "norm_bwd"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op.startswith("norm"):
        C = _log(rng, 16, 16384)
        C = C if rng.random() < 0.4 else max(16, C // 8 * 8)
        most = 16384 * 2048 // (2 if case["dtype"] == "f32" else 1)
        return {**case, "rows": _log(rng, 1, most // C), "C": C}
    Hk, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 4])
    Hk = max(1, min(Hk, 16 // group))
    Dk, Dv = (rng.choice([32, 64, 64, 96, 128, 128, 128]) if rng.random() < 0.7 else rng.randint(8, 128) for _ in range(2))
    case.update(Hk=Hk, Hv=Hk * group, Dk=Dk, Dv=Dv, unit=rng.random() < 0.6)
    if op == "delta_step":
        return {**case, "B": _log(rng, 1, 64)}
    most = 16384 * 16 // (2 if case["dtype"] == "f32" else 1)
    tokens = _log(rng, 16, min(32768, most // case["Hv"]))
    case["B"] = min(tokens, _log(rng, 1, 32))
    if rng.random() < 0.35:
        case.update(T=0, tokens=tokens)
    else:
        case["T"] = max(1, tokens // case["B"])
    if op == "delta_fwd":
        case["states"] = case["T"] > 0 and rng.random() < 0.5
    return case


def lengths(case):
    """The lengths of the sequences: all T, or odd ones that add up to `tokens`, an empty one and one of one token among them."""
    if case["T"]:
        return [case["T"]] * case["B"]
    n, left = case["B"], case["tokens"]
    rng = random.Random(1000 * n + left)
    cuts = sorted(rng.randrange(left + 1) for _ in range(n - 1))
    got = [b - a for a, b in zip([0] + cuts, cuts + [left])]
    if n > 3:
        k = max(range(2, n), key=got.__getitem__)
        got[k] += got[0] + got[1] - 1
        got[0], got[1] = 0, 1
        if got[k] < 0:
            got[k], got[1] = 0, got[1] + got[k]
    return got


def work(case):
    op = case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    if op.startswith("norm"):
        n, rows, C = case["rows"] * case["C"], case["rows"], case["C"]
        if op == "norm_fwd":
            return {"bytes": 2 * n * e + 8 * rows + 8 * C, "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * rows + 12 * C, "flops": 14 * n}
    Hk, Hv, Dk, Dv, B = (case[k] for k in ("Hk", "Hv", "Dk", "Dv", "B"))
    lens = [1] * B if op == "delta_step" else lengths(case)
    n, state = sum(lens), Hv * Dk * Dv
    rows = n * (2 * Hk * Dk + 2 * Hv * Dv) * e + n * 8 * Hv
    # decay of the state, what it holds at k, the new outer product, what it holds at q
    if op != "delta_bwd":
        saved = sum(-(-v // BLOCK) for v in lens) * state * 4 if case.get("states") else 0
        return {"bytes": rows + 8 * B * state + saved, "flops": 7 * n * state}
    saved = sum(-(-v // BLOCK) for v in lens) * state * 4
    return {"bytes": rows + n * (2 * Hk * Dk + Hv * Dv) * e + n * 8 * Hv + 8 * B * state + saved, "flops": 20 * n * state}


# ---- inputs ------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    op = case["op"]
    st = {"case": case, "op": op}
    if op.startswith("norm"):
        rows, C = case["rows"], case["C"]
        # rows of a residual stream: each with an offset and a size of its own
        st["x"] = (normal(rows, C) * (0.5 + uniform(rows, 1)) + normal(rows, 1, std=0.5)).to(dt)
        st["weight"], st["bias"] = 1 + normal(C, std=0.2), normal(C, std=0.2)
        if op == "norm_bwd":
            st["dy"] = normal(rows, C, dtype=dt)
            xf = st["x"].double()
            st["mean"] = xf.mean(1).float()
            st["rstd"] = (1 / torch.sqrt((xf - xf.mean(1, keepdim=True)).square().mean(1) + NORM_EPS)).float()
        return st
    B, Hk, Hv, Dk, Dv = (case[k] for k in ("B", "Hk", "Hv", "Dk", "Dv"))
    step = op == "delta_step"
    lens = [1] * B if step else lengths(case)
    n = sum(lens)
    packed = not step and not case["T"]
    rows = (n,) if packed or step else (B, case["T"])
    st.update(n=n, lens=lens, packed=packed, max_len=max(lens), scale=1 / math.sqrt(Dk), offsets=None)
    first = [0]
    for v in lens:
        first.append(first[-1] + v)
    st["first"] = first[:-1]
    if packed:
        st["offsets"] = torch.tensor(first, dtype=torch.int32, device="cuda")
    # activations of a convolution in front of them; where the call does not bring them to unit length, they are near it already
    std = 1.0 if case["unit"] else 1 / math.sqrt(Dk)
    st["q"], st["k"], st["v"] = normal(*rows, Hk, Dk, dtype=dt, std=std), normal(*rows, Hk, Dk, dtype=dt, std=std), normal(*rows, Hv, Dv, dtype=dt)
    # decays: heads that remember for hundreds of tokens and heads that forget within a few
    rate = torch.exp(math.log(0.003) + uniform(Hv) * math.log(300.0))
    st["g"] = -rate * torch.nn.functional.softplus(normal(*rows, Hv))
    st["beta"] = torch.sigmoid(normal(*rows, Hv))
    st["s"] = normal(B, Hv, Dk, Dv, std=0.1)
    if op == "delta_bwd":
        st["dy"] = normal(*rows, Hv, Dv, dtype=dt)
        st["ds"] = normal(B, Hv, Dk, Dv, std=0.1)
        # the states that a forward pass saved
        st["saved"] = _delta_blocks(st, _delta_read(st))[2]
    return st


# ---- one pass ----------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    from cnn_convolution_forward_amd import binding as B
    op = st["op"]
    if op == "norm_fwd":
        return dict(zip(("y", "mean", "rstd"), B.layer_norm(st["x"], st["weight"], st["bias"], eps=NORM_EPS, with_stats=True)))
    if op == "norm_bwd":
        return dict(zip(("dx", "dweight", "dbias"), B.layer_norm_backward(st["x"], st["weight"], st["dy"], st["mean"], st["rstd"])))
    data = (st["q"], st["k"], st["v"], st["g"], st["beta"])
    opts = {"scale": st["scale"], "unit": st["case"]["unit"], "eps": UNIT_EPS}
    if op == "delta_step":
        return {"y": B.delta_rule_step(*data, st["s"], **opts), "s": st["s"]}
    if st["packed"]:
        opts.update(offsets=st["offsets"], max_len=st["max_len"])
    if op == "delta_fwd":
        got = B.delta_rule(*data, s0=st["s"], with_states=st["case"]["states"], **opts)
        return dict(zip(("y", "s", "saved"), got))
    got = B.delta_rule_backward(*data, st["dy"], st["saved"], ds=st["ds"], **opts)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), got))


def _run_plain(st):
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "delta_fwd": _delta_fwd, "delta_bwd": _delta_bwd, "delta_step": _delta_step}[st["op"]](st)


def _norm_fwd(st):
    x = st["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt(c.square().mean(1) + NORM_EPS)
    return {"y": (c * rstd[:, None] * st["weight"] + st["bias"]).to(st["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_bwd(st):
    x, dy, r = st["x"].float(), st["dy"].float(), st["rstd"][:, None]
    xh = (x - st["mean"][:, None]) * r
    wdy = dy * st["weight"]
    dx = r * (wdy - wdy.mean(1, keepdim=True) - xh * (wdy * xh).mean(1, keepdim=True))
    return {"dx": dx.to(st["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _unit(st, x):
    """x with rows of unit length where the case asks for it, and the factor of each row."""
    f = 1 / torch.sqrt(x.square().sum(-1, keepdim=True) + UNIT_EPS) if st["case"]["unit"] else torch.ones_like(x[..., :1])
    return x * f, f


def _delta_step(st):
    case = st["case"]
    group = case["Hv"] // case["Hk"]
    q, k = (_unit(st, st[n].float())[0].repeat_interleave(group, 1) for n in ("q", "k"))
    S = st["s"] * torch.exp(st["g"])[..., None, None]
    u = st["beta"][..., None] * (st["v"].float() - (S * k[..., None]).sum(2))
    S = S + k[..., None] * u[:, :, None]
    st["s"].copy_(S)
    return {"y": (st["scale"] * (S * q[..., None]).sum(2)).to(st["v"].dtype), "s": st["s"]}


def _places(st):
    """The row of each place of the padded layout (B, blocks * 64), and whether there is one."""
    N = -(-st["max_len"] // BLOCK)
    t = torch.arange(N * BLOCK, device="cuda")
    lens, first = torch.tensor(st["lens"], device="cuda"), torch.tensor(st["first"], device="cuda")
    return first[:, None] + t, t < lens[:, None], N


def _spread(st, x, where):
    """Rows of a tensor (..., H, D) as (B, H, blocks, 64, D) in float32, zeros where there is no row."""
    rows, on, N = where
    x = x.reshape(st["n"], *x.shape[-2:]).float()
    x = x[rows.clamp(max=max(st["n"] - 1, 0))] * on[..., None, None]
    return x.reshape(x.shape[0], N, BLOCK, *x.shape[2:]).permute(0, 3, 1, 2, 4).contiguous()


def _gather(st, x, where, dtype):
    """The reverse: (B, H, blocks, 64, D) as rows (n, H, D)."""
    x = x.permute(0, 2, 3, 1, 4)
    x = x.reshape(x.shape[0], -1, *x.shape[3:])[where[1]]
    return x.to(dtype)


def _delta_read(st):
    """What blocks of 64 tokens make of the inputs before any state is known."""
    case, d = st["case"], {}
    group = case["Hv"] // case["Hk"]
    d["where"] = w = _places(st)
    q, k = (_spread(st, st[n], w) for n in ("q", "k"))
    (d["q"], d["fq"]), (d["k"], d["fk"]) = ([t.repeat_interleave(group, 1) for t in _unit(st, x)] for x in (q, k))
    d["v"] = _spread(st, st["v"], w)
    d["beta"] = _spread(st, st["beta"][..., None], w)
    G = torch.cumsum(_spread(st, st["g"][..., None], w)[..., 0].double(), -1)
    diff = G[..., :, None] - G[..., None, :]
    i = torch.arange(BLOCK, device="cuda")
    low = i[:, None] >= i
    d["D"] = torch.where(low, torch.exp(torch.where(low, diff, torch.zeros((), device="cuda", dtype=diff.dtype))).float(), torch.zeros((), device="cuda"))
    d["E"], d["F"] = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    strict = d["D"] * (i[:, None] > i)
    A = d["beta"] * strict * (d["k"] @ d["k"].transpose(-1, -2).contiguous())
    T = torch.zeros_like(A)
    T[..., 0, 0] = 1
    for r in range(1, BLOCK):       # rows of (I + A)^-1
        T[..., r:r + 1, :] = -(A[..., r:r + 1, :r] @ T[..., :r, :])
        T[..., r, r] = 1
    d["T"] = T
    d["P"] = st["scale"] * d["D"] * (d["q"] @ d["k"].transpose(-1, -2).contiguous())
    d["strict"] = strict
    return d


def _delta_blocks(st, d):
    """Outputs, the last state, and the states in front of the blocks; block after block."""
    S, N = st["s"], d["where"][2]
    lens = torch.tensor(st["lens"], device="cuda")
    kF = (d["k"] * d["F"]).transpose(-1, -2).contiguous()
    out, saved = [], []
    for n in range(N):
        saved.append(torch.where((n * BLOCK < lens)[:, None, None, None], S, torch.zeros((), device="cuda")))
        u = d["T"][:, :, n] @ (d["beta"][:, :, n] * (d["v"][:, :, n] - d["E"][:, :, n] * (d["k"][:, :, n] @ S)))
        out.append(st["scale"] * d["E"][:, :, n] * (d["q"][:, :, n] @ S) + d["P"][:, :, n] @ u)
        S = S * d["E"][:, :, n, -1:] + kF[:, :, n] @ u
    if not N:
        return d["v"], S.clone(), S.new_zeros(S.shape[0], 0, *S.shape[1:])
    return torch.stack(out, 2), S, torch.stack(saved, 1)


def _delta_fwd(st):
    d = _delta_read(st)
    y, S, saved = _delta_blocks(st, d)
    got = {"y": _gather(st, y, d["where"], st["v"].dtype).reshape(st["v"].shape), "s": S}
    if st["case"]["states"]:
        got["saved"] = saved
    return got


def _delta_bwd(st):
    case, d, s = st["case"], _delta_read(st), st["scale"]
    group, dt, where = case["Hv"] // case["Hk"], st["v"].dtype, d["where"]
    t = lambda x: x.transpose(-1, -2).contiguous()
    S0 = st["saved"].transpose(1, 2).contiguous()
    do = _spread(st, st["dy"], where)
    N = where[2]
    kE, qE = t(d["k"] * d["E"] * d["beta"]), t(s * d["q"] * d["E"])
    Tt, Pdo = t(d["T"]), t(d["P"]) @ do
    dS, ends, zs = st["ds"], [None] * N, [None] * N
    for n in range(N - 1, -1, -1):
        ends[n] = dS
        z = Tt[:, :, n] @ (Pdo[:, :, n] + d["F"][:, :, n] * (d["k"][:, :, n] @ dS))
        zs[n] = z
        dS = dS * d["E"][:, :, n, -1:] + qE[:, :, n] @ do[:, :, n] - kE[:, :, n] @ z
    dSL, Z = torch.stack(ends, 2), torch.stack(zs, 2)
    U = d["T"] @ (d["beta"] * (d["v"] - d["E"] * (d["k"] @ S0)))
    Y = s * d["D"] * (do @ t(U))
    M = -d["strict"] * (Z @ t(U))               # times beta of its row
    dq = s * d["E"] * (do @ t(S0)) + Y @ d["k"]
    read = M @ d["k"] - d["E"] * (Z @ t(S0))     # times beta of its row
    write = t(Y) @ d["q"] + t(M * d["beta"]) @ d["k"] + d["F"] * (U @ t(dSL))
    at = (d["k"] * read).sum(-1, keepdim=True)
    dbeta = (Z * d["v"]).sum(-1, keepdim=True) + at
    dG = ((d["q"] * dq).sum(-1, keepdim=True) + d["beta"] * at - (d["k"] * write).sum(-1, keepdim=True)).double()
    kept = d["E"][..., -1, 0].double() * (S0 * dSL).sum((-1, -2), dtype=torch.float64)
    kept = kept + (d["F"] * U * (d["k"] @ dSL)).sum((-1, -2), dtype=torch.float64)
    dg = torch.flip(torch.cumsum(torch.flip(dG, (-2,)), -2), (-2,)) + kept[..., None, None]
    dk = d["beta"] * read + write

    def back(dx, x, f):
        """Through the unit length, and summed over the value heads that share a head."""
        if case["unit"]:
            dx = f * (dx - x * (x * dx).sum(-1, keepdim=True))
        return dx.reshape(dx.shape[0], case["Hk"], group, *dx.shape[2:]).sum(2)

    rows = lambda x, like, kind=dt: _gather(st, x, where, kind).reshape(like.shape)
    return {"dq": rows(back(dq, d["q"], d["fq"]), st["q"]), "dk": rows(back(dk, d["k"], d["fk"]), st["k"]), "dv": rows(d["beta"] * Z, st["v"]),
            "dg": rows(dg, st["g"], torch.float32), "dbeta": rows(dbeta, st["beta"], torch.float32), "ds0": dS}


# ---- the definition in 64 bits -----------------------------------------------

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    f = torch.float64
    if case["op"].startswith("norm"):
        x, w = st["x"].to(f), st["weight"].to(f)
        if case["op"] == "norm_fwd":
            mean, var = x.mean(1, keepdim=True), x.var(1, keepdim=True, unbiased=False)
            rstd = torch.rsqrt(var + NORM_EPS)
            return {"y": (x - mean) * rstd * w + st["bias"].to(f), "mean": mean[:, 0], "rstd": rstd[:, 0]}
        dy, rstd = st["dy"].to(f), st["rstd"].to(f)[:, None]
        z = (x - st["mean"].to(f)[:, None]) * rstd
        e = w * dy
        C = case["C"]
        return {"dx": rstd / C * (C * e - e.sum(1, keepdim=True) - z * (e * z).sum(1, keepdim=True)), "dweight": (z * dy).sum(0), "dbias": dy.sum(0)}
    return _exact_delta(st, case)


def _exact_delta(st, case):
    """Token by token over all sequences and heads at once; a sequence that has ended keeps its state."""
    f, B, Hv, group = torch.float64, case["B"], case["Hv"], case["Hv"] // case["Hk"]
    op, top = case["op"], st["max_len"]
    raw = {n: st[n].reshape(st["n"], *st[n].shape[-2:]).to(f) for n in ("q", "k", "v")}
    raw.update({n: st[n].reshape(st["n"], Hv).to(f) for n in ("g", "beta")})
    size = {n: torch.sqrt((raw[n] ** 2).sum(-1, keepdim=True) + UNIT_EPS) if case["unit"] else torch.ones(st["n"], case["Hk"], 1, device="cuda", dtype=f)
            for n in ("q", "k")}
    q, k = ((raw[n] / size[n]).repeat_interleave(group, 1) for n in ("q", "k"))
    v, alpha, beta, scale = raw["v"], torch.exp(raw["g"]), raw["beta"], st["scale"]
    lens, at = torch.tensor(st["lens"], device="cuda"), torch.tensor(st["first"], device="cuda")
    equal = not st["packed"]
    S = (st["saved"][:, 0] if op == "delta_bwd" and top else st["s"]).to(f).clone()
    if op == "delta_bwd":
        S = torch.where((lens > 0)[:, None, None, None], S, torch.zeros((), device="cuda", dtype=f))
    y, e, before, kept, saved = torch.zeros_like(v), torch.zeros_like(v), [], [], []
    for t in range(top):
        on = slice(None) if equal else torch.nonzero(lens > t)[:, 0]
        r = at[on] + t
        if t % BLOCK == 0 and case.get("states"):
            saved.append(S.clone())
        D = S[on] * alpha[r][:, :, None, None]
        e[r] = v[r] - (D * k[r][..., None]).sum(2)
        new = D + k[r][..., None] * (beta[r][..., None] * e[r])[:, :, None]
        if op == "delta_bwd":
            before.append(D)
            kept.append((on, r))
        else:
            y[r] = scale * (new * q[r][..., None]).sum(2)
        S[on] = new
    if op != "delta_bwd":
        got = {"y": y.reshape(st["v"].shape), "s": S}
        if case.get("states"):
            got["saved"] = torch.stack(saved, 1)
        return got
    dS, dy = st["ds"].to(f).clone(), st["dy"].reshape(st["n"], Hv, -1).to(f)
    dq, dk, dv, dg, db = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(alpha), torch.zeros_like(beta)
    for t in range(top - 1, -1, -1):
        (on, r), D = kept[t], before[t]
        before[t] = None
        kr, u = k[r][..., None], beta[r][..., None] * e[r]
        new = D + kr * u[:, :, None]
        d = dS[on] + scale * q[r][..., None] * dy[r][:, :, None]
        dq[r] = scale * (new * dy[r][:, :, None]).sum(3)
        du = (d * kr).sum(2)
        db[r] = (du * e[r]).sum(2)
        de = beta[r][..., None] * du
        dv[r] = de
        dk[r] = (d * u[:, :, None]).sum(3) - (D * de[:, :, None]).sum(3)
        d = d - kr * de[:, :, None]
        dg[r] = (d * D).sum((2, 3))
        dS[on] = d * alpha[r][:, :, None, None]

    def back(dx, x, n):
        if case["unit"]:
            dx = (dx - x * (x * dx).sum(-1, keepdim=True)) / size[n].repeat_interleave(group, 1)
        return dx.reshape(st["n"], case["Hk"], group, -1).sum(2).reshape(st[n].shape)

    return {"dq": back(dq, q, "q"), "dk": back(dk, k, "k"), "dv": dv.reshape(st["v"].shape), "dg": dg.reshape(st["g"].shape),
            "dbeta": db.reshape(st["beta"].shape), "ds0": dS}
