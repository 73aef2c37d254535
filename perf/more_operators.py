"""Cases, plain forms and 64-bit definitions of further operators of hybrid models.

Three operators of layers that stand next to long convolutions and the gated
delta rule:

* ``decay``: linear attention with a decay for each head over whole sequences
  (forward, and forward + backward), equal lengths or ragged sequences packed
  in one batch row, the decay fixed for a head or given for each token;
* ``step``: the same for one new token per request, on a pool of states that
  is updated in place;
* ``layernorm``: layer norm of token rows (forward, and forward + backward with
  the reduction of the weight's and bias's gradients).

``run`` is one pass through an operator: in elementary torch operations where
``own`` is false, through the library's entry points where it is true.
``exact`` is the operator's definition in 64 bits, token by token.

Sizes follow this repository's workloads (64 x 1024 x 768, 16 x 8192 x 768,
4 x 32768 x 512), their channels taken as heads of 64 or 128.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
CHUNK = 64


# ---------------------------------------------------------------- the cases

def _layernorm(name, B, T, D, weight, wide, grad, dtype):
    return {"name": name, "op": "layernorm", "B": B, "T": T, "D": D, "weight": weight,
            "wide": wide, "grad": grad, "dtype": dtype}


def _decay(name, B, T, Hk, Hv, Dk, Dv, seqs, fixed, init, grad, dtype):
    return {"name": name, "op": "decay", "B": B, "T": T, "Hk": Hk, "Hv": Hv, "Dk": Dk, "Dv": Dv,
            "seqs": seqs, "fixed": fixed, "init": init, "grad": grad, "dtype": dtype}


def _step(name, N, pool, Hk, Hv, Dk, Dv, fixed, dtype):
    return {"name": name, "op": "step", "N": N, "pool": pool, "Hk": Hk, "Hv": Hv, "Dk": Dk,
            "Dv": Dv, "fixed": fixed, "dtype": dtype}


def listed():
    return [
        # one new token for each of 24 requests while serving: latency counts
        _layernorm("layernorm decode", 24, 1, 768, True, False, False, "bf16"),
        # prefill of the 64 x 1024 x 768 workload
        _layernorm("layernorm prefill", 64, 1024, 768, True, False, False, "bf16"),
        # a training step's norm at 16 x 8192 x 768
        _layernorm("layernorm train", 16, 8192, 768, True, False, True, "f16"),
        # training in 32 bits on an odd number of tokens and an odd width
        _layernorm("layernorm odd f32", 3, 1237, 1029, True, False, True, "f32"),
        # one request being answered: a single token against one state
        _step("step single", 1, 4, 6, 6, 128, 128, True, "bf16"),
        # a full serving batch, its states scattered over a pool, keys shared by two value heads
        _step("step batch", 192, 256, 4, 8, 128, 128, False, "bf16"),
        # a short prompt
        _decay("decay prompt", 1, 77, 6, 6, 128, 128, 0, True, True, False, "bf16"),
        # prefill of ragged prompts packed in one row, shared keys, some prompts empty or one token long
        _decay("decay ragged", 1, 9001, 4, 8, 64, 128, 23, False, True, False, "f16"),
        # the 64 x 1024 x 768 workload, six heads of 128, forward only
        _decay("decay prefill", 64, 1024, 6, 6, 128, 128, 0, True, False, False, "bf16"),
        # the 4 x 32768 x 512 workload: few rows, long sequences
        _decay("decay long", 4, 32768, 4, 4, 128, 128, 0, False, False, False, "bf16"),
        # a training step of the 64 x 1024 x 768 workload
        _decay("decay train", 64, 1024, 6, 6, 128, 128, 0, False, False, True, "bf16"),
        # training in 32 bits on an odd length, shared keys, one decay a head
        _decay("decay train f32", 2, 1501, 2, 4, 64, 64, 0, True, True, True, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    op = rng.choice(["layernorm", "layernorm", "step", "decay", "decay", "decay"])
    if op == "layernorm":
        D = _log(rng, 32, 8192)
        if rng.random() < 0.7:
            D = (D + 63) // 64 * 64
        tokens = _log(rng, 1, 90e6 / D)
        B = min(tokens, _log(rng, 1, 64))
        c = _layernorm("", B, max(1, tokens // B), D, rng.random() < 0.8, rng.random() < 0.3,
                       rng.random() < 0.5, dtype)
    elif op == "step":
        Hk = rng.randint(1, 8)
        Hv = Hk * rng.choice([1, 1, 2])
        N = _log(rng, 1, 192)
        c = _step("", N, N + rng.randint(0, 64), Hk, Hv, rng.choice([64, 96, 128, 128]),
                  rng.choice([64, 128, 128, 256]), rng.random() < 0.5, dtype)
    else:
        Hk = rng.randint(1, 6)
        Hv = Hk * rng.choice([1, 1, 2])
        Dk, Dv = rng.choice([(64, 64), (64, 128), (96, 96), (128, 128), (128, 128), (128, 256)])
        grad = rng.random() < 0.4
        B, seqs = 1, 0
        if rng.random() < 0.3:
            seqs = rng.randint(1, 40)
            T = _log(rng, 8, 16384)
        else:
            T = _log(rng, 1, 16384)
            B = _log(rng, 1, max(1, min(64, 40e6 / (T * Hv * (Dk + Dv)))))
        c = _decay("", B, T, Hk, Hv, Dk, Dv, seqs, rng.random() < 0.5, rng.random() < 0.5, grad,
                   dtype)
    del c["name"]
    return c


# --------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)


def _log_decays(gen, case, lead):
    """Log decays as trained layers have them: one a head, memories of a few tokens to
    thousands; or one a token, a head's rate times a softplus of a projection of the token."""
    Hv = case["Hv"]
    if case["fixed"]:
        return -torch.exp(torch.empty(Hv, device="cuda").uniform_(math.log(2.0 ** -12),
                                                                  math.log(0.5), generator=gen))
    rate = torch.exp(torch.empty(Hv, device="cuda").uniform_(math.log(0.003), math.log(3.0),
                                                             generator=gen))
    return -rate * torch.nn.functional.softplus(_randn(gen, *lead, Hv))


def _bounds(case, seed):
    """Bounds of the packed sequences: random cuts, some sequences empty or one token long."""
    n, T = case["seqs"], case["T"]
    gen = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, T + 1, (n - 1,), generator=gen).sort().values
    if n > 3:
        cuts[1] = cuts[0]                              # an empty sequence
        cuts[-1] = min(T, int(cuts[-2]) + 1)           # one of at most one token
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts,
                      torch.full((1,), T, dtype=torch.int64)])


def prepare(case, seed):
    gen, dt, op = _gen(seed), DTYPES[case["dtype"]], case["op"]
    s = {"case": case}
    if op == "layernorm":
        B, T, D = case["B"], case["T"], case["D"]
        # wide: x is a view of rows that hold another layer's values beside it
        x = _randn(gen, B, T, (2 if case["wide"] else 1) * D)
        # a residual stream: channels and tokens with means and sizes of their own
        x = x * (0.5 + _randn(gen, B, T, 1).abs()) + 0.5 * _randn(gen, x.shape[-1])
        s["x"] = x.to(dt)[..., :D]
        s["w"] = s["b"] = None
        if case["weight"]:
            s["w"] = 1 + 0.2 * _randn(gen, D)
            s["b"] = 0.1 * _randn(gen, D)
        if case["grad"]:
            s["dy"] = _randn(gen, B, T, D).to(dt)
        return s
    Hk, Hv, Dk, Dv = (case[x] for x in ("Hk", "Hv", "Dk", "Dv"))
    if op == "step":
        N = case["N"]
        s["q"] = _unit(_randn(gen, N, Hk, Dk)).to(dt)
        s["k"] = _unit(_randn(gen, N, Hk, Dk)).to(dt)
        s["v"] = _randn(gen, N, Hv, Dv).to(dt)
        s["g"] = _log_decays(gen, case, (N,))
        s["state"] = 0.3 * _randn(gen, case["pool"], Hv, Dk, Dv)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device="cuda")[:N]
        return s
    B, T = case["B"], case["T"]
    s["q"] = _unit(_randn(gen, B, T, Hk, Dk)).to(dt)
    s["k"] = _unit(_randn(gen, B, T, Hk, Dk)).to(dt)
    # v is a view of a projection that holds the output gate beside it
    s["v"] = _randn(gen, B, T, 2 * Hv, Dv).to(dt)[:, :, :Hv]
    s["g"] = _log_decays(gen, case, (B, T))
    s["cu"], rows = None, B
    if case["seqs"]:
        s["cu"], rows = _bounds(case, seed).to("cuda"), case["seqs"]
    s["init"] = 0.3 * _randn(gen, rows, Hv, Dk, Dv) if case["init"] else None
    if case["grad"]:
        s["do"] = _randn(gen, B, T, Hv, Dv).to(dt)
        s["dstate"] = 0.1 * _randn(gen, rows, Hv, Dk, Dv)
    return s


# ---------------------------------------------------------- the plain forms

def _plain_layernorm(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    x = s["x"].float()
    x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    y = (n if s["w"] is None else n * s["w"] + s["b"]).to(dt)
    if not case["grad"]:
        return {"y": y}
    dy = s["dy"].float()
    h = dy if s["w"] is None else dy * s["w"]
    dx = r * (h - h.mean(-1, keepdim=True) - n * (h * n).mean(-1, keepdim=True))
    return {"y": y, "dx": dx.to(dt), "dw": None if s["w"] is None else (dy * n).sum((0, 1)),
            "db": None if s["w"] is None else dy.sum((0, 1))}


def _plain_step(s):
    case, at = s["case"], s["slots"]
    group = case["Hv"] // case["Hk"]
    q = s["q"].float().repeat_interleave(group, 1)
    k = s["k"].float().repeat_interleave(group, 1)
    a = torch.exp(s["g"]).expand(case["N"], case["Hv"])
    S = s["state"][at] * a[..., None, None] + k[..., None] * s["v"].float()[..., None, :]
    o = case["Dk"] ** -0.5 * (q[..., None] * S).sum(-2)
    s["state"][at] = S
    return {"o": o.to(DTYPES[case["dtype"]]), "state": s["state"]}


def _places(s):
    """Row and column of each token where every sequence is a row, and the longest row."""
    case = s["case"]
    cu = s["cu"]
    size = cu[1:] - cu[:-1]
    row = torch.repeat_interleave(torch.arange(len(size), device=cu.device), size)
    return row, torch.arange(case["T"], device=cu.device) - cu[row], int(size.max())


def _chunked(s, at, x):
    """[B, T, H, ...] as [rows, H, chunks, CHUNK, ...], padded with zeros."""
    B, T = x.shape[:2]
    rows, most = (B, T) if at is None else (s["case"]["seqs"], at[2])
    n = -(-most // CHUNK)
    y = x.new_zeros(rows, n * CHUNK, *x.shape[2:])
    if at is None:
        y[:, :T] = x
    else:
        y[at[0], at[1]] = x[0]
    return y.unflatten(1, (n, CHUNK)).movedim(3, 1)


def _plain_forward(s, at, q, k, v, g, S):
    """The chunked form: scores within 64 tokens, a state from chunk to chunk (the recurrence
    over the chunks is the one loop).  Sums of log decays are of 64 bits."""
    case = s["case"]
    group = case["Hv"] // case["Hk"]
    q, k, v, g = (_chunked(s, at, x) for x in (q, k, v, g))
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    G = g.double().cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=G.device).tril()
    gam = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~lower, -math.inf).float())
    P = torch.matmul(q, k.transpose(-1, -2)) * gam
    inner = torch.matmul(P, v)
    eG = torch.exp(G.float())[..., None]
    end = torch.exp((G[..., -1:] - G).float())[..., None]
    N = torch.matmul((end * k).transpose(-1, -2), v)
    before = []
    for c in range(q.shape[2]):
        before.append(S)
        S = eG[:, :, c, -1:] * S + N[:, :, c]
    if before:
        inner = inner + eG * torch.matmul(q, torch.stack(before, 2))
    o = (case["Dk"] ** -0.5 * inner).movedim(1, 3).flatten(1, 2)
    return (o[:, :case["T"]] if at is None else o[at[0], at[1]][None]), S


def _plain_decay(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    at = None if s["cu"] is None else _places(s)
    rows = case["seqs"] or case["B"]
    S0 = s["init"] if s["init"] is not None else \
        torch.zeros(rows, case["Hv"], case["Dk"], case["Dv"], device="cuda")
    ins = [x.float() for x in (s["q"], s["k"], s["v"])] + [s["g"], S0]
    if case["grad"]:
        ins = [x.detach().requires_grad_() for x in ins]
    q, k, v, g, S0 = ins
    o, S = _plain_forward(s, at, q, k, v, g.expand(case["B"], case["T"], case["Hv"]), S0)
    if not case["grad"]:
        return {"o": o.to(dt), "state": S}
    d = torch.autograd.grad([o, S], ins, [s["do"].float(), s["dstate"]])
    return {"o": o.detach().to(dt), "state": S.detach(), "dq": d[0].to(dt), "dk": d[1].to(dt),
            "dv": d[2].to(dt), "dg": d[3], "dinit": d[4] if s["init"] is not None else None}


# ------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if not own:
        return {"layernorm": _plain_layernorm, "step": _plain_step,
                "decay": _plain_decay}[case["op"]](s)
    from fft_long_convolution_amd.decay import DecayAttention, LayerNorm
    if case["op"] == "layernorm":
        op = LayerNorm(case["D"], eps=EPS, dtype=case["dtype"])
        y = op.forward(s["x"], s["w"], s["b"])
        if not case["grad"]:
            return {"y": y}
        dx, dw, db = op.backward(s["x"], s["dy"], s["w"], s["b"])
        return {"y": y, "dx": dx, "dw": dw, "db": db}
    op = DecayAttention(case["Dk"], case["Dv"], dtype=case["dtype"])
    if case["op"] == "step":
        o = op.step(s["q"], s["k"], s["v"], s["g"], s["state"], slots=s["slots"])
        return {"o": o, "state": s["state"]}
    args = (s["q"], s["k"], s["v"], s["g"])
    o, S = op.forward(*args, initial_state=s["init"], cu_seqlens=s["cu"])
    if not case["grad"]:
        return {"o": o, "state": S}
    dq, dk, dv, dg, dinit = op.backward(*args, s["do"], d_final_state=s["dstate"],
                                        initial_state=s["init"], cu_seqlens=s["cu"])
    return {"o": o, "state": S, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dinit": dinit}


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "layernorm":
        x = case["B"] * case["T"] * case["D"]
        # forward: x in, y out; backward: x and dy in, dx out
        return {"bytes": x * e * (5 if case["grad"] else 2) + 8 * case["D"],
                "flops": x * (24 if case["grad"] else 8)}
    Hk, Hv, Dk, Dv = (case[x] for x in ("Hk", "Hv", "Dk", "Dv"))
    gates = 0 if case["fixed"] else 4 * Hv
    token = (2 * Hk * Dk + 2 * Hv * Dv) * e + gates
    if case["op"] == "step":
        return {"bytes": case["N"] * (token + 8 * Hv * Dk * Dv + 8),
                "flops": case["N"] * Hv * 5 * Dk * Dv}
    n, rows = case["B"] * case["T"], case["seqs"] or case["B"]
    states = rows * Hv * Dk * Dv * 4 * (2 if case["init"] else 1)
    # products of a token and head: with the state and into it, and the recurrence needs no more
    flops = n * Hv * 4 * Dk * Dv
    if not case["grad"]:
        return {"bytes": n * token + states, "flops": flops}
    # forward, then inputs and do in, the gradients out
    more = (4 * Hk * Dk + 3 * Hv * Dv) * e + 2 * gates
    return {"bytes": n * (token + more) + 2 * states, "flops": 3.5 * flops}


# ---------------------------------------- the definitions, in 64 bits

def _exact_layernorm(s):
    case = s["case"]
    D, shape = case["D"], s["x"].shape
    w = torch.ones(D, dtype=torch.float64, device="cuda") if s["w"] is None else s["w"].double()
    y, dx = (torch.empty(shape, dtype=torch.float64, device="cuda").view(-1, D) for _ in "yx")
    dw, db = torch.zeros_like(w), torch.zeros_like(w)
    x, dy = s["x"].reshape(-1, D), s["dy"].view(-1, D) if case["grad"] else None
    for i in range(0, x.shape[0], 1 << 16):
        z = x[i:i + (1 << 16)].double()
        var, mean = torch.var_mean(z, -1, correction=0, keepdim=True)
        sd = torch.sqrt(var + EPS)
        n = (z - mean) / sd
        y[i:i + (1 << 16)] = w * n if s["b"] is None else w * n + s["b"].double()
        if case["grad"]:
            d = dy[i:i + (1 << 16)].double()
            dw += (d * n).sum(0)
            db += d.sum(0)
            # y depends on x through x - mean and through sd: d sd / dx = (x - mean) / (D sd)
            c = d * w / sd
            dsd = -(c * n).sum(-1, keepdim=True)
            dx[i:i + (1 << 16)] = c - c.mean(-1, keepdim=True) + dsd * n / D
    out = {"y": y.view(shape)}
    if case["grad"]:
        out.update(dx=dx.view(shape), dw=None if s["w"] is None else dw,
                   db=None if s["w"] is None else db)
    return out


def _exact_step(s):
    case, at = s["case"], s["slots"]
    head = torch.arange(case["Hv"], device="cuda") // (case["Hv"] // case["Hk"])
    q, k, v = s["q"].double()[:, head], s["k"].double()[:, head], s["v"].double()
    state = s["state"].double()
    S = torch.exp(s["g"].double()).expand(case["N"], -1)[..., None, None] * state[at]
    S = S + torch.einsum("nhk,nhv->nhkv", k, v)
    state[at] = S
    return {"o": case["Dk"] ** -0.5 * torch.einsum("nhkv,nhk->nhv", S, q), "state": state}


def _exact_decay(s):
    """Token by token: S_t = e^g_t S_{t-1} + k_t v_t^T, o_t = c S_t^T q_t, and its adjoint."""
    case = s["case"]
    B, T, Hk, Hv, Dk, Dv = (case[x] for x in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    head = torch.arange(Hv, device="cuda") // (Hv // Hk)
    c = Dk ** -0.5
    if s["cu"] is None:
        spans = [(b, 0, T) for b in range(B)]
    else:
        cu = s["cu"].tolist()
        spans = [(0, a, z) for a, z in zip(cu[:-1], cu[1:])]
    rows, most = len(spans), max(z - a for _, a, z in spans)
    if most * (26 if case["grad"] else 6) > 1200000:
        return None

    def by_time(x):
        y = torch.zeros(most, rows, *x.shape[2:], dtype=torch.float64, device="cuda")
        for r, (b, a, z) in enumerate(spans):
            y[:z - a, r] = x[b, a:z].double()
        return y

    def by_row(y):
        x = torch.zeros(B, T, *y.shape[2:], dtype=torch.float64, device="cuda")
        for r, (b, a, z) in enumerate(spans):
            x[b, a:z] = y[:z - a, r]
        return x

    q, k, v = (by_time(s[x]) for x in ("q", "k", "v"))
    decay = torch.exp(by_time(s["g"].expand(B, T, Hv)))[..., None, None]
    # behind a sequence's end nothing may change: tokens of zeros that decay nothing
    q, k = q[:, :, head], k[:, :, head]
    S = s["init"].double() if s["init"] is not None else \
        torch.zeros(rows, Hv, Dk, Dv, dtype=torch.float64, device="cuda")
    o, every, kept = torch.zeros_like(v), 128, []
    for t in range(most):
        if t % every == 0:
            kept.append(S)
        S = torch.addcmul(decay[t] * S, k[t][..., None], v[t][..., None, :])
        o[t] = c * torch.matmul(q[t][..., None, :], S)[..., 0, :]
    out = {"o": by_row(o), "state": S}
    if not case["grad"]:
        return out
    do, dS = by_time(s["do"]), s["dstate"].double()
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    dg = torch.zeros(most, rows, Hv, dtype=torch.float64, device="cuda")
    for first in reversed(range(0, most, every)):
        S, seen = kept[first // every], []
        for t in range(first, min(most, first + every)):
            old = decay[t] * S
            S = torch.addcmul(old, k[t][..., None], v[t][..., None, :])
            seen.append((S, old))
        for t in reversed(range(first, first + len(seen))):
            S, old = seen.pop()
            dq[t] = c * torch.matmul(S, do[t][..., None])[..., 0]
            dS = torch.addcmul(dS, q[t][..., None], do[t][..., None, :], value=c)
            dk[t] = torch.matmul(dS, v[t][..., None])[..., 0]
            dv[t] = torch.matmul(k[t][..., None, :], dS)[..., 0, :]
            dg[t] = (dS * old).sum((-1, -2))
            dS = decay[t] * dS
    shared = lambda x: by_row(x).unflatten(2, (Hk, Hv // Hk)).sum(3)  # noqa: E731
    dg = by_row(dg)
    out.update(dq=shared(dq), dk=shared(dk), dv=by_row(dv),
               dg=dg.sum((0, 1)) if case["fixed"] else dg,
               dinit=dS if s["init"] is not None else None)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"layernorm": _exact_layernorm, "step": _exact_step,
            "decay": _exact_decay}[case["op"]](s)
