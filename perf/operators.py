"""Cases, plain forms and 64-bit definitions of the token-mixer operators.

Three operators of layers that stand next to long convolutions in hybrid
models:

* ``norm``: norms of queries and keys for each head with the position
  rotation in the same pass (forward, and forward + backward);
* ``delta``: the gated delta rule over whole sequences (forward, and forward +
  backward), equal lengths or ragged sequences packed in one batch row;
* ``step``: the gated delta rule for one new token per request, on a pool of
  states that is updated in place.

``run`` is one pass through an operator: in elementary torch operations in 32
bits where ``own`` is false, through the library's entry points where it is
true.  ``exact`` is the operator's definition in 64 bits, token by token.

Sizes follow this repository's workloads (64 x 1024 x 768, 16 x 8192 x 768,
4 x 32768 x 512), their channels taken as heads of 64 or 128.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
CHUNK = 64


# ---------------------------------------------------------------- the cases

def _norm(name, B, T, Hq, Hk, D, R, kind, weight, interleaved, grad, dtype):
    return {"name": name, "op": "norm", "B": B, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R,
            "kind": kind, "weight": weight, "interleaved": interleaved, "grad": grad,
            "dtype": dtype}


def _delta(name, B, T, Hk, Hv, Dk, Dv, seqs, init, grad, dtype):
    return {"name": name, "op": "delta", "B": B, "T": T, "Hk": Hk, "Hv": Hv, "Dk": Dk,
            "Dv": Dv, "seqs": seqs, "init": init, "grad": grad, "dtype": dtype}


def _step(name, N, pool, Hk, Hv, Dk, Dv, dtype):
    return {"name": name, "op": "step", "N": N, "pool": pool, "Hk": Hk, "Hv": Hv, "Dk": Dk,
            "Dv": Dv, "dtype": dtype}


def listed():
    return [
        # one new token for each of 24 requests while serving: latency counts
        _norm("norm decode", 24, 1, 6, 6, 128, 128, "rms", True, False, False, "bf16"),
        # prefill of the 64 x 1024 x 768 workload, six heads of 128
        _norm("norm prefill", 64, 1024, 6, 6, 128, 128, "l2", False, False, False, "bf16"),
        # a training step's norms at 16 x 8192 x 768 with shared keys, part of each head rotated
        _norm("norm train", 16, 8192, 12, 4, 64, 32, "rms", True, True, True, "f16"),
        # evaluation in 32 bits of an odd number of tokens, heads of 96
        _norm("norm odd f32", 3, 1237, 8, 8, 96, 96, "rms", True, False, True, "f32"),
        # one request being answered: a single token against one state
        _step("step single", 1, 4, 6, 6, 128, 128, "bf16"),
        # a full serving batch, its states scattered over a pool, keys shared by two value heads
        _step("step batch", 192, 256, 4, 8, 128, 128, "bf16"),
        # a short prompt
        _delta("delta prompt", 1, 77, 6, 6, 128, 128, 0, True, False, "bf16"),
        # prefill of ragged prompts packed in one row, shared keys, some prompts empty or one token long
        _delta("delta ragged", 1, 9001, 4, 8, 64, 128, 23, True, False, "f16"),
        # the 64 x 1024 x 768 workload, six heads of 128, forward only
        _delta("delta prefill", 64, 1024, 6, 6, 128, 128, 0, False, False, "bf16"),
        # the 4 x 32768 x 512 workload: few rows, long sequences
        _delta("delta long", 4, 32768, 4, 4, 128, 128, 0, False, False, "bf16"),
        # a training step of the 64 x 1024 x 768 workload
        _delta("delta train", 64, 1024, 6, 6, 128, 128, 0, False, True, "bf16"),
        # training in 32 bits on an odd length, shared keys
        _delta("delta train f32", 2, 1501, 2, 4, 64, 64, 0, True, True, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    op = rng.choice(["norm", "norm", "step", "delta", "delta", "delta"])
    if op == "norm":
        D = rng.choice([64, 96, 128, 128, 256])
        inter = rng.random() < 0.4
        R = rng.choice([0, 16, 32, D // 2, D, D])
        Hk = rng.randint(1, 8)
        Hq = Hk * rng.choice([1, 1, 2, 4])
        grad = rng.random() < 0.5
        kind = rng.choice(["rms", "rms", "l2"])
        tokens = _log(rng, 1, 90e6 / (D * (Hq + Hk)))
        B = min(tokens, _log(rng, 1, 64))
        c = _norm("", B, max(1, tokens // B), Hq, Hk, D, R, kind, kind == "rms", inter, grad,
                  dtype)
    elif op == "step":
        Hk = rng.randint(1, 8)
        Hv = Hk * rng.choice([1, 1, 2])
        N = _log(rng, 1, 192)
        c = _step("", N, N + rng.randint(0, 64), Hk, Hv, rng.choice([64, 96, 128, 128]),
                  rng.choice([64, 128, 128, 256]), dtype)
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
        c = _delta("", B, T, Hk, Hv, Dk, Dv, seqs, rng.random() < 0.5, grad, dtype)
    del c["name"]
    return c


# --------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _unit(x):
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)


def _gates(gen, lead, Hv):
    """Log decays and write strengths as a trained layer has them: each head with a rate of its
    own over three decades, a softplus of a projection of the token, a sigmoid."""
    rate = torch.exp(torch.empty(Hv, device="cuda").uniform_(math.log(0.003), math.log(3.0),
                                                             generator=gen))
    g = -rate * torch.nn.functional.softplus(_randn(gen, *lead, Hv))
    beta = torch.sigmoid(1.5 * _randn(gen, *lead, Hv))
    return g, beta


def _lengths(case, seed):
    """Bounds of the packed sequences: random cuts, so some sequences are empty or one token
    long."""
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
    if op == "norm":
        B, T, Hq, Hk, D, R = (case[x] for x in ("B", "T", "Hq", "Hk", "D", "R"))
        # q, k and v come out of one projection: q and k are views of its columns
        qkv = (1.5 * _randn(gen, B, T, Hq + 2 * Hk, D)).to(dt)
        s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        s["wq"] = s["wk"] = s["cos"] = s["sin"] = s["pos"] = None
        if case["weight"]:
            s["wq"] = 1 + 0.2 * _randn(gen, D)
            s["wk"] = 1 + 0.2 * _randn(gen, D)
        if R:
            P = 8192
            freq = 10000.0 ** (-torch.arange(R // 2, dtype=torch.float64, device="cuda") * 2 / R)
            ang = torch.arange(P, dtype=torch.float64, device="cuda")[:, None] * freq
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            first = torch.randint(0, P - T + 1, (B, 1), generator=gen, device="cuda") \
                if T < P else torch.zeros(B, 1, dtype=torch.int64, device="cuda")
            s["pos"] = (first + torch.arange(T, device="cuda")) % P
        if case["grad"]:
            s["dq"] = _randn(gen, B, T, Hq, D).to(dt)
            s["dk"] = _randn(gen, B, T, Hk, D).to(dt)
        return s
    Hk, Hv, Dk, Dv = (case[x] for x in ("Hk", "Hv", "Dk", "Dv"))
    if op == "step":
        N = case["N"]
        s["q"] = _unit(_randn(gen, N, Hk, Dk)).to(dt)
        s["k"] = _unit(_randn(gen, N, Hk, Dk)).to(dt)
        s["v"] = _randn(gen, N, Hv, Dv).to(dt)
        s["g"], s["beta"] = _gates(gen, (N,), Hv)
        s["state"] = 0.3 * _randn(gen, case["pool"], Hv, Dk, Dv)
        s["slots"] = torch.randperm(case["pool"], generator=gen, device="cuda")[:N]
        return s
    B, T = case["B"], case["T"]
    s["q"] = _unit(_randn(gen, B, T, Hk, Dk)).to(dt)
    s["k"] = _unit(_randn(gen, B, T, Hk, Dk)).to(dt)
    # v is a view of a projection that holds the output gate beside it
    s["v"] = _randn(gen, B, T, 2 * Hv, Dv).to(dt)[:, :, :Hv]
    s["g"], s["beta"] = _gates(gen, (B, T), Hv)
    s["cu"], rows = None, B
    if case["seqs"]:
        s["cu"], rows = _lengths(case, seed).to("cuda"), case["seqs"]
    s["init"] = 0.3 * _randn(gen, rows, Hv, Dk, Dv) if case["init"] else None
    if case["grad"]:
        s["do"] = _randn(gen, B, T, Hv, Dv).to(dt)
        s["dstate"] = 0.1 * _randn(gen, rows, Hv, Dk, Dv)
    return s


# ---------------------------------------------------------- the plain forms

def _rotate(x, cos, sin, R, interleaved):
    if not R:
        return x
    c, n = cos[:, :, None], sin[:, :, None]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_norm(s):
    case = s["case"]
    D, R, dt = case["D"], case["R"], DTYPES[case["dtype"]]
    scale = 1.0 / D if case["kind"] == "rms" else 1.0
    cos, sin = (s["cos"][s["pos"]], s["sin"][s["pos"]]) if R else (None, None)

    def one(x, w):
        x = x.float()
        r = torch.rsqrt(scale * (x * x).sum(-1, keepdim=True) + EPS)
        n = x * r if w is None else x * r * w
        return x, r, _rotate(n, cos, sin, R, case["interleaved"]).to(dt)

    def back(x, r, w, dy):
        dn = _rotate(dy.float(), cos, None if sin is None else -sin, R, case["interleaved"])
        dw = None if w is None else (x * r * dn).sum((0, 1, 2))
        dn = dn if w is None else dn * w
        dx = r * dn - x * (r * r * r) * (scale * (x * dn).sum(-1, keepdim=True))
        return dx.to(dt), dw

    xq, rq, yq = one(s["q"], s["wq"])
    xk, rk, yk = one(s["k"], s["wk"])
    if not case["grad"]:
        return {"q": yq, "k": yk}
    dq, dwq = back(xq, rq, s["wq"], s["dq"])
    dk, dwk = back(xk, rk, s["wk"], s["dk"])
    return {"q": yq, "k": yk, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _plain_step(s):
    case, at = s["case"], s["slots"]
    group = case["Hv"] // case["Hk"]
    q = s["q"].float().repeat_interleave(group, 1)
    k = s["k"].float().repeat_interleave(group, 1)
    S = s["state"][at] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (k[..., None] * S).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    o = case["Dk"] ** -0.5 * (q[..., None] * S).sum(-2)
    s["state"][at] = S
    return {"o": o.to(DTYPES[case["dtype"]]), "state": s["state"]}


def _rows(s, x):
    """[B, T, ...] to [rows, H, chunks, CHUNK, ...], rows of equal length padded with tokens
    that write nothing; and where each token went."""
    if s["cu"] is None:
        B, T = x.shape[:2]
        n = -(-T // CHUNK)
        y = x.new_zeros(B, n * CHUNK, *x.shape[2:])
        y[:, :T] = x
    else:
        cu = s["cu"]
        size = cu[1:] - cu[:-1]
        n = -(-s["case"]["T"] // CHUNK) if len(size) == 1 else -(-int(s["most"]) // CHUNK)
        y = x.new_zeros(len(size), n * CHUNK, *x.shape[2:])
        row, col = s["at"]
        y[row, col] = x[0]
    y = y.view(y.shape[0], n, CHUNK, *y.shape[2:])
    return y.movedim(3, 1)


def _plain_forward(s, q, k, v, g, beta, S):
    """The chunked form: within a chunk of 64 tokens the writes solve a unit lower triangular
    system; the chunks follow one another (the recurrence over them is the one loop)."""
    case = s["case"]
    group = case["Hv"] // case["Hk"]
    q, k, v, g, beta = (_rows(s, x) for x in (q, k, v, g, beta))
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    G = g.cumsum(-1)
    lower = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=G.device).tril()
    gam = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~lower, -math.inf))
    kk = torch.matmul(k, k.transpose(-1, -2))
    A = (beta[..., None] * gam * kk).tril(-1)
    unit = torch.eye(CHUNK, device=G.device).expand_as(A)
    Tb = torch.linalg.solve_triangular(unit + A, unit, upper=False, unitriangular=True)
    Tb = Tb * beta[..., None, :]
    P = torch.matmul(q, k.transpose(-1, -2)) * gam
    eG = torch.exp(G)[..., None]
    end = torch.exp(G[..., -1:] - G)[..., None]
    outs = []
    for c in range(q.shape[2]):
        X = v[:, :, c] - eG[:, :, c] * torch.matmul(k[:, :, c], S)
        U = torch.matmul(Tb[:, :, c], X)
        outs.append(eG[:, :, c] * torch.matmul(q[:, :, c], S) + torch.matmul(P[:, :, c], U))
        S = eG[:, :, c, -1:] * S + torch.matmul((end[:, :, c] * k[:, :, c]).transpose(-1, -2), U)
    o = case["Dk"] ** -0.5 * torch.stack(outs, 2)
    o = o.movedim(1, 3).flatten(1, 2)
    return (o[:, :case["T"]] if s["cu"] is None else o[s["at"]][None]), S


def _plain_delta(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if s["cu"] is not None:
        cu = s["cu"]
        size = cu[1:] - cu[:-1]
        row = torch.repeat_interleave(torch.arange(len(size), device=cu.device), size)
        s = dict(s, at=(row, torch.arange(case["T"], device=cu.device) - cu[row]),
                 most=size.max())
    rows = case["seqs"] or case["B"]
    S0 = s["init"] if s["init"] is not None else \
        torch.zeros(rows, case["Hv"], case["Dk"], case["Dv"], device="cuda")
    if not case["grad"]:
        o, S = _plain_forward(s, s["q"].float(), s["k"].float(), s["v"].float(), s["g"],
                              s["beta"], S0)
        return {"o": o.to(dt), "state": S}
    ins = [x.float().detach().requires_grad_() for x in
           (s["q"], s["k"], s["v"], s["g"], s["beta"], S0)]
    o, S = _plain_forward(s, *ins)
    d = torch.autograd.grad([o, S], ins, [s["do"].float(), s["dstate"]])
    return {"o": o.detach().to(dt), "state": S.detach(), "dq": d[0].to(dt), "dk": d[1].to(dt),
            "dv": d[2].to(dt), "dg": d[3], "dbeta": d[4],
            "dinit": d[5] if s["init"] is not None else None}


# ------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    if not own:
        return {"norm": _plain_norm, "step": _plain_step, "delta": _plain_delta}[case["op"]](s)
    from fft_long_convolution_amd.delta import GatedDelta, QKNorm
    if case["op"] == "norm":
        op = QKNorm(case["D"], rotary_dim=case["R"], norm=case["kind"], eps=EPS,
                    interleaved=case["interleaved"], dtype=case["dtype"])
        extra = dict(q_weight=s["wq"], k_weight=s["wk"], cos=s["cos"], sin=s["sin"],
                     positions=s["pos"])
        q, k = op.forward(s["q"], s["k"], **extra)
        if not case["grad"]:
            return {"q": q, "k": k}
        dq, dk, dwq, dwk = op.backward(s["q"], s["k"], s["dq"], s["dk"], **extra)
        return {"q": q, "k": k, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    op = GatedDelta(case["Dk"], case["Dv"], dtype=case["dtype"])
    if case["op"] == "step":
        o = op.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"])
        return {"o": o, "state": s["state"]}
    args = (s["q"], s["k"], s["v"], s["g"], s["beta"])
    if not case["grad"]:
        o, S = op.forward(*args, initial_state=s["init"], cu_seqlens=s["cu"])
        return {"o": o, "state": S}
    o, S, saved = op.forward_train(*args, initial_state=s["init"], cu_seqlens=s["cu"])
    dq, dk, dv, dg, dbeta, dinit = op.backward(*args, s["do"], saved, d_final_state=s["dstate"],
                                               initial_state=s["init"], cu_seqlens=s["cu"])
    return {"o": o, "state": S, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta,
            "dinit": dinit}


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        tokens, Hq, Hk, D, R = case["B"] * case["T"], case["Hq"], case["Hk"], case["D"], case["R"]
        x = tokens * (Hq + Hk) * D
        table = min(tokens, 8192) * R * 4 + (8 * tokens if R else 0)
        # forward: x in, y out; backward: x and dy in, dx out
        return {"bytes": x * e * (5 if case["grad"] else 2) + table,
                "flops": x * (20 if case["grad"] else 8)}
    Hk, Hv, Dk, Dv = (case[x] for x in ("Hk", "Hv", "Dk", "Dv"))
    token = (2 * Hk * Dk + 2 * Hv * Dv) * e + 8 * Hv
    if case["op"] == "step":
        return {"bytes": case["N"] * (token + 8 * Hv * Dk * Dv + 8),
                "flops": case["N"] * Hv * 7 * Dk * Dv}
    n, rows = case["B"] * case["T"], case["seqs"] or case["B"]
    states = rows * Hv * Dk * Dv * 4 * (2 if case["init"] else 1)
    # products of a token and head in the chunked form: with the state, with the chunk's
    # 64 x 64 matrices (half of them zero) and with its triangular inverse
    flops = n * Hv * (6 * Dk * Dv + CHUNK * (2 * Dk + 2 * Dv) + CHUNK * CHUNK / 3)
    if not case["grad"]:
        return {"bytes": n * token + states, "flops": flops}
    # forward, then inputs and do in, five gradients out
    more = (4 * Hk * Dk + 3 * Hv * Dv) * e + 16 * Hv
    return {"bytes": n * (token + more) + 2 * states, "flops": 3.5 * flops}


# ---------------------------------------- the definitions, in 64 bits

def _exact_norm(s):
    case = s["case"]
    D, R = case["D"], case["R"]
    c = 1.0 / D if case["kind"] == "rms" else 1.0
    first = torch.arange(0, R, 2) if case["interleaved"] else torch.arange(0, R // 2)
    second = first + (1 if case["interleaved"] else R // 2)
    # a rotation as a product with a complex number of unit modulus
    turn = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"]][:, :, None] if R else None

    def rotated(x, turn):
        y = x.clone()
        if R:
            z = torch.complex(x[..., first], x[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        w = torch.ones(D, dtype=torch.float64, device="cuda") if s["w" + name] is None \
            else s["w" + name].double()
        m = c * x.square().sum(-1, keepdim=True) + EPS
        out[name] = rotated(w * x / m.sqrt(), turn)
        if case["grad"]:
            dn = rotated(s["d" + name].double(), turn.conj() if R else None)
            # d(x / sqrt(m)) = (dx m - x c <x, dx>) / m^(3/2)
            h = dn * w
            out["d" + name] = (h * m - x * c * (x * h).sum(-1, keepdim=True)) / m ** 1.5
            out["dw" + name] = (dn * x / m.sqrt()).flatten(0, 2).sum(0) \
                if s["w" + name] is not None else None
    return out


def _exact_step(s):
    case, at = s["case"], s["slots"]
    head = torch.arange(case["Hv"], device="cuda") // (case["Hv"] // case["Hk"])
    q, k, v = s["q"].double()[:, head], s["k"].double()[:, head], s["v"].double()
    S, _, o = _token(s["state"][at].double(), q, k, v, s["g"].double(), s["beta"].double(),
                     case["Dk"] ** -0.5)
    state = s["state"].double()
    state[at] = S
    return {"o": o, "state": state}


def _token(S, q, k, v, g, beta, scale):
    """One token of the recurrence: the new state, the decayed old one and the output."""
    old = torch.exp(g)[..., None, None] * S
    u = beta[..., None] * (v - torch.einsum("nhkv,nhk->nhv", old, k))
    S = old + torch.einsum("nhk,nhv->nhkv", k, u)
    return S, old, scale * torch.einsum("nhkv,nhk->nhv", S, q)


def _exact_delta(s):
    case = s["case"]
    B, T, Hk, Hv, Dk, Dv = (case[x] for x in ("B", "T", "Hk", "Hv", "Dk", "Dv"))
    head = torch.arange(Hv, device="cuda") // (Hv // Hk)
    scale = Dk ** -0.5
    if s["cu"] is None:
        bounds = [(b, 0, T) for b in range(B)]
    else:
        cu = s["cu"].tolist()
        bounds = [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]
    rows, most = len(bounds), max(b - a for _, a, b in bounds)
    # the adjoint of the recurrence is some 45 small kernels a token
    if most * (45 if case["grad"] else 8) > 1200000:
        return None

    def table(x):
        y = torch.zeros(most, rows, *x.shape[2:], dtype=torch.float64, device="cuda")
        for r, (b, a, z) in enumerate(bounds):
            y[:z - a, r] = x[b, a:z].double()
        return y

    def back(y):
        x = torch.zeros(B, T, *y.shape[2:], dtype=torch.float64, device="cuda")
        for r, (b, a, z) in enumerate(bounds):
            x[b, a:z] = y[:z - a, r]
        return x

    q, k, v, g, beta = (table(s[x]) for x in ("q", "k", "v", "g", "beta"))
    q, k = q[:, :, head], k[:, :, head]
    S = s["init"].double() if s["init"] is not None else \
        torch.zeros(rows, Hv, Dk, Dv, dtype=torch.float64, device="cuda")
    o, every, kept = torch.zeros_like(v), 128, []
    for t in range(most):
        if t % every == 0:
            kept.append(S)
        S, _, o[t] = _token(S, q[t], k[t], v[t], g[t], beta[t], scale)
    out = {"o": back(o), "state": S}
    if not case["grad"]:
        return out
    do, dS = table(s["do"]), s["dstate"].double()
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, g, beta))
    for first in reversed(range(0, most, every)):
        last, S, seen = min(most, first + every), kept[first // every], []
        for t in range(first, last):
            S, old, _ = _token(S, q[t], k[t], v[t], g[t], beta[t], scale)
            seen.append((S, old))
        for t in reversed(range(first, last)):
            S, old = seen[t - first]
            dq[t] = scale * torch.einsum("nhkv,nhv->nhk", S, do[t])
            dS = dS + scale * torch.einsum("nhk,nhv->nhkv", q[t], do[t])
            miss = v[t] - torch.einsum("nhkv,nhk->nhv", old, k[t])
            du = torch.einsum("nhkv,nhk->nhv", dS, k[t])
            db[t] = (du * miss).sum(-1)
            dv[t] = beta[t][..., None] * du
            dk[t] = torch.einsum("nhkv,nhv->nhk", dS, beta[t][..., None] * miss) \
                - torch.einsum("nhkv,nhv->nhk", old, dv[t])
            dS = dS - torch.einsum("nhk,nhv->nhkv", k[t], dv[t])
            dg[t] = (dS * old).sum((-1, -2))
            dS = torch.exp(g[t])[..., None, None] * dS
    shared = lambda x: back(x).unflatten(2, (Hk, Hv // Hk)).sum(3)  # noqa: E731
    out.update(dq=shared(dq), dk=shared(dk), dv=back(dv), dg=back(dg), dbeta=back(db),
               dinit=dS if s["init"] is not None else None)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "step": _exact_step, "delta": _exact_delta}[case["op"]](s)
