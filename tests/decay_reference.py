"""Plain 64-bit forms of linear attention with a decay for each head (token by
token, differentiable) and of layer norm, on the CPU.  Nothing here is shared
with the library.

TOL: relative 2-norm error allowed for an output of each type.  16-bit outputs
are rounded once to p significant bits, which is off by at most 2^-p of each
value: 2^-8 (bf16) or 2^-11 (f16); what meets only such outputs has at least 17
bits, for which 2^-13 more is allowed.  fp32 outputs are sums of products that
keep 22 bits or more over chunks of 64 tokens, joined by decays of at most one: 64
roundings of 2^-24 in a row would be 4e-6; 1e-5 allows for two such sums in a row.
"""
from __future__ import annotations

import torch

from tests.mixer_reference import DT, TOL, rel  # noqa: F401


def sequence(q, k, v, g, S, scale):
    """One sequence: q, k [T, Hv, Dk], v [T, Hv, Dv], g [T, Hv], S [Hv, Dk, Dv]."""
    outs = []
    for t in range(q.shape[0]):
        S = torch.exp(g[t])[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        outs.append(scale * (q[t][:, :, None] * S).sum(1))
    return torch.stack(outs) if outs else v, S


def decay(q, k, v, g, init, cu, scale):
    """The batch or the packed sequences; inputs as DecayAttention takes them, in
    double on the CPU.  Tokens that no sequence holds have outputs of 0."""
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    head = torch.arange(Hv) // (Hv // Hk)
    q, k, g = q[:, :, head], k[:, :, head], g.expand(B, T, Hv)
    spans = [(b, 0, T) for b in range(B)] if cu is None else \
        [(0, int(a), int(z)) for a, z in zip(cu[:-1], cu[1:])]
    o, states = [], []
    for i, (b, a, z) in enumerate(spans):
        S = torch.zeros(Hv, Dk, Dv, dtype=torch.float64) if init is None else init[i]
        y, S = sequence(q[b, a:z], k[b, a:z], v[b, a:z], g[b, a:z], S, scale)
        o.append(y)
        states.append(S)
    if cu is None:
        o = torch.stack(o)
    else:
        before, behind = v.new_zeros(int(cu[0]), Hv, Dv), v.new_zeros(T - int(cu[-1]), Hv, Dv)
        o = torch.cat([before, *o, behind])[None]
    return o, torch.stack(states)


def decay_inputs(seed, B, T, Hk, Hv, Dk, Dv, dtype, rows=None, init=True, fixed=False, rate=0.3):
    """Inputs on the CPU, in their own types."""
    gen = torch.Generator().manual_seed(seed)

    def unit(*shape):
        x = torch.randn(*shape, generator=gen)
        return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)

    q, k = unit(B, T, Hk, Dk).to(DT[dtype]), unit(B, T, Hk, Dk).to(DT[dtype])
    v = torch.randn(B, T, Hv, Dv, generator=gen).to(DT[dtype])
    g = -rate * (torch.rand(Hv, generator=gen) if fixed else
                 torch.rand(B, T, Hv, generator=gen) * (1 + torch.arange(Hv)))
    S = 0.3 * torch.randn(rows or B, Hv, Dk, Dv, generator=gen) if init else None
    return q, k, v, g, S


def layer_norm(x, w, b, eps):
    x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w
    return y if b is None else y + b
