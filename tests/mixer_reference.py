"""Plain 64-bit forms of the token mixers beside the long convolution, on the
CPU: norms of queries and keys with the rotation, and the gated delta rule
token by token with its adjoint.  Nothing here is shared with the library.

TOL: relative 2-norm error allowed for an output of each type.  16-bit
outputs are rounded once to p significant bits, which is off by at most 2^-p of
each value: 2^-8 (bf16) or 2^-11 (f16); the products behind them keep at least
16 bits, for which 2^-13 more is allowed.  fp32 outputs are sums of products that keep 24 bits
over chunks of 64 tokens, joined by decays of at most one: 64 roundings of
2^-24 in a row would be 4e-6; 1e-5 allows for two such sums in a row.
"""
from __future__ import annotations

import torch

TOL = {"bf16": 2.0 ** -8 + 2.0 ** -13, "f16": 2.0 ** -11 + 2.0 ** -13, "f32": 1e-5}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rel(got, want):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    n = want.norm().item()
    return (got - want).norm().item() / n if n else got.norm().item()


def rotate(x, cos, sin, R, interleaved):
    """x [B, T, H, D]; cos, sin [B, T, R/2]."""
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    c, s = cos[:, :, None], sin[:, :, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def qk_norm(x, w, cos, sin, R, interleaved, kind, eps):
    c = 1.0 / x.shape[-1] if kind == "rms" else 1.0
    n = x / torch.sqrt(c * (x * x).sum(-1, keepdim=True) + eps)
    if w is not None:
        n = n * w
    return rotate(n, cos, sin, R, interleaved) if R else n


def delta_sequence(q, k, v, g, beta, S, scale):
    """One sequence: q, k [T, Hv, Dk], v [T, Hv, Dv], S [Hv, Dk, Dv]; all
    double.  Differentiable."""
    outs = []
    for t in range(q.shape[0]):
        S = torch.exp(g[t])[:, None, None] * S
        u = beta[t][:, None] * (v[t] - (k[t][:, :, None] * S).sum(1))
        S = S + k[t][:, :, None] * u[:, None, :]
        outs.append(scale * (q[t][:, :, None] * S).sum(1))
    o = torch.stack(outs) if outs else v
    return o, S


def delta(q, k, v, g, beta, init, cu, scale):
    """The batch or the packed sequences; inputs as GatedDelta takes them, in
    double on the CPU."""
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    head = torch.arange(Hv) // (Hv // Hk)
    q, k = q[:, :, head], k[:, :, head]
    spans = [(b, 0, T) for b in range(B)] if cu is None else \
        [(0, int(a), int(z)) for a, z in zip(cu[:-1], cu[1:])]
    o, states = [], []
    for i, (b, a, z) in enumerate(spans):
        S = torch.zeros(Hv, Dk, Dv, dtype=torch.float64) if init is None else init[i]
        y, S = delta_sequence(q[b, a:z], k[b, a:z], v[b, a:z], g[b, a:z], beta[b, a:z], S, scale)
        o.append(y)
        states.append(S)
    o = torch.stack(o) if cu is None else torch.cat(o)[None]
    return o, torch.stack(states)


def delta_inputs(seed, B, T, Hk, Hv, Dk, Dv, dtype, rows=None, init=True, decay=0.3):
    """Inputs on the CPU, in their own types."""
    gen = torch.Generator().manual_seed(seed)

    def unit(*shape):
        x = torch.randn(*shape, generator=gen)
        return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)

    q, k = unit(B, T, Hk, Dk).to(DT[dtype]), unit(B, T, Hk, Dk).to(DT[dtype])
    v = torch.randn(B, T, Hv, Dv, generator=gen).to(DT[dtype])
    g = -decay * torch.rand(B, T, Hv, generator=gen) * (1 + torch.arange(Hv))
    beta = torch.rand(B, T, Hv, generator=gen)
    S = 0.3 * torch.randn(rows or B, Hv, Dk, Dv, generator=gen) if init else None
    return q, k, v, g, beta, S
