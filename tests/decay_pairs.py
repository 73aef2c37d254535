"""Linear attention with a decay for each head as sums over all pairs of tokens, in 64
bits on the tensors' device: one sequence of one head, with all gradients.  Nothing here
is shared with the library or with the token recurrence of decay_reference.py."""
from __future__ import annotations

import torch


def head(q, k, v, do, S, dS, g):
    """q, k [T, Dk], v, do [T, Dv], S, dS [Dk, Dv], g [T], all double.  Returns o, final
    state, dq, dk, dv, dg, d initial state."""
    c, G = q.shape[1] ** -0.5, g.cumsum(0)
    w = c * torch.exp((G[:, None] - G).clamp_max(0)).tril()
    to, end, all = c * torch.exp(G)[:, None], torch.exp(G[-1] - G)[:, None], torch.exp(G[-1])
    scores, owed = w * (q @ k.t()), w * (do @ v.t())
    o = to * (q @ S) + scores @ v
    fin = all * S + (end * k).t() @ v
    dq = to * (do @ S.t()) + owed @ k
    dk = end * (v @ dS.t()) + owed.t() @ q
    dv = end * (k @ dS) + scores.t() @ do
    dinit = all * dS + (to * q).t() @ do
    # dg of a token: the pairs that end at it or behind, but for those that begin there
    pairs = (owed * (q @ k.t())).tril(-1)
    ends = pairs.sum(1) + to[:, 0] * ((q @ S) * do).sum(1)
    begins = pairs.sum(0) + end[:, 0] * ((k @ dS) * v).sum(1)
    at_end = end[:, 0] @ ((k @ dS) * v).sum(1) + all * (S * dS).sum()
    dg = (ends - begins).flip(0).cumsum(0).flip(0) + at_end
    return o, fin, dq, dk, dv, dg, dinit


def batch(q, k, v, do, S, dS, g, cu=None):
    """All rows (or packed sequences) and heads, as DecayAttention takes them, of any type;
    gradients of shared heads summed, dg of g's shape."""
    B, T, Hk, Dk = q.shape
    Hv, fixed = v.shape[2], g.dim() == 1
    q, k, v, do, S, dS, g = (x.double() for x in (q, k, v, do, S, dS, g))
    o, dq, dk, dv = (torch.zeros(B, T, Hv, x.shape[-1], dtype=q.dtype, device=q.device)
                     for x in (v, q, k, v))
    dg, fin, dinit = torch.zeros_like(o[..., 0]), torch.empty_like(S), torch.empty_like(S)
    spans = [(b, 0, T) for b in range(B)] if cu is None else \
        [(0, a, z) for a, z in zip(cu[:-1], cu[1:])]
    for i, (b, a, z) in enumerate(spans):
        for h in range(Hv):
            if a == z:
                fin[i, h], dinit[i, h] = S[i, h], dS[i, h]
                continue
            j, at = h * Hk // Hv, slice(a, z)
            outs = head(q[b, at, j], k[b, at, j], v[b, at, h], do[b, at, h], S[i, h], dS[i, h],
                        g[h].expand(z - a) if fixed else g[b, at, h])
            for x, y in zip((o[b, at, h], fin[i, h], dq[b, at, h], dk[b, at, h], dv[b, at, h],
                             dg[b, at, h], dinit[i, h]), outs):
                x.copy_(y)
    dq, dk = (x.unflatten(2, (Hk, Hv // Hk)).sum(3) for x in (dq, dk))
    return dict(o=o, state=fin, dq=dq, dk=dk, dv=dv, dg=dg.sum((0, 1)) if fixed else dg,
                dinit=dinit)
