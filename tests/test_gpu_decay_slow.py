"""Decays so slow that a state lives through a thousand chunks of 32 tokens, against
sums over all pairs of tokens in 64 bits.

A chunk rounds each element of the state once, by 2^-24 of it at most and either
way: after n chunks the 2-norm is off by sqrt(n / 3) 2^-24, 1.1e-6 for n = 1024.  A
factor e^(32 g) rounded to fp32 is the same number in each chunk of a fixed decay: its
error, up to 2^-25, would count n times in one direction, 3e-5.  The decays are those
whose factors 1 - (n + 1/2) 2^-24 lie half-way between two numbers.  1e-5 is allowed,
as for other fp32 outputs."""
import math

import pytest
import torch

from tests.decay_reference import DT, TOL, rel

pytestmark = pytest.mark.gpu
T, D = 32768, 16
DECAYS = [-(n + 0.5) * 2.0 ** -29 for n in (536, 1024, 8192)]


def attend(dtype):
    from fft_long_convolution_amd.decay import DecayAttention
    return DecayAttention(D, D, dtype=dtype)


def inputs(dtype):
    """One head's; rows have a direction in common, so sums over tokens do not cancel."""
    gen = torch.Generator().manual_seed(3)
    rows = [((0.5 + torch.randn(T, D, generator=gen)) / 4).to(DT[dtype]) for _ in range(4)]
    return [x.cuda() for x in (*rows, torch.randn(D, D, generator=gen), torch.randn(D, D, generator=gen))]


def wanted(q, k, v, do, S, dS, g):
    """o, final state, dv, dg of each token, d initial state; g one number, all double."""
    c, t = D ** -0.5, torch.arange(T, dtype=torch.float64, device="cuda")
    to = torch.exp(g * (t + 1))[:, None]              # from the first state to the token
    end = torch.exp(g * (T - 1 - t))[:, None]         # from the token to the last state
    fin = math.exp(g * T) * S + (end * k).t() @ v
    dinit = math.exp(g * T) * dS + c * (to * q).t() @ do
    o, dv = c * to * (q @ S), end * (k @ dS)
    # what a token's output owes to the tokens before it, and what those behind owe to it
    owes, owed = c * to[:, 0] * ((q @ S) * do).sum(-1), end[:, 0] * ((k @ dS) * v).sum(-1)
    for i in range(0, T, 2048):
        u = t[i:i + 2048, None]
        w = torch.where(u >= t, torch.exp(g * (u - t).clamp_min(0)), 0)
        p = c * w * (q[i:i + 2048] @ k.t())
        o[i:i + 2048] += p @ v
        dv += p.t() @ do[i:i + 2048]
        p *= do[i:i + 2048] @ v.t()
        p = torch.where(u > t, p, 0)
        owes[i:i + 2048] += p.sum(-1)
        owed += p.sum(0)
    # the pairs around a token: those that end at it or behind, but for those that begin there
    last = (end[:, 0] * ((k @ dS) * v).sum(-1)).sum() + math.exp(g * T) * (S * dS).sum()
    dg = owes.flip(0).cumsum(0).flip(0) + last - owed.flip(0).cumsum(0).flip(0)
    return [x.cpu() for x in (o, fin, dv, dg, dinit)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [3, 513])
@pytest.mark.parametrize("fixed", [True, False])
def test_slow_decays(fixed, heads, dtype):
    """Three heads in segments, 513 (three again and again) whole."""
    q, k, v, do, S, dS = inputs(dtype)
    op = attend(dtype)
    g = torch.tensor(DECAYS, device="cuda").repeat(heads // 3)
    if not fixed:
        g = g.expand(1, T, heads)
    args = [q[None, :, None], k[None, :, None], v[None, :, None].expand(1, T, heads, D), g]
    S0, dS0 = (x.expand(1, heads, D, D) for x in (S, dS))
    cut = op._lib.fftconv_decay_workspace_bytes(op._describe(*args, None, None)[0][1][0])
    assert (cut > 0) == (heads == 3)
    o, fin = op.forward(*args, initial_state=S0)
    d = op.backward(*args, do[None, :, None].expand(1, T, heads, D), d_final_state=dS0,
                    initial_state=S0)
    for i, h in enumerate((0, 1, heads - 1)):
        want = wanted(*(x.double() for x in (q, k, v, do, S, dS)), DECAYS[i])
        if fixed:
            want[3] = want[3].sum()
        got = (o[0, :, h], fin[0, h], d[2][0, :, h], d[3][h] if fixed else d[3][0, :, h], d[4][0, h])
        for name, x, y in zip(("o", "state", "dv", "dg", "dinit"), got, want):
            assert rel(x, y) <= TOL[dtype if name in ("o", "dv") else "f32"], (name, DECAYS[i])
