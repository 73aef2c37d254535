"""Gradients of linear attention with a decay for each head against the adjoint of
the token recurrence in 64 bits, and against differences of it."""
import math

import pytest
import torch

from tests.decay_reference import DT, TOL, decay, decay_inputs, rel

pytestmark = pytest.mark.gpu
NAMES = ("dq", "dk", "dv", "dg", "dinit")


def attend(Dk, Dv, dtype, **kw):
    from fft_long_convolution_amd.decay import DecayAttention
    return DecayAttention(Dk, Dv, dtype=dtype, **kw)


def gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def gradients(ins, do, dfin, cu, dtype):
    q, k, v, g, init = gpu(*ins)
    op = attend(q.shape[-1], v.shape[-1], dtype)
    return op.backward(q, k, v, g, do.cuda(), d_final_state=gpu(dfin)[0], initial_state=init,
                       cu_seqlens=gpu(cu)[0])


def wanted(ins, do, dfin, cu):
    leaves = [t.double().requires_grad_() for t in ins if t is not None]
    args = leaves if len(leaves) == 5 else leaves + [None]
    o, S = decay(*args, cu, ins[0].shape[-1] ** -0.5)
    outs, ds = [o], [do.double()]
    if dfin is not None:
        outs, ds = outs + [S], ds + [dfin.double()]
    d = torch.autograd.grad(outs, leaves, ds, allow_unused=True)
    return [torch.zeros_like(x) if y is None else y for x, y in zip(leaves, d)]


def tangents(seed, ins, rows, dfin):
    v = ins[2]
    gen = torch.Generator().manual_seed(seed)
    do = torch.randn(v.shape, generator=gen).to(v.dtype)
    d = 0.3 * torch.randn(rows, v.shape[2], ins[0].shape[3], v.shape[3], generator=gen)
    return do, d if dfin else None


def check(ins, cu, dtype, dfin):
    rows = ins[0].shape[0] if cu is None else len(cu) - 1
    do, d = tangents(7, ins, rows, dfin)
    got, want = gradients(ins, do, d, cu, dtype), wanted(ins, do, d, cu)
    for name, x, y in zip(NAMES, got, want):
        assert x.dtype == (torch.float32 if name in ("dg", "dinit") else DT[dtype])
        assert rel(x, y) <= TOL["f32" if name in ("dg", "dinit") else dtype], name
    if ins[4] is None:
        assert got[4] is None


# B, T, Hk, Hv, Dk, Dv
SHAPES = [
    (1, 1, 1, 1, 64, 64),
    (2, 2, 1, 2, 8, 8),
    (1, 31, 1, 1, 16, 24),
    (1, 63, 2, 2, 128, 128),
    (2, 64, 1, 1, 64, 128),
    (1, 65, 1, 3, 96, 72),
    (2, 200, 2, 4, 128, 128),
    (1, 131, 1, 1, 40, 256),
    (1, 100, 1, 2, 256, 64),
    (1, 97, 1, 1, 200, 248),
    (1, 517, 1, 1, 128, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients(shape, dtype):
    n = sum(shape)
    ins = decay_inputs(n, *shape, dtype, init=n % 3 > 0, fixed=n % 2 == 0)
    check(ins, None, dtype, n % 5 > 0)
    ins = decay_inputs(n, *shape, dtype, init=n % 3 == 0, fixed=n % 2 == 1)
    check(ins, None, dtype, n % 5 == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bounds", [
    [0, 1], [0, 0, 5, 5, 6, 70, 70], [0, 64, 128, 129, 300], [0, 3, 67, 131, 195, 196],
    [0, 10, 10, 10, 11, 12, 13, 14, 80], [7, 7, 40, 140]], ids=str)
def test_packed_gradients(bounds, dtype):
    cu, T = torch.tensor(bounds), bounds[-1] + (9 if bounds[0] else 0)
    ins = decay_inputs(T, 1, T, 1, 2, 64, 72, dtype, rows=len(bounds) - 1, fixed=T % 2 == 0)
    check(ins, cu, dtype, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rate", [0.0, 1e-3, 0.05, 1.0, 4.0, 8.0, 16.0])
def test_decay_gradients_at_every_rate(rate, dtype):
    """dg of a head by itself: strong decays leave little of it, and no more error."""
    ins = list(decay_inputs(3, 1, 300, 1, 1, 64, 64, dtype))
    ins[3] = -rate * (0.9 + 0.2 * torch.rand(ins[3].shape, generator=torch.Generator().manual_seed(1)))
    do, d = tangents(5, ins, 1, True)
    got, want = gradients(ins, do, d, None, dtype)[3], wanted(ins, do, d, None)[3]
    assert rel(got, want) <= TOL["f32"]
    # and away from the last state's part and the first's
    assert rel(got[:, 64:-64], want[:, 64:-64]) <= TOL["f32"]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_gradients_at_a_reset(dtype):
    """e^-inf = 0: nothing before the token reaches it, and its own dg is 0."""
    ins = list(decay_inputs(4, 1, 150, 1, 2, 64, 64, dtype))
    ins[3][:, 70, 0] = -math.inf
    do, d = tangents(5, ins, 1, True)
    got = gradients(ins, do, d, None, dtype)
    assert got[3][0, 70, 0] == 0
    finite = list(ins)
    finite[3] = ins[3].clamp_min(-1e3)            # e^-1000 = 0 in 64 bits too
    for name, x, y in zip(NAMES, got, wanted(finite, do, d, None)):
        assert rel(x, y) <= TOL["f32" if name in ("dg", "dinit") else dtype], name


@pytest.mark.parametrize("fixed", [False, True])
def test_against_differences(fixed):
    """The derivative along a direction in every input, from central differences
    of the recurrence in 64 bits (their error is of h^2, below 1e-6)."""
    ins = decay_inputs(8, 1, 90, 1, 2, 32, 40, "f32", fixed=fixed)
    do, d = tangents(2, ins, 1, True)
    got = gradients(ins, do, d, None, "f32")
    gen = torch.Generator().manual_seed(9)
    for i, name in enumerate(NAMES):
        way = torch.randn(ins[i].shape, generator=gen, dtype=torch.float64)

        def loss(h):
            at = [t.double() for t in ins]
            at[i] = at[i] + h * way
            o, S = decay(*at, None, 32 ** -0.5)
            return (o * do.double()).sum() + (S * d.double()).sum()

        h = 1e-5
        want = ((loss(h) - loss(-h)) / (2 * h)).item()
        # sums of n products of random signs, each off by the gradient's 1e-5
        size = (got[i].cpu().double() * way).norm().item()
        assert abs((got[i].cpu().double() * way).sum().item() - want) <= 2e-5 * size + 1e-6 * abs(want), name
