"""Linear attention with a decay for each head (sequences, single tokens) against
the token recurrence in 64 bits."""
import math

import pytest
import torch

from tests.decay_reference import DT, TOL, decay, decay_inputs, rel

pytestmark = pytest.mark.gpu


def attend(Dk, Dv, dtype, **kw):
    from fft_long_convolution_amd.decay import DecayAttention
    return DecayAttention(Dk, Dv, dtype=dtype, **kw)


def gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def double(*ts):
    return [None if t is None else t.double() for t in ts]


def check_forward(ins, cu, dtype, Dk, Dv):
    o, S = attend(Dk, Dv, dtype).forward(*gpu(*ins[:4]), initial_state=gpu(ins[4])[0],
                                         cu_seqlens=None if cu is None else cu.cuda())
    want_o, want_S = decay(*double(*ins), cu, Dk ** -0.5)
    assert o.dtype == DT[dtype] and S.dtype == torch.float32
    assert rel(o, want_o) <= TOL[dtype]
    assert rel(S, want_S) <= TOL["f32"]


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
    (1, 97, 1, 1, 200, 264),
    (1, 517, 1, 1, 128, 64),
]


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype, init):
    ins = decay_inputs(sum(shape), *shape, dtype, init=init, fixed=sum(shape) % 2 == 0)
    check_forward(ins, None, dtype, shape[4], shape[5])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bounds", [
    [0, 1], [0, 0, 5, 5, 6, 70, 70], [0, 64, 128, 129, 300], [0, 3, 67, 131, 195, 196],
    [0, 0, 0], [0, 10, 10, 10, 11, 12, 13, 14, 80], [7, 7, 40, 140]], ids=str)
def test_packed_sequences(bounds, dtype):
    cu, T = torch.tensor(bounds), bounds[-1] + (9 if bounds[0] else 0)
    ins = decay_inputs(T, 1, T, 1, 2, 64, 72, dtype, rows=len(bounds) - 1, fixed=T % 2 == 0)
    check_forward(ins, cu, dtype, 64, 72)


@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Dk, Dv", [(64, 64), (128, 128), (96, 40), (256, 136), (8, 8)])
def test_step(Dk, Dv, dtype, fixed):
    N, pool, Hk, Hv = 5, 9, 2, 4
    q, k, v, g, _ = decay_inputs(Dk + Dv, N, 1, Hk, Hv, Dk, Dv, dtype, init=False, fixed=fixed)
    gen = torch.Generator().manual_seed(1)
    state = torch.randn(pool, Hv, Dk, Dv, generator=gen)
    slots = torch.tensor([3, -1, 8, 0, pool])
    held = [0, 2, 3]
    gs = g if fixed else g[:, 0]
    S = state.cuda()
    o = attend(Dk, Dv, dtype).step(*gpu(q[:, 0], k[:, 0], v[:, 0], gs), S, slots=slots.cuda())
    want_o, want_S = torch.zeros(N, Hv, Dv, dtype=torch.float64), state.double()
    y, s = decay(*double(q[held], k[held], v[held], g if fixed else g[held], state[slots[held]]),
                 None, Dk ** -0.5)
    want_o[held], want_S[slots[held]] = y[:, 0], s
    assert rel(o, want_o) <= TOL[dtype]
    assert rel(S, want_S) <= TOL["f32"]
    assert (o[[1, 4]] == 0).all()
    untouched = [i for i in range(pool) if i not in slots.tolist()]
    assert torch.equal(S.cpu()[untouched], state[untouched])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_steps_continue_a_sequence(dtype):
    ins = decay_inputs(5, 2, 100, 1, 2, 64, 64, dtype)
    q, k, v, g, init = gpu(*ins)
    op = attend(64, 64, dtype)
    _, S = op.forward(q[:, :90], k[:, :90], v[:, :90], g[:, :90], initial_state=init)
    o = torch.stack([op.step(q[:, t], k[:, t], v[:, t], g[:, t], S) for t in range(90, 100)], 1)
    want_o, want_S = decay(*double(*ins), None, 64 ** -0.5)
    assert rel(o, want_o[:, 90:]) <= TOL[dtype]
    assert rel(S, want_S) <= TOL["f32"]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_resets_and_strong_decays(dtype):
    """A log decay of -inf drops the state, large ones leave nothing of it; each
    head by itself, so that no head hides another's error."""
    ins = list(decay_inputs(11, 1, 150, 1, 4, 64, 64, dtype))
    g = ins[3]
    g[:, 70, 0] = -math.inf
    g[:, 0, 0] = -math.inf
    g[..., 1] = -8.0
    g[..., 2] = -50.0
    g[..., 3] = 0.0
    o, S = attend(64, 64, dtype).forward(*gpu(*ins[:4]), initial_state=ins[4].cuda())
    want_o, want_S = decay(*double(*ins), None, 0.125)
    for h in range(4):
        assert rel(o[:, :, h], want_o[:, :, h]) <= TOL[dtype]
        assert rel(S[:, h], want_S[:, h]) <= TOL["f32"]
