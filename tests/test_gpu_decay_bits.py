"""Linear attention with decays keeps the bits of fp32 in states and scores, whatever
the I/O type: sums of which all but the last bits cancel.

Every value and every partial sum below is a multiple of 2^-17 and below 2^5, at most 22
bits, so sums in fp32 are exact in any order: what is allowed is the rounding to the
output's type, half a step."""
import pytest
import torch

from tests.decay_reference import DT, decay

pytestmark = pytest.mark.gpu
TYPES = ["bf16", "f16", "f32"]
T = 40
# 1 + 2^-9 and the same with one more bit; as a product of rows (1, 2^-9, 2^-17) and
# ones, and as elements of a state
FINE = (1.0, 2.0 ** -9, 2.0 ** -17)


def attend(Dk, Dv, dtype):
    from fft_long_convolution_amd.decay import DecayAttention
    return DecayAttention(Dk, Dv, dtype=dtype, scale=1.0)


def zeros(Dk, Dv, dtype):
    return (torch.zeros(1, T, 1, Dk, dtype=DT[dtype]), torch.zeros(1, T, 1, Dk, dtype=DT[dtype]),
            torch.zeros(1, T, 1, Dv, dtype=DT[dtype]), torch.zeros(1, T, 1, Dv, dtype=DT[dtype]),
            torch.zeros(1, T, 1), torch.zeros(1, 1, Dk, Dv))


def results(q, k, v, do, g, S, dS, dtype):
    """Outputs and gradients, and the same in 64 bits."""
    op = attend(q.shape[-1], v.shape[-1], dtype)
    on = [x.cuda() for x in (q, k, v, g)]
    o, fin = op.forward(*on, initial_state=S.cuda())
    d = op.backward(*on, do.cuda(), d_final_state=dS.cuda(), initial_state=S.cuda())
    ins = [x.double().requires_grad_() for x in (q, k, v, g, S)]
    want, want_S = decay(*ins, None, 1.0)
    grads = torch.autograd.grad([want, want_S], ins, [do.double(), dS.double()])
    names = ("o", "state", "dq", "dk", "dv", "dg", "dinit")
    return dict(zip(names, (o, fin, *d))), dict(zip(names, (want.detach(), want_S.detach(), *grads)))


def close(got, want, dtype):
    got = got.cpu().double()
    assert want.any()
    assert ((got - want).abs() <= torch.finfo(DT[dtype]).eps / 2 * want.abs()).all()


def signs(n):
    """1 and -1 in turn in the last 40 elements, 0 before."""
    x = torch.tensor([1.0, -1.0]).repeat(n // 2)
    x[:-40] = 0
    return x


def fine_state(n, m):
    """[n, m]: alternately with the last bit and without it along n."""
    return (FINE[0] + FINE[1] + FINE[2] * (signs(n) > 0).float())[:, None].expand(n, m)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk, Dv", [(64, 64), (128, 72), (40, 128), (256, 200)])
@pytest.mark.parametrize("name", ["o", "dq", "dk", "dv"])
def test_products_with_a_state(name, Dk, Dv, dtype):
    q, k, v, do, g, S = zeros(Dk, Dv, dtype)
    dS = torch.zeros_like(S)
    if name == "o":                     # S^T q
        S[0, 0] = fine_state(Dk, Dv)
        q[:] = signs(Dk)
    elif name == "dq":                  # S do
        S[0, 0] = fine_state(Dv, Dk).t()
        do[:] = signs(Dv)
    elif name == "dk":                  # dS v
        dS[0, 0] = fine_state(Dv, Dk).t()
        v[:] = signs(Dv)
    else:                               # dS^T k
        dS[0, 0] = fine_state(Dk, Dv)
        k[:] = signs(Dk)
    got, want = results(q, k, v, do, g, S, dS, dtype)
    close(got[name], want[name], dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Dk, Dv", [(64, 64), (128, 72), (40, 128), (256, 200)])
@pytest.mark.parametrize("name", ["o", "dq", "dk", "dv"])
def test_products_with_scores(name, Dk, Dv, dtype):
    """Two tokens whose scores differ in the last bit, with values of opposite signs."""
    q, k, v, do, g, S = zeros(Dk, Dv, dtype)
    # rows whose products are the scores, and the values: of two tokens and of the one
    # token (the last, or for gradients behind it the first) that adds them up
    two, one, values, first = {"o": (k, q, v, True), "dq": (v, do, k, True),
                               "dk": (do, v, q, False), "dv": (q, k, do, False)}[name]
    a, b, at = (1, 17, 30) if first else (7, 30, 5)         # in one chunk
    two[0, a, 0, :3] = 1
    two[0, b, 0, :2] = 1
    one[0, at, 0, :3] = torch.tensor(FINE)
    values[0, a], values[0, b] = 1, -1
    got, want = results(q, k, v, do, g, S, torch.zeros_like(S), dtype)
    assert want[name][0, at].abs().max() == FINE[2]
    close(got[name][0, at], want[name][0, at], dtype)
