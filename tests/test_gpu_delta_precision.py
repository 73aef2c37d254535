"""How exact the gated delta rule's outputs are before they are rounded to
their type.

fp32 operands of the products are two f16 terms, off by at most 2^-23 of the
largest value of their row or column, the product of the two low terms (2^-22) is left
out, and sums are fp32.  A chain of them over a chunk leaves some 3e-7 of a
result's norm; 1e-5, what fp32 outputs are allowed, is the bound here.
"""
import pytest
import torch

from tests.mixer_reference import TOL, delta, delta_inputs
from tests.test_gpu_delta import double, gpu, rule

pytestmark = pytest.mark.gpu

# Of normally distributed exact values, rounded to 8 bits (spacing at least 2^-8
# of a value x), an error of e times their rms moves a share of min(1, a / |x|),
# a = 2 e 2^8, to a neighbour: 0.8 a (1 + ln(1 / a)) on average, 2.5 % at 1e-5.
MOVED = 0.025


def moved(got, want):
    """Share of the values that are not the exact ones rounded once."""
    return (got.cpu() != want.to(got.dtype)).double().mean().item()


@pytest.mark.parametrize("shape", [(1, 130, 2, 2, 128, 128), (2, 100, 1, 3, 64, 72)], ids=str)
def test_bf16_results_are_rounded_once(shape):
    ins = delta_inputs(sum(shape), *shape, "bf16")
    Dk = shape[4]
    do = torch.randn(ins[2].shape, generator=torch.Generator().manual_seed(3)).bfloat16()
    op, a = rule(Dk, shape[5], "bf16"), gpu(*ins)
    o, _, saved = op.forward_train(*a[:5], initial_state=a[5])
    d = op.backward(*a[:5], do.cuda(), saved, initial_state=a[5])
    leaf = [x.requires_grad_() for x in double(*ins)]
    want, _ = delta(*leaf, None, Dk ** -0.5)
    grads = torch.autograd.grad((want * do.double()).sum(), leaf[:3])
    for name, x, y in zip(("o", "dq", "dk", "dv"), (o, *d[:3]), (want.detach(), *grads)):
        share = moved(x, y)
        assert share <= MOVED, name


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_queries_beside_a_strong_pair(dtype):
    # the first token stores a value 2^11 times the others', which the later
    # keys and queries are orthogonal to but for their rounding: |S| |q| is some
    # 2^10 times |o|, and the outputs' error beyond their rounding has to be
    # small against o.  2^-20 |S| |q| allows eight times an operand's 2^-23.
    T, D = 200, 64
    q, k, v, g, beta, _ = delta_inputs(41, 1, T, 1, 1, D, D, dtype, init=False, decay=0.001)
    k0 = k[0, 0, 0].double()
    for x in (q, k):
        y = x[0, 1:, 0].double()
        y = y - (y @ k0)[:, None] * k0 / (k0 @ k0)
        x[0, 1:, 0] = (y / y.norm(dim=-1, keepdim=True)).to(x.dtype)
    v[0, 0] *= 2.0 ** 11
    beta[0, 0] = 1.0
    ins = (q, k, v, g, beta, None)
    o, _ = rule(D, D, dtype, scale=1.0).forward(*gpu(*ins[:5]))
    want, S = delta(*double(*ins), None, 1.0)
    strong = S.norm().item() * T ** 0.5
    assert strong > 2.0 ** 7 * want[0, 1:].norm().item()
    o, want = o.cpu()[0, 1:], want[0, 1:]
    rounding = (want.to(o.dtype).double() - want).norm().item()
    error = (o.double() - want).norm().item()
    assert error <= rounding + 2.0 ** -20 * strong


def test_fp32_terms_of_columns_of_all_sizes():
    # columns of v and S spread over 2^12 and 2^16, those of the gradients
    # against them: a value 2^-16 of the largest has all its bits
    T, D = 130, 64
    for spread in (12, 16):
        q, k, v, g, beta, S = delta_inputs(spread, 1, T, 1, 2, D, D, "f32")
        cols = 2.0 ** torch.linspace(0, spread, D).round()
        v, S = v * cols, S * cols
        do = torch.randn(v.shape, generator=torch.Generator().manual_seed(3)) / cols
        op, a = rule(D, D, "f32"), gpu(q, k, v, g, beta, S)
        o, F, saved = op.forward_train(*a[:5], initial_state=a[5])
        d = op.backward(*a[:5], do.cuda(), saved, initial_state=a[5])
        leaf = [x.requires_grad_() for x in double(q, k, v, g, beta, S)]
        want, Fw = delta(*leaf, None, D ** -0.5)
        grads = torch.autograd.grad((want * do.double()).sum(), leaf)
        # column by column where columns differ in size
        pairs = [("o", o, want.detach(), 1 / cols), ("state", F, Fw.detach(), 1 / cols),
                 ("dq", d[0], grads[0], 1), ("dk", d[1], grads[1], 1), ("dv", d[2], grads[2], cols),
                 ("dg", d[3], grads[3], 1), ("dbeta", d[4], grads[4], 1),
                 ("dinit", d[5], grads[5], cols)]
        for name, x, y, s in pairs:
            e = ((x.cpu().double() - y) * s).norm() / (y * s).norm()
            assert e <= TOL["f32"], (spread, name, e.item())


def test_fp32_terms_of_tokens_of_all_sizes():
    # the outputs' gradients spread over 2^16 from token to token; a token's dq
    # follows its own alone
    T, D = 130, 64
    q, k, v, g, beta, S = delta_inputs(14, 1, T, 1, 1, D, D, "f32")
    size = 2.0 ** -torch.randint(0, 17, (T,), generator=torch.Generator().manual_seed(4)).float()
    do = torch.randn(v.shape, generator=torch.Generator().manual_seed(3)) * size[:, None, None]
    op, a = rule(D, D, "f32"), gpu(q, k, v, g, beta, S)
    _, _, saved = op.forward_train(*a[:5], initial_state=a[5])
    dq = op.backward(*a[:5], do.cuda(), saved, initial_state=a[5])[0].cpu().double()
    leaf = double(q, k, v, g, beta, S)
    leaf[0].requires_grad_()
    want, _ = delta(*leaf, None, D ** -0.5)
    want, = torch.autograd.grad((want * do.double()).sum(), leaf[:1])
    e = (dq - want) / size[:, None, None]
    assert e.norm() <= TOL["f32"] * (want / size[:, None, None]).norm()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decay_gradients_of_each_head(dtype):
    # g around -rate: dg is e^g times something of order one, head by head.  The
    # factors e^(G_i - G_j) are off by the rounding of their exponents, 23 / 2^24
    # of themselves where e^-16 is the largest: within what fp32 outputs may be off.
    rates = torch.tensor([0.01, 1.0, 4.0, 8.0, 16.0])
    T, H, D = 150, len(rates), 64
    q, k, v, g, beta, S = delta_inputs(51, 1, T, H, H, D, D, dtype)
    g = -rates * (0.9 + 0.2 * torch.rand(1, T, H, generator=torch.Generator().manual_seed(2)))
    gen = torch.Generator().manual_seed(3)
    do = torch.randn(v.shape, generator=gen).to(v.dtype)
    dS = torch.randn(S.shape, generator=gen)
    op, a = rule(D, D, dtype), gpu(q, k, v, g, beta, S)
    _, _, saved = op.forward_train(*a[:5], initial_state=a[5])
    dg = op.backward(*a[:5], do.cuda(), saved, d_final_state=dS.cuda(), initial_state=a[5])[3]
    leaf = double(q, k, v, g, beta, S)
    leaf[3].requires_grad_()
    o, F = delta(*leaf, None, D ** -0.5)
    want, = torch.autograd.grad((o * do.double()).sum() + (F * dS.double()).sum(), leaf[3:4])
    for h in range(H):
        e = (dg[0, :, h].cpu().double() - want[0, :, h]).norm() / want[0, :, h].norm()
        assert e <= TOL["f32"], (rates[h].item(), e.item())
