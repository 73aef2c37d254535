"""Values that are not finite in the gated delta rule: what comes before them
stays, what they reach is never a finite number that looks like a result."""
import math

import pytest
import torch

from tests.mixer_reference import TOL, delta, delta_inputs
from tests.test_gpu_delta import double, gpu, rule

pytestmark = pytest.mark.gpu

Q, K, V, G, BETA = range(5)


def spoil(ins, which, value, t):
    """Inputs with `value` at token t: one element of q, k or v, one gate."""
    bad = [x.clone() for x in ins]
    if which in (Q, K, V):
        bad[which][0, t, 0, 3] = value
    else:
        bad[which][0, t, 0] = value
    return bad


def agree(got, want, dtype, scale):
    """Finite exactly where the definition is, and its values there."""
    got, ok = got.cpu().double(), torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), ok)
    if ok.any():
        assert (got - want)[ok].norm() <= TOL[dtype] * scale


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("which", [Q, K, V, G, BETA], ids=["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_tokens_before_are_those_of_the_definition(dtype, which, value):
    if which == G and value == -math.inf:
        return                          # a reset
    # the chunk's first token, inside its first and its second 32, its last
    for T, t in ((140, 64), (140, 69), (140, 101), (140, 127), (140, 0), (40, 39)):
        ins = delta_inputs(t, 1, T, 1, 2, 64, 40, dtype)
        bad = spoil(ins, which, value, t)
        o, S = rule(64, 40, dtype).forward(*gpu(*bad[:5]), initial_state=bad[5].cuda())
        want, Sw = delta(*double(*bad), None, 0.125)
        clean, Sc = delta(*double(*ins), None, 0.125)
        agree(o, want, dtype, clean.norm())
        agree(S, Sw, "f32", Sc.norm())


@pytest.mark.parametrize("which", [K, V, G], ids=["k", "v", "g"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_before_in_a_cut_sequence(dtype, which):
    T = 1300
    for t in (600, 1290):
        ins = delta_inputs(t, 1, T, 1, 1, 64, 64, dtype, decay=0.02)
        bad = spoil(ins, which, math.nan, t)
        o, S = rule(64, 64, dtype).forward(*gpu(*bad[:5]), initial_state=bad[5].cuda())
        want, Sw = delta(*double(*bad), None, 0.125)
        clean, Sc = delta(*double(*ins), None, 0.125)
        agree(o, want, dtype, clean.norm())
        agree(S, Sw, "f32", Sc.norm())


def test_states_that_are_not_finite():
    for value in (math.nan, math.inf):
        ins = list(delta_inputs(3, 1, 70, 1, 2, 64, 40, "f32"))
        ins[5][0, 1, 7, 5] = value
        o, S = rule(64, 40, "f32").forward(*gpu(*ins[:5]), initial_state=ins[5].cuda())
        want, Sw = delta(*double(*ins), None, 0.125)
        clean = torch.nan_to_num(want, 0, 0, 0).norm()
        agree(o, want, "f32", clean)
        # an infinity's column: the other rows of the state stay finite in the
        # definition until their first token
        agree(S, Sw, "f32", torch.nan_to_num(Sw, 0, 0, 0).norm())


@pytest.mark.parametrize("value", [math.nan, math.inf], ids=str)
@pytest.mark.parametrize("which", [Q, K, V, G, BETA, "do", "dS"],
                         ids=["q", "k", "v", "g", "beta", "do", "dS"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_gradient_looks_like_a_result(dtype, which, value):
    # what is finite is right; a chunk's gradients may be NaN beyond what the
    # definition loses, those of chunks it leaves alone may not
    T, t = 200, 70
    ins = delta_inputs(5, 1, T, 1, 2, 64, 64, dtype)
    gen = torch.Generator().manual_seed(6)
    do = torch.randn(ins[2].shape, generator=gen).to(ins[2].dtype)
    dS = torch.randn(ins[5].shape, generator=gen)

    def reference(ins, do, dS):
        leaf = [x.requires_grad_() for x in double(*ins)]
        o, S = delta(*leaf, None, 0.125)
        return torch.autograd.grad((o * do.double()).sum() + (S * dS.double()).sum(), leaf)

    clean = reference(ins, do, dS)
    bad = list(ins)
    if which == "do":
        do = do.clone()
        do[0, t, 0, 3] = value
    elif which == "dS":
        dS = dS.clone()
        dS[0, 0, 3, 3] = value
    else:
        bad = spoil(ins, which, value, t)
    want = reference(bad, do, dS)
    op, a = rule(64, 64, dtype), gpu(*bad)
    _, _, saved = op.forward_train(*a[:5], initial_state=a[5])
    got = op.backward(*a[:5], do.cuda(), saved, d_final_state=dS.cuda(), initial_state=a[5])
    for i, (x, w, c) in enumerate(zip(got, want, clean)):
        x, fin = x.cpu().double(), torch.isfinite(w)
        there = torch.isfinite(x)
        assert not (there & ~fin).any(), i
        assert (x - w)[there].norm() <= TOL[dtype if i < 3 else "f32"] * c.norm(), i
        if i < 5:
            # chunks other than the token's: lost only where the definition loses
            rest = [j for j in range(T) if j // 64 != t // 64]
            if which in (Q, V):
                assert torch.equal(there[0, rest], fin[0, rest]), i


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(3, 200, 96, 96, 16, 24), (2, 130, 24, 72, 128, 128)], ids=str)
def test_other_heads_of_many(shape, dtype):
    # chains in pieces, and eight waves of 128 columns: all chains but one have
    # the bits of the call without NaN, that one's tokens before it their values
    b, t, h = 1, 101, 5
    ins = gpu(*delta_inputs(sum(shape), *shape, dtype))
    op = rule(shape[4], shape[5], dtype)
    d = torch.randn(ins[2].shape, device="cuda").to(ins[2].dtype)

    def run(v):
        a = (*ins[:2], v, *ins[3:5])
        o, S = op.forward(*a, initial_state=ins[5])
        o2, S2, saved = op.forward_train(*a, initial_state=ins[5])
        return [o, o2, S, S2], op.backward(*a, d, saved, d_final_state=S, initial_state=ins[5])

    (clean, _), bad = run(ins[2]), ins[2].clone()
    bad[b, t, h, 3] = math.nan
    got, grads = run(bad)
    for x, y in zip(got[:2], clean[:2]):
        lost = torch.zeros(x.shape, dtype=torch.bool, device="cuda")
        lost[b, t:, h, 3] = True
        assert torch.equal(torch.isnan(x), lost)
        e = (x[b, :t, h, 3].double() - y[b, :t, h, 3].double()).norm()
        assert e <= TOL[dtype] * y[b, :t, h, 3].double().norm()
        lost[b, :, h, 3] = True
        assert torch.equal(x[~lost], y[~lost])
    for x, y in zip(got[2:], clean[2:]):
        lost = torch.zeros(x.shape, dtype=torch.bool, device="cuda")
        lost[b, h, :, 3] = True
        assert torch.equal(torch.isnan(x), lost) and torch.equal(x[~lost], y[~lost])
    assert not torch.isfinite(grads[0][b, t, h // (shape[3] // shape[2])]).any()
    assert torch.isfinite(grads[2][0]).all()
