"""The gated delta rule (sequences, single tokens) against the token
recurrence in 64 bits."""
import math

import pytest
import torch

from tests.mixer_reference import DT, TOL, delta, delta_inputs, rel

pytestmark = pytest.mark.gpu


def rule(Dk, Dv, dtype, **kw):
    from fft_long_convolution_amd.delta import GatedDelta
    return GatedDelta(Dk, Dv, dtype=dtype, **kw)


def gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


def double(*ts):
    return [None if t is None else t.double() for t in ts]


def check_forward(ins, cu, dtype, Dk, Dv):
    o, S = rule(Dk, Dv, dtype).forward(*gpu(*ins[:5]), initial_state=gpu(ins[5])[0],
                                       cu_seqlens=None if cu is None else cu.cuda())
    want_o, want_S = delta(*double(*ins), cu, Dk ** -0.5)
    assert o.dtype == DT[dtype] and S.dtype == torch.float32
    assert rel(o, want_o) <= TOL[dtype]
    assert rel(S, want_S) <= TOL["f32"]


# B, T, Hk, Hv, Dk, Dv
SHAPES = [
    (1, 1, 1, 1, 64, 64),
    (2, 2, 1, 2, 8, 8),
    (1, 63, 2, 2, 128, 128),
    (2, 64, 1, 1, 64, 128),
    (1, 65, 1, 3, 96, 72),
    (2, 200, 2, 4, 128, 128),
    (1, 131, 1, 1, 40, 256),
    (1, 517, 1, 1, 128, 64),
]


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype, init):
    ins = delta_inputs(sum(shape), *shape, dtype, init=init)
    check_forward(ins, None, dtype, shape[4], shape[5])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bounds", [
    [0, 1], [0, 0, 5, 5, 6, 70, 70], [0, 64, 128, 129, 300], [0, 3, 67, 131, 195, 196],
    [0, 0, 0], [0, 10, 10, 10, 11, 12, 13, 14, 80]], ids=str)
def test_packed_sequences(bounds, dtype):
    cu = torch.tensor(bounds)
    ins = delta_inputs(len(bounds), 1, bounds[-1], 1, 2, 64, 64, dtype, rows=len(bounds) - 1)
    if bounds[-1] == 0:
        o, S = rule(64, 64, dtype).forward(*gpu(*ins[:5]), initial_state=ins[5].cuda(),
                                           cu_seqlens=cu.cuda())
        assert o.shape[1] == 0 and torch.equal(S.cpu(), ins[5])
        return
    check_forward(ins, cu, dtype, 64, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_decay_and_strong_decay(dtype):
    for decay in (0.0, 40.0):
        ins = delta_inputs(5, 1, 300, 1, 2, 64, 64, dtype, decay=decay)
        check_forward(ins, None, dtype, 64, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_resets_and_silent_tokens(dtype):
    # g = -inf drops the state; beta = 0 writes nothing
    ins = list(delta_inputs(6, 1, 150, 1, 2, 64, 64, dtype))
    g, beta = ins[3].clone(), ins[4].clone()
    g[0, 10] = -math.inf
    g[0, 63, 0] = -math.inf
    g[0, 64, 1] = -1e30
    g[0, 100:103] = -math.inf
    beta[0, 20:90] = 0
    ins[3], ins[4] = g, beta
    check_forward(ins, None, dtype, 64, 64)
    beta.zero_()
    check_forward(ins, None, dtype, 64, 64)


def test_nan_stays_in_its_sequence():
    cu = torch.tensor([0, 70, 140])
    ins = delta_inputs(7, 1, 140, 1, 1, 64, 64, "f32", rows=2)
    for i, t in ((2, 69), (3, 69), (0, 69), (1, 69), (4, 69)):
        bad = list(ins)
        bad[i] = ins[i].clone()
        bad[i][0, t] = math.nan
        o, S = rule(64, 64, "f32").forward(*gpu(*bad[:5]), initial_state=bad[5].cuda(),
                                           cu_seqlens=cu.cuda())
        good, Sg = rule(64, 64, "f32").forward(*gpu(*ins[:5]), initial_state=ins[5].cuda(),
                                               cu_seqlens=cu.cuda())
        assert torch.isnan(o[0, 69]).any()
        assert torch.equal(o[0, :64], good[0, :64]) and torch.equal(o[0, 70:], good[0, 70:])
        assert torch.equal(S[1], Sg[1])


def test_large_and_small_scales():
    # bf16 terms have fp32's range: inputs far from one lose nothing
    for s in (1e-12, 1e12):
        q, k, v, g, beta, S = delta_inputs(8, 1, 100, 1, 1, 64, 64, "f32")
        check_forward((q, k, v * s, g, beta, S * s), None, "f32", 64, 64)


def test_strided_views_and_streams():
    q, k, v, g, beta, S = gpu(*delta_inputs(9, 2, 100, 2, 2, 64, 64, "bf16"))
    op = rule(64, 64, "bf16")
    want = op.forward(q, k, v, g, beta, initial_state=S)
    wide = torch.zeros(100, 2, 6, 64, dtype=q.dtype, device="cuda").transpose(0, 1)
    for i, x in enumerate((q, k, v)):
        wide[:, :, 2 * i:2 * i + 2] = x
    a = [wide[:, :, 2 * i:2 * i + 2] for i in range(3)]
    got = op.forward(*a, g, beta, initial_state=S)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # head-major tensors, misaligned ones, broken inner strides
    hm = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
    got = op.forward(*hm, g, beta, initial_state=S)
    assert torch.equal(got[0], want[0])
    odd = [torch.empty(x.numel() + 3, dtype=x.dtype, device="cuda")[3:].view_as(x).copy_(x)
           for x in (q, k, v)]
    s = torch.cuda.Stream()
    got = op.forward(*odd, g, beta, initial_state=S, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0])
    inner = [x.transpose(2, 3).contiguous().transpose(2, 3) for x in (q, k, v)]
    assert torch.equal(op.forward(*inner, g, beta, initial_state=S)[0], want[0])


def test_bounds_out_of_order_stay_in_the_tensors():
    # clamped on the device: any result, but nothing outside is read or written
    ins = gpu(*delta_inputs(10, 1, 100, 1, 1, 64, 64, "bf16", rows=3))
    cu = torch.tensor([-5, 90, 40, 1000], device="cuda")
    o, S = rule(64, 64, "bf16").forward(*ins[:5], initial_state=ins[5], cu_seqlens=cu)
    assert torch.isfinite(S).all()


STEPS = [(1, 1, 1, 8, 8), (3, 2, 4, 64, 64), (2, 1, 1, 96, 40), (5, 3, 3, 128, 128),
         (1, 1, 2, 128, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", STEPS, ids=str)
def test_step(shape, dtype):
    N, Hk, Hv, Dk, Dv = shape
    q, k, v, g, beta, _ = delta_inputs(sum(shape), N, 1, Hk, Hv, Dk, Dv, dtype)
    gen = torch.Generator().manual_seed(1)
    pool = torch.randn(N + 3, Hv, Dk, Dv, generator=gen)
    slots = torch.randperm(N + 3, generator=gen)[:N]
    state = pool.cuda()
    o = rule(Dk, Dv, dtype).step(*gpu(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0]), state,
                                 slots=slots.cuda())
    want_o, want_S = delta(*double(q, k, v, g, beta, pool[slots]), None, Dk ** -0.5)
    assert rel(o, want_o[:, 0]) <= TOL[dtype]
    assert rel(state[slots.cuda()], want_S) <= TOL["f32"]
    rest = [i for i in range(N + 3) if i not in slots.tolist()]
    assert torch.equal(state.cpu()[rest], pool[rest])


def test_step_padding_and_reset():
    q, k, v, g, beta, _ = delta_inputs(2, 4, 1, 1, 1, 64, 64, "f32")
    g[3] = -math.inf
    state = torch.randn(4, 1, 64, 64).cuda()
    was = state.clone()
    o = rule(64, 64, "f32").step(*gpu(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0]), state,
                                 slots=torch.tensor([0, -1, 4, 2]).cuda())
    assert torch.equal(o[1:3], torch.zeros_like(o[1:3]))
    assert torch.equal(state[1], was[1]) and torch.equal(state[3], was[3])
    w = delta(*double(q[3:], k[3:], v[3:], g[3:], beta[3:], was.cpu()[2:3]), None, 0.125)
    assert rel(state[2:3], w[1]) <= TOL["f32"] and rel(o[3:], w[0][:, 0]) <= TOL["f32"]


def test_steps_continue_a_prompt():
    ins = gpu(*delta_inputs(11, 2, 90, 1, 2, 64, 64, "f32"))
    op = rule(64, 64, "f32")
    o, S = op.forward(*ins[:5], initial_state=ins[5])
    _, state = op.forward(*(x[:, :80] for x in ins[:5]), initial_state=ins[5])
    for t in range(80, 90):
        y = op.step(*(x[:, t] for x in ins[:5]), state)
        assert rel(y, o[:, t].cpu()) <= 2 * TOL["f32"]
    assert rel(state, S.cpu()) <= 2 * TOL["f32"]


def test_refusals():
    from fft_long_convolution_amd.delta import GatedDelta
    from fft_long_convolution_amd.fftconv import FFTConvError
    q, k, v, g, beta, S = gpu(*delta_inputs(3, 1, 4, 2, 4, 64, 64, "bf16"))
    op = rule(64, 64, "bf16")
    for bad in ((q.float(), k, v, g, beta), (q, k[:, :3], v, g, beta), (q, k, v, g.half(), beta),
                (q, k, v, g[:, :, :2], beta), (q.cpu(), k, v, g, beta), (q[0], k, v, g, beta)):
        with pytest.raises(ValueError):
            op.forward(*bad)
    with pytest.raises(ValueError):
        op.forward(q, k, v, g, beta, initial_state=S[:, :2])
    with pytest.raises(ValueError):
        op.forward(q, k, v, g, beta, cu_seqlens=torch.tensor([0, 4], dtype=torch.int32).cuda())
    with pytest.raises(FFTConvError) as e:      # 4 heads of v over 3 of k
        op.forward(*(torch.cat([x, x[:, :, :1]], 2) for x in (q, k)), v, g, beta)
    assert e.value.status == 1
    with pytest.raises(FFTConvError) as e:
        op.forward(q, k, v, g, beta, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(FFTConvError) as e:
        op.forward(q, k, v, g, beta, out=v.view(v.shape))
    assert e.value.status == 1
    with pytest.raises(FFTConvError) as e:
        op.forward(q, k, v, g, beta, initial_state=S, final_state=S)
    assert e.value.status == 1
    for Dk, Dv in ((136, 64), (60, 64), (64, 1032)):
        ins = gpu(*delta_inputs(4, 1, 2, 1, 1, Dk, Dv, "bf16"))
        with pytest.raises(FFTConvError) as e:
            GatedDelta(Dk, Dv).forward(*ins[:5])
        assert e.value.status == 2
    with pytest.raises(ValueError):
        op.step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], S.transpose(2, 3))


# ------------------------------------------------------------- gradients

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinit")


def run_backward(ins, cu, dtype, Dk, Dv, do, dS):
    op = rule(Dk, Dv, dtype)
    a = gpu(*ins[:5])
    kw = dict(initial_state=gpu(ins[5])[0], cu_seqlens=None if cu is None else cu.cuda())
    o, S, saved = op.forward_train(*a, **kw)
    o2, S2 = op.forward(*a, **kw)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    return op.backward(*a, do.cuda(), saved, d_final_state=gpu(dS)[0], **kw)


def check_backward(ins, cu, dtype, Dk, Dv, with_final=True):
    gen = torch.Generator().manual_seed(77)
    do = torch.randn(ins[2].shape, generator=gen).to(DT[dtype])
    rows = ins[0].shape[0] if cu is None else len(cu) - 1
    dS = torch.randn(rows, ins[2].shape[2], Dk, Dv, generator=gen) if with_final else None
    got = run_backward(ins, cu, dtype, Dk, Dv, do, dS)
    again = run_backward(ins, cu, dtype, Dk, Dv, do, dS)
    leaf = [None if x is None else x.requires_grad_() for x in double(*ins)]
    o, S = delta(*leaf, cu, Dk ** -0.5)
    loss = (o * do.double()).sum() + (0 if dS is None else (S * dS.double()).sum())
    want = torch.autograd.grad(loss, [x for x in leaf if x is not None])
    assert (got[5] is None) == (ins[5] is None)
    for i, (n, w) in enumerate(zip(NAMES, want)):
        assert got[i].dtype == ins[i].dtype
        assert torch.equal(got[i], again[i]), n
        t = TOL[dtype if i < 3 else "f32"]
        assert rel(got[i], w) <= t, (n, rel(got[i], w))


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype, init):
    ins = delta_inputs(sum(shape) + 1, *shape, dtype, init=init)
    check_backward(ins, None, dtype, shape[4], shape[5], with_final=init)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bounds", [[0, 1], [0, 0, 5, 5, 6, 70, 70], [0, 64, 128, 129, 300],
                                    [0, 10, 10, 10, 11, 12, 13, 14, 80]], ids=str)
def test_backward_packed(bounds, dtype):
    cu = torch.tensor(bounds)
    ins = delta_inputs(len(bounds), 1, bounds[-1], 1, 2, 64, 64, dtype, rows=len(bounds) - 1)
    check_backward(ins, cu, dtype, 64, 64)


def test_backward_resets_and_silent_tokens():
    ins = list(delta_inputs(6, 1, 150, 1, 2, 64, 64, "f32"))
    g, beta = ins[3].clone(), ins[4].clone()
    g[0, 10] = -200.0
    g[0, 63, 0] = -1e30
    g[0, 100:103] = -1e4
    beta[0, 20:90] = 0
    ins[3], ins[4] = g, beta
    check_backward(ins, None, "f32", 64, 64)
    # -inf: the factor is 0 and so is its gradient; the 64-bit form would
    # multiply 0 by inf, so its log decay there is a large finite one
    got = []
    for low in (-math.inf, -1e30):
        g[0, 10] = low
        ins[3] = g
        got.append(run_backward(ins, None, "f32", 64, 64, torch.ones_like(ins[2]), None))
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    assert (got[0][3][0, 10] == 0).all()


def test_backward_of_empty_sequences():
    op = rule(64, 64, "bf16")
    q, k, v, g, beta, S = gpu(*delta_inputs(3, 1, 0, 1, 2, 64, 64, "bf16", rows=2))
    cu = torch.zeros(3, dtype=torch.int64, device="cuda")
    o, F, saved = op.forward_train(q, k, v, g, beta, initial_state=S, cu_seqlens=cu)
    assert torch.equal(F, S)
    d = op.backward(q, k, v, g, beta, o, saved, d_final_state=2 * S, initial_state=S,
                    cu_seqlens=cu)
    assert torch.equal(d[5], 2 * S)


def test_gradient_against_differences():
    # fp32 kernels: central differences of the library's own forward.  With
    # h = 2^-6 the third derivative leaves about h^2 / 6 = 4e-5 of a value of
    # order one, and rounding 1e-6 * |loss| / h = 6e-5 |loss|; |loss| < 10.
    ins = gpu(*delta_inputs(12, 1, 70, 1, 2, 16, 16, "f32"))
    op = rule(16, 16, "f32")
    gen = torch.Generator().manual_seed(5)
    do = (0.1 * torch.randn(ins[2].shape, generator=gen)).cuda()
    dS = (0.1 * torch.randn(ins[5].shape, generator=gen)).cuda()

    def loss(a):
        o, S = op.forward(*a[:5], initial_state=a[5])
        return ((o.double() * do).sum() + (S.double() * dS).sum()).item()

    o, S, saved = op.forward_train(*ins[:5], initial_state=ins[5])
    d = op.backward(*ins[:5], do, saved, d_final_state=dS, initial_state=ins[5])
    h = 2.0 ** -6
    for i, x in enumerate(ins):
        for j in torch.randint(0, x.numel(), (8,), generator=gen).tolist():
            up, down = list(ins), list(ins)
            for a, s in ((up, h), (down, -h)):
                a[i] = x.clone()
                a[i].view(-1)[j] += s
            diff = (loss(up) - loss(down)) / (2 * h)
            assert abs(diff - d[i].reshape(-1)[j].item()) <= 2e-3, NAMES[i]


def test_backward_refusals():
    from fft_long_convolution_amd.fftconv import FFTConvError
    q, k, v, g, beta, S = gpu(*delta_inputs(3, 1, 4, 2, 4, 64, 64, "bf16"))
    op = rule(64, 64, "bf16")
    o, F, saved = op.forward_train(q, k, v, g, beta)
    with pytest.raises(ValueError):
        op.backward(q, k, v, g, beta, o.float(), saved)
    with pytest.raises(ValueError):
        op.backward(q, k, v, g, beta, o, saved, d_final_state=F[:, :2])
    with pytest.raises(FFTConvError) as e:
        op.backward(q, k, v, g, beta, o, saved[:-16])
    assert e.value.status == 1
    with pytest.raises(FFTConvError) as e:
        op.backward(q, k, v, g, beta, o, saved,
                    workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
