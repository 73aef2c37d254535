"""Linear attention with decays and layer norm as a model uses them: views of one
projection, long sequences, tokens that no sequence holds, values that are not
finite, other streams, graphs, states past 4 GiB, and a layer of all of them."""
import math

import pytest
import torch

from tests.decay_reference import DT, TOL, decay, decay_inputs, layer_norm, rel
from tests.test_gpu_decay import attend, check_forward, double, gpu
from tests.test_gpu_decay_grad import NAMES, check, gradients, tangents, wanted
from tests.test_gpu_layernorm import norm

pytestmark = pytest.mark.gpu
TYPES = ["bf16", "f16", "f32"]


def kind(name, dtype):
    return "f32" if name in ("dg", "dinit") else dtype


# ------------------------------------------------------------------- views

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [0, 8, 3])
def test_views_of_one_projection(dtype, offset):
    B, T, Hk, Hv, Dk, Dv = 2, 75, 2, 4, 64, 40
    ins = gpu(*decay_inputs(offset, B, T, Hk, Hv, Dk, Dv, dtype))
    q, k, v, g, S = ins
    wide = torch.full((B, T, offset + 2 * Hk * Dk + Hv * Dv + 16), math.nan,
                      dtype=DT[dtype], device="cuda")
    at, views = offset, []
    for x in (q, k, v):
        n = x.shape[2] * x.shape[3]
        views.append(wide[..., at:at + n].unflatten(-1, x.shape[2:]))
        views[-1].copy_(x)
        at += n
    op = attend(Dk, Dv, dtype)
    do = torch.randn(v.shape, device="cuda").to(DT[dtype])
    want = op.forward(q, k, v, g, initial_state=S)
    got = op.forward(*views, g, initial_state=S)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want = op.backward(q, k, v, g, do, initial_state=S)
    got = op.backward(*views, g, do, initial_state=S)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    a, b = S.clone(), S.clone()
    want = op.step(q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), g[:, 0], a)
    got = op.step(*(x[:, 0] for x in views), g[:, 0], b)
    assert torch.equal(got, want) and torch.equal(a, b)


def test_broadcast_inputs():
    """One row of q and k for the whole batch; gradients are those of each row."""
    q, k, v, g, S = gpu(*decay_inputs(3, 3, 70, 1, 2, 64, 64, "bf16"))
    q, k = q[:1].expand(3, -1, -1, -1), k[:1].expand(3, -1, -1, -1)
    op, do = attend(64, 64, "bf16"), torch.randn(v.shape, device="cuda").bfloat16()
    for fn in (lambda q, k: op.forward(q, k, v, g, initial_state=S),
               lambda q, k: op.backward(q, k, v, g, do, initial_state=S)):
        assert all(torch.equal(a, b) for a, b in zip(fn(q, k), fn(q.contiguous(), k.contiguous())))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 768, 333])
def test_layer_norm_views(D, dtype):
    gen = torch.Generator().manual_seed(D)
    wide = torch.randn(3, 5, D + 32, generator=gen).to(DT[dtype]).cuda()
    w, b = (1 + 0.1 * torch.randn(D, generator=gen)).cuda(), torch.randn(D, generator=gen).cuda()
    dy = torch.randn(3, 5, D, generator=gen).to(DT[dtype]).cuda()
    op = norm(D, dtype)
    for x in (wide[..., :D], wide[..., 3:3 + D], wide[:, :1, 16:16 + D].expand(3, 5, D)):
        y, g = op.forward(x, w, b), op.backward(x, dy, w, b)
        z = x.contiguous()
        assert torch.equal(y, op.forward(z, w, b))
        assert all(torch.equal(a, c) for a, c in zip(g, op.backward(z, dy, w, b)))
        assert rel(y, layer_norm(*double(x.cpu(), w.cpu(), b.cpu()), 1e-5)) <= TOL[dtype]


# ------------------------------------------------- long sequences, many heads

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1300, 4000])
def test_cut_sequences(T, dtype):
    ins = decay_inputs(T, 1, T, 1, 2, 64, 64, dtype, rate=0.01)
    op = attend(64, 64, dtype)
    assert op._lib.fftconv_decay_workspace_bytes(
        op._describe(*gpu(*ins[:4]), None, None)[0][1][0]) > 0
    check_forward(ins, None, dtype, 64, 64)
    check(ins, None, dtype, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_sequences_that_are_cut(dtype):
    bounds = [5, 5, 700, 701, 2100, 2100, 2164]
    ins = decay_inputs(9, 1, 2200, 1, 2, 64, 128, dtype, rows=6, rate=0.02)
    check_forward(ins, torch.tensor(bounds), dtype, 64, 128)
    check(ins, torch.tensor(bounds), dtype, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_heads(dtype):
    """More workgroups than the card holds at once, sequences walked whole."""
    ins = decay_inputs(2, 20, 70, 8, 16, 64, 128, dtype)
    check_forward(ins, None, dtype, 64, 128)
    check(ins, None, dtype, True)


def test_a_cut_sequence_is_the_whole_one():
    """The same sequences as rows of a large batch, walked whole, and alone, cut."""
    q, k, v, g, S = gpu(*decay_inputs(4, 1, 640, 1, 1, 64, 64, "f32", rate=0.02))
    op, n = attend(64, 64, "f32"), 600
    o, fin = op.forward(q, k, v, g, initial_state=S)
    many = [x.expand(n, *x.shape[1:]) for x in (q, k, v)]
    O, F = op.forward(*many, g.expand(n, -1, -1), initial_state=S.expand(n, -1, -1, -1))
    for x, y in ((o, O), (fin, F)):
        assert all(torch.equal(y[i], y[0]) for i in (1, n // 2, n - 1))
        assert rel(x[0], y[0].cpu().double()) <= TOL["f32"]


# ------------------------------------------------------ tokens nobody holds

@pytest.mark.parametrize("T, first, last", [(64, 10, 40), (3000, 64, 2000), (40, 40, 40),
                                            (100, 0, 0)])
def test_tokens_that_no_sequence_holds(T, first, last):
    ins = list(decay_inputs(T, 1, T, 1, 2, 64, 64, "bf16", rows=2))
    cu = torch.tensor([first, (first + last) // 2, last]).cuda()
    q, k, v, g, S = gpu(*ins)
    out = torch.zeros(T, dtype=torch.bool)
    out[:first], out[last:] = True, True
    for x in (q, k, v, g):
        x[:, out] = math.nan                 # padding holds anything
    op = attend(64, 64, "bf16")
    o, fin = op.forward(q, k, v, g, initial_state=S, cu_seqlens=cu)
    given = torch.full_like(v, 7.0)
    o2, _ = op.forward(q, k, v, g, initial_state=S, cu_seqlens=cu, out=given)
    assert o2 is given and (o[:, out] == 0).all() and (given[:, out] == 7).all()
    assert torch.equal(o[:, ~out], given[:, ~out])
    want, want_S = decay(*double(*ins), cu.cpu(), 0.125)
    assert rel(fin, want_S) <= TOL["f32"]
    if first < last:
        assert rel(o, want) <= TOL["bf16"]
    do = torch.randn(v.shape, device="cuda").bfloat16()
    do[:, out] = math.nan
    d = op.backward(q, k, v, g, do, initial_state=S, cu_seqlens=cu)
    assert all((x[:, out] == 0).all() for x in d[:4])
    want = wanted(ins, torch.where(out[None, :, None, None], 0, do.cpu()), None, cu.cpu())
    for name, x, y in zip(NAMES, d, want):
        assert (x == 0).all() if not y.any() else rel(x, y) <= TOL[kind(name, "bf16")], name


@pytest.mark.parametrize("bounds", [[-5, 30, 300, 400], [-9, -3, -1, 200], [90, 95, 95, 99]], ids=str)
def test_bounds_outside_are_clamped(bounds):
    T = 90
    q, k, v, g, S = gpu(*decay_inputs(1, 1, T, 1, 1, 64, 64, "f32", rows=3))
    op, runs = attend(64, 64, "f32"), []
    for cu in (torch.tensor(bounds), torch.tensor(bounds).clamp(0, T)):
        runs.append([*op.forward(q, k, v, g, initial_state=S, cu_seqlens=cu.cuda()),
                     *op.backward(q, k, v, g, v, initial_state=S, cu_seqlens=cu.cuda())])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


# ------------------------------------------------------- nothing and little

def test_empty():
    op, ln = attend(64, 64, "bf16"), norm(64, "bf16")
    for B, T in ((0, 5), (2, 0), (0, 0)):
        q, v, g = (torch.empty(B, T, 2, 64, dtype=torch.bfloat16, device="cuda"),
                   torch.empty(B, T, 4, 64, dtype=torch.bfloat16, device="cuda"),
                   torch.empty(B, T, 4, device="cuda"))
        S = torch.randn(B, 4, 64, 64, device="cuda")
        o, fin = op.forward(q, q, v, g, initial_state=S)
        assert o.shape == v.shape and torch.equal(fin, S)
        assert (op.forward(q, q, v, g)[1] == 0).all()
        d = op.backward(q, q, v, g, v, d_final_state=S, initial_state=S)
        assert [x.shape for x in d] == [x.shape for x in (q, q, v, g, S)]
        assert torch.equal(d[4], S)
        d = op.backward(q, q, v, torch.full((4,), -0.1, device="cuda"), v)
        assert (d[3] == 0).all()
    for n in (0, 3):
        q, v = (torch.empty(n, h, 64, dtype=torch.bfloat16, device="cuda") for h in (2, 4))
        slots = torch.full((n,), -1, device="cuda")
        o = op.step(q, q, v, torch.zeros(4, device="cuda"), torch.empty(0, 4, 64, 64, device="cuda"),
                    slots=slots)
        assert (o == 0).all()
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    assert ln.forward(x, w, w).shape == x.shape
    dx, dw, db = ln.backward(x, x, w, w)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all()


# ------------------------------------------------------ values not finite

Q, K, V, G = range(4)


def agree(got, want, dtype, scale):
    """Finite exactly where the definition is, and its values there."""
    got, ok = got.cpu().double(), torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), ok)
    if ok.any():
        assert (got - want)[ok].norm() <= TOL[dtype] * scale


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("which", [Q, K, V, G], ids=["q", "k", "v", "g"])
@pytest.mark.parametrize("dtype", TYPES)
def test_not_finite(dtype, which, value):
    if which == G and value == -math.inf:
        return                          # a reset
    # a chunk's first and last token, one inside it, the sequence's first and last; cut
    for T, t in ((140, 64), (140, 69), (140, 95), (140, 0), (40, 39), (1300, 600)):
        ins = decay_inputs(t, 1, T, 1, 2, 64, 40, dtype, rate=0.02 if T > 1000 else 0.3)
        bad = [x.clone() for x in ins]
        bad[which][(0, t, 0, 3)[:bad[which].dim()]] = value
        o, S = attend(64, 40, dtype).forward(*gpu(*bad[:4]), initial_state=bad[4].cuda())
        want, want_S = decay(*double(*bad), None, 0.125)
        clean, clean_S = decay(*double(*ins), None, 0.125)
        agree(o, want, dtype, clean.norm())
        agree(S, want_S, "f32", clean_S.norm())


@pytest.mark.parametrize("which", [Q, K, V, G, 5], ids=["q", "k", "v", "g", "do"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_not_finite(dtype, which):
    """Other sequences of the batch and other heads do not see it; where the
    definition has no finite gradient, there is none."""
    B, T, t = 3, 200, 77
    ins = list(decay_inputs(t, B, T, 2, 2, 64, 40, dtype))
    do, _ = tangents(1, ins, B, False)
    clean = gradients(ins, do, None, None, dtype)
    (ins[which] if which < 5 else do)[(1, t, 0, 3)[:3 if which == G else 4]] = math.nan
    got, want = gradients(ins, do, None, None, dtype), wanted(ins, do, None, None)
    for name, x, y, z in zip(NAMES, got, want, clean):
        assert torch.equal(x[[0, 2]], z[[0, 2]]), name
        if name == "dinit":
            assert torch.equal(x[:, 1], z[:, 1])
        else:
            assert torch.equal(x[:, :, 1], z[:, :, 1]), name
        assert not torch.isfinite(x.cpu()[~torch.isfinite(y)]).any(), name


def test_layer_norm_not_finite():
    x = torch.randn(5, 96)
    x[1, 3], x[3, 0] = math.nan, math.inf
    w = torch.ones(96).cuda()
    y = norm(96, "f32").forward(x.cuda(), w, w)
    dx, dw, _ = norm(96, "f32").backward(x.cuda(), x.cuda().nan_to_num(0, 1, -1), w, w)
    for a in (y, dx):
        assert torch.isfinite(a[[0, 2, 4]]).all() and not torch.isfinite(a[[1, 3]]).any()
    assert not torch.isfinite(dw).any()


# ------------------------------------------- streams, graphs, long addresses

def layer(dtype="bf16", D=64, H=2, T=1100, B=1, project=True):
    """Layer norm, projections, norm of q and k, attention, gradients of all of it,
    and a step, on given tensors: as a training step and a server would."""
    from fft_long_convolution_amd.delta import QKNorm
    width = H * D if project else 3 * H * D
    ln, qk, op = norm(width, dtype), QKNorm(D, dtype=dtype), attend(D, D, dtype)
    w, b = torch.ones(width).cuda(), torch.zeros(width).cuda()
    S = torch.randn(B, H, D, D, device="cuda")

    def inputs(seed):
        gen = torch.Generator().manual_seed(seed)
        return [torch.randn(B, T, width, generator=gen).to(DT[dtype]).cuda(),
                (torch.randn(width, 3 * width, generator=gen) / width ** 0.5).to(DT[dtype]).cuda(),
                (-0.05 * torch.rand(B, T, H, generator=gen)).cuda(),
                torch.randn(B, T, H, D, generator=gen).to(DT[dtype]).cuda()]

    def run(x, W, g, do, state):
        y = ln.forward(x, w, b)
        q, k, v = (y @ W if project else y).unflatten(-1, (3 * H, D)).split(H, 2)
        nq, nk = qk.forward(q, k)
        o, fin = op.forward(nq, nk, v, g, initial_state=S)
        d = op.backward(nq, nk, v, g, do, d_final_state=fin, initial_state=S)
        n = qk.backward(q, k, d[0], d[1])
        dqkv = torch.cat([n[0], n[1], d[2]], 2).flatten(2)
        dy = dqkv @ W.t().contiguous() if project else dqkv
        state.copy_(fin)
        z = op.step(nq[:, -1], nk[:, -1], v[:, -1], g[:, -1], state)
        return [y, o, fin, *d, dqkv, *ln.backward(x, dy, w, b), z, state]
    return inputs, run, S


def test_graph_of_a_layer_is_replayed():
    # the framework's own calls only: no library product in the graph
    inputs, run, S = layer(project=False)
    static, state = inputs(1), torch.empty_like(S)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            run(*static, state)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(*static, state)
    for seed in (2, 3, 2, 4):
        fresh = inputs(seed)
        for x, y in zip(static, fresh):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        seen = [x.clone() for x in got]
        want = run(*fresh, torch.empty_like(S))
        torch.cuda.synchronize()
        for a, b in zip(seen, want):
            assert torch.equal(a, b)


def test_a_layer_against_64_bits():
    """All of it in fp32 against automatic gradients of the plain forms in 64 bits."""
    D, H, T = 64, 2, 150
    inputs, run, S = layer("f32", D, H, T)
    x, W, g, do = inputs(5)
    got = run(x, W, g, do, torch.empty_like(S))
    x, W, g, do = (t.cpu().double() for t in (x, W, g, do))
    x.requires_grad_()
    y = layer_norm(x, None, None, 1e-5)
    q, k, v = (y @ W).unflatten(-1, (3 * H, D)).split(H, 2)
    q, k = (t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) for t in (q, k))
    o, fin = decay(q, k, v, g, S.cpu().double(), None, D ** -0.5)
    dx, = torch.autograd.grad([o, fin], [x], [do, fin.detach()])
    # two fp32 matrix products of the library and eight operators one after the other
    for a, b in ((got[1], o), (got[2], fin), (got[9], dx)):
        assert rel(a, b.detach()) <= 8 * TOL["f32"]


def test_other_streams():
    """Calls on a stream of their own, at the same time as others on the default one."""
    inputs, run, S = layer(T=300)
    ins = [inputs(i) for i in (1, 2)]
    want = [run(*x, torch.empty_like(S)) for x in ins]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(3):
        with torch.cuda.stream(side):
            got[0] = run(*ins[0], torch.empty_like(S))
        got[1] = run(*ins[1], torch.empty_like(S))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    # a stream that is given, not the current one
    q, k, v, g, init = gpu(*decay_inputs(1, 1, 500, 1, 1, 64, 64, "bf16"))
    op = attend(64, 64, "bf16")
    want = op.forward(q, k, v, g, initial_state=init)
    torch.cuda.synchronize()
    got = op.forward(q, k, v, g, initial_state=init, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_equal_calls_give_equal_bits():
    for dtype in TYPES:
        q, k, v, g, S = gpu(*decay_inputs(2, 2, 900, 2, 4, 64, 64, dtype, rate=0.02))
        op, ln = attend(64, 64, dtype), norm(700, dtype)
        x = torch.randn(900, 700, device="cuda").to(DT[dtype])
        w = torch.ones(700, device="cuda")
        runs = [[*op.forward(q, k, v, g, initial_state=S),
                 *op.backward(q, k, v, g, v, initial_state=S), *op.backward(q, k, v, g[0, 0], v)[:4],
                 *ln.backward(x, x, w, w)] for _ in range(3)]
        for other in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_a_pool_past_4_gib():
    H, D = 4, 128
    pool = (1 << 32) // (H * D * D * 4) + 40
    q, k, v, g, S = decay_inputs(3, 3, 1, H, H, D, D, "bf16")
    state = torch.empty(pool, H, D, D, device="cuda")
    slots = torch.tensor([pool - 1, 0, pool - 17], device="cuda")
    state[slots] = S.cuda()
    o = attend(D, D, "bf16").step(*gpu(q[:, 0], k[:, 0], v[:, 0], g[:, 0]), state, slots=slots)
    want_o, want_S = decay(*double(q, k, v, g, S), None, D ** -0.5)
    assert rel(o, want_o[:, 0]) <= TOL["bf16"] and rel(state[slots], want_S) <= TOL["f32"]


def test_tokens_past_4_gib():
    """A row of q, k and v past 4 GiB of one tensor: the last sequence of a batch."""
    B, T, H, D = 3, 40, 1, 64
    far = (1 << 30) + 8                     # 2-byte elements between rows
    wide = torch.empty((B - 1) * far + T * 3 * H * D, dtype=torch.bfloat16, device="cuda")
    ins = decay_inputs(6, B, T, H, H, D, D, "bf16")
    views = []
    for i, x in enumerate(gpu(*ins[:3])):
        views.append(torch.as_strided(wide, x.shape, (far, 3 * H * D, D, 1), i * H * D))
        views[-1].copy_(x)
    assert (B - 1) * far * 2 >= 1 << 32
    o, S = attend(D, D, "bf16").forward(*views, ins[3].cuda(), initial_state=ins[4].cuda())
    want_o, want_S = decay(*double(*ins), None, 0.125)
    assert rel(o, want_o) <= TOL["bf16"] and rel(S, want_S) <= TOL["f32"]


def test_layer_norm_past_4_gib():
    D, rows = 64, 3
    far = (1 << 31) // (rows - 1) + 8
    wide = torch.empty((rows - 1) * far + D, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(wide, (rows, D), (far, 1))
    x.copy_(torch.randn(rows, D))
    w = torch.ones(D, device="cuda")
    y, z = norm(D, "bf16").forward(x, w, w), x.contiguous()
    assert torch.equal(y, norm(D, "bf16").forward(z, w, w))
    assert all(torch.equal(a, b) for a, b in zip(norm(D, "bf16").backward(x, z, w, w),
                                                 norm(D, "bf16").backward(z, z, w, w)))


def test_more_rows_than_a_launch_takes():
    """16 rows a workgroup of 256 threads: 2^28 rows are 2^32 threads."""
    base = torch.randn(1 << 14, 8, device="cuda").bfloat16()
    n, w = (1 << 14) + 1, torch.ones(8, device="cuda")
    x = base.repeat(n, 1)
    y = norm(8, "bf16").forward(x, w, w).view(n, 1 << 14, 8)
    want = norm(8, "bf16").forward(base, w, w)
    for i in (0, 1, n // 2, n - 2, n - 1):
        assert torch.equal(y[i], want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_states_are_joined(dtype):
    """Cut sequences of so many states that a thread joins several elements: each row
    as it is by itself (other segments, so other roundings)."""
    B, T, H, D = 20, 1000, 2, 128
    assert B * H * D * D // 256 > 2048
    q, k, v, g, S = gpu(*decay_inputs(8, B, T, H, H, D, D, dtype, rate=0.02))
    op = attend(D, D, dtype)
    assert op._lib.fftconv_decay_workspace_bytes(op._describe(q, k, v, g, None, None)[0][1][0]) > 0
    do = torch.randn(v.shape, device="cuda").to(DT[dtype])
    got = [*op.forward(q, k, v, g, initial_state=S),
           *op.backward(q, k, v, g, do, d_final_state=S, initial_state=S)]
    for i in (0, 7, B - 1):
        r = [x[i:i + 1] for x in (q, k, v, g, S, do)]
        want = [*op.forward(*r[:4], initial_state=r[4]),
                *op.backward(*r[:4], r[5], d_final_state=r[4], initial_state=r[4])]
        for name, x, y in zip(("o", "state", *NAMES), got, want):
            t = "f32" if name == "state" else kind(name, dtype)
            assert rel(x[i:i + 1], y.cpu().double()) <= 2 * TOL[t], name
