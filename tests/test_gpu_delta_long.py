"""The gated delta rule where its launches take other forms than at the sizes
of a few chunks: few long sequences, cut into segments that are walked side by
side and joined, and many short ones, walked by wider workgroups.  Against the
token recurrence in 64 bits, in the tolerances of the short sequences: the
segments change the order of the same sums only.  Graphs are replayed."""
import math

import pytest
import torch

from tests.mixer_reference import DT, TOL, delta, delta_inputs, rel
from tests.test_gpu_delta import check_backward, check_forward, gpu, rule

pytestmark = pytest.mark.gpu

# B, T, Hk, Hv, Dk, Dv
LONG = [
    (1, 1024, 1, 2, 128, 128),
    (2, 1500, 1, 2, 64, 72),
    (1, 2049, 1, 1, 96, 40),
    (1, 1700, 2, 2, 128, 264),
    (3, 1111, 1, 2, 24, 16),
]


def is_cut(op, ins, cu):
    """Whether a call keeps states of segments in its workspace."""
    a = [*ins[:5], cu, ins[5]]
    need = op._describe(*a)[0][3][0]
    B, T, Hv = ins[3].shape
    rows = B if cu is None else len(cu) - 1
    slots = B * -(-T // 64) if cu is None else -(-T // 64) + rows
    one = op._describe(*(x[:1, :1] for x in ins[:5]), None, None)[0][3][0] // Hv
    return need > slots * Hv * one


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_long_sequences(shape, dtype):
    for init in (False, True):
        ins = delta_inputs(sum(shape), *shape, dtype, init=init, decay=0.02)
        assert is_cut(rule(shape[4], shape[5], dtype), gpu(*ins), None)
        check_forward(ins, None, dtype, shape[4], shape[5])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bounds", [
    [0, 1600], [0, 5, 1400, 1400, 2001], [0, 64, 128, 2048], [0, 1023, 1024, 1025, 2300, 2364],
    [0, 0, 1999, 2000]], ids=str)
def test_long_packed_sequences(bounds, dtype):
    cu = torch.tensor(bounds)
    ins = delta_inputs(len(bounds), 1, bounds[-1], 1, 1, 64, 128, dtype, rows=len(bounds) - 1,
                       decay=0.02)
    check_forward(ins, cu, dtype, 64, 128)


def test_long_packed_sequences_are_cut():
    cu = torch.tensor([0, 1600])
    ins = delta_inputs(1, 1, 1600, 1, 1, 64, 128, "bf16")
    assert is_cut(rule(64, 128, "bf16"), gpu(*ins), cu.cuda())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_sequence_decays(dtype):
    # no decay at all, a state that is gone within a chunk, and one reset
    for decay in (0.0, 20.0):
        ins = delta_inputs(3, 1, 1300, 1, 2, 64, 64, dtype, decay=decay)
        check_forward(ins, None, dtype, 64, 64)
    ins = list(delta_inputs(3, 1, 1300, 1, 2, 64, 64, dtype, decay=0.02))
    ins[3] = ins[3].clone()
    ins[3][0, 700] = -math.inf
    ins[3][0, 64 * 5, 1] = -1e30
    check_forward(ins, None, dtype, 64, 64)


def test_nan_stays_in_a_long_sequence():
    cu = torch.tensor([0, 1200, 2400])
    ins = delta_inputs(7, 1, 2400, 1, 1, 64, 64, "f32", rows=2)
    bad = list(ins)
    bad[2] = ins[2].clone()
    bad[2][0, 600] = math.nan
    op = rule(64, 64, "f32")
    o, S = op.forward(*gpu(*bad[:5]), initial_state=bad[5].cuda(), cu_seqlens=cu.cuda())
    good, Sg = op.forward(*gpu(*ins[:5]), initial_state=ins[5].cuda(), cu_seqlens=cu.cuda())
    assert torch.isnan(o[0, 600]).any()
    assert torch.equal(o[0, :576], good[0, :576]) and torch.equal(o[0, 1200:], good[0, 1200:])
    assert torch.equal(S[1], Sg[1])


def test_bounds_of_long_sequences_stay_in_the_tensors():
    # not from 0 to T: the tokens outside the sequences keep what they hold
    ins = gpu(*delta_inputs(10, 1, 2000, 1, 1, 64, 64, "bf16", rows=2))
    cu = torch.tensor([900, 1500, 1800], device="cuda")
    out = torch.full_like(ins[2], 7.0)
    op = rule(64, 64, "bf16")
    o, S = op.forward(*ins[:5], initial_state=ins[5], cu_seqlens=cu, out=out)
    assert (o[0, :900] == 7).all() and (o[0, 1800:] == 7).all()
    want, Sw = op.forward(*(x[:, 900:1800].contiguous() for x in ins[:5]),
                          initial_state=ins[5], cu_seqlens=cu - 900)
    assert rel(o[0, 900:1800], want[0].cpu()) <= TOL["bf16"] and rel(S, Sw.cpu()) <= TOL["f32"]
    for bounds in ([-5, 1900, 40], [1999, 3, 10 ** 12], [2000, 0, 2000]):
        o, S = op.forward(*ins[:5], initial_state=ins[5],
                          cu_seqlens=torch.tensor(bounds, device="cuda"))
        assert o.shape == out.shape


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_long_sequence_backward(dtype):
    shape = (1, 1100, 1, 2, 32, 40)
    ins = delta_inputs(21, *shape, dtype, decay=0.02)
    check_backward(ins, None, dtype, 32, 40)
    cu = torch.tensor([0, 3, 3, 1100])
    ins = delta_inputs(22, *shape, dtype, rows=3, decay=0.02)
    check_backward(ins, cu, dtype, 32, 40)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 2100, 1, 1, 128, 24), (2, 1300, 1, 2, 24, 72)], ids=str)
def test_cut_sequence_backward(shape, dtype):
    ins = delta_inputs(23, *shape, dtype, decay=0.02)
    assert is_cut(rule(shape[4], shape[5], dtype), gpu(*ins), None)
    check_backward(ins, None, dtype, shape[4], shape[5])
    check_backward(ins[:5] + (None,), None, dtype, shape[4], shape[5], with_final=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cut_packed_sequences_backward(dtype):
    cu = torch.tensor([0, 0, 10, 3000])
    ins = delta_inputs(24, 1, 3000, 1, 1, 16, 24, dtype, rows=3, decay=0.02)
    check_backward(ins, cu, dtype, 16, 24)
    cu = torch.tensor([0, 900, 3000])
    ins = delta_inputs(25, 1, 3000, 1, 1, 16, 24, dtype, rows=2, decay=0.02)
    assert is_cut(rule(16, 24, dtype), gpu(*ins), cu.cuda())
    check_backward(ins, cu, dtype, 16, 24)


# more workgroups of 64 columns than CUs, fewer of 128
MANY = [(2, 130, 24, 72, 128, 128), (3, 70, 48, 48, 40, 128), (150, 65, 1, 1, 128, 104)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_many_heads(shape, dtype):
    ins = delta_inputs(sum(shape), *shape, dtype)
    check_forward(ins, None, dtype, shape[4], shape[5])


@pytest.mark.parametrize("shape,dtype", [
    ((2, 70, 24, 72, 24, 128), "bf16"), ((3, 66, 48, 48, 24, 104), "f16"),
    ((2, 66, 72, 72, 24, 128), "f32"), ((1, 65, 72, 144, 72, 128), "bf16"),
    ((145, 20, 1, 1, 128, 128), "f32")], ids=str)
def test_many_heads_backward(shape, dtype):
    ins = delta_inputs(sum(shape), *shape, dtype)
    check_backward(ins, None, dtype, shape[4], shape[5])


# chains in pieces: more of them than CUs, several chunks long
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(3, 700, 96, 96, 16, 128), (5, 1030, 60, 60, 8, 24),
                                   (2, 777, 60, 60, 72, 264)], ids=str)
def test_chains_in_pieces(shape, dtype):
    for init in (False, True):
        ins = delta_inputs(sum(shape), *shape, dtype, init=init, decay=0.001)
        assert is_cut(rule(shape[4], shape[5], dtype), gpu(*ins), None)
        check_forward(ins, None, dtype, shape[4], shape[5])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(3, 800, 96, 96, 16, 24), (1, 700, 2, 300, 8, 104)], ids=str)
def test_chains_in_pieces_backward(shape, dtype):
    ins = delta_inputs(sum(shape), *shape, dtype, decay=0.001)
    assert is_cut(rule(shape[4], shape[5], dtype), gpu(*ins), None)
    check_backward(ins, None, dtype, shape[4], shape[5])


def test_tensors_over_4_gib():
    # two batch rows 2^32 bytes apart, tokens and heads with gaps
    B, T, H, D = 2, 70, 2, 64
    ins = delta_inputs(31, B, T, H, H, D, D, "bf16")
    op = rule(D, D, "bf16")
    a = gpu(*ins)
    far = 1 << 31           # elements of 2 bytes
    wide = []
    for i in range(3):
        base = torch.empty(far + 2 * T * H * D + 64, dtype=torch.bfloat16, device="cuda")
        x = base.as_strided((B, T, H, D), (far, 2 * H * D, 2 * D, 1))
        x.copy_(a[i])
        wide.append(x)
    want = op.forward(*a[:5], initial_state=a[5])
    got = op.forward(*wide, a[3], a[4], initial_state=a[5])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_state_pool_over_4_gib():
    # states past 2^32 bytes of a pool
    H, D = 2, 128
    per = H * D * D
    pool = (1 << 30) // per + 3
    q, k, v, g, beta, S = delta_inputs(5, 2, 1, 1, H, D, D, "bf16")
    state = torch.empty(pool, H, D, D, device="cuda")
    slots = torch.tensor([pool - 1, 0], device="cuda")
    state[slots] = S.cuda()
    o = rule(D, D, "bf16").step(*gpu(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0]), state,
                                slots=slots)
    want_o, want_S = delta(*(x.double() for x in (q, k, v, g, beta, S)), None, D ** -0.5)
    assert rel(o, want_o[:, 0]) <= TOL["bf16"] and rel(state[slots], want_S) <= TOL["f32"]


def test_graph_of_a_layer_is_replayed():
    """Norms, a prompt in segments, its gradients and a step, captured
    once; every replay on new inputs against the same calls made eagerly."""
    from fft_long_convolution_amd.delta import QKNorm
    D, H, T, dev = 64, 2, 1100, "cuda"
    norm, op = QKNorm(D, norm="l2", rotary_dim=32), rule(D, D, "bf16")
    tab = torch.rand(T, 16, device=dev)
    cos, sin, pos = tab.cos(), tab.sin(), torch.arange(T, device=dev)[None]
    S = torch.randn(1, H, D, D, device=dev)
    w = torch.rand(D, device=dev)

    def inputs(seed):
        q, k, v, g, beta, _ = delta_inputs(seed, 1, T, H, H, D, D, "bf16", decay=0.02)
        return gpu(q, k, v, g, beta)

    def run(q, k, v, g, beta, state):
        nq, nk = norm.forward(q, k, w, w, cos, sin, pos)
        o, fin, saved = op.forward_train(nq, nk, v, g, beta, initial_state=S)
        d = op.backward(nq, nk, v, g, beta, o, saved, d_final_state=fin, initial_state=S)
        n = norm.backward(q, k, d[0], d[1], w, w, cos, sin, pos)
        state.copy_(fin)
        y = op.step(nq[:, -1], nk[:, -1], v[:, -1], g[:, -1], beta[:, -1], state)
        return [nq, nk, o, fin, *d, *n, y, state]

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
