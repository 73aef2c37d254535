"""Host side of linear attention with decays and of layer norm (no GPU): sizes of
their buffers, refusals before anything reaches the device, and the binding."""
import ctypes

import pytest
import torch

from fft_long_convolution_amd import decay, delta
from fft_long_convolution_amd import fftconv as fc
from tests.test_mixer_host import ALIGNMENT, INVALID, OK, UNSUPPORTED, WORKSPACE, addr, strides
from tests.test_mixer_binding import calls, projection  # noqa: F401


def desc(dtype="bf16", B=2, T=100, Hk=2, Hv=4, Dk=64, Dv=128, sequences=0, fixed=0, **kw):
    d = decay.DecayDesc(fc.DTYPES[dtype], B, T, Hk, Hv, Dk, Dv, sequences, 0.125, fixed,
                        strides(T, Hk, Dk), strides(T, Hk, Dk), strides(T, Hv, Dv), 0)
    for k, x in kw.items():
        setattr(d, k, x)
    return d


def sizes(d):
    L, r = decay.lib(), ctypes.byref(d)
    return L.fftconv_decay_workspace_bytes(r), L.fftconv_decay_backward_workspace_bytes(r)


FORWARD = ["q", "k", "v", "g", "cu", "init", "o", "fin", "ws"]
BACKWARD = ["q", "k", "v", "g", "cu", "init", "do", "dfin", "dq", "dk", "dv", "dg", "dinit", "ws"]


def call(d, backward=False, ws_bytes=1 << 36, **at):
    """Every pointer an address of its own unless given."""
    names = BACKWARD if backward else FORWARD
    a = {n: addr(i) for i, n in enumerate(names)}
    a["cu"] = addr(len(names)) if d.sequences else None
    a.update(at)
    L = decay.lib()
    fn = L.fftconv_decay_backward if backward else L.fftconv_decay_forward
    return fn(ctypes.byref(d), *(a[n] for n in names), ws_bytes, None)


def step(d, pool=8, **at):
    names = ["q", "k", "v", "g", "state", "slots", "o"]
    a = {n: addr(i) for i, n in enumerate(names)}
    a.update(at)
    return decay.lib().fftconv_decay_step(
        ctypes.byref(d), *(a[n] for n in names[:5]), pool, a["slots"], a["o"], None)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_buffer_sizes(dtype):
    for d in (desc(dtype), desc(dtype, B=1, T=1000, sequences=7), desc(dtype, fixed=1)):
        assert all(x % 16 == 0 for x in sizes(d)) and sizes(d)[1] > 0
    # the gradients' buffer grows with the tokens
    assert sizes(desc(dtype, T=4000))[1] > sizes(desc(dtype, T=400))[1]
    # short sequences of many heads are walked whole: no buffer
    assert sizes(desc(dtype, B=256, T=128, Hk=8, Hv=8))[0] == 0
    # long ones of few heads in segments: their states
    few = desc(dtype, B=1, T=64 * 64, Hk=1, Hv=1)
    assert sizes(few)[0] >= 2 * 64 * 128 * 4 and sizes(few)[1] > 2 * sizes(few)[0]
    assert sizes(desc(dtype, B=0))[0] == 0
    assert sizes(desc(dtype, Dv=264))[1] == 0       # forward only


BAD_SIZES = [
    (UNSUPPORTED, dict(dtype=7)), (UNSUPPORTED, dict(Dk=60)), (UNSUPPORTED, dict(Dk=264)),
    (UNSUPPORTED, dict(Dk=0)), (UNSUPPORTED, dict(Dv=1032)), (UNSUPPORTED, dict(Dv=4)),
    (INVALID, dict(Hk=3)), (INVALID, dict(Hk=0)), (INVALID, dict(Hv=0)),
    (INVALID, dict(sequences=2)), (UNSUPPORTED, dict(T=1 << 40)), (UNSUPPORTED, dict(T=0x7fffffff)),
    (UNSUPPORTED, dict(B=1 << 40)), (UNSUPPORTED, dict(Hv=1 << 20, Hk=1)),
    (UNSUPPORTED, dict(B=1 << 30, T=1 << 30)), (UNSUPPORTED, dict(B=1 << 22, T=1)),
    (ALIGNMENT, dict(q_stride=delta._LL3(12804, 128, 64))),
    (ALIGNMENT, dict(v_stride=delta._LL3(51200, 516, 128))),
    (INVALID, dict(k_stride=delta._LL3(12800, -128, 64))),
    (INVALID, dict(k_stride=delta._LL3(1 << 60, 128, 64))),
    (UNSUPPORTED, dict(q_stride=delta._LL3(12800, 1 << 24, 64)))]


@pytest.mark.parametrize("want,kw", BAD_SIZES, ids=[str(sorted(kw)) + str(i)
                                                    for i, (_, kw) in enumerate(BAD_SIZES)])
def test_sizes_are_refused(want, kw):
    d = desc()
    for k, x in kw.items():
        setattr(d, k, x)
    assert call(d) == want and call(d, backward=True) == want
    if not any(k.endswith("stride") for k in kw):
        assert sizes(d) == (0, 0)


@pytest.mark.parametrize("backward", [False, True])
def test_pointers_are_refused(backward):
    d = desc(B=1, T=4096, Hk=1, Hv=1)               # one that asks for a workspace
    names = BACKWARD if backward else FORWARD
    optional = {"cu", "init", "fin", "dfin", "dinit"}
    for n in names:
        if n not in optional:
            assert call(d, backward, **{n: None}) == (WORKSPACE if n == "ws" else INVALID), n
        if n != "cu":
            assert call(d, backward, **{n: addr(20) + 8}) == ALIGNMENT, n
    assert call(d, backward, cu=addr(20)) == INVALID        # bounds that nothing asked for
    packed = desc(B=1, sequences=2)
    assert call(packed, backward, cu=None) == INVALID
    assert call(packed, backward, cu=addr(20) + 4) == ALIGNMENT
    assert call(d, backward, ws_bytes=sizes(d)[backward] - 1) == WORKSPACE
    pairs = [("dq", "q"), ("dk", "dq"), ("dv", "do"), ("dinit", "dfin"), ("ws", "init"),
             ("dg", "g"), ("dinit", "ws")] if backward else \
        [("o", "q"), ("o", "v"), ("fin", "init"), ("o", "fin"), ("fin", "ws"), ("o", "g")]
    for a, b in pairs:
        assert call(d, backward, **{a: addr(20), b: addr(20)}) == INVALID, (a, b)
    if backward:
        assert call(desc(Dv=264), True) == UNSUPPORTED
    assert decay.lib().fftconv_decay_forward(None, *[None] * 9, 0, None) == INVALID
    assert decay.lib().fftconv_decay_backward(None, *[None] * 14, 0, None) == INVALID


def test_step_refusals():
    d = desc(T=1, B=4)
    assert step(desc(T=2)) == INVALID
    assert step(desc(T=1, B=1, sequences=1)) == INVALID
    for n in ("q", "k", "v", "g", "state", "o"):
        assert step(d, **{n: None}) == INVALID, n
        assert step(d, **{n: addr(20) + 8}) == ALIGNMENT, n
    assert step(d, slots=addr(20) + 4) == ALIGNMENT
    assert step(d, pool=3, slots=None) == INVALID
    assert step(d, pool=1 << 40) == UNSUPPORTED
    assert step(d, o=addr(4)) == INVALID            # on the states
    assert step(d, v=addr(4)) == INVALID
    assert step(desc(T=1, B=0)) == OK


def test_empty_calls_need_no_device():
    for d in (desc(B=0), desc("f32", B=0, T=0)):
        assert call(d, **{n: None for n in FORWARD}) == OK
        assert call(d, True, **{n: None for n in BACKWARD if n != "ws"}) == OK


def ln_desc(dtype="bf16", rows=10, D=768, eps=1e-5, stride=768):
    return decay.LayerNormDesc(fc.DTYPES.get(dtype, 9), rows, D, eps, stride)


def ln(d, backward=False, ws_bytes=1 << 30, **at):
    names = ["x", "w", "dy", "dx", "dw", "db", "ws"] if backward else ["x", "w", "b", "y"]
    a = {n: addr(i) for i, n in enumerate(names)}
    a.update(at)
    v = [a[n] for n in names]
    L = decay.lib()
    if backward:
        return L.fftconv_layernorm_backward(ctypes.byref(d), *v, ws_bytes, None)
    return L.fftconv_layernorm_forward(ctypes.byref(d), *v, None)


def test_layer_norm_refusals():
    for want, kw in ((UNSUPPORTED, dict(D=16385, stride=16385)), (INVALID, dict(D=0)),
                     (UNSUPPORTED, dict(dtype="f64")), (INVALID, dict(eps=-1.0)),
                     (INVALID, dict(eps=float("nan"))), (UNSUPPORTED, dict(rows=1 << 40)),
                     (INVALID, dict(stride=767)), (INVALID, dict(stride=-768)),
                     (INVALID, dict(stride=1 << 60))):
        assert ln(ln_desc(**kw)) == want and ln(ln_desc(**kw), True) == want, kw
    d = ln_desc()
    for n in ("x", "y"):
        assert ln(d, **{n: None}) == INVALID
    for n in ("x", "w", "b", "y"):
        assert ln(d, **{n: addr(20) + 4}) == ALIGNMENT, n
    for n in ("x", "dy", "dx"):
        assert ln(d, True, **{n: None}) == INVALID, n
    for n in ("x", "w", "dy", "dx", "dw", "db", "ws"):
        assert ln(d, True, **{n: addr(20) + 8}) == ALIGNMENT, n
    need = decay.lib().fftconv_layernorm_workspace_bytes(ctypes.byref(d))
    assert need > 0 and need % 16 == 0
    assert ln(d, True, ws_bytes=need - 1) == WORKSPACE and ln(d, True, ws=None) == WORKSPACE
    for a, b in (("y", "x"), ("y", "w"), ("y", "b")):
        assert ln(d, **{a: addr(20), b: addr(20)}) == INVALID, (a, b)
    for a, b in (("dx", "dy"), ("dx", "x"), ("dw", "db"), ("dw", "w"), ("ws", "dx")):
        assert ln(d, True, **{a: addr(20), b: addr(20)}) == INVALID, (a, b)
    assert ln(ln_desc(rows=0), x=None, y=None) == OK


# ------------------------------------------------------------------ binding

def run(name, q, k, v):
    B, T, _, D = q.shape
    Hv, op = v.shape[2], decay.DecayAttention(q.shape[3], v.shape[3])
    g = torch.zeros(B, T, Hv)
    if name == "forward":
        op.forward(q, k, v, g)
    elif name == "backward":
        op.backward(q, k, v, g, torch.zeros(v.shape, dtype=v.dtype))
    else:
        op.step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], torch.zeros(B, Hv, D, v.shape[3]))


@pytest.mark.parametrize("twice", [False, True])
@pytest.mark.parametrize("name", ["forward", "backward", "step"])
def test_descriptor_has_the_strides_of_the_tensors_passed(calls, name, twice):  # noqa: F811
    for offset in (0, 4):
        q, k, v = projection(2, 5, (6, 6, 6), 128, offset, 8)
        for _ in range(1 + twice):
            run(name, q, k, v)
    # aligned views go in as they are
    assert not calls[0][2][0].is_contiguous()
    for _, d, kept, args in calls:
        for x, ptr, st in zip(kept, args, (d.q_stride, d.k_stride, d.v_stride)):
            want = list(x.stride()[:3]) if x.dim() == 4 else [x.stride(0), 0, x.stride(1)]
            assert list(st) == want and x.stride(-1) == 1
            assert ptr == x.data_ptr() and ptr % 16 == 0


def rows_of(x):
    """x as LayerNorm hands it on, of a tensor on the CPU."""
    class OnDevice(torch.Tensor):
        is_cuda = True
    return x.as_subclass(OnDevice)


def test_layer_norm_strides(calls):  # noqa: F811
    op = decay.LayerNorm(40)
    wide = torch.zeros(3, 5, 96, dtype=torch.bfloat16)
    for x, stride in ((torch.zeros(3, 5, 40, dtype=torch.bfloat16), 40), (wide[0, :, 8:48], 96),
                      (wide[0, :1, :40].expand(7, 40), 40), (wide[0, 0, :40], 40),
                      (torch.zeros(40, 6, dtype=torch.bfloat16).t(), 40)):
        op.forward(rows_of(x))
        name, d, kept, args = calls[-1]
        assert d.x_stride == stride and d.rows == x.numel() // 40 and d.D == 40
        assert args[0] == kept[0].data_ptr() and args[0] % 16 == 0


def test_settings_changed_after_the_first_call(calls):  # noqa: F811
    q, k, v = projection(1, 4, (2, 2, 2), 64, 0, 0)
    g = torch.zeros(1, 4, 2)
    a, b = decay.DecayAttention(64, 64), decay.DecayAttention(64, 64)
    a.forward(q, k, v, g)
    a.scale = 3.0
    a.forward(q, k, v, g)
    assert calls[-1][1].scale == 3.0
    b.forward(q, k, v, g)
    assert calls[-1][1].scale == 0.125
    # a fixed decay is another descriptor; so is a given output
    b.forward(q, k, v, g[0, 0])
    assert calls[-1][1].fixed_decay == 1 and calls[-1][1].clear_unheld == 1
    b.forward(q, k, v, g, out=torch.zeros(v.shape, dtype=v.dtype))
    assert calls[-1][1].fixed_decay == 0 and calls[-1][1].clear_unheld == 0


def test_binding_refuses(calls):  # noqa: F811
    q, k, v = projection(1, 4, (2, 2, 2), 64, 0, 0)
    g, op = torch.zeros(1, 4, 2), decay.DecayAttention(64, 64)
    cu, S = torch.tensor([0, 4]), torch.zeros(1, 2, 64, 64)
    bad = [dict(q=q[:, :3]), dict(k=k[..., :32]), dict(v=v.float()), dict(g=g.double()),
           dict(g=torch.zeros(3)), dict(g=g[:, :, :1]), dict(cu_seqlens=cu.int()),
           dict(cu_seqlens=cu[:1]), dict(initial_state=S[:, :1]), dict(initial_state=S.half()),
           dict(out=torch.zeros(1, 4, 2, 32, dtype=v.dtype)),
           dict(out=torch.zeros(1, 2, 4, 64, dtype=v.dtype).transpose(1, 2)),
           dict(final_state=S.transpose(2, 3))]
    for kw in bad:
        with pytest.raises(ValueError):
            op.forward(**{**dict(q=q, k=k, v=v, g=g), **kw})
    with pytest.raises(ValueError, match="B = 1"):
        op.forward(*(x.expand(2, *x.shape[1:]) for x in (q, k, v)), g.expand(2, 4, 2),
                   cu_seqlens=cu)
    with pytest.raises(ValueError):
        op.backward(q, k, v, g, v[:, :2])
    with pytest.raises(ValueError, match="contiguous"):
        op.step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], S.transpose(2, 3))
    assert not calls
    with pytest.raises(ValueError, match="CUDA"):
        decay.LayerNorm(64).forward(torch.zeros(2, 64, dtype=torch.bfloat16))
    for D, x in ((64, torch.zeros(2, 32)), (0, torch.zeros(2, 0)), (1, torch.zeros(()))):
        with pytest.raises(ValueError, match="must be"):
            decay.LayerNorm(D).forward(x)
    with pytest.raises(ValueError, match="dtype"):
        decay.DecayAttention(64, 64, dtype="f64")


def test_binding_marshals_only():
    src = open(decay.__file__).read()
    for bad in ("matmul", "einsum", "bmm", "torch.exp", "softmax", ".sum(", "rsqrt", "oracle",
                ".mean("):
        assert bad not in src


def test_missing_library_fails_loudly(monkeypatch):
    monkeypatch.setattr(fc, "_lib", None)
    monkeypatch.setattr(delta, "_ready", None)
    monkeypatch.setattr(decay, "_ready", None)
    monkeypatch.setattr(fc, "LIB_PATH", "/nonexistent/libfftconv.so")
    for make in (lambda: decay.LayerNorm(64), lambda: decay.DecayAttention(64, 64)):
        with pytest.raises(RuntimeError, match="not built"):
            make()


def test_more_segments_than_a_launch_takes():
    # sequences that could be cut are walked whole where the segments, or the threads
    # that join them, would be more than one launch takes
    for kw in (dict(T=8000 * 192, sequences=8000, Hk=64, Hv=64, Dk=8, Dv=8),
               dict(T=8000 * 192, sequences=8000, Hk=64, Hv=64, Dk=128, Dv=128),
               dict(T=7000 * 300, sequences=7000, Hk=64, Hv=64, Dk=128, Dv=128)):
        d = desc(B=1, **kw)
        assert sizes(d)[0] == 0 and sizes(d)[1] > 0
        assert call(d, ws_bytes=0, ws=None, q=None) == INVALID       # not UNSUPPORTED
