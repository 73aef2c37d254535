"""Host side of the token mixers (no GPU): sizes of their buffers, refusals
before anything reaches the device, and the binding."""
import ctypes

import pytest

from fft_long_convolution_amd import delta
from fft_long_convolution_amd import fftconv as fc

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
BASE = 1 << 44          # addresses that are only compared, far from each other


def addr(i):
    return BASE + (i << 38)


def strides(T, H, D):
    return delta._LL3(T * H * D, H * D, D)


def delta_desc(dtype="bf16", B=2, T=100, Hk=2, Hv=4, Dk=64, Dv=128, sequences=0, **kw):
    d = delta.DeltaDesc(fc.DTYPES[dtype], B, T, Hk, Hv, Dk, Dv, sequences, 0.125,
                        strides(T, Hk, Dk), strides(T, Hk, Dk), strides(T, Hv, Dv))
    for k, x in kw.items():
        setattr(d, k, x)
    return d


def norm_desc(dtype="bf16", B=2, T=10, Hq=4, Hk=2, D=64, R=32, **kw):
    d = delta.QKNormDesc(fc.DTYPES[dtype], B, T, Hq, Hk, D, R, 0, 0, 1e-6, 100,
                         strides(T, Hq, D), strides(T, Hk, D))
    for k, x in kw.items():
        setattr(d, k, x)
    return d


def sizes(d):
    L, r = delta.lib(), ctypes.byref(d)
    return (L.fftconv_delta_workspace_bytes(r), L.fftconv_delta_saved_bytes(r),
            L.fftconv_delta_backward_workspace_bytes(r))


def forward(d, ws_bytes=1 << 36, saved_bytes=1 << 36, **at):
    """q k v g beta cu init o fin saved workspace, each an address of its own
    unless given."""
    names = ["q", "k", "v", "g", "beta", "cu", "init", "o", "fin", "saved", "ws"]
    a = {n: addr(i) for i, n in enumerate(names)}
    a["cu"] = addr(5) if d.sequences else None
    a.update(at)
    return delta.lib().fftconv_delta_forward(
        ctypes.byref(d), *(a[n] for n in names[:10]), saved_bytes, a["ws"], ws_bytes, None)


def step(d, pool=8, **at):
    names = ["q", "k", "v", "g", "beta", "state", "slots", "o"]
    a = {n: addr(i) for i, n in enumerate(names)}
    a.update(at)
    return delta.lib().fftconv_delta_step(
        ctypes.byref(d), *(a[n] for n in names[:6]), pool, a["slots"], a["o"], None)


def norm(d, backward=False, ws_bytes=1 << 30, **at):
    names = ["q", "k", "wq", "wk", "cos", "sin", "pos"]
    names += ["dqo", "dko", "dq", "dk", "dwq", "dwk", "ws"] if backward else ["qo", "ko"]
    a = {n: addr(i) for i, n in enumerate(names)}
    a.update(at)
    v = [a[n] for n in names]
    L = delta.lib()
    if backward:
        return L.fftconv_qknorm_backward(ctypes.byref(d), *v, ws_bytes, None)
    return L.fftconv_qknorm_forward(ctypes.byref(d), *v, None)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_buffer_sizes(dtype):
    small = sizes(delta_desc(dtype))
    assert all(x > 0 and x % 16 == 0 for x in small)
    # two chunks a row: four times the rows, four times the bytes
    assert sizes(delta_desc(dtype, B=8)) == tuple(4 * x for x in small)
    # a state and 64 values of each token of a chunk are kept in fp32
    assert small[1] >= 2 * 2 * 4 * (64 * 128 + 64 * 128) * 4
    # a packed row has at most one chunk more for each of its sequences
    one = sizes(delta_desc(dtype, B=1, T=64))
    assert sizes(delta_desc(dtype, B=1, T=128, sequences=3)) == tuple(5 * x for x in one)
    for empty in (delta_desc(dtype, B=0), delta_desc(dtype, T=0)):
        assert sizes(empty) == (0, 0, 0)
    L = delta.lib()
    assert L.fftconv_qknorm_workspace_bytes(ctypes.byref(norm_desc(dtype))) % 16 == 0


def test_long_sequences_ask_for_their_segments():
    # few heads: states and matrices of segments besides the chunks' data
    chunk = sizes(delta_desc(B=1, T=64, Hk=1, Hv=1))[0]
    assert sizes(delta_desc(B=1, T=64 * 64, Hk=1, Hv=1))[0] > 64 * chunk
    # many: none
    assert sizes(delta_desc(B=64, T=64 * 64, Hk=8, Hv=8))[0] == 64 * 64 * 8 * chunk


BAD_SIZES = [
    (UNSUPPORTED, dict(dtype=7)), (UNSUPPORTED, dict(Dk=60)), (UNSUPPORTED, dict(Dk=136)),
    (UNSUPPORTED, dict(Dk=0)), (UNSUPPORTED, dict(Dv=1032)), (UNSUPPORTED, dict(Dv=4)),
    (INVALID, dict(Hk=3)), (INVALID, dict(Hk=0)), (INVALID, dict(Hv=0)),
    (INVALID, dict(sequences=2)), (UNSUPPORTED, dict(T=1 << 40)), (UNSUPPORTED, dict(B=1 << 40)),
    (UNSUPPORTED, dict(Hv=1 << 20, Hk=1)), (UNSUPPORTED, dict(B=1 << 30, T=1 << 30)),
    (ALIGNMENT, dict(q_stride=delta._LL3(12804, 128, 64))),
    (ALIGNMENT, dict(v_stride=delta._LL3(51200, 516, 128))),
    (INVALID, dict(k_stride=delta._LL3(12800, -128, 64))),
    (INVALID, dict(k_stride=delta._LL3(1 << 60, 128, 64))),
    (UNSUPPORTED, dict(q_stride=delta._LL3(12800, 1 << 24, 64)))]


@pytest.mark.parametrize("want,kw", BAD_SIZES, ids=[str(sorted(kw)) + str(i)
                                                    for i, (_, kw) in enumerate(BAD_SIZES)])
def test_delta_sizes_are_refused(want, kw):
    d = delta_desc()
    for k, x in kw.items():
        setattr(d, k, x)
    assert forward(d) == want
    if not any(k.endswith("stride") for k in kw):
        assert sizes(d) == (0, 0, 0)


def test_delta_pointers_are_refused():
    d = delta_desc()
    for n in ("q", "k", "v", "g", "beta", "o"):
        assert forward(d, **{n: None}) == INVALID, n
        assert forward(d, **{n: addr(20) + 4}) == ALIGNMENT, n
    for n in ("init", "fin", "saved", "ws"):
        assert forward(d, **{n: addr(20) + 8}) == ALIGNMENT, n
    assert forward(d, cu=addr(20)) == INVALID       # bounds that nothing asked for
    packed = delta_desc(B=1, sequences=2)
    assert forward(packed, cu=None) == INVALID
    assert forward(packed, cu=addr(20) + 4) == ALIGNMENT
    assert forward(d, ws_bytes=sizes(d)[0] - 1) == WORKSPACE
    assert forward(d, ws=None) == WORKSPACE
    assert forward(d, saved_bytes=sizes(d)[1] - 1) == INVALID
    # outputs on inputs, on each other and on the workspace
    for a, b in (("o", "q"), ("o", "v"), ("fin", "init"), ("o", "fin"), ("saved", "ws"),
                 ("fin", "ws"), ("o", "g")):
        assert forward(d, **{a: addr(20), b: addr(20)}) == INVALID, (a, b)
    assert forward(d, o=addr(20), v=addr(20) + 16) == INVALID
    assert delta.lib().fftconv_delta_forward(None, *[None] * 10, 0, None, 0, None) == INVALID


def test_step_refusals():
    d = delta_desc(T=1, B=4)
    assert step(delta_desc(T=2)) == INVALID
    assert step(delta_desc(T=1, B=1, sequences=1)) == INVALID
    for n in ("q", "k", "v", "g", "beta", "state", "o"):
        assert step(d, **{n: None}) == INVALID, n
        assert step(d, **{n: addr(20) + 8}) == ALIGNMENT, n
    assert step(d, slots=addr(20) + 4) == ALIGNMENT
    assert step(d, pool=3, slots=None) == INVALID
    assert step(d, pool=1 << 40) == UNSUPPORTED
    assert step(d, o=addr(5)) == INVALID            # on the states
    assert step(d, v=addr(5)) == INVALID
    assert step(delta_desc(T=1, B=0)) == OK


def test_delta_backward_refusals():
    d = delta_desc()
    names = ["q", "k", "v", "g", "beta", "cu", "saved", "do", "dfin", "dq", "dk", "dv", "dg",
             "dbeta", "dinit", "ws"]

    def call(saved_bytes=1 << 36, ws_bytes=1 << 36, **at):
        a = {n: addr(i) for i, n in enumerate(names)}
        a["cu"] = None
        a.update(at)
        return delta.lib().fftconv_delta_backward(
            ctypes.byref(d), *(a[n] for n in names[:7]), saved_bytes, *(a[n] for n in names[7:]),
            ws_bytes, None)
    for n in names:
        if n not in ("cu", "dfin", "dinit", "ws"):
            assert call(**{n: None}) == INVALID, n
        if n != "cu":
            assert call(**{n: addr(20) + 8}) == ALIGNMENT, n
    assert call(saved_bytes=sizes(d)[1] - 1) == INVALID
    assert call(ws_bytes=sizes(d)[2] - 1) == WORKSPACE
    assert call(ws=None) == WORKSPACE
    for a, b in (("dq", "q"), ("dk", "dq"), ("dv", "do"), ("dinit", "dfin"), ("ws", "saved")):
        assert call(**{a: addr(20), b: addr(20)}) == INVALID, (a, b)


def test_norm_refusals():
    for want, kw in ((UNSUPPORTED, dict(D=60)), (UNSUPPORTED, dict(D=264)),
                     (UNSUPPORTED, dict(R=24)), (INVALID, dict(R=80)),
                     (UNSUPPORTED, dict(dtype=5)), (INVALID, dict(norm=2)),
                     (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))),
                     (UNSUPPORTED, dict(B=1 << 40)), (UNSUPPORTED, dict(table_rows=1 << 40)),
                     (ALIGNMENT, dict(q_stride=delta._LL3(2560, 257, 64))),
                     (INVALID, dict(k_stride=delta._LL3(1280, 128, -64)))):
        R, kw2 = kw.get("R"), {k: x for k, x in kw.items() if k != "R"}
        d = norm_desc()
        for k, x in kw2.items():
            setattr(d, k, x)
        if R is not None:
            d.rotary_dim = R
        assert norm(d) == want and norm(d, backward=True) == want, kw
    d = norm_desc()
    for n in ("q", "k", "cos", "sin", "pos"):
        assert norm(d, **{n: None}) == INVALID, n
        assert norm(d, **{n: addr(20) + 4}) == ALIGNMENT, n
    for a, b in (("qo", "q"), ("ko", "qo"), ("ko", "cos"), ("qo", "wq")):
        assert norm(d, **{a: addr(20), b: addr(20)}) == INVALID, (a, b)
    need = delta.lib().fftconv_qknorm_workspace_bytes(ctypes.byref(d))
    assert need > 0
    assert norm(d, backward=True, ws_bytes=need - 1) == WORKSPACE
    assert norm(d, backward=True, ws=None) == WORKSPACE
    assert norm(d, backward=True, ws=addr(20) + 8) == ALIGNMENT
    for a, b in (("dq", "q"), ("dk", "dqo"), ("dwq", "dwk")):
        assert norm(d, backward=True, **{a: addr(20), b: addr(20)}) == INVALID, (a, b)


def test_empty_calls_need_no_device():
    for d in (delta_desc(B=0), delta_desc("f32", B=0, T=0)):
        assert forward(d, q=None, k=None, v=None, g=None, beta=None, o=None, init=None,
                       fin=None, saved=None) == OK
    for d in (norm_desc(B=0), norm_desc(T=0)):
        assert norm(d, q=None, k=None, cos=None, sin=None, pos=None, qo=None, ko=None) == OK


def test_binding_checks_before_the_library():
    import torch
    op = delta.GatedDelta(64, 64)
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    g = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        op.forward(q, q, q, g, g)
    with pytest.raises(ValueError, match="CUDA"):
        delta.QKNorm(64).forward(q, q)
    with pytest.raises(ValueError, match="dtype"):
        delta.GatedDelta(64, 64, dtype="f64")
    with pytest.raises(ValueError, match="norm"):
        delta.QKNorm(64, norm="max")


def test_binding_marshals_only():
    src = open(delta.__file__).read()
    for bad in ("matmul", "einsum", "bmm", "torch.exp", "softmax", ".sum(", "rsqrt", "oracle"):
        assert bad not in src


def test_missing_library_fails_loudly(monkeypatch):
    monkeypatch.setattr(fc, "_lib", None)
    monkeypatch.setattr(delta, "_ready", None)
    monkeypatch.setattr(fc, "LIB_PATH", "/nonexistent/libfftconv.so")
    for make in (lambda: delta.QKNorm(64), lambda: delta.GatedDelta(64, 64)):
        with pytest.raises(RuntimeError, match="not built"):
            make()


def test_more_chains_than_a_launch_takes():
    # 512 threads and more for each chain, fewer than 2^32 in all: refused before
    # anything is launched, not by the launch of the walk
    for B in (8388609, 9000000, 16 << 20):
        d = delta_desc(B=B, T=1, Hk=1, Hv=1, Dk=8, Dv=8)
        assert sizes(d) == (0, 0, 0)
        assert forward(d, ws_bytes=1 << 50, saved_bytes=1 << 50) == UNSUPPORTED
    assert min(sizes(delta_desc(B=8388000, T=1, Hk=1, Hv=1, Dk=8, Dv=8))) > 0
