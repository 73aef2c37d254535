"""Norms of queries and keys with the rotation against their 64-bit form."""
import pytest
import torch

from tests.mixer_reference import DT, TOL, qk_norm, rel

pytestmark = pytest.mark.gpu

EPS = 1e-6
# B, T, Hq, Hk, D, R, kind, weight, interleaved
SHAPES = [
    (1, 1, 1, 1, 8, 0, "rms", True, False),
    (2, 3, 3, 2, 64, 64, "rms", True, False),
    (1, 17, 5, 1, 96, 48, "l2", False, False),
    (3, 5, 2, 4, 128, 128, "l2", True, True),
    (1, 33, 4, 4, 128, 32, "rms", False, False),
    (2, 9, 7, 1, 256, 256, "rms", True, False),
    (1, 4, 1, 1, 40, 8, "rms", True, True),
    (1, 20000, 2, 1, 64, 16, "rms", True, False),
]


def make(shape, dtype, seed=0):
    B, T, Hq, Hk, D, R, kind, weight, inter = shape
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    qkv = (2.0 * r(B, T, Hq + 2 * Hk, D)).to(DT[dtype])
    a = {"q": qkv[:, :, :Hq], "k": qkv[:, :, Hq:Hq + Hk],
         "q_weight": 1 + 0.3 * r(D) if weight else None,
         "k_weight": 1 + 0.3 * r(D) if weight else None,
         "cos": None, "sin": None, "positions": None}
    if R:
        ang = 6.3 * torch.rand(50, R // 2, generator=gen)
        a.update(cos=ang.cos(), sin=ang.sin(),
                 positions=torch.randint(0, 50, (B, T), generator=gen))
    return a


def cuda(a):
    # the views of q and k keep their strides
    out = {}
    for n, x in a.items():
        if n == "k":
            continue
        if n == "q":
            B, T, H, D = x.shape
            base = torch.empty(B, T, H + 2 * a["k"].shape[2], D, dtype=x.dtype, device="cuda")
            out["q"], out["k"] = base[:, :, :H], base[:, :, H:H + a["k"].shape[2]]
            out["q"].copy_(x)
            out["k"].copy_(a["k"])
        else:
            out[n] = None if x is None else x.cuda()
    return out


def op_of(shape, dtype):
    from fft_long_convolution_amd.delta import QKNorm
    return QKNorm(shape[4], rotary_dim=shape[5], norm=shape[6], eps=EPS, interleaved=shape[8],
                  dtype=dtype)


def reference(shape, a, grads=None):
    R, kind, inter = shape[5], shape[6], shape[8]
    cos = a["cos"].double()[a["positions"]] if R else None
    sin = a["sin"].double()[a["positions"]] if R else None
    out = []
    for n in ("q", "k"):
        x = a[n].double().requires_grad_()
        w = None if a[n + "_weight"] is None else a[n + "_weight"].double().requires_grad_()
        y = qk_norm(x, w, cos, sin, R, inter, kind, EPS)
        if grads is None:
            out.append(y.detach())
        else:
            d = torch.autograd.grad(y, [x] + ([] if w is None else [w]), grads[n].double())
            out.append((d[0], d[1] if w is not None else None))
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(shape, dtype):
    a = make(shape, dtype)
    q, k = op_of(shape, dtype).forward(**cuda(a))
    assert q.dtype == DT[dtype] and q.is_contiguous()
    want = reference(shape, a)
    assert rel(q, want[0]) <= TOL[dtype]
    assert rel(k, want[1]) <= TOL[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(shape, dtype):
    a = make(shape, dtype)
    gen = torch.Generator().manual_seed(9)
    gr = {n: torch.randn(a[n].shape, generator=gen).to(DT[dtype]) for n in ("q", "k")}
    c = cuda(a)
    op = op_of(shape, dtype)
    q, k = c.pop("q"), c.pop("k")
    got = op.backward(q, k, gr["q"].cuda(), gr["k"].cuda(), **c)
    again = op.backward(q, k, gr["q"].cuda(), gr["k"].cuda(), **c)
    want = reference(shape, a, gr)
    for i in (0, 1):
        assert got[i].dtype == DT[dtype]
        assert rel(got[i], want[i][0]) <= TOL[dtype]
        if want[i][1] is None:
            assert got[2 + i] is None
        else:
            assert rel(got[2 + i], want[i][1]) <= TOL["f32"]
            assert torch.equal(got[2 + i], again[2 + i])


def test_gradient_against_differences():
    # the fp32 kernels' gradient against central differences of the fp32
    # forward: h = 2^-6 leaves h^2/6 of the third derivative (about 1e-4 of a
    # first derivative of order one) and 2^-24 / h = 4e-6 of rounding
    shape = (1, 2, 2, 1, 16, 16, "rms", True, False)
    a = cuda(make(shape, "f32", seed=3))
    op = op_of(shape, "f32")
    q, k = a.pop("q").contiguous(), a.pop("k").contiguous()
    gen = torch.Generator().manual_seed(4)
    gq = torch.randn(q.shape, generator=gen).cuda()
    gk = torch.randn(k.shape, generator=gen).cuda()
    loss = lambda q: sum((x.double() * y).sum() for x, y in  # noqa: E731
                         zip(op.forward(q, k, **a), (gq, gk))).item()
    dq = op.backward(q, k, gq, gk, **a)[0].flatten()
    h = 2.0 ** -6
    for i in range(0, q.numel(), 5):
        e = torch.zeros(q.numel(), device="cuda")
        e[i] = h
        e = e.view_as(q)
        assert abs((loss(q + e) - loss(q - e)) / (2 * h) - dq[i].item()) <= 2e-3


def test_zero_rows_and_positions_outside_the_tables():
    from fft_long_convolution_amd.delta import QKNorm
    op = QKNorm(64, rotary_dim=32, dtype="f32")
    q = torch.zeros(1, 3, 2, 64, device="cuda")
    k = torch.ones(1, 3, 1, 64, device="cuda")
    cos, sin = torch.ones(4, 16, device="cuda"), torch.zeros(4, 16, device="cuda")
    pos = torch.tensor([[0, 4, -1]], device="cuda")
    y, z = op.forward(q, k, cos=cos, sin=sin, positions=pos)
    assert torch.equal(y[:, :1], torch.zeros_like(y[:, :1]))
    assert torch.isfinite(z[:, 0]).all()
    assert torch.isnan(z[:, 1:, :, :32]).all()
    assert torch.isfinite(z[:, 1:, :, 32:]).all()


def test_empty_and_other_stream():
    from fft_long_convolution_amd.delta import QKNorm
    op = QKNorm(64, dtype="bf16")
    q = torch.empty(2, 0, 3, 64, dtype=torch.bfloat16, device="cuda")
    y, z = op.forward(q, q[:, :, :1])
    assert y.shape == (2, 0, 3, 64) and z.shape == (2, 0, 1, 64)
    w = torch.ones(64, device="cuda")
    d = op.backward(q, q[:, :, :1], y, z, q_weight=w, k_weight=w)
    assert torch.equal(d[2], torch.zeros_like(w)) and torch.equal(d[3], torch.zeros_like(w))
    x = torch.randn(1, 100, 4, 64, device="cuda").bfloat16()
    want = op.forward(x, x)[0]
    s = torch.cuda.Stream()
    # a misaligned view: the binding copies it, and keeps the copy alive
    odd = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view_as(x)
    odd.copy_(x)
    got = op.forward(odd, odd, stream=s)[0]
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    from fft_long_convolution_amd.delta import QKNorm
    from fft_long_convolution_amd.fftconv import FFTConvError
    x = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        QKNorm(64, norm="max")
    with pytest.raises(ValueError):
        QKNorm(64, dtype="f64")
    op = QKNorm(64)
    with pytest.raises(ValueError):
        op.forward(x, x.float())
    with pytest.raises(ValueError):
        op.forward(x, x[:, :1])
    with pytest.raises(ValueError):
        op.forward(x.cpu(), x)
    with pytest.raises(ValueError):
        op.forward(x, x, q_weight=torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        QKNorm(64, rotary_dim=32).forward(x, x)
    for bad in (QKNorm(64, rotary_dim=24), QKNorm(64, rotary_dim=80)):
        t = torch.zeros(4, bad.rotary_dim // 2, device="cuda")
        with pytest.raises(FFTConvError):
            bad.forward(x, x, cos=t, sin=t, positions=torch.zeros(1, 2, dtype=torch.int64,
                                                                  device="cuda"))
    with pytest.raises(FFTConvError) as e:
        op.forward(x, x, out=(x, torch.empty_like(x)))
    assert e.value.status == 1
    y = torch.zeros(1, 2, 2, 12, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(FFTConvError) as e:
        QKNorm(12).forward(y, y)
    assert e.value.status == 2


def test_backward_without_heads_reads_no_token():
    # the weights' gradients are sums over no heads; positions and tables may be missing
    import ctypes
    from fft_long_convolution_amd import delta
    for B, T in ((3, 5), (0, 5)):
        d = delta.QKNormDesc(2, B, T, 0, 0, 64, 32, 0, 0, 1e-6, 100, delta._LL3(0, 64, 64),
                             delta._LL3(0, 64, 64))
        ref, L = ctypes.byref(d), delta.lib()
        ws = torch.empty(L.fftconv_qknorm_workspace_bytes(ref), dtype=torch.uint8, device="cuda")
        dw = torch.full((2, 64), 7.0, device="cuda")
        status = L.fftconv_qknorm_backward(ref, *[None] * 11, dw[0].data_ptr(), dw[1].data_ptr(),
                                           ws.data_ptr(), ws.numel(),
                                           torch.cuda.current_stream().cuda_stream)
        assert status == 0
        assert torch.equal(dw, torch.zeros_like(dw))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_tensors_have_the_bits_of_their_parts(dtype):
    # past the caches: loads and stores of another kind, the same sums
    from fft_long_convolution_amd.delta import QKNorm
    T = 120001
    q = torch.randn(1, T, 5, 128, device="cuda").to(DT[dtype])
    k = torch.randn(1, T, 1, 128, device="cuda").to(DT[dtype])
    assert (q.numel() + k.numel()) * 2 > 160 << 20
    angle = torch.rand(64, 32, device="cuda")
    w = 1 + torch.rand(128, device="cuda")
    pos = torch.randint(0, 64, (1, T), device="cuda")
    op = QKNorm(128, rotary_dim=64, dtype=dtype)
    whole = op.forward(q, k, w, w, angle.cos(), angle.sin(), pos)
    grads = op.backward(q, k, whole[0], whole[1], w, w, angle.cos(), angle.sin(), pos)
    for a, z in ((0, 60000), (60000, T)):
        part = [x[:, a:z] for x in (q, k)]
        y = op.forward(*part, w, w, angle.cos(), angle.sin(), pos[:, a:z])
        d = op.backward(*part, whole[0][:, a:z], whole[1][:, a:z], w, w, angle.cos(),
                        angle.sin(), pos[:, a:z])
        for x, p in zip((*whole, *grads[:2]), (*y, *d[:2])):
            assert torch.equal(x[:, a:z], p)
