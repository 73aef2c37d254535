"""Layer norm, forward and backward, against its formulas in 64 bits."""
import pytest
import torch

from tests.decay_reference import DT, TOL, layer_norm, rel

pytestmark = pytest.mark.gpu


def norm(D, dtype, eps=1e-5):
    from fft_long_convolution_amd.decay import LayerNorm
    return LayerNorm(D, eps=eps, dtype=dtype)


def inputs(rows, D, dtype, weight=True, wide=False):
    gen = torch.Generator().manual_seed(rows + D)
    x = torch.randn(rows, 2 * D if wide else D, generator=gen) + torch.randn(rows, 1, generator=gen)
    x = x.to(DT[dtype])[:, :D]
    dy = torch.randn(rows, D, generator=gen).to(DT[dtype])
    w = 1 + 0.2 * torch.randn(D, generator=gen) if weight else None
    b = 0.1 * torch.randn(D, generator=gen) if weight else None
    return x, dy, w, b


def check(x, dy, w, b, dtype, eps=1e-5):
    D = x.shape[-1]
    op = norm(D, dtype, eps)
    on = [None if t is None else t.cuda() for t in (x, dy, w, b)]
    y = op.forward(on[0], on[2], on[3])
    dx, dw, db = op.backward(*on)
    ins = [t.double().requires_grad_() for t in (x, w, b) if t is not None]
    full = ins + [None] * (3 - len(ins))
    want = layer_norm(*full, eps)
    d = torch.autograd.grad(want, ins, dy.double())
    assert y.dtype == DT[dtype] and y.shape == x.shape and dx.shape == x.shape
    assert rel(y, want.detach()) <= TOL[dtype]
    # dx = r (h - mean(h) - n mean(h n)) may be far smaller than its terms (at D = 2
    # all but eps / s of it cancels).  n is off by four roundings of 2^-24 at most
    # (mean, difference, r, product), the two means by three (products, sum, factor),
    # and three more come with the two differences and r: some 12 roundings of terms
    # that are at most r max|h|, beside the rounding of dx itself.
    z = x.double()
    h = dy.double() if w is None else dy.double() * w.double()
    r = (z.var(-1, correction=0) + eps).rsqrt()
    terms = (D * (r * h.abs().amax(-1)).square().sum()).sqrt().item()
    off = (dx.cpu().double() - d[0]).norm().item()
    assert off <= TOL[dtype] * d[0].norm().item() + 12 * 2.0 ** -24 * terms
    if w is None:
        assert dw is None and db is None
    else:
        assert rel(dw, d[1]) <= TOL["f32"]
        assert rel(db, d[2]) <= TOL["f32"]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows, D", [
    (1, 8), (3, 2), (5, 64), (17, 96), (70, 512), (9, 520), (33, 768), (1, 1024), (13, 1032),
    (21, 1029), (6, 2048), (7, 2056), (5, 5003), (3, 8192), (2, 16384), (2, 16383), (2000, 40),
    (3001, 129)])
def test_sizes(rows, D, dtype):
    check(*inputs(rows, D, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows, D", [(5, 64), (33, 768), (7, 333)])
def test_without_weights_and_views(rows, D, dtype):
    check(*inputs(rows, D, dtype, weight=False), dtype)
    check(*inputs(rows, D, dtype, wide=True), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_one_element(dtype):
    """D = 1: x equals its mean, y is the bias and dx is 0."""
    op = norm(1, dtype)
    x = torch.randn(10, 1).to(DT[dtype]).cuda()
    b = torch.full((1,), 0.5, device="cuda")
    assert (op.forward(x, None, b) == 0.5).all()
    assert (op.backward(x, x, None, b)[0] == 0).all()


def test_many_rows():
    check(*inputs(40000, 256, "bf16"), "bf16")


def test_large_means():
    """The variance is of differences from the mean: a mean 1000 times the
    spread costs the bits of x itself and no more."""
    x, dy, w, b = inputs(50, 768, "f32")
    x = x + 1000
    check(x, dy, w, b, "f32")
