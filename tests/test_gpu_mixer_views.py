"""Views of wide tensors through every entry point of the token mixers: the
bits of the calls on contiguous tensors."""
import pytest
import torch

from tests.mixer_reference import delta_inputs

pytestmark = pytest.mark.gpu


def ops(D, dtype="bf16"):
    from fft_long_convolution_amd.delta import GatedDelta, QKNorm
    return GatedDelta(D, D, dtype=dtype), QKNorm(D, rotary_dim=D // 2, norm="l2", dtype=dtype)


def inputs(B, T, Hk, Hv, D, dtype="bf16"):
    return [x.cuda() for x in delta_inputs(B * T + Hv, B, T, Hk, Hv, D, D, dtype)]


def views(xs, offset, layout):
    """q, k, v as parts of one projection, `offset` elements off a 16-byte
    boundary: token-major, or with the heads outside."""
    B, T = xs[0].shape[:2]
    H = sum(x.shape[2] for x in xs)
    D = xs[0].shape[3]
    base = torch.zeros(B * T * (H * D + 8) + offset, dtype=xs[0].dtype, device="cuda")[offset:]
    if layout == "tokens":
        wide = base.view(B, T, H * D + 8)[..., :H * D].unflatten(-1, (H, D))
    else:
        wide = base[:B * T * H * D].view(B, H, T, D).transpose(1, 2)
    out, at = [], 0
    for x in xs:
        out.append(wide[:, :, at:at + x.shape[2]])
        out[-1].copy_(x)
        at += x.shape[2]
    return out


def spread(x):
    """x with gaps between its rows, misaligned."""
    y = torch.zeros(x.numel() * 2 + 4, dtype=x.dtype, device="cuda")[4:].view(*x.shape[:-1], -1)
    y = y[..., :x.shape[-1]]
    return y.copy_(x)


def everything(q, k, v, g, beta, S, d, stream=None):
    """All outputs of the six entry points, on `stream`."""
    rule, norm = ops(q.shape[3])
    B, T, D = q.shape[0], q.shape[1], q.shape[3]
    angle = torch.arange(T, device="cuda")[:, None] * torch.ones(D // 4, device="cuda") / 7
    table = dict(cos=angle.cos(), sin=angle.sin(),
                 positions=torch.arange(T, device="cuda").expand(B, T))
    w = torch.linspace(0.5, 1.5, D, device="cuda")
    kw = dict(stream=stream)
    out = [*norm.forward(q, k, w, w, **table, **kw)]
    dq, dk = d[:, :, :q.shape[2]], d[:, :, :k.shape[2]]
    out += norm.backward(q, k, dq, dk, w, w, **table, **kw)
    out += rule.forward(q, k, v, g, beta, initial_state=S, **kw)
    o, F, saved = rule.forward_train(q, k, v, g, beta, initial_state=S, **kw)
    out += [o, F]
    out += rule.backward(q, k, v, g, beta, d, saved, d_final_state=F, initial_state=S, **kw)
    state = S.clone()
    if stream is not None:
        stream.synchronize()
    out.append(rule.step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], state, **kw))
    if stream is not None:
        stream.synchronize()
    return out + [state]


@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("offset", [0, 4])
@pytest.mark.parametrize("heads", [(2, 2), (1, 3)], ids=str)
def test_views_of_a_projection(heads, offset, layout):
    q, k, v, g, beta, S = inputs(2, 70, *heads, 64)
    d = torch.randn(v.shape, device="cuda").to(v.dtype)
    want = everything(q, k, v, g, beta, S, d)
    wide = views([q, k, v], offset, layout)
    assert not any(x.is_contiguous() for x in wide)
    assert (wide[0].data_ptr() % 16 != 0) == (offset != 0)
    got = everything(*wide, g, beta, S, d)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("heads", [(2, 2), (1, 3)], ids=str)
def test_views_of_everything_on_another_stream(heads):
    q, k, v, g, beta, S = inputs(2, 70, *heads, 64)
    d = torch.randn(v.shape, device="cuda").to(v.dtype)
    want = everything(q, k, v, g, beta, S, d)
    wide = views([q, k, v], 4, "tokens")
    torch.cuda.synchronize()
    got = everything(*wide, spread(g), spread(beta), spread(S).contiguous(), spread(d),
                     stream=torch.cuda.Stream())
    for a, b in zip(got, want):
        assert torch.equal(a, b)
