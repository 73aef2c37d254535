"""The token mixers' binding without a GPU: what it hands to the library, with
the calls recorded in place of run."""
import pytest
import torch

from fft_long_convolution_amd import delta


@pytest.fixture
def calls(monkeypatch):
    """Calls as (name, descriptor, tensors kept, arguments), of CPU tensors."""
    seen = []

    def call(self, fn, device, stream, kept, ref, *args):
        seen.append((fn.__name__, ref._obj, kept, args))

    monkeypatch.setattr(delta._Op, "_known", {})
    monkeypatch.setattr(delta._Op, "_first", lambda self, q, dims: q.device)
    monkeypatch.setattr(delta._Op, "_call", call)
    return seen


def projection(B, T, heads, D, offset, pad, dtype=torch.bfloat16):
    """Views [B, T, heads, D] of one wide projection, `offset` elements off a
    16-byte boundary; strides are multiples of eight elements."""
    x = torch.arange(B * T * (sum(heads) * D + pad) + 8, dtype=torch.float32).to(dtype)
    start = next(i for i in range(8) if (x[i:].data_ptr() - 2 * offset) % 16 == 0)
    x = x[start:start + B * T * (sum(heads) * D + pad)].view(B, T, -1)
    out, at = [], 0
    for h in heads:
        out.append(x[..., at:at + h * D].unflatten(-1, (h, D)))
        at += h * D
    return out


def run(name, q, k, v):
    """The entry point `name` on these tensors."""
    B, T, Hk, D = q.shape
    Hv = v.shape[2]
    rule, norm = delta.GatedDelta(D, D), delta.QKNorm(D)
    g = torch.zeros(B, T, Hv)
    if name == "norm.forward":
        norm.forward(q, k)
    elif name == "norm.backward":
        norm.backward(q, k, torch.zeros(q.shape, dtype=q.dtype), torch.zeros(k.shape, dtype=q.dtype))
    elif name == "forward":
        rule.forward(q, k, v, g, g)
    elif name == "forward_train":
        rule.forward_train(q, k, v, g, g)
    elif name == "backward":
        saved = torch.zeros(16, dtype=torch.uint8)
        rule.backward(q, k, v, g, g, torch.zeros(v.shape, dtype=v.dtype), saved)
    else:
        rule.step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], g[:, 0], torch.zeros(B, Hv, D, D))


NAMES = ["norm.forward", "norm.backward", "forward", "forward_train", "backward", "step"]


@pytest.mark.parametrize("twice", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_descriptor_has_the_strides_of_the_tensors_passed(calls, name, twice):
    for offset in (0, 4):
        q, k, v = projection(2, 5, (6, 6, 6), 128, offset, 8)
        assert q.data_ptr() % 16 == 2 * offset and not q.is_contiguous()
        for _ in range(1 + twice):
            run(name, q, k, v)
    aligned, copied = calls[0][2][:3], calls[-1][2][:3]
    # the aligned views go in as they are
    assert aligned[0].data_ptr() == calls[0][3][0] and not aligned[0].is_contiguous()
    for _, desc, kept, args in calls:
        strides = [desc.q_stride, desc.k_stride]
        if not name.startswith("norm"):
            strides.append(desc.v_stride)
        for x, ptr, st in zip(kept, args, strides):
            want = list(x.stride()[:3]) if x.dim() == 4 else [x.stride(0), 0, x.stride(1)]
            assert list(st) == want and x.stride(-1) == 1
            assert ptr == x.data_ptr() and ptr % 16 == 0
    q, k, v = projection(2, 5, (6, 6, 6), 128, 4, 8)
    for x, y in zip(copied, (q, k, v) if not name.startswith("norm") else (q, k)):
        assert torch.equal(x, y if x.dim() == 4 else y[:, 0])


def test_settings_changed_after_the_first_call(calls):
    # descriptors are kept by the settings they were made with: neither the
    # changed operator nor another of the old settings gets the wrong one
    q, k, v = projection(1, 4, (2, 2, 2), 64, 0, 0)
    g = torch.zeros(1, 4, 2)
    for change_first in (False, True):
        a, b = delta.GatedDelta(64, 64), delta.GatedDelta(64, 64)
        if not change_first:
            a.forward(q, k, v, g, g)
        a.scale = 3.0
        a.forward(q, k, v, g, g)
        assert calls[-1][1].scale == 3.0
        b.forward(q, k, v, g, g)
        assert calls[-1][1].scale == 0.125
        delta._Op._known.clear()
        a, b = delta.QKNorm(64, eps=1e-6), delta.QKNorm(64, eps=1e-6)
        if not change_first:
            a.forward(q, k)
        a.eps, a.norm = 0.5, "l2"
        a.forward(q, k)
        assert calls[-1][1].eps == 0.5 and calls[-1][1].norm == delta.NORMS["l2"]
        b.forward(q, k)
        assert abs(calls[-1][1].eps - 1e-6) < 1e-12 and calls[-1][1].norm == 0
        delta._Op._known.clear()
    with pytest.raises(AttributeError):
        delta.GatedDelta(64, 64).dtype = "f16"
