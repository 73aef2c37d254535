"""Tokens of a packed row before the first and behind the last sequence: no
part of any result, and zeros in the tensors that the calls make."""
import pytest
import torch

from tests.mixer_reference import delta_inputs
from tests.test_gpu_delta import gpu, rule

pytestmark = pytest.mark.gpu

# T, bounds
ROWS = [(200, [70, 130, 131, 180]), (200, [64, 64, 128, 128]), (200, [0, 10, 60]), (77, [3, 77]),
        (300, [299, 300]), (300, [100, 100, 100]), (130, [0, 0]), (64, [64, 64]), (500, [1, 2, 250])]


def poison():
    """Memory that the allocator hands out next holds NaN."""
    blocks = [torch.full((n,), float("nan"), device="cuda")
              for n in (1 << 10, 1 << 13, 1 << 15, 1 << 16, 1 << 17, 1 << 20) for _ in range(12)]
    del blocks


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(2, 2), (1, 3)], ids=str)
@pytest.mark.parametrize("T,bounds", ROWS, ids=str)
def test_tokens_outside_the_bounds(T, bounds, heads, dtype):
    a, z = bounds[0], bounds[-1]
    rows = len(bounds) - 1
    ins = gpu(*delta_inputs(T, 1, T, *heads, 64, 40, dtype, rows=rows))
    # what stands there must not matter
    for x in ins[:5]:
        x[:, :a] = float("nan")
        x[:, z:] = float("nan")
    cu = torch.tensor(bounds, device="cuda")
    d = torch.randn(ins[2].shape, device="cuda").to(ins[2].dtype)
    op = rule(64, 40, dtype)

    def everything(xs, d, cu):
        o, F = op.forward(*xs, initial_state=ins[5], cu_seqlens=cu)
        o2, F2, saved = op.forward_train(*xs, initial_state=ins[5], cu_seqlens=cu)
        g = op.backward(*xs, d, saved, d_final_state=F, initial_state=ins[5], cu_seqlens=cu)
        return [o, o2, *g[:5]], [F, F2, g[5]]

    poison()
    rowwise, states = everything(ins[:5], d, cu)
    held = [x[:, a:z].contiguous() for x in ins[:5]]
    want, want_states = everything(held, d[:, a:z].contiguous(), cu - a)
    for x, y in zip(rowwise, want):
        assert torch.equal(x[:, :a], torch.zeros_like(x[:, :a]))
        assert torch.equal(x[:, z:], torch.zeros_like(x[:, z:]))
        assert torch.equal(x[:, a:z], y)
    for x, y in zip(states, want_states):
        assert torch.equal(x, y)
    # a tensor of the caller keeps what it holds there
    out = torch.full_like(ins[2], 7.0)
    op.forward(*ins[:5], initial_state=ins[5], cu_seqlens=cu, out=out)
    assert (out[:, :a] == 7).all() and (out[:, z:] == 7).all()
    assert torch.equal(out[:, a:z], want[0])
