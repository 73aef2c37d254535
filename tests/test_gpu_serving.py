"""The example block's decoding sees the tokens up to its own."""
import pytest
import torch

from tests.test_gpu_example import example

pytestmark = pytest.mark.gpu


def test_decoding_does_not_see_later_tokens():
    m = example()
    torch.manual_seed(1)
    block = m.HybridBlock(128, 2, 256).cuda()
    x = torch.randn(2, 256, 128, device="cuda").bfloat16()
    late = x.clone()
    late[0, 200 + 4:] = 7.0
    late[1, 100 + 4:] = -7.0
    with torch.no_grad():
        a, b = (m.serve(block, y, (200, 100), 8) for y in (x, late))
    # two prompts and four tokens that both runs were given alike
    for (y, _), (z, _) in zip(a[:6], b[:6]):
        assert torch.equal(y, z)
    assert not torch.equal(a[6][0], b[6][0])
