"""The measure that the example block's serving check uses (no GPU)."""
import torch

from tests.test_gpu_example import example


def test_one_wrong_token_shows():
    # a decoded token that is 5 % off is an error of 5 %, among however many
    # tokens that are right
    m = example()
    gen = torch.Generator().manual_seed(1)
    want = torch.randn(256, 128, generator=gen)
    pairs = [(want[:200], want[:200])] + [(want[i:i + 2], want[i:i + 2]) for i in range(200, 250)]
    assert m.worst_error(pairs) == 0
    pairs[7] = (1.05 * pairs[7][1], pairs[7][1])
    assert abs(m.worst_error(pairs) - 0.05) < 1e-5
