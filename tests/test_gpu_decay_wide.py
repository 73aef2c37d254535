"""Linear attention with decays at every width of the kernels where sequences are cut
into segments: effects of segments, the states they begin with, and states kept inside a
sequence for dg, against sums over pairs in 64 bits."""
import pytest
import torch

from tests import decay_pairs
from tests.decay_reference import TOL, decay_inputs, rel

pytestmark = pytest.mark.gpu
TYPES = ["bf16", "f16", "f32"]


def check(dtype, T, Hk, Hv, Dk, Dv, fixed, cu=None, rate=0.02):
    from fft_long_convolution_amd.decay import DecayAttention
    rows = 1 if cu is None else len(cu) - 1
    q, k, v, g, S = (x.cuda() for x in decay_inputs(T + Dk + Dv, 1, T, Hk, Hv, Dk, Dv, dtype,
                                                    rows=rows, fixed=fixed, rate=rate))
    gen = torch.Generator().manual_seed(2)
    do = torch.randn(v.shape, generator=gen).to(v.dtype).cuda()
    dS = (0.3 * torch.randn(S.shape, generator=gen)).cuda()
    op, bounds = DecayAttention(Dk, Dv, dtype=dtype), None if cu is None else torch.tensor(cu).cuda()
    # cut, not walked whole
    assert op._lib.fftconv_decay_workspace_bytes(op._describe(q, k, v, g, bounds, None)[0][1][0]) > 0
    o, fin = op.forward(q, k, v, g, initial_state=S, cu_seqlens=bounds)
    d = op.backward(q, k, v, g, do, d_final_state=dS, initial_state=S, cu_seqlens=bounds)
    want = decay_pairs.batch(q, k, v, do, S, dS, g, cu)
    for name, x in zip(("o", "state", "dq", "dk", "dv", "dg", "dinit"), (o, fin, *d)):
        assert rel(x, want[name].cpu()) <= TOL["f32" if name in ("state", "dg", "dinit") else dtype], name


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("T, Hk, Hv, Dk, Dv", [
    (1300, 1, 2, 128, 256), (1111, 1, 2, 200, 72), (1300, 2, 2, 256, 248), (1037, 1, 1, 40, 136),
    (1200, 1, 2, 96, 128), (1501, 2, 4, 64, 64)])
def test_cut_sequences_of_every_width(T, Hk, Hv, Dk, Dv, fixed, dtype):
    check(dtype, T, Hk, Hv, Dk, Dv, fixed)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("Dk, Dv", [(64, 128), (256, 136), (128, 200)])
def test_packed_sequences_of_every_width(Dk, Dv, fixed, dtype):
    check(dtype, 2600, 1, 2, Dk, Dv, fixed, cu=[5, 5, 900, 901, 2500, 2500, 2564])


@pytest.mark.parametrize("dtype", TYPES)
def test_values_wider_than_gradients_take(dtype):
    """Heads of values up to 1024, forward."""
    from fft_long_convolution_amd.decay import DecayAttention
    q, k, v, g, S = (x.cuda() for x in decay_inputs(6, 1, 1600, 1, 1, 136, 520, dtype, rate=0.02))
    op = DecayAttention(136, 520, dtype=dtype)
    o, fin = op.forward(q, k, v, g, initial_state=S)
    want = decay_pairs.batch(q, k, v, torch.zeros_like(v), S, torch.zeros_like(S), g)
    assert rel(o, want["o"].cpu()) <= TOL[dtype] and rel(fin, want["state"].cpu()) <= TOL["f32"]
