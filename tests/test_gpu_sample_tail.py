"""The tail of a distribution: probabilities far below the largest, whose differences of logits round most."""
import pytest
import torch

from tests.test_gpu_sample import _sample, _settings

pytestmark = pytest.mark.gpu

# the special-function unit's 2^-22, the correction, its product, the sum's conversion, the quotient and the last product: five of 2^-24
BOUND = 2.0 ** -22 + 5.1 * 2.0 ** -24


@pytest.mark.parametrize("V", [4001, 151936])
@pytest.mark.parametrize("top,temperature", [(77.3, 1.0), (0.1, 1.47), (-50.7, 0.63), (150.2, 1.9), (3.3, 0.05)])
def test_the_tail_of_a_distribution(top, temperature, V):
    """Logits down to 2^-120 of the largest.  A difference of 64 or more rounds by 2^-18, which alone is 2^-18 of a probability."""
    rows = 3
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    s = _settings(rows, temperature=temperature)
    c = s["temperature"][0].double()
    z = top - 120.0 * 0.6931 * c.item() * torch.rand((rows, V), generator=g, device="cuda")
    z[:, 11] = top
    probs, status = torch.full((rows, V), -7.0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    _sample()(z, status, probs=probs, **s)
    assert status.item() == 0
    want = (z.double() / c).softmax(1)
    there = want > 2.0 ** -125
    assert there.float().mean() > 0.9
    assert ((probs.double() - want).abs() / want)[there].max().item() <= BOUND
