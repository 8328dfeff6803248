"""Sampling of long rows, whose tokens are told from a sampled threshold, a streamed sum and lists."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import _sample, _settings

pytestmark = pytest.mark.gpu


def _run(z, u, settings):
    rows = z.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens, probs = torch.full((rows,), -7, dtype=torch.int32, device="cuda"), torch.full((rows, z.shape[1]), -7.0, device="cuda")
    _sample()(z, status, uniforms=u, tokens=tokens, probs=probs, **settings)
    assert status.item() == 0
    return tokens, probs


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("steps_off", [150000, -150000])
def test_what_lies_below_half_a_step_adds_nothing(rows, steps_off):
    """A million tokens between 2^-43 and 2^-44 of the largest round to 0 each, though they add up to 390 thousand steps of 2^-42.  A bound
    `steps_off` such steps above a token's end (of what the sum is by its definition: below it) leaves that token alone or takes the next."""
    n = 1 << 20
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    z = -(43.1 + 0.8 * torch.rand((1, n), generator=g, device="cuda")) * 0.6931472
    p = float(np.float32(0.6))
    want = (1.0 / p - 1.0) - steps_off * 2.0 ** -42              # the second token's weight
    z[0, 0], z[0, 1] = 0.0, float(np.float32(np.log(want)))
    got = (float(np.exp(np.float64(z[0, 1].item()))) - (1.0 / p - 1.0)) * 2.0 ** 42
    assert abs(got + steps_off) < 60000                          # (z itself comes in steps of 2^-25)
    assert z[0, 2:].max().item() < -43.02 * 0.6931472
    tokens, probs = _run(z.expand(rows, n).contiguous(), torch.full((rows,), 0.99, device="cuda"), _settings(rows, top_p=p))
    assert (probs > 0).sum(1).tolist() == [1 if steps_off > 0 else 2] * rows
    assert tokens.tolist() == [0 if steps_off > 0 else 1] * rows
