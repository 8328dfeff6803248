"""Where sampling's distributions may lie: beside the logits in one buffer, never over them."""
import pytest
import torch

from tests.test_gpu_sample import _check, _logits, _sample, _settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [3001, 151936])
def test_probs_beside_logits_in_one_buffer(V):
    """Columns of rows of one pitch share no byte, so they are taken; rows without a setting are read more than once."""
    rows = 6
    x, u = _logits(rows, V, torch.float32, seed=3)
    buf = torch.full((rows, 2 * V + 1), 5.0, device="cuda")
    z, probs = buf[:, :V], buf[:, V + 1:]
    z.copy_(x)
    status, tokens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    s = _settings(rows, temperature=[1.0, 0.7, 1.5, 1.0, 0.0, 1.0], top_p=[1.0, 0.9, 0.97, 1.0, 1.0, 0.5], top_k=[0, 40, 0, 900, 0, 0])
    _sample()(z, status, uniforms=u, tokens=tokens, probs=probs, **s)
    assert status.item() == 0 and torch.equal(z, x) and (buf[:, V] == 5.0).all()
    _check(x, u, s, tokens.cpu().numpy(), probs.double().cpu().numpy())


def test_probs_over_logits_are_refused():
    from speculative_decoding_verify_ragged_gb300 import SdvError
    rows, V = 4, 2000
    z, u = _logits(rows, V + 8, torch.float32, seed=4)
    before = z.clone()
    status, tokens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    half = z.view(torch.bfloat16)
    for logits, probs in ((z, z), (z[:, :V], z[:, 8:]), (half[:, : V], z[:, :V]), (z[:2], z[1:3]), (z[1:2], z[1:2])):
        with pytest.raises(SdvError):
            _sample()(logits, status, uniforms=u[: len(logits)], tokens=tokens[: len(logits)], probs=probs)
    torch.cuda.synchronize()
    assert torch.equal(z, before) and status.item() == 0 and (tokens == -7).all()
