"""Adapters of rows with infinities, NaN and values past bf16's largest."""
import pytest
import torch

from tests.test_gpu_adapters import _adapters, _apply, _make, _want

pytestmark = pytest.mark.gpu
KINDS = [("bf16", "fp32"), ("fp32", "fp32"), ("bf16", "bf16"), ("fp32", "bf16")]


@pytest.mark.parametrize("x,y", KINDS)
@pytest.mark.parametrize("counts,K,N,rank", [([5], 64, 48, 8), ([3, 40, 1], 264, 96, 24), ([70, 2], 512, 72, 16), ([9], 128, 40, 72)])
def test_infinities_do_what_they_do_in_their_own_rows(counts, K, N, rank, x, y):
    """Every rank value of the row is +-inf; features whose B has one sign become +-inf, others NaN (inf - inf).  Ranks that the kernel
    rounds up to and rows beside it take no part."""
    s = _make(counts, [0] * len(counts), K, N, rank, 1, x, y, seed=rank)
    s["a"][0, :, 7] = s["a"][0, :, 7].abs() + 0.125
    b = s["b"][0].abs() + 0.125
    sign = torch.tensor([1.0, -1.0, 1.0], device="cuda").repeat(N)[:N, None].expand(N, rank).clone()
    sign[2::3, ::2] = -1.0
    s["b"][0] = b * sign
    hit = {0: float("inf"), 2: -float("inf")}
    if sum(counts) > 4:
        hit[4] = float("nan")
    for r, v in hit.items():
        s["x"][r, 7] = v
    _apply(_adapters(s), s)
    assert s["status"].item() == 0
    want, tol = _want(s)
    for r, v in hit.items():
        got = s["out"][r].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want[r])) and torch.equal(got.nan_to_num(0.0, 1.0, -1.0), want[r].nan_to_num(0.0, 1.0, -1.0))
        if v == v:
            assert got[0] == v and got[1] == -v and torch.isnan(got[2])
    rest = [r for r in range(s["T"]) if r not in hit]
    assert ((s["out"].double() - want).abs() <= tol)[rest].all()


@pytest.mark.parametrize("x,y", KINDS)
@pytest.mark.parametrize("rank", [8, 16, 64])
def test_finite_values_past_bf16s_largest(rank, x, y):
    """x (fp32) and rank values between bf16's largest value and fp32's, brought back by small A and B."""
    s = _make([6], [0], 64, 32, rank, 1, x, y, seed=1)
    s["scales"].fill_(1.0)
    if x == "fp32":
        s["x"][1, 3], s["x"][4, 3] = 3.4e38, -3.4e38
        s["a"][0, :, 3] *= 2.0 ** -120
    # row 2's first rank value: (2 - 2^-9) 2^127, of three products
    s["x"][2] = 0.0
    s["a"][0, :, 8:11] = 0.0
    s["a"][0, 0, 8:11] = torch.tensor([2.0 ** 63, 2.0 ** 60, 2.0 ** 60], device="cuda").to(torch.bfloat16)
    s["x"][:, 8:11] = 0.0
    s["x"][2, 8:11] = torch.tensor([1.9921875 * 2.0 ** 64, 2.0 ** 59, 2.0 ** 58], device="cuda").to(s["x"].dtype)
    s["b"][0, :, 0] *= 2.0 ** -120
    _apply(_adapters(s), s)
    assert s["status"].item() == 0
    want, tol = _want(s)
    assert torch.isfinite(want).all() and torch.isfinite(s["out"]).all()
    assert ((s["out"].double() - want).abs() <= tol).all()
    assert (want - s["base"].double())[2].abs().max() > 1.0
