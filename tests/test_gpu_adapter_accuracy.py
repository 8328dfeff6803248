"""How far the adapters' fp32 outs are off as a whole, and the batches whose clusters and items the small ones do not meet.

Bound of the relative error (root mean square over the batch): of a request of up to 16 rows a warp's products of a slab are two MMAs of
x's first part (those of the others are 2^-9 and less of it), which may cut two steps of 2^-23 each (what is added up and what it
is added to), as may the one of the second product: 3 * 2 * 2^-23 = 7.2e-7 where all cut alike.  Rounded sums, 2^-24 / sqrt(3) each and
independent: 40 slabs at 0.7 of the sum on average, then 8 warps and up to 8 blocks: 2.1e-7 in all.  Three parts hold x and the
rank values to 2^-27.  Together below 2^-20.  With two parts it is 2.4e-6: each leaves 2^-8 / (1.44 sqrt(3)) on average."""
import pytest
import torch

from tests.test_gpu_adapters import _adapters, _apply, _check, _make

BOUND = 2.0 ** -20
KINDS = [("bf16", "fp32"), ("fp32", "fp32"), ("bf16", "bf16"), ("fp32", "bf16")]


def _parts(x, n):
    out = torch.zeros_like(x)
    for _ in range(n):
        out = out + (x - out).to(torch.bfloat16).float()
    return out


@pytest.mark.parametrize("lost", ["x", "v"])
def test_two_parts_would_be_told(lost):
    """The bound is one that a lost third part of x or of the rank values does not keep (everything else in 64 bits)."""
    g = torch.Generator()
    g.manual_seed(1)
    x, a, b = (torch.randn(s, generator=g) for s in ((32, 2000), (16, 2000), (64, 16)))
    a, b = (t.to(torch.bfloat16).double() for t in (a, b))
    want = (x.double() @ a.T) @ b.T
    for n, told in ((2, True), (3, False)):
        v = (_parts(x, n) if lost == "x" else x).double() @ a.T
        v = _parts(v.float(), n).double() if lost == "v" else v
        err = (v @ b.T - want).norm() / want.norm()
        assert (err > 2 * BOUND) == told


@pytest.mark.gpu
@pytest.mark.parametrize("x", ["fp32", "bf16"])
@pytest.mark.parametrize("counts", [[16] * 4, [16] * 40, [16] * 130, [1] * 3])
def test_the_error_of_a_batch(counts, x):
    """Clusters of 8, 4 and 2 blocks (items: half the requests more than there are); long sums of each block's slabs."""
    s = _make(counts, [b % 3 for b in range(len(counts))], 10000, 64, 16, 3, x, "fp32", seed=len(counts))
    s["base"].zero_()
    _apply(_adapters(s), s)
    want = torch.zeros_like(s["out"], dtype=torch.float64)
    for b, i in enumerate(s["ids"]):
        rows = slice(s["off"][b], s["off"][b + 1])
        want[rows] = s["scales"][i].double() * (s["x"][rows].double() @ s["a"][i].double().T) @ s["b"][i].double().T
    assert s["status"].item() == 0
    assert ((s["out"].double() - want).norm() / want.norm()).item() < BOUND


@pytest.mark.gpu
@pytest.mark.parametrize("x,y", KINDS)
@pytest.mark.parametrize("rank", [32, 64])
@pytest.mark.parametrize("counts", [[300], [1000] * 4, [1000, 999] * 4], ids=["8 blocks", "4 blocks", "2 blocks"])
def test_items_of_64_rows(counts, rank, x, y):
    s = _make(counts, [(b % 4) - (b == 2) * 3 for b in range(len(counts))], 520, 264, rank, 4, x, y, seed=rank)
    _apply(_adapters(s), s)
    _check(s, s["out"])


@pytest.mark.gpu
@pytest.mark.parametrize("x,y", KINDS)
@pytest.mark.parametrize("counts,rank", [([40, 3], 128), ([40, 3], 96), ([700] * 3, 128), ([500] * 8, 72)])
def test_wide_ranks_and_many_features(counts, rank, x, y):
    """Several groups of features a warp at ranks above 64, by 8, 4 and 2 blocks to an item."""
    s = _make(counts, [1, 0, 1, 1, 0, -1, 0, 1][:len(counts)], 264, 4104, rank, 2, x, y, seed=rank)
    _apply(_adapters(s), s)
    _check(s, s["out"])


@pytest.mark.gpu
def test_more_long_items_than_clusters():
    s = _make([500] * 90, [b % 3 for b in range(90)], 64, 40, 16, 3, seed=2)
    _apply(_adapters(s), s)
    _check(s, s["out"])
