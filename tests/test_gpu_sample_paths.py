"""Sampling of long rows, whose tokens are told from a sampled threshold, a streamed sum and lists, by 8, 4, 2 and 1 blocks to a row.

With 152 SMs a call takes 8 blocks to a row up to 19 rows, 4 up to 76, 2 up to 209, else one (vocabularies of this length); a row's
beginning and what its blocks find differ, its answer may not."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import FINE, TAIL, _logits, _sample, _settings

pytestmark = pytest.mark.gpu
V = 151936
BATCHES = (70, 200, 512)
INF = float("inf")


def _run(z, u, settings):
    rows = z.shape[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tokens, probs = torch.full((rows,), -7, dtype=torch.int32, device="cuda"), torch.full((rows, z.shape[1]), -7.0, device="cuda")
    _sample()(z, status, uniforms=u, tokens=tokens, probs=probs, **settings)
    assert status.item() == 0
    return tokens, probs


def _tile(x, rows):
    return x.repeat((rows + x.shape[0] - 1) // x.shape[0], *[1] * (x.dim() - 1))[:rows].contiguous()


def _told(z, u, settings, tokens, probs):
    """Rows against their definition in 64 bits.  Below 2^-13 of the largest (t = 13) a weight is off by its exponential and two roundings,
    2^-22 + 2^-23, and by the difference's in t, t 2^-24 ln 2; above by 2^-34, and all by half a step of 2^-42.  What that comes to of the
    row's sum is how far a bound may lie from a token's end and take it or leave it, and likewise the token drawn."""
    d = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    st = {n: settings[n].double().tolist() if n in settings else [v] * z.shape[0] for n, v in d.items()}
    for r in range(z.shape[0]):
        t, k, p, m = (st[n][r] for n in d)
        x = z[r].double()
        order = torch.argsort(x, descending=True, stable=True)
        order = order[: int((x > -INF).sum())]
        if t == 0.0 or k > 0:
            order = order[: 1 if t == 0.0 else int(k)]
        v = x[order]
        w = torch.where(v == v[0], 0.0, (v - v[0]) / (t or 1.0)).exp()
        bits = torch.where(v == v[0], 0.0, (v[0] - v) / (t or 1.0) * 1.442695).clamp(max=64.0)
        e = (w * torch.where(bits < 13.0, 2.0 ** -34, bits * 2.0 ** -24 * 0.6932 + 2.0 ** -22 + 2.0 ** -23)).sum().item() / w.sum().item()
        e += v.numel() * 2.0 ** -43
        got = int((probs[r] > 0).sum())
        n = order.numel()
        if p < 1.0 and t > 0.0:
            reach = w.cumsum(0)
            least, most = (min(n, int(torch.searchsorted(reach, (p + s * e) * reach[-1])) + 1) for s in (-1, 1))
            n = max(least, min(got, most))
        if t > 0.0:
            n = min(n, int((w >= m).sum()))
        want = torch.zeros_like(x)
        want[order[:n]] = w[:n] / w[:n].sum()
        tol = torch.where(want > want.max() * 2.0 ** -12.9, FINE, TAIL) * want + 1e-37
        assert ((probs[r].double() - want).abs() <= tol).all(), (r, got, n)
        run, i, point = want.cumsum(0), int(tokens[r]), float(u[r])
        assert probs[r][i] > 0 and run[i] - want[i] <= point + e and point <= run[i] + e, (r, i)


def _unlike_rows(io):
    """Rows that a sample of their beginnings says little of, ties, masks and infinities."""
    g = torch.Generator(device="cuda")
    g.manual_seed(17)
    x, _ = _logits(14, V, torch.float32, seed=40)
    x[1] = 4.25
    x[2] = torch.where(torch.rand(V, generator=g, device="cuda") < 0.3, 1.0, 0.5)
    x[3] = torch.randint(0, 40, (V,), generator=g, device="cuda") / 1024.0
    x[4] = torch.where(torch.rand(V, generator=g, device="cuda") < 0.5, 0.0, -0.0)
    x[5] = x[5].sort().values                       # the beginnings of runs are their smallest
    x[6] = x[6].sort(descending=True).values        # all of it in the first block
    x[7, ::2] = -INF
    x[8] = -INF
    x[8, 140001] = -3.0e38
    x[9, [0, 77, 100003, V - 1]] = INF
    x[10] = -3.4e38
    x[10, 90007] = 3.4e38
    x[11, 40:] = -INF
    x[12, 5:V - 9] = torch.finfo(io).min
    x[13] = 1e-3 * x[13]
    return x.to(io), torch.rand(14, generator=g, device="cuda")


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", [dict(), dict(top_p=0.9), dict(temperature=0.0), dict(top_k=40, top_p=0.95), dict(top_k=1000), dict(min_p=0.3),
                                dict(top_k=9001, top_p=0.37, temperature=1.5)], ids=lambda kw: "-".join(f"{k}{v}" for k, v in kw.items()) or "none")
def test_unlike_rows_in_every_batch(io, kw):
    """Each row is its definition's, and the same bit for bit however many blocks take it."""
    z, u = _unlike_rows(io)
    s = _settings(14, **kw)
    tokens, probs = _run(z, u, s)
    _told(z, u, s, tokens, probs)
    for rows in BATCHES:
        many, p = _run(_tile(z, rows), _tile(u, rows), {n: _tile(v, rows) for n, v in s.items()})
        assert torch.equal(many, _tile(tokens, rows))
        for r in range(0, rows, 14):
            n = min(14, rows - r)
            assert torch.equal(p[r:r + n], probs[:n])


@pytest.mark.parametrize("rows", (3,) + BATCHES)
@pytest.mark.parametrize("at", [0, 70001, V - 1])
def test_a_nan_is_found_wherever_it_is(rows, at):
    z, u = _logits(rows, V, torch.float32, seed=rows)
    z[rows - 2, at] = float("nan")
    for kw in (dict(), dict(top_p=0.9), dict(top_k=5), dict(temperature=0.0)):
        status, tokens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
        _sample()(z, status, uniforms=u, tokens=tokens, **_settings(rows, **kw))
        assert status.item() == 6


@pytest.mark.parametrize("rows", (15,) + BATCHES)
@pytest.mark.parametrize("temperature", [1.0, 1.3])
def test_bounds_about_the_ends_of_tokens(rows, temperature):
    """Top-p bounds from 2^-19 to 2^-14 of the row's sum off a token's end: within the streamed sum's bound (2^-15 of what is not kept) the
    row has to be read again, beyond it not.  The sum of weights as defined lies nearer than 2^-19 to the real one."""
    z, _ = _logits(1, V, torch.float32, seed=23)
    c = float(np.float32(temperature))
    w = (z.double()[0] / c).softmax(0)
    t = (z.double().max() - z.double()[0]) / c * 1.442695
    assert (w * torch.where(t < 13.0, 2.0 ** -34, t * 2.0 ** -24 * 0.6932 + 2.0 ** -22 + 2.0 ** -23)).sum().item() < 2.0 ** -20
    order = torch.argsort(w, descending=True, stable=True)
    reach = w[order].cumsum(0)
    ps = []
    for k in (0, 3, 10, 40, 200, 700, 2000):
        e = reach[k].item()
        ps += [np.float32(e + sign * 2.0 ** -n) for n in range(19, 13, -1) for sign in (1, -1)]
    ps = [float(p) for p in ps if p < 0.9999]
    p = _tile(torch.tensor(ps, dtype=torch.float32, device="cuda"), max(rows, len(ps)))
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    u = torch.rand(p.numel(), generator=g, device="cuda")
    for r0 in range(0, p.numel(), rows):
        pp, uu = p[r0:r0 + rows], u[r0:r0 + rows]
        n = pp.numel()
        tokens, probs = _run(z.expand(n, V).contiguous(), uu, _settings(n, temperature=temperature, top_p=pp.tolist()))
        kept = torch.searchsorted(reach, pp.double()) + 1
        assert torch.equal((probs > 0).sum(1), kept)
        for r in range(n):
            mine = torch.zeros(V, dtype=torch.float64, device="cuda")
            stay = order[:kept[r]]
            mine[stay] = w[stay]
            assert torch.equal(probs[r] > 0, mine > 0)
            run = mine.cumsum(0)
            t, point = int(tokens[r]), uu[r].item() * run[-1].item()
            assert mine[t] > 0 and run[t].item() - mine[t].item() <= point + 2.0 ** -20 and point <= run[t].item() + 2.0 ** -20


@pytest.mark.parametrize("rows", (4,) + BATCHES)
def test_borders_are_met_exactly(rows):
    z = torch.full((rows, V), -2.5, device="cuda")
    ps = [0.25, 0.5, 1.0, 0.75]
    _, probs = _run(z, torch.zeros(rows, device="cuda"), _settings(rows, top_p=[ps[r % 4] for r in range(rows)]))
    assert (probs > 0).sum(1).tolist() == [int(ps[r % 4] * V) for r in range(rows)]


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


@pytest.mark.parametrize("top,temperature", [(0.0, 1.0), (0.1, 1.0), (3.7, 0.7), (-11.3, 3.3)])
def test_weights_are_good_to_two_to_the_minus_34(top, temperature):
    """128 equal largest tokens and 64872 of one other weight w: under top-p of p stay ceil(p (128 + 64872 w)) of the largest.  p is taken
    next to where that changes, as near as fp32 comes (2^-24 of it); w is within 2^-34 and half a step of 2^-42, 2^-32.4 of itself
    together (t is 10 at most), so bounds nearer than 2^-31 are left out."""
    first, n = 128, 65000
    rng = np.random.default_rng(5)
    top, c = float(np.float32(top)), float(np.float32(temperature))
    for t in rng.uniform(8.05, 9.95, 6):
        low = float(np.float32(top - t * np.log(2.0) * c))
        w = np.exp((low - top) / c)
        total = first + (n - first) * w
        ps, want = [], []
        for m in range(1, first):
            p = np.float32(m / total)
            for q in (np.nextafter(p, np.float32(0)), p, np.nextafter(p, np.float32(1))):
                if abs(float(q) * total / m - 1.0) > 2.0 ** -31:
                    ps.append(float(q))
                    want.append(int(np.ceil(float(q) * total)))
        rows = len(ps)
        z = torch.full((rows, n), low, device="cuda")
        z[:, 7:7 + 500 * first:500] = top
        _, probs = _run(z, torch.zeros(rows, device="cuda"), _settings(rows, temperature=temperature, top_p=ps))
        assert (probs > 0).sum(1).tolist() == want, t


def test_random_rows_and_settings():
    """Unlike lengths, kinds of rows and settings in one call each."""
    rng = np.random.default_rng(8)
    for case in range(12):
        n, rows = int(np.exp(rng.uniform(np.log(60), np.log(160000)))), int(rng.integers(1, 24))
        io = (torch.float32, torch.bfloat16)[case % 2]
        z, u = _logits(rows, n, io, seed=100 + case, spread=float(rng.choice([0.3, 2.2, 6.0])), peaks=int(rng.choice([0, 60, 400])))
        if case % 3 == 0:
            z[:, rng.integers(0, n, n // 3)] = -INF
            z[:, n // 2] = 0.5
        s = _settings(rows, temperature=rng.choice([0.0, 0.4, 1.0, 1.7], rows).tolist(), top_k=rng.choice([0, 1, 30, 700, 20000], rows).tolist(),
                      top_p=rng.choice([1.0, 0.3, 0.9, 0.99], rows).tolist(), min_p=rng.choice([0.0, 0.01, 0.2], rows).tolist())
        tokens, probs = _run(z, u, s)
        _told(z, u, s, tokens, probs)
