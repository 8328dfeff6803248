"""How the chunk attention over codes rounds its weights: rows with one key far above the rest.

The first key of a sequence (the sink) is `gap` nats above the others' mean logit and its value is 0, so the
output is made of the small weights alone; the values have one sign, so that weight lost shows as a shift of the
whole row.  The definition is in 64 bits.  The bounds count, beside what
tests/cache_helpers.py counts for every row, the weights that fall below fp16's normal range: those are off by
2^-25 of the unit that the kernel carries them in.

Few rows (mma.sync): a weight goes in times its value's scale 2^e.  On the first page of a row its largest such product
stands at 2^15, so the unit is 2^-15 of it; on every later page the largest is at least 2^-9 units.
Many rows (tcgen05): steps of 64 keys.  The first step's largest weight stands at 2^4, and every later step's
weights add up to at least 2^-8 units.
"""
import math

import pytest
import torch

from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu

N_Q, N_KV, D = 4, 2, 128


def _sunk(q_len, kv, gap, size, seed, steps=0):
    """One sequence over codes: the sink at position 0, the other values size * (1 + randn / 4).  With `steps`, every
    that many keys stand `gap` times a number in [-1, 1] nats off the mean instead, and the values above it are 0."""
    s = ch.make([q_len], [kv], N_Q, N_KV, D, "e4m3", seed=seed, tail=0.0)
    g = torch.Generator(device="cuda").manual_seed(seed + 50)
    page, slot = s["table"][0].long()[torch.arange(kv, device="cuda") // 16], torch.arange(kv, device="cuda") % 16
    k = torch.randn((kv, N_KV, D), generator=g, device="cuda")
    k[:, :, 0] = 0.0
    k[0] = 0.0
    k[0, :, 0] = gap * math.sqrt(D) / 4.0
    v = size * (1.0 + 0.25 * torch.randn((kv, N_KV, D), generator=g, device="cuda"))
    v[0] = 0.0
    if steps:
        off = gap * (2.0 * torch.rand(-(-kv // steps), generator=g, device="cuda") - 1.0)
        off = off.repeat_interleave(steps)[:kv]
        k[:, :, 0] = (off * math.sqrt(D) / 4.0)[:, None]
        v[off > 0] = 0.0
    exps = []
    for which, x in ((0, k), (1, v)):
        e = ch.exponent(x.abs().amax(-1))
        e = torch.where(x.abs().amax(-1) == 0, torch.full_like(e, -15.0), e)
        codes = (x * torch.exp2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["pool"][page, :, which, slot] = codes.view(torch.uint8)
        s["scales"][page, :, which, slot] = (e + 127).to(torch.uint8)
        s["values"][page, :, which, slot] = codes.double() * torch.exp2(e.double())[..., None]
        exps.append(e)
    s["q"] = torch.randn((q_len, N_Q, D), generator=g, device="cuda").to(torch.bfloat16)
    s["q"][:, :, 0] = 4.0
    return s, exps[1].double()


def _bound(s, e, few):
    """(out, how far it may be off): the weights by blocks of 16 keys (few rows) or 64."""
    n, kv = s["q_lens"][0], s["kv_lens"][0]
    out = torch.zeros((n, N_Q, D), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    at, pos = torch.arange(kv, device="cuda"), ch.positions(s, 0)
    see = at[None] <= pos[:, None]
    width = 16 if few else 64
    for j in range(N_Q):
        k, v = ch.cached(s, 0, j // 2)
        q = s["q"][:, j].double()
        z = ((q @ k.T) / math.sqrt(D)).masked_fill(~see, -math.inf)
        p = torch.softmax(z, -1)
        out[:, j] = p @ v
        size = ((q.abs() @ k.abs().T) / math.sqrt(D)).masked_fill(~see, 0).amax(-1, keepdim=True)
        tol[:, j] = (p @ v.abs()) * (ch.FP16_HALF + 2 * (D * 2.0 ** -23 * size + 2.0 ** -20)) + ch.BF16_HALF * out[:, j].abs()
        scale = torch.exp2(e[:, j // 2])
        for b0 in range(0, kv, width):
            b = slice(b0, min(kv, b0 + width))
            if few:    # against codes: v / scale
                top = (p[:, b] * scale[b]).amax(-1, keepdim=True)
                unit = top * (2.0 ** -15 if b0 == 0 else 2.0 ** 9)
                small = (v[b].abs() / scale[b][:, None]).sum(0)
            else:
                unit = p[:, b].amax(-1, keepdim=True) * 2.0 ** -4 if b0 == 0 else p[:, b].sum(-1, keepdim=True) * 2.0 ** 8
                small = v[b].abs().sum(0)
            tol[:, j] += 2.0 ** -25 * unit * small
    return out, tol


def _check(rows, size, gap, copies, few, steps=0):
    from speculative_decoding_verify_ragged_gb300.cache import PagedCache
    s, e = _sunk(rows, 4096 + rows, gap, size, seed=rows + gap, steps=steps)
    want, tol = _bound(s, e, few)
    c = PagedCache(dict(n_q=N_Q, n_kv=N_KV, head_dim=D, cache_format="e4m3"), max_rows=rows * copies, max_slots=copies)
    q = s["q"].repeat(copies, 1, 1)
    out = torch.full_like(q, 7.0)
    offsets = torch.arange(copies + 1, device="cuda", dtype=torch.int32) * rows
    c.attention(c.chunk(rows=rows * copies, max_q=rows, row_offsets=offsets, kv_lens=s["lens"].repeat(copies),
                        page_table=s["table"].repeat(copies, 1), kv_pool=s["pool"], kv_scales=s["scales"]), q, out, s["status"])
    assert s["status"].item() == 0
    off = (out.double().view(copies, rows, N_Q, D) - want).abs()
    worst = (off / tol).max().item()
    shift = (off.norm() / (want.norm() * copies ** 0.5)).item()
    assert worst <= 1.0, f"{worst:.3g} of the bound, relative 2-norm {shift:.3g}"


# one sequence, cut over the whole GPU, and as many that whole ones are a block's
@pytest.mark.parametrize("copies", [1, 300])
@pytest.mark.parametrize("rows", [1, 7])           # 2 and 14 packed rows
@pytest.mark.parametrize("size", [0.1, 0.01, 0.003])
@pytest.mark.parametrize("gap", [10, 12, 14, 16])
def test_few_rows_beside_a_sink(rows, size, gap, copies):
    _check(rows, size, gap, copies, True)


@pytest.mark.parametrize("copies", [1, 160])
@pytest.mark.parametrize("rows", [9, 64, 200])     # 18, 128 and 400 packed rows
@pytest.mark.parametrize("size", [0.1, 0.01])
@pytest.mark.parametrize("gap", [10, 12, 14, 16, 18])
def test_many_rows_beside_a_sink(rows, size, gap, copies):
    _check(rows, size, gap, copies, False)


@pytest.mark.parametrize("copies", [1, 160])
@pytest.mark.parametrize("rows", [1, 7, 9, 64])
@pytest.mark.parametrize("gap", [3, 8, 15])
def test_steps_up_and_down(rows, gap, copies):
    """The bound follows pages (few rows) or steps of 64 keys that lie up to 30 nats apart, up and down in any
    order; only those below the middle have values."""
    few = rows * 2 <= 16
    _check(rows, 0.1, gap, copies, few, steps=16 if few else 64)
