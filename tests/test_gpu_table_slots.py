"""Steps of fewer requests than the tables have slots: the others have no rows in them."""
import pytest
import torch

from tests.test_gpu_tables import Model, _i32, _same, _tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slots,rows", [(5, 50), (40, 3000), (1024, 2000)])
def test_offsets_and_last_rows_of_the_other_slots(slots, rows):
    t, m = _tables(slots, rows, 4, 4 * slots), Model(slots, rows, 4, 4 * slots)
    status = _i32([0])
    for B in (slots, 2, slots - 1, 1, slots):
        new = [(7 * b + B) % 3 for b in range(B)]
        lens = [min(64, 20 + n) for n in new]
        t.row_offsets.fill_(99)
        t.last_rows.fill_(99)
        t.plan(_i32(new), _i32(lens), status)
        assert status.item() == 0
        _same(t, m, m.plan(new, lens), B)
        assert t.row_offsets.tolist()[B:] == [sum(new)] * (slots + 1 - B)
        assert t.last_rows.tolist()[B:] == [-1] * (slots - B)


def test_one_chunk_serves_steps_of_any_number_of_requests():
    """A chunk over all slots: a step of two requests writes their positions and nothing of the others'."""
    from speculative_decoding_verify_ragged_gb300.cache import PagedCache
    B, T, W = 5, 24, 3
    t = _tables(B, T, W, B * W)
    c = PagedCache(dict(n_q=2, n_kv=1, head_dim=64), max_rows=T, max_slots=B)
    pool, _ = c.new_pool(B * W)
    status, lens = _i32([0]), _i32([6, 4, 17, 5, 3])
    chunk = c.chunk(rows=T, max_q=T, row_offsets=t.row_offsets, kv_lens=lens, page_table=t.page_table, kv_pool=pool)
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    k, v = (torch.randn((T, 1, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    t.plan(_i32([6, 4, 8, 3, 3]), lens, status)
    c.append(chunk, k, v, status)
    before, table = pool.clone(), t.page_table.tolist()
    for x in (k, v):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    lens[:2] = _i32([7, 6])
    t.plan(_i32([1, 2]), lens[:2].contiguous(), status)
    c.append(chunk, k, v, status)
    q, out = (torch.zeros((T, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out.fill_(7.0)
    c.attention(chunk, q, out, status)
    assert status.item() == 0
    want = before.clone()
    for row, slot, pos in ((0, 0, 6), (1, 1, 4), (2, 1, 5)):
        want[table[slot][0], 0, 0, pos], want[table[slot][0], 0, 1, pos] = k[row, 0], v[row, 0]
    assert torch.equal(pool, want)
    assert (out[3:] == 7.0).all() and not (out[:3] == 7.0).any()
