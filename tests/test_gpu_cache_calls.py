"""Calls of the paged cache's operators that the headers allow at their edges, on the GPU."""
import pytest
import torch

from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu


def _cache(s, **kw):
    from speculative_decoding_verify_ragged_gb300.cache import PagedCache
    a = dict(max_rows=max(1, s["T"]), max_slots=len(s["q_lens"]))
    a.update(kw)
    return PagedCache(dict(n_q=s["n_q"], n_kv=s["n_kv"], head_dim=s["d"], cache_format=s["fmt"]), **a)


def _chunk(c, s, **kw):
    a = dict(rows=s["T"], max_q=max(s["q_lens"]), row_offsets=s["row_offsets"], kv_lens=s["lens"], page_table=s["table"],
             kv_pool=s["pool"], kv_scales=s["scales"], window=s["window"])
    a.update(kw)
    return c.chunk(**a)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_step_without_rows(fmt):
    """T = 0: empty tensors (null pointers) are taken, the cache and the status word stay as they are."""
    s = ch.make([0, 0], [40, 7], 4, 2, 64, fmt, seed=1, tail=0.0)
    c = _cache(s)
    chunk = _chunk(c, s)
    pool = s["pool"].clone()
    for dtype in (torch.bfloat16, torch.float32):
        q, kv = torch.zeros((0, 4, 64), dtype=dtype, device="cuda"), torch.zeros((0, 2, 64), dtype=dtype, device="cuda")
        out = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
        assert q.data_ptr() == 0
        c.append(chunk, kv, kv.clone(), s["status"], q=q, q_out=out)
        c.append(chunk, kv, kv.clone(), s["status"])
        c.read(chunk, kv, kv.clone(), s["status"])
        c.read(chunk, None, kv, s["status"])
        c.attention(chunk, out, out.clone(), s["status"])
    assert s["status"].item() == 0 and torch.equal(s["pool"], pool)
    with pytest.raises(ValueError):
        c.read(chunk, None, None, s["status"])
