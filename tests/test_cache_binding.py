"""The paged cache's Python binding on the CPU: what it hands to the library, and what it refuses before that.

The library is a recorder in place of libsdv.so, so nothing here needs a device."""
import types

import pytest
import torch

from speculative_decoding_verify_ragged_gb300 import cache as pc
from speculative_decoding_verify_ragged_gb300._abi import SdvCacheConfig


class Recorder:
    """Stands in for the library: counts the calls of each entry point and accepts them."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


STREAM = types.SimpleNamespace(cuda_stream=0)


def make_cache(n_q=4, n_kv=2, head_dim=64, fmt="bf16"):
    c = pc.PagedCache.__new__(pc.PagedCache)
    c.lib = Recorder()
    c._setup(SdvCacheConfig(n_q, n_kv, head_dim, 16, pc.FORMATS[fmt], 0.0), fmt, torch.empty(256, dtype=torch.uint8))
    c._streams.add(STREAM.cuda_stream)
    c.handle = 1
    return c


def make_chunk(c, rows=3, pages=4, **kw):
    pool, scales = c.new_pool(pages)
    i32 = dict(dtype=torch.int32)
    a = dict(rows=rows, max_q=3, row_offsets=torch.tensor([0, 3], **i32), kv_lens=torch.tensor([3], **i32),
             page_table=torch.zeros((1, 2), **i32), kv_pool=pool, kv_scales=scales)
    a.update(kw)
    return c.chunk(**a)


def operators(c, chunk, rows=3):
    """The three calls, with rows that fit the cache `c`."""
    n_q, n_kv, d = c.cfg.n_q, c.cfg.n_kv, c.cfg.head_dim
    q, kv = torch.zeros((rows, n_q, d), dtype=torch.bfloat16), torch.zeros((rows, n_kv, d), dtype=torch.bfloat16)
    st = torch.zeros(1, dtype=torch.int32)
    return [lambda: c.append(chunk, kv, kv, st, stream=STREAM), lambda: c.attention(chunk, q, q.clone(), st, stream=STREAM),
            lambda: c.read(chunk, kv, kv.clone(), st, stream=STREAM)]


@pytest.mark.parametrize("other", [dict(n_kv=1), dict(n_kv=4), dict(head_dim=128), dict(fmt="e4m3")])
def test_a_chunk_of_another_geometry_is_refused(other):
    """A chunk's pool was checked against the cache that made it; a cache of other heads, sizes or format would
    run past its end."""
    mine, theirs = make_cache(), make_cache(**other)
    for owner, user in ((mine, theirs), (theirs, mine)):
        chunk = make_chunk(owner)
        for call in operators(user, chunk):
            with pytest.raises(ValueError, match="chunk"):
                call()
        assert user.lib.calls == []
        for call in operators(owner, chunk):
            call()
        assert len(owner.lib.calls) == 3
        owner.lib.calls.clear()


def test_a_chunk_of_the_same_geometry_serves():
    """Another cache of the same heads, size and format may use it: the layers of a model share their chunk's words."""
    mine, twin = make_cache(), make_cache(n_q=8)
    for call in operators(twin, make_chunk(mine)):
        call()
    assert [n for n, _ in twin.lib.calls] == ["sdv_cache_append", "sdv_cache_attention", "sdv_cache_read"]


def test_numbers_past_32_bits_keep_their_meaning():
    """The C fields have 32 bits: a window or a bound longer than that stays one that covers all, a count is refused
    by the library as too large, and a number below 0 stays below 0."""
    c = make_cache()
    top = 2 ** 31 - 1
    s = make_chunk(c, window=2 ** 32 + 5, max_q=2 ** 32 + 1).struct
    assert (s.window, s.max_q) == (top, top)
    assert make_chunk(c, window=2 ** 31).struct.window == top
    assert make_chunk(c, rows=2 ** 32 + 3).struct.T == top
    s = make_chunk(c, window=-2 ** 32 + 5, max_q=-2 ** 31 - 1).struct
    assert s.window < 0 and s.max_q < 0
    # a handle: the library sees the sizes it is asked for, or larger ones than it takes
    seen = []

    class Sizes(Recorder):
        def sdv_cache_workspace_size(self, cfg, rows, slots):
            c = cfg._obj
            seen.append((c.n_q, c.n_kv, c.head_dim, c.page_size, rows, slots))
            return 0

    real, pc.load_library = pc.load_library, lambda *a: Sizes()
    try:
        with pytest.raises(Exception, match="rejected"):
            pc.PagedCache(dict(n_q=2 ** 32 + 4, n_kv=2 ** 32 + 2, head_dim=2 ** 32 + 64, page_size=2 ** 32 + 16), 2 ** 32 + 8, 2 ** 32 + 2)
    finally:
        pc.load_library = real
    assert seen == [(top,) * 6]


def test_one_row_has_no_stride():
    """The stride of a tensor of one row says nothing; the library, which wants 16 bytes of it, gets the row's width."""
    c = make_cache(n_q=4, n_kv=2, head_dim=64)
    chunk = make_chunk(c, rows=1)
    row = lambda heads, st: torch.zeros(1024, dtype=torch.bfloat16).as_strided((1, heads, 64), (st, 64, 1))  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32)
    for odd in (1, 3, 515):
        c.attention(chunk, row(4, odd), row(4, odd), st, stream=STREAM)
        c.append(chunk, row(2, odd), row(2, odd), st, q=row(4, odd), q_out=row(4, odd), stream=STREAM)
        c.read(chunk, row(2, odd), row(2, odd), st, stream=STREAM)
        (_, at), (_, ap), (_, rd) = c.lib.calls[-3:]
        r = ap[2]._obj
        assert (at[3], at[5]) == (256, 256) and (rd[3], rd[5]) == (128, 128)
        assert (r.k_stride, r.v_stride, r.q_stride, r.q_out_stride) == (128, 128, 256, 256)
