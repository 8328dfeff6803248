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


@pytest.mark.parametrize("how", ["argument", "current"])
def test_a_workspace_let_go_while_another_stream_uses_it(how):
    """The handle is dropped while its call waits on a side stream: its workspace's memory is not handed
    to anyone before that call has ended."""
    s = ch.make([2], [300], 8, 2, 128, "bf16", seed=3)
    want, tol = ch.attention(s)
    out = torch.zeros_like(s["q"])
    c = _cache(s)
    at, size = c.workspace.data_ptr(), c.workspace.numel()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)                  # a fifth of a second or so
    chunk = _chunk(c, s)
    if how == "argument":
        c.attention(chunk, s["q"], out, s["status"], stream=side)
    else:
        with torch.cuda.stream(side):
            c.attention(chunk, s["q"], out, s["status"])
    del c
    taken = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(3)]
    waiting = not side.query()
    assert waiting and at not in [t.data_ptr() for t in taken]
    side.synchronize()
    assert s["status"].item() == 0
    assert ((out.double() - want).abs() <= tol).all()


def _mixed(B, n_kv, d, fmt, pieces=2, seed=5):
    """B - `pieces` next tokens and as many pieces of 40 rows, spread over the batch."""
    g = torch.Generator().manual_seed(seed)
    kv = torch.randint(1, 200, (B,), generator=g).tolist()
    q = [1] * B
    for i in range(pieces):
        at = i * (B - 1) // max(1, pieces - 1)
        q[at], kv[at] = 40, 90 + i
    return ch.make(q, kv, 4 * n_kv, n_kv, d, fmt, seed=seed)


@pytest.mark.parametrize("fmt,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("e4m3", 64)])
def test_a_mixed_step_takes_a_second_kernel_only_where_it_pays(fmt, d):
    """Next tokens beside pieces of prompts: with few of them a second kernel's launch costs more than it saves, so
    one takes all (it and the join, 2 launches); with many, both run (3).  The outputs are right either way."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per_sm = {64: 1.0, 128: 1.25, 256: 8.0}[d * (2 if fmt == "bf16" else 1)]
    edge = -(-int(per_sm * sms * 4) // 4)
    for n_kv in (8, 2):
        least = -(-edge // n_kv)
        for B, launches in ((least - 1, 2), (least, 3), (8, 2)):
            if B > 400:
                continue
            s = _mixed(B, n_kv, d, fmt)
            want, tol = ch.attention(s)
            c = _cache(s)
            out = torch.full_like(s["q"], 7.0)
            chunk = _chunk(c, s)
            before = c.lib.sdv_kernel_launches()
            c.attention(chunk, s["q"], out, s["status"])
            assert c.lib.sdv_kernel_launches() - before == launches, (B, n_kv)
            assert s["status"].item() == 0
            assert ((out.double() - want).abs() <= tol).all(), (B, n_kv)
    # half of the sequences pieces or more: one kernel
    s = _mixed(64, 8, d, fmt, pieces=33)
    c = _cache(s)
    before = c.lib.sdv_kernel_launches()
    c.attention(_chunk(c, s), s["q"], torch.empty_like(s["q"]), s["status"])
    assert c.lib.sdv_kernel_launches() - before == 2 and s["status"].item() == 0


@pytest.mark.parametrize("window", [0, 33])
@pytest.mark.parametrize("fmt,d,n_q,n_kv", [("bf16", 64, 8, 4), ("e4m3", 64, 8, 4), ("e4m3", 128, 8, 4), ("bf16", 128, 16, 16)])
def test_both_kernels_of_a_mixed_step(fmt, d, n_q, n_kv, window):
    """Next tokens, sequences without rows, more rows than positions and pieces, each in both kernels' shares; then
    the captured call over other lengths."""
    B = 90
    g = torch.Generator().manual_seed(7)
    kv = torch.randint(1, 700, (B,), generator=g).tolist()
    q = [1] * B
    q[3], q[40], q[B - 1] = 300, 150, 40
    q[5], q[6], q[7], kv[7], q[8], kv[8] = 0, 3, 2, 0, 30, 9
    kv[3], kv[40], kv[B - 1] = 650, 150, 41
    s = ch.make(q, kv, n_q, n_kv, d, fmt, seed=11, window=window)
    c = _cache(s)
    chunk, out = _chunk(c, s), torch.full_like(s["q"], 7.0)
    before = c.lib.sdv_kernel_launches()
    c.attention(chunk, s["q"], out, s["status"])
    assert c.lib.sdv_kernel_launches() - before == 3 and s["status"].item() == 0
    want, tol = ch.attention(s)
    assert ((out.double() - want).abs() <= tol).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attention(chunk, s["q"], out, s["status"])
    for k in range(2):
        lens = [max(0, n - 5 * k - b % 7) for b, n in enumerate(kv)]
        s["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        want, tol = ch.attention(dict(s, kv_lens=lens))
        assert s["status"].item() == 0
        assert ((out.double() - want).abs() <= tol).all()


def test_no_second_kernel_for_groups_past_its_rows():
    """A single token of a group of 17 is past the 16 packed rows of the few-row kernel: it is not launched for nothing."""
    s = ch.make([30, 30] + [1] * 158, [40, 60] + list(range(1, 159)), 34, 2, 64, "e4m3", seed=2)
    c = _cache(s)
    out = torch.full_like(s["q"], 7.0)
    before = c.lib.sdv_kernel_launches()
    c.attention(_chunk(c, s), s["q"], out, s["status"])
    assert c.lib.sdv_kernel_launches() - before == 2 and s["status"].item() == 0
    want, tol = ch.attention(s)
    assert ((out.double() - want).abs() <= tol).all()
