"""The paged cache's operators (include/sdv_cache.h) on the GPU, against their definition in 64 bits."""
import pytest
import torch

from tests import cache_helpers as ch

pytestmark = pytest.mark.gpu


def _cache(s, theta=0.0, rows=None, slots=None):
    from speculative_decoding_verify_ragged_gb300.cache import PagedCache
    return PagedCache(dict(n_q=s["n_q"], n_kv=s["n_kv"], head_dim=s["d"], cache_format=s["fmt"], rope_theta=theta),
                      max_rows=rows or max(1, s["T"]), max_slots=slots or len(s["q_lens"]))


def _chunk(c, s, **kw):
    a = dict(rows=s["T"], max_q=max(s["q_lens"]), row_offsets=s["row_offsets"], kv_lens=s["lens"], page_table=s["table"],
             kv_pool=s["pool"], kv_scales=s["scales"], window=s["window"])
    a.update(kw)
    return c.chunk(**a)


def _close(got, want, tol):
    assert torch.isfinite(got).all()
    off = (got.double() - want).abs()
    worst = (off / tol).max().item()
    assert worst <= 1.0, f"{worst:.3g} of the bound; max off {off.max().item():.3g}"


def _attend(s, c=None):
    c = c or _cache(s)
    out = torch.full_like(s["q"], 7.0)
    c.attention(_chunk(c, s), s["q"], out, s["status"])
    torch.cuda.synchronize()
    assert s["status"].item() == 0
    return out


HEADS = [(32, 8, 128), (4, 2, 64), (6, 6, 128), (16, 1, 64), (20, 4, 128), (7, 1, 128), (64, 2, 64)]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("lens", [
    ([1], [1]),
    ([1, 1, 1, 1], [1, 15, 16, 17]),
    ([1, 3, 0, 2, 16, 17], [513, 3, 40, 129, 16, 300]),
    ([5, 33], [2, 33]),                       # more rows than positions: the first are empty
    ([0, 1, 0], [7, 0, 0]),                   # no rows, no positions
    ([130, 1, 61], [130, 700, 255]),
], ids=["one", "page_ends", "ragged", "empty_rows", "nothing", "prompts"])
def test_attention(fmt, heads, lens):
    s = ch.make(*lens, *heads, fmt, seed=len(lens[0]))
    want, tol = ch.attention(s)
    _close(_attend(s), want, tol)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 7, 16, 100, 5000, 2 ** 31 - 1])
def test_attention_window(fmt, window):
    s = ch.make([1, 40, 257, 2], [300, 40, 600, 33], 8, 2, 128, fmt, seed=window, window=window)
    want, tol = ch.attention(s)
    # entries before every row's window may be anything: they are not read
    for b, (n, m) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        s["table"][b, :max(0, m - n - window + 1) // 16] = -5
    _close(_attend(s), want, tol)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q,kv", [(1, 20000), (4, 9001), (700, 5000), (1500, 1500), (64, 12345)])
def test_attention_long(fmt, d, q, kv):
    s = ch.make([q], [kv], 8, 2, d, fmt, seed=q)
    want, tol = ch.attention(s)
    _close(_attend(s), want, tol)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_many_sequences(fmt):
    g = torch.Generator().manual_seed(4)
    kv = torch.randint(1, 900, (300,), generator=g).tolist()
    q = [min(int(n), m) for n, m in zip(torch.randint(0, 6, (300,), generator=g).tolist(), kv)]
    s = ch.make(q, kv, 8, 2, 64, fmt, seed=9)
    want, tol = ch.attention(s)
    _close(_attend(s), want, tol)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_extreme_values(fmt):
    """Large and tiny queries, a row of zeros, logits far apart: the running maximum carries them."""
    s = ch.make([6, 40], [200, 300], 8, 2, 128, fmt, seed=5)
    s["q"][0] *= 2.0 ** 6
    s["q"][1] = 0
    s["q"][2] *= 2.0 ** -60
    s["q"][3, :, ::2] = 0
    s["q"][7:20] *= 2.0 ** 5
    want, tol = ch.attention(s)
    _close(_attend(s), want, tol)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 9, 3], [50, 9, 777]), ([200, 1], [431, 90])])
def test_attention_strides_and_rows_behind(fmt, q_lens, kv_lens):
    """q and out as parts of wider rows; rows behind the last sequence and the rest of the wide rows stay."""
    s = ch.make(q_lens, kv_lens, 8, 2, 64, fmt, seed=3)
    want, tol = ch.attention(s)
    T = s["T"]
    wide = torch.full((T + 5, 13, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:T, 2:10] = s["q"]
    out = torch.full((T + 5, 11, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    c = _cache(s, rows=T + 5)
    c.attention(_chunk(c, s, rows=T + 5), wide[:, 2:10], out[:, 1:9], s["status"])
    assert s["status"].item() == 0
    _close(out[:T, 1:9], want, tol)
    assert (out[T:] == 3.0).all() and (out[:, 0] == 3.0).all() and (out[:, 9:] == 3.0).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q,kv", [(1, 700), (300, 900)])
def test_attention_offsets_past_32_bits(fmt, q, kv):
    """Pages whose element offset passes 2^31 (and 2^32 bytes)."""
    n_kv, d = 8, 128
    s = ch.make([q], [kv], 16, n_kv, d, fmt, seed=2)
    want, tol = ch.attention(s)
    far = (1 << 31) // (n_kv * 2 * 16 * d) + 9
    n = s["pool"].shape[0]
    pool = torch.empty((far + n,) + tuple(s["pool"].shape[1:]), dtype=s["pool"].dtype, device="cuda")
    pool[far:] = s["pool"]
    if s["scales"] is not None:
        scales = torch.full((far + n,) + tuple(s["scales"].shape[1:]), 127, dtype=torch.uint8, device="cuda")
        scales[far:] = s["scales"]
        s["scales"] = scales
    s["pool"] = pool
    s["table"] = torch.where(s["table"] >= 0, s["table"] + far, s["table"])
    _close(_attend(s), want, tol)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 4], [3000, 900]), ([600, 1, 20], [1800, 700, 20])])
def test_attention_same_bits_again(q_lens, kv_lens):
    s = ch.make(q_lens, kv_lens, 32, 8, 128, "bf16", seed=6)
    c = _cache(s)
    first = _attend(s, c)
    for _ in range(3):
        assert torch.equal(_attend(s, c), first)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_read(fmt, d):
    s = ch.make([1, 40, 0, 9, 33], [5, 40, 17, 4, 500], 4, 2, d, fmt, seed=1)
    T = s["T"]
    c = _cache(s, rows=T + 2)
    for dtype in (torch.float32, torch.bfloat16):
        k = torch.full((T + 2, 2, d), 3.0, dtype=dtype, device="cuda")
        wide = torch.full((T + 2, 5, d), 3.0, dtype=dtype, device="cuda")
        c.read(_chunk(c, s, rows=T + 2), k, wide[:, 1:3], s["status"])
        assert s["status"].item() == 0
        r0 = 0
        for b, n in enumerate(s["q_lens"]):
            pos = ch.positions(s, b)
            there = pos >= 0
            for h in range(2):
                kk, vv = ch.cached(s, b, h)
                assert torch.equal(k[r0:r0 + n, h][there].double(), kk[pos[there]])
                assert torch.equal(wide[r0:r0 + n, 1 + h][there].double(), vv[pos[there]])
                assert (k[r0:r0 + n, h][~there] == 0).all() and (wide[r0:r0 + n, 1 + h][~there] == 0).all()
            r0 += n
        assert (k[T:] == 3.0).all() and (wide[T:] == 3.0).all() and (wide[:, 0] == 3.0).all() and (wide[:, 3:] == 3.0).all()
        only = torch.zeros((T, 2, d), dtype=dtype, device="cuda")
        c.read(_chunk(c, s), None, only, s["status"])
        assert torch.equal(only, wide[:T, 1:3])


def _append_case(q_lens, kv_lens, n_q, n_kv, d, fmt, dtype, seed):
    s = ch.make(q_lens, kv_lens, n_q, n_kv, d, fmt, seed=seed, tail=0.0)
    if s["scales"] is not None:
        s["scales"].clamp_(max=134)
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    x = torch.randn((s["T"] + 2, n_q + 2 * n_kv, d), generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-6, 7, (s["T"] + 2, n_q + 2 * n_kv, 1), generator=g, device="cuda").float())
    s["x"] = x.to(dtype)
    return s


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("theta", [0.0, 1e6])
@pytest.mark.parametrize("heads", [(32, 8, 128), (4, 2, 64), (5, 1, 128), (3, 3, 64)], ids=lambda h: "x".join(map(str, h)))
def test_append(fmt, dtype, theta, heads):
    """Each stored value against the rotation in 64 bits: half a step of the format, and of fp32 for the
    rotation (cosine, sine, two products and their sum: at most 8 half steps of the larger of the pair); every other place
    of the cache as it was."""
    n_q, n_kv, d = heads
    s = _append_case([1, 40, 0, 9, 300], [5000, 40, 17, 4, 70000], n_q, n_kv, d, fmt, dtype, 7)
    T, x = s["T"], s["x"]
    q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    before = (s["pool"].clone(), None if s["scales"] is None else s["scales"].clone())
    q_out = torch.full((T + 2, n_q, d), 5.0, dtype=torch.bfloat16, device="cuda")
    c = _cache(s, theta, rows=T + 2)
    c.append(_chunk(c, s, rows=T + 2), k, v, s["status"], q=q, q_out=q_out)
    assert s["status"].item() == 0
    touched = torch.zeros(s["pool"].shape[:1] + (16,), dtype=torch.bool, device="cuda")
    r0 = 0
    pair = lambda t: torch.maximum(t[..., :d // 2].abs(), t[..., d // 2:].abs()).repeat(1, 1, 2).double()  # noqa: E731
    for b, n in enumerate(s["q_lens"]):
        pos = ch.positions(s, b)
        there = pos >= 0
        pos = pos[there]
        page, slot = s["table"][b].long()[pos // 16], pos % 16
        touched[page, slot] = True
        rows = slice(r0 + n - len(pos), r0 + n)
        assert (q_out[r0:rows.start] == 5.0).all()
        turn = (lambda t: ch.rotate(t, pos, theta, d)) if theta else (lambda t: t.double())
        slip = 8 * 2.0 ** -24 if theta else 0.0
        want = turn(q[rows])
        assert ((q_out[rows].double() - want).abs() <= ch.BF16_HALF * want.abs() + 1.01 * slip * pair(q[rows])).all()
        for which, (t, f) in enumerate(((k[rows], turn), (v[rows], lambda t: t.double()))):
            want, fp32 = f(t), (slip if which == 0 else 0.0) * pair(t)
            if fmt == "bf16":
                got = s["pool"][page, :, which, slot].double()
                assert ((got - want).abs() <= ch.BF16_HALF * want.abs() + 1.01 * fp32).all()
            else:
                byte = s["scales"][page, :, which, slot].double()
                e = byte - 127
                amax = want.abs().amax(-1)
                near = fp32.amax(-1)
                assert ((e >= ch.exponent(amax - near)) & (e <= ch.exponent(amax + near))).all()
                got = s["pool"].view(torch.float8_e4m3fn)[page, :, which, slot].double() * torch.exp2(e)[..., None]
                # a half step is 2^-4 relative, or half of the subnormal step 2^-9, of the scale
                assert ((got - want).abs() <= torch.maximum(ch.E4M3_HALF * want.abs(), 2.0 ** -10 * torch.exp2(e)[..., None])
                        + 1.07 * fp32).all()
        r0 += n
    assert (q_out[T:] == 5.0).all()
    for got, was in zip((s["pool"], s["scales"]), before):
        if got is not None:
            keep = ~touched
            a, w = got.movedim(3, 1), was.movedim(3, 1)
            assert torch.equal(a[keep], w[keep])


def test_append_values_at_the_format_s_edges():
    """Zeros, the largest value of each exponent, saturation, infinities and NaN, by hand."""
    d = 64
    s = _append_case([8], [8], 1, 1, d, "e4m3", torch.float32, 1)
    rows = torch.zeros((8, 1, d), device="cuda")
    rows[1, 0, 0] = 448.0                      # e = 0 exactly
    rows[2, 0, 0] = 448.0 * (1 + 2.0 ** -20)   # just above: e = 1
    rows[3, 0, :2] = torch.tensor([1e9, -1.0])
    rows[4, 0, :3] = torch.tensor([float("inf"), float("-inf"), 2.0 ** 7])
    rows[5, 0, :2] = torch.tensor([float("nan"), 1.0])
    rows[6, 0, 0] = 2.0 ** -24                 # the smallest value of the smallest scale
    rows[7, 0, 0] = 2.0 ** -26                 # below half of it: 0
    c = _cache(s)
    c.append(_chunk(c, s), rows, rows.clone(), s["status"])
    k = torch.zeros((8, 1, d), device="cuda")
    c.read(_chunk(c, s), k, None, s["status"])
    page = int(s["table"][0, 0])
    e = s["scales"][page, 0, 0, :8].int().cpu() - 127
    assert e.tolist() == [-15, 0, 1, 7, 7, -8, -15, -15]
    k = k[:, 0].cpu()
    assert k[1, 0] == 448.0 and k[2, 0] == 448.0 and k[3, 0] == 57344.0 and k[3, 1] == -1.0
    assert k[4, 0] == 57344.0 and k[4, 1] == -57344.0 and k[4, 2] == 128.0
    assert torch.isnan(k[5, 0]) and k[5, 1] == 1.0
    assert k[6, 0] == 2.0 ** -24 and k[7, 0] == 0.0 and (k[0] == 0).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_bad_chunks_are_reported_and_write_nothing(fmt):
    base = ch.make([3, 2], [40, 20], 4, 2, 64, fmt, seed=2)
    T = base["T"]
    c = _cache(base, rows=T + 8)
    from speculative_decoding_verify_ragged_gb300._abi import SDV_ERR_BAD_INPUT, SDV_ERR_PAGE_RANGE
    bad = [("row_offsets", [1, 3, 5], SDV_ERR_BAD_INPUT), ("row_offsets", [0, 4, 3], SDV_ERR_BAD_INPUT),
           ("row_offsets", [0, 3, T + 9], SDV_ERR_BAD_INPUT), ("row_offsets", [0, 5, 5], SDV_ERR_BAD_INPUT),
           ("lens", [-1, 20], SDV_ERR_BAD_INPUT), ("lens", [40, 16 * base["table"].shape[1] + 1], SDV_ERR_PAGE_RANGE)]
    for key, words, code in bad:
        s = dict(base)
        s[key] = torch.tensor(words, dtype=torch.int32, device="cuda")
        chunk = _chunk(c, s, rows=T, max_q=4)
        pool = s["pool"].clone()
        q, out = s["q"], torch.full_like(s["q"], 3.0)
        kv = torch.full((T, 2, 64), 3.0, device="cuda")
        for call in (lambda st: c.attention(chunk, q, out, st), lambda st: c.read(chunk, kv, kv.clone(), st),
                     lambda st: c.append(chunk, kv, kv, st)):
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            call(st)
            assert st.item() == code, (key, words)
        assert (out == 3.0).all() and (kv == 3.0).all()
        assert torch.equal(s["pool"].view(torch.int16 if fmt == "bf16" else torch.uint8),
                           pool.view(torch.int16 if fmt == "bf16" else torch.uint8))
    # the handle serves the next call as ever, and a failed call's status stops the ones behind it
    want, tol = ch.attention(base)
    _close(_attend(base, c), want, tol)
    st = torch.full((1,), 6, dtype=torch.int32, device="cuda")
    out = torch.full_like(base["q"], 3.0)
    c.attention(_chunk(c, base), base["q"], out, st)
    assert st.item() == 6 and (out == 3.0).all()
    _close(_attend(base, c), want, tol)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_page_ids_outside_the_pool(fmt):
    from speculative_decoding_verify_ragged_gb300._abi import SDV_ERR_PAGE_RANGE
    for q_lens, kv_lens in (([3, 2], [40, 900]), ([300, 2], [400, 900])):
        s = ch.make(q_lens, kv_lens, 4, 2, 64, fmt, seed=2)
        T = s["T"]
        c = _cache(s)
        good, tol = ch.attention(s)
        for wrong in (-1, s["pool"].shape[0], 1 << 30):
            t = dict(s, table=s["table"].clone())
            t["table"][0, (kv_lens[0] - 1) // 16] = wrong
            chunk = _chunk(c, t)
            kv = torch.full((T, 2, 64), 3.0, device="cuda")
            for call in (lambda st: c.attention(chunk, s["q"], torch.empty_like(s["q"]), st),
                         lambda st: c.read(chunk, kv.clone(), kv.clone(), st)):
                st = torch.zeros(1, dtype=torch.int32, device="cuda")
                call(st)
                assert st.item() == SDV_ERR_PAGE_RANGE
        _close(_attend(s, c), good, tol)


def test_refusals():
    from speculative_decoding_verify_ragged_gb300 import SdvError
    from speculative_decoding_verify_ragged_gb300.cache import PagedCache
    s = ch.make([3, 2], [40, 20], 4, 2, 64, "bf16", seed=2)
    c = _cache(s)
    ok = _chunk(c, s)
    out = torch.empty_like(s["q"])
    for kw in (dict(rows=-1), dict(max_q=-1), dict(window=-1)):
        with pytest.raises(SdvError):
            c.attention(_chunk(c, s, **kw), s["q"], out, s["status"])
    with pytest.raises(SdvError):                       # more sequences than the handle holds
        _cache(s, slots=1).attention(ok, s["q"], out, s["status"])
    with pytest.raises(SdvError):                       # more rows than the handle holds
        _cache(s, rows=3).attention(ok, s["q"], out, s["status"])
    with pytest.raises(SdvError):                       # rows that do not begin on 16 bytes
        flat = torch.empty(s["T"] * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")
        c.attention(ok, s["q"], flat[1:].view(s["T"], 4, 64), s["status"])
    for q in (s["q"].float(), s["q"][:3], s["q"][:, :2], s["q"].cpu(), s["q"].transpose(1, 2)):
        with pytest.raises(ValueError):
            c.attention(ok, q, out, s["status"])
    with pytest.raises(ValueError):
        _chunk(c, s, kv_lens=s["lens"].long())
    with pytest.raises(ValueError):
        _chunk(c, s, kv_scales=torch.zeros(3, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        _chunk(c, s, kv_pool=s["pool"][:, :, :, :8])
    kv = torch.zeros((s["T"], 2, 64), device="cuda")
    with pytest.raises(ValueError):
        c.append(ok, kv, kv.to(torch.bfloat16), s["status"])
    with pytest.raises(ValueError):
        c.append(ok, kv, kv, s["status"], q=s["q"].float())
    with pytest.raises(ValueError):
        c.read(ok, None, None, s["status"])
    for cfg in (dict(head_dim=96), dict(page_size=32), dict(n_q=3), dict(rope_theta=0.5), dict(rope_theta=-1.0)):
        with pytest.raises(SdvError):
            PagedCache({**dict(n_q=4, n_kv=2, head_dim=64), **cfg}, 8, 2)
    with pytest.raises(ValueError):
        PagedCache(dict(n_q=4, n_kv=2, head_dim=64, cache_format="fp8"), 8, 2)
    with pytest.raises(SdvError):
        PagedCache(dict(n_q=4, n_kv=2, head_dim=64), 8, 1025)
    assert s["status"].item() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_other_streams_and_graphs(fmt):
    """Two handles on two streams at once; a captured chunk replayed over lengths that move."""
    many = [ch.make([1, 3, 200], [900, 30, 700], 8, 2, 128, fmt, seed=i) for i in range(2)]
    want = [ch.attention(s) for s in many]
    caches = [_cache(s) for s in many]
    outs = [torch.zeros_like(s["q"]) for s in many]
    streams = [torch.cuda.Stream() for _ in many]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, c, o, st in zip(many, caches, outs, streams):
            c.attention(_chunk(c, s), s["q"], o, s["status"], stream=st)
    torch.cuda.synchronize()
    for o, (w, tol) in zip(outs, want):
        _close(o, w, tol)
    s, c = many[0], caches[0]
    chunk, out = _chunk(c, s), torch.zeros_like(s["q"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attention(chunk, s["q"], out, s["status"])
    for lens in ([900, 30, 700], [500, 7, 666], [33, 3, 200]):
        s["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        t = dict(s, kv_lens=lens)
        graph.replay()
        torch.cuda.synchronize()
        w, tol = ch.attention(t)
        _close(out, w, tol)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_prompt_in_pieces_then_drafts(fmt):
    """A prompt appended and attended piece by piece, then a step of few rows: each piece's output is
    the definition's over the cache as it then stands, and the bf16 cache serves the verify step's
    own attention with the same result."""
    n_q, n_kv, d, theta = 8, 2, 128, 1e6
    pieces = [100, 1, 60, 4]
    total = sum(pieces)
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((total, n_q + 2 * n_kv, d), generator=g, device="cuda")
    s = ch.make([total], [total], n_q, n_kv, d, fmt, seed=1)
    c = _cache(s, theta)
    s["pool"].zero_()
    if fmt == "e4m3":
        s["scales"].fill_(127)
    done = 0
    for n in pieces:
        t = dict(s, q_lens=[n], kv_lens=[done + n], T=n,
                 row_offsets=torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                 lens=torch.tensor([done + n], dtype=torch.int32, device="cuda"),
                 q=torch.zeros((n, n_q, d), dtype=torch.bfloat16, device="cuda"))
        chunk = _chunk(c, t)
        rows = x[done:done + n]
        c.append(chunk, rows[:, n_q:n_q + n_kv], rows[:, n_q + n_kv:], t["status"], q=rows[:, :n_q], q_out=t["q"])
        out = torch.zeros_like(t["q"])
        c.attention(chunk, t["q"], out, t["status"])
        assert t["status"].item() == 0
        if fmt == "bf16":
            t["values"] = t["pool"].double()
        else:
            t["values"] = t["pool"].view(torch.float8_e4m3fn).double() * torch.exp2(t["scales"].double() - 127)[..., None]
        want, tol = ch.attention(t)
        _close(out, want, tol)
        done += n
    if fmt == "bf16":
        import workloads as wl
        from speculative_decoding_verify_ragged_gb300 import VerifyEngine
        from workloads import device as wd
        dims = dict(wl.TINY, n_q=n_q, n_kv=n_kv, head_dim=d)
        eng = VerifyEngine(wd.config(dims, 3), wd.weights_to_device(wl.make_weights(dims, 1)), max_rows=16, max_slots=4)
        i32 = dict(dtype=torch.int32, device="cuda")
        batch = dict(B=1, R=4, G=3, seq_lens=torch.tensor([total - 4], **i32), draft_lens=torch.tensor([3], **i32),
                     kv_pool=s["pool"], num_pool_pages=s["pool"].shape[0], page_table=s["table"],
                     num_pages=torch.tensor([-(-total // 16)], **i32))
        out32, st = torch.zeros((4, n_q * d), device="cuda"), torch.zeros(1, **i32)
        eng.attention(t["q"].float().contiguous(), batch, out32, st)
        assert st.item() == 0
        _close(out32.view(4, n_q, d), want, tol)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_next_tokens_beside_pieces_of_prompts(fmt, d):
    """A step that mixes single tokens with long pieces (both kernels take a share), one without the
    hint of it (one kernel takes all), and a batch of pieces whose last tiles are nearly empty."""
    for q, kv in (([1] * 10 + [200, 40, 0, 3], [700, 16, 33, 5, 900, 1, 250, 64, 129, 400, 1000, 41, 9, 800]),
                  ([1, 300, 2], [500, 650, 2]), ([65, 129, 33, 257], [65, 1000, 70, 257])):
        s = ch.make(q, kv, 8, 2, d, fmt, seed=sum(q))
        want, tol = ch.attention(s)
        _close(_attend(s), want, tol)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_one_handle_over_many_shapes(fmt):
    """Calls of unlike shapes one after another on one handle, nothing waited for between them: what one leaves
    in the workspace (parts, counters) is never seen by the next."""
    shapes = [([1], [3000]), ([300, 2], [900, 40]), ([1] * 40, list(range(1, 4001, 100))), ([64], [9000]), ([1000], [1000]),
              ([3, 1], [20, 7000]), ([128, 16], [128, 2000])]
    cases = [ch.make(q, kv, 16, 4, 128, fmt, seed=i) for i, (q, kv) in enumerate(shapes)]
    c = _cache(cases[0], rows=1200, slots=64)
    chunks = [_chunk(c, s) for s in cases]
    first = []
    for s, k in zip(cases, chunks):
        out = torch.empty_like(s["q"])
        c.attention(k, s["q"], out, s["status"])
        torch.cuda.synchronize()
        want, tol = ch.attention(s)
        _close(out, want, tol)
        first.append(out)
    g = torch.Generator().manual_seed(1)
    order = [int(i) for _ in range(20) for i in torch.randperm(len(cases), generator=g)]
    outs = [torch.empty_like(cases[i]["q"]) for i in order]
    for i, out in zip(order, outs):
        c.attention(chunks[i], cases[i]["q"], out, cases[i]["status"])
    torch.cuda.synchronize()
    for i, out in zip(order, outs):
        assert cases[i]["status"].item() == 0 and torch.equal(out, first[i])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,kv_lens", [([4, 1], [300, 90]), ([150, 9], [700, 90])])
def test_rows_that_are_not_numbers_stay_alone(fmt, q_lens, kv_lens):
    """NaN and infinite queries give NaN in their own rows and heads and nothing elsewhere; keys that are
    NaN where no earlier row sees them change no earlier row."""
    s = ch.make(q_lens, kv_lens, 8, 2, 128, fmt, seed=4)
    want, tol = ch.attention(s)
    q = s["q"].clone()
    s["q"][1, 3] = float("nan")
    s["q"][2, 5, 7] = float("inf")
    out = torch.empty_like(q)
    c = _cache(s)
    c.attention(_chunk(c, s), s["q"], out, s["status"])
    assert s["status"].item() == 0
    odd = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    odd[1, 3] = odd[2, 5] = True
    assert torch.isnan(out[odd]).all()
    _close(out[~odd], want[~odd], tol[~odd])
    # the newest key of sequence 0 is a NaN: the rows before the newest are as they were
    s["q"].copy_(q)
    at = kv_lens[0] - 1
    page = int(s["table"][0, at // 16])
    if fmt == "bf16":
        s["pool"][page, :, 0, at % 16] = float("nan")
    else:
        s["pool"][page, :, 0, at % 16] = 0x7F
    c.attention(_chunk(c, s), s["q"], out, s["status"])
    keep = torch.ones(s["T"], dtype=torch.bool, device="cuda")
    keep[q_lens[0] - 1] = False
    assert torch.isnan(out[q_lens[0] - 1]).all()
    _close(out[keep], want[keep], tol[keep])


@pytest.mark.parametrize("q,kv", [(1, 600), (200, 700)])
@pytest.mark.parametrize("e", [-15, 7])
def test_attention_at_the_scales_ends(q, kv, e):
    """Keys and values under the smallest and the largest scale."""
    s = ch.make([q], [kv], 8, 2, 128, "e4m3", seed=8, tail=0.0)
    used = s["scales"] <= 134
    byte = torch.full_like(s["scales"], e + 127)
    shift = torch.exp2(e - (s["scales"].double() - 127))
    s["values"] = s["values"] * torch.where(used, shift, torch.ones_like(shift))[..., None]
    s["scales"] = torch.where(used, byte, s["scales"])
    s["q"] = (s["q"].float() * 2.0 ** (-6 - e)).to(torch.bfloat16)
    want, tol = ch.attention(s)
    out = _attend(s)
    # (tol's term for small weights is of a value of 448 at scale 2^0)
    _close(out, want, tol * max(1.0, 2.0 ** e))
