"""The paged key/value cache's operators: writing a chunk of new tokens into the
cache (rotary embedding, and in 8 bits where the cache holds 8 bits), attention
of that chunk over the cache, and reading the cache back.

Every sequence b of a batch has kv_lens[b] positions in the cache, the chunk's
own among them, and owns the rows row_offsets[b] .. row_offsets[b + 1) of the
chunk: its i-th row sits at position kv_lens[b] - q_len + i.  Rows at positions
below 0 are empty.  A page holds 16 positions of every key/value head, keys
then values: [pages, n_kv, 2, 16, head_dim].

The 8-bit cache holds e4m3 codes and one power-of-two scale 2^e per (position,
head, key or value): e is the smallest exponent in [-15, 7] with
max|x| <= 448 * 2^e, kept as the byte e + 127; larger values saturate.
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 16
E_MIN, E_MAX, CODE_MAX = -15, 7, 448.0
THETA = 1.0e6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, name=None, **kw):
    c = dict(op=op, n_q=32, n_kv=8, head_dim=128, cache="bf16", batch=1, q_min=1, q_max=1, kv_min=1, kv_max=1,
             window=0, io="bf16", rope=False, with_q=False, whole=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user's next token at a short context: the smallest call, all latency
        _case("attention", "decode_1_bf16", kv_min=517, kv_max=517),
        # a decode step of a full batch at unlike lengths over the 8-bit cache
        _case("attention", "decode_64_e4m3", cache="e4m3", batch=64, kv_min=1000, kv_max=9000),
        # the verify rows of 128 sequences, 3 drafts each, at the bench's context of 2048
        _case("attention", "verify_128x4_bf16", batch=128, q_min=4, q_max=4, kv_min=2048, kv_max=2056),
        # one step of a continuous batch: next tokens and drafts beside pieces of prompts
        _case("attention", "mixed_24_e4m3", cache="e4m3", batch=24, q_min=1, q_max=515, kv_min=600, kv_max=6000),
        # fresh prompts of unlike lengths, as many key heads as query heads, a sliding window
        _case("attention", "prompts_5_window_bf16", n_q=16, n_kv=16, head_dim=64, batch=5, q_min=37, q_max=2500,
              window=700, whole=True),
        # a piece of a long document over what is cached already
        _case("attention", "prefill_2048_bf16", q_min=2048, q_max=2048, kv_min=32749, kv_max=32749),
        # the same over the 8-bit cache
        _case("attention", "prefill_1024_e4m3", cache="e4m3", q_min=1024, q_max=1024, kv_min=16411, kv_max=16411),
        # a decode step's new keys and values, rotated and quantised, with the step's queries
        _case("append", "append_64_e4m3", cache="e4m3", batch=64, kv_min=300, kv_max=9000, io="fp32", rope=True,
              with_q=True),
        # a long prompt piece's fused q, k, v rows at far positions into the 8-bit cache
        _case("append", "append_8192_e4m3", cache="e4m3", q_min=8192, q_max=8192, kv_min=121003, kv_max=121003,
              io="fp32", rope=True, with_q=True),
        # prompts' keys and values as they are into the 16-bit cache
        _case("append", "append_3_prompts_bf16", batch=3, q_min=500, q_max=3000, whole=True),
        # the newest positions of a few sequences, to be looked at in 32 bits
        _case("read", "read_4_e4m3", cache="e4m3", batch=4, q_min=60, q_max=130, kv_min=200, kv_max=900, io="fp32"),
        # a whole long sequence leaves for another machine
        _case("read", "read_32k_bf16", q_min=32749, q_max=32749, whole=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "append", "read"])
    d = rng.choice([64, 128])
    n_kv = rng.choice([1, 2, 4, 8])
    c = dict(n_q=n_kv * rng.choice([1, 2, 4, 5, 8]), n_kv=n_kv, head_dim=d, cache=rng.choice(["bf16", "e4m3"]))
    if op == "attention":
        kind = rng.choice(["decode", "mixed", "prefill", "prompts"])
        if kind == "decode":
            batch = _log(rng, 1, 128)
            hi = _log(rng, 16, min(9000, 400000 // batch))
            q = rng.choice([1, 1, 2, 5, 8])
            c.update(batch=batch, q_min=q, q_max=q, kv_min=max(1, hi // 3), kv_max=hi)
        elif kind == "mixed":
            batch = _log(rng, 2, 24)
            c.update(batch=batch, q_min=1, q_max=_log(rng, 8, 500), kv_min=_log(rng, 100, 600), kv_max=_log(rng, 700, 6000))
        elif kind == "prefill":
            q = _log(rng, 20, 2000)
            kv = q + _log(rng, 1, 30000)
            c.update(batch=1, q_min=q, q_max=q, kv_min=kv, kv_max=kv)
        else:
            c.update(batch=_log(rng, 1, 6), q_min=_log(rng, 1, 40), q_max=_log(rng, 50, 2500), whole=True)
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 3000)])
    else:
        batch = _log(rng, 1, 64)
        q_max = _log(rng, 1, 8000 // batch)
        c.update(batch=batch, q_min=max(1, q_max // 3), q_max=q_max, kv_min=1, kv_max=_log(rng, 1, 40000),
                 io=rng.choice(["bf16", "fp32"]))
        if op == "append":
            c.update(rope=rng.choice([True, False]), with_q=rng.choice([True, False]))
    return _case(op, **c)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lens(case):
    """(rows, cached positions) of each sequence: the case's ranges, spread by a fixed rule."""
    q, kv = [], []
    for b in range(case["batch"]):
        u = (b * 0.6180339887) % 1.0
        w = (b * 0.7548776662 + 0.37) % 1.0
        if case["batch"] > 4 and case["q_min"] == 1 and case["q_max"] > 16:
            u = u * 4 - 3 if u > 0.75 else 0.0        # a mixed step: three of four sequences bring one token
        n = int(round(case["q_min"] + (case["q_max"] - case["q_min"]) * u))
        if case["batch"] == 1:
            n = case["q_max"]
        m = int(round(case["kv_min"] + (case["kv_max"] - case["kv_min"]) * w))
        if case["batch"] == 1:
            m = case["kv_max"]
        q.append(n)
        kv.append(n if case["whole"] else max(m, n))
    return q, kv


def _quantise(x):
    """Codes (as float8 e4m3) and exponents (int32) of rows x [..., d] in fp32."""
    a = x.abs()
    a = torch.where(a.isnan(), torch.zeros_like(a), a).amax(-1).clamp(max=CODE_MAX * 2.0 ** E_MAX)
    m, e = torch.frexp(a / CODE_MAX)                  # a / 448 = m 2^e with m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e).clamp(E_MIN, E_MAX)
    e = torch.where(a > 0, e, torch.full_like(e, E_MIN)).to(torch.int32)
    e = torch.where((a > CODE_MAX * torch.exp2(e.float())) & (e < E_MAX), e + 1, e)
    y = (x * torch.exp2(-e.float())[..., None]).clamp(-CODE_MAX, CODE_MAX)
    return y.to(torch.float8_e4m3fn), e


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    n_q, n_kv, d = case["n_q"], case["n_kv"], case["head_dim"]
    q_lens, kv_lens = _lens(case)
    B, T = case["batch"], sum(q_lens)
    i32 = dict(dtype=torch.int32, device=dev)
    offsets = [0]
    for n in q_lens:
        offsets.append(offsets[-1] + n)
    # pages: each sequence's own, in a shuffled pool; operators that touch only the
    # chunk's rows get pages for those, the blocks before them are not there (-1)
    blocks = [-(-n // PAGE) for n in kv_lens]
    first = [0 if case["op"] == "attention" else (kv_lens[b] - q_lens[b]) // PAGE for b in range(B)]
    used = sum(blocks[b] - first[b] for b in range(B))
    pool_pages = used + 3
    perm = torch.randperm(pool_pages, generator=g, device=dev)[:used].to(torch.int32)
    table = torch.full((B, max(blocks)), -1, **i32)
    at = 0
    for b in range(B):
        n = blocks[b] - first[b]
        table[b, first[b]:blocks[b]] = perm[at:at + n]
        at += n
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    # keys have a few strong channels, the same for every position of a head
    channel = 1.0 + 3.0 * (torch.rand((n_kv, 1, d), generator=g, device=dev) > 0.95).float()
    pool = torch.empty((pool_pages, n_kv, 2, PAGE, d), dtype=torch.bfloat16 if case["cache"] == "bf16" else torch.uint8,
                       device=dev)
    scales = torch.full((pool_pages, n_kv, 2, PAGE), 127, dtype=torch.uint8, device=dev) if case["cache"] == "e4m3" else None
    step = max(1, (1 << 26) // (n_kv * 2 * PAGE * d))
    for p0 in range(0, pool_pages, step):
        x = rnd(min(step, pool_pages - p0), n_kv, 2, PAGE, d)
        x[:, :, 0] *= channel
        if case["cache"] == "bf16":
            pool[p0:p0 + step] = x.to(torch.bfloat16)
        else:
            codes, e = _quantise(x)
            pool[p0:p0 + step] = codes.view(torch.uint8)
            scales[p0:p0 + step] = (e + 127).to(torch.uint8)
    s = dict(case=case, q_lens=q_lens, kv_lens=kv_lens, T=T, pool=pool, scales=scales, table=table,
             row_offsets=torch.tensor(offsets, **i32), lens=torch.tensor(kv_lens, **i32),
             seq=torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(q_lens, device=dev)),
             status=torch.zeros(1, **i32))
    io = torch.bfloat16 if case["io"] == "bf16" else torch.float32
    if case["op"] == "attention":
        if case["cache"] == "bf16":                    # what lies behind a sequence's end is anything
            ends = torch.tensor([b for b in range(B) if kv_lens[b] % PAGE], device=dev, dtype=torch.long)
            for b in ends.tolist():
                pool[table[b, blocks[b] - 1].long(), :, :, kv_lens[b] % PAGE:] = float("nan")
        s["q"] = (2.0 * rnd(T, n_q, d)).to(torch.bfloat16)
        s["out"] = torch.zeros_like(s["q"])
    elif case["op"] == "append":
        # the rows of one fused projection: query heads, key heads, value heads
        x = rnd(T, n_q + 2 * n_kv, d)
        x[:, n_q:n_q + n_kv] *= channel[:, 0]
        x = x.to(io)
        s["q"], s["k"], s["v"] = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
        s["q_out"] = torch.zeros((T, n_q, d), dtype=torch.bfloat16, device=dev) if case["with_q"] else None
    else:
        s["k_out"] = torch.zeros((T, n_kv, d), dtype=io, device=dev)
        s["v_out"] = torch.zeros((T, n_kv, d), dtype=io, device=dev)
    if own:
        from speculative_decoding_verify_ragged_gb300.cache import PagedCache
        s["cache"] = PagedCache(dict(n_q=n_q, n_kv=n_kv, head_dim=d, page_size=PAGE, cache_format=case["cache"],
                                     rope_theta=THETA if case["rope"] else 0.0), max_rows=T, max_slots=B)
        s["chunk"] = s["cache"].chunk(rows=T, max_q=max(q_lens), row_offsets=s["row_offsets"], kv_lens=s["lens"],
                                      page_table=table, kv_pool=pool, kv_scales=scales, window=case["window"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return dict(attention=_attention, append=_append, read=_read)[s["case"]["op"]](s)


def _run_own(s):
    op = s["case"]["op"]
    if op == "attention":
        s["cache"].attention(s["chunk"], s["q"], s["out"], s["status"])
        return s["out"]
    if op == "append":
        s["cache"].append(s["chunk"], s["k"], s["v"], s["status"], q=s["q"] if s["case"]["with_q"] else None,
                          q_out=s["q_out"])
        return _stored(s)
    s["cache"].read(s["chunk"], s["k_out"], s["v_out"], s["status"])
    return dict(k=s["k_out"], v=s["v_out"])


def _stored(s):
    """The cache as the values that its bytes stand for, and the rotated queries."""
    r = dict(pool=s["pool"]) if s["scales"] is None else dict(codes=s["pool"].view(torch.float8_e4m3fn),
                                                              scales=s["scales"].view(torch.float8_e8m0fnu))
    if s["case"]["with_q"]:
        r["q"] = s["q_out"]
    return r


def _values(s, pages):
    """The keys and values of pages [...] in fp32: [..., n_kv, 2, 16, d]."""
    x = s["pool"][pages]
    if s["scales"] is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * torch.exp2(s["scales"][pages].float() - 127.0)[..., None]


def _attention(s):
    """softmax(q k^T / sqrt(d)) v over the positions each row sees, in fp32, all sequences padded to the longest."""
    case = s["case"]
    n_q, n_kv, d, B = case["n_q"], case["n_kv"], case["head_dim"], case["batch"]
    Q, nb = max(s["q_lens"]), s["table"].shape[1]
    kv = _values(s, s["table"].clamp(min=0).long())                               # [B, nb, n_kv, 2, 16, d]
    kv = kv.permute(3, 0, 2, 1, 4, 5).reshape(2, B, n_kv, nb * PAGE, d)
    at = torch.arange(nb * PAGE, device=kv.device)
    there = (at < s["lens"][:, None])[:, None, :, None]                           # behind the end: anything
    k, v = torch.where(there, kv[0], 0.0), torch.where(there, kv[1], 0.0)
    row = torch.arange(Q, device=kv.device)
    q_len = s["row_offsets"][1:] - s["row_offsets"][:-1]
    idx = (s["row_offsets"][:-1, None] + row).clamp(max=s["T"] - 1).long()        # [B, Q]
    q = s["q"].float()[idx].reshape(B, Q, n_kv, n_q // n_kv, d).permute(0, 2, 3, 1, 4).reshape(B, n_kv, -1, d)
    z = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(B, n_kv, n_q // n_kv, Q, nb * PAGE)
    pos = (s["lens"] - q_len)[:, None] + row                                      # [B, Q]
    hide = at > pos[..., None]
    if case["window"]:
        hide |= at <= pos[..., None] - case["window"]
    z.masked_fill_(hide[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, n_kv, -1, nb * PAGE) @ v).view(B, n_kv, n_q // n_kv, Q, d) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Q, n_q, d)
    s["out"][:] = o[row < q_len[:, None]].to(torch.bfloat16)
    return s["out"]


def _places(s):
    """(row indices, pages, slots) of the chunk's rows that have a position."""
    q_len = s["row_offsets"][1:] - s["row_offsets"][:-1]
    rows = torch.arange(s["T"], device=s["pool"].device)
    pos = (s["lens"] - q_len)[s["seq"]] + rows - s["row_offsets"][:-1][s["seq"]]
    rows = rows[pos >= 0]
    p = pos[rows].long()
    return rows, p, s["table"][s["seq"][rows], p // PAGE].long(), p % PAGE


def _rotate(x, pos, d):
    """Rotate-half rotary embedding of x [rows, heads, d] at positions pos; the angles in 64 bits."""
    f = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d)
    a = pos.double()[:, None] * f
    c, n = a.cos().float()[:, None], a.sin().float()[:, None]
    lo, hi = x[..., :d // 2].float(), x[..., d // 2:].float()
    return torch.cat([lo * c - hi * n, hi * c + lo * n], -1)


def _append(s):
    case = s["case"]
    d = case["head_dim"]
    rows, pos, page, slot = _places(s)
    k, v = s["k"][rows].float(), s["v"][rows].float()
    if case["rope"]:
        k = _rotate(k, pos, d)
    for which, x in ((0, k), (1, v)):
        if s["scales"] is None:
            s["pool"][page, :, which, slot] = x.to(torch.bfloat16)
        else:
            codes, e = _quantise(x)
            s["pool"][page, :, which, slot] = codes.view(torch.uint8)
            s["scales"][page, :, which, slot] = (e + 127).to(torch.uint8)
    if case["with_q"]:
        q = s["q"][rows]
        s["q_out"][rows] = (_rotate(q, pos, d) if case["rope"] else q).to(torch.bfloat16)
    return _stored(s)


def _read(s):
    rows, _, page, slot = _places(s)
    for which, out in ((0, s["k_out"]), (1, s["v_out"])):
        x = s["pool"][page, :, which, slot]
        if s["scales"] is not None:
            x = x.view(torch.float8_e4m3fn).float() * torch.exp2(s["scales"][page, :, which, slot].float() - 127.0)[..., None]
        out[rows] = x.to(out.dtype)
    return dict(k=s["k_out"], v=s["v_out"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    n_q, n_kv, d, w = case["n_q"], case["n_kv"], case["head_dim"], case["window"]
    q_lens, kv_lens = _lens(case)
    T = sum(q_lens)
    place = n_kv * 2 * (2 * d if case["cache"] == "bf16" else d + 1)               # one cached position
    io = 2 if case["io"] == "bf16" else 4
    if case["op"] == "read":
        return dict(bytes=T * (place + n_kv * 2 * d * io), flops=0)
    if case["op"] == "append":
        heads = n_kv * 2 + (n_q if case["with_q"] else 0)
        turned = n_kv + (n_q if case["with_q"] else 0) if case["rope"] else 0
        return dict(bytes=T * (place + heads * d * io + (n_q * d * 2 if case["with_q"] else 0)), flops=T * turned * d * 3)
    pairs = seen = 0
    for n, m in zip(q_lens, kv_lens):
        lo, hi = m - n, m                                                          # positions of the rows
        if w:
            pairs += sum(min(w, p + 1) for p in range(lo, hi))
            seen += hi - max(0, lo - w + 1)
        else:
            pairs += (lo + 1 + hi) * n // 2
            seen += hi
    return dict(bytes=seen * place + 2 * T * n_q * d * 2, flops=4 * d * n_q * pairs)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _code64(x):
    """(nearest e4m3 value of each x / 2^e, the scale 2^e), by the grid's spacing; x fp64 [rows, heads, d]."""
    big = x.abs().amax(-1).clamp(max=CODE_MAX * 2.0 ** E_MAX)
    e = torch.full_like(big, float(E_MAX))
    for t in range(E_MAX - 1, E_MIN - 1, -1):
        e = torch.where(big <= CODE_MAX * 2.0 ** t, torch.full_like(e, float(t)), e)
    y = (x / (2.0 ** e)[..., None]).clamp(-CODE_MAX, CODE_MAX)
    binade = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    grid = 2.0 ** (binade - 3)
    return torch.round(y / grid) * grid, 2.0 ** e


def exact(case, seed):
    s = prepare(case, seed)
    n_q, n_kv, d = case["n_q"], case["n_kv"], case["head_dim"]
    G = n_q // n_kv
    off = 0
    pool = s["pool"].double() if s["scales"] is None else None
    if s["scales"] is not None:
        pool = s["pool"].view(torch.float8_e4m3fn).double() if case["op"] == "append" else (
            s["pool"].view(torch.float8_e4m3fn).double() * (2.0 ** (s["scales"].double() - 127))[..., None])
        scales = 2.0 ** (s["scales"].double() - 127)
    if case["op"] == "attention":
        out = torch.zeros((s["T"], n_q, d), dtype=torch.float64, device="cuda")
    elif case["op"] == "append":
        q_out = s["q_out"].double() if case["with_q"] else None
    else:
        outs = [torch.zeros((s["T"], n_kv, d), dtype=torch.float64, device="cuda") for _ in range(2)]
    for b, (n, m) in enumerate(zip(s["q_lens"], s["kv_lens"])):
        at = torch.arange(max(0, m - n) if case["op"] != "attention" else 0, m, device="cuda")
        page, slot = s["table"][b].long()[at // PAGE], at % PAGE
        skip = n - min(n, m)
        if case["op"] == "attention":
            p = torch.arange(m - n, m, device="cuda")
            see = at[None] <= p[:, None]
            if case["window"]:
                see &= at[None] > p[:, None] - case["window"]
            for h in range(n_kv):
                k, v = pool[page, h, 0, slot], pool[page, h, 1, slot]
                for j in range(h * G, h * G + G):
                    for r in range(0, n, 2048):
                        z = (s["q"][off + r:off + min(n, r + 2048), j].double() @ k.T) / math.sqrt(d)
                        z = z.masked_fill(~see[r:r + 2048], -math.inf)
                        z = torch.softmax(z, -1)
                        out[off + r:off + min(n, r + 2048), j] = torch.nan_to_num(z) @ v
        elif case["op"] == "append":
            rows = slice(off + skip, off + n)
            k, v, q = s["k"][rows].double(), s["v"][rows].double(), s["q"][rows].double()
            if case["rope"]:
                a = at.double()[:, None, None] * torch.exp(
                    -torch.arange(d // 2, device="cuda", dtype=torch.float64) * (2.0 / d) * math.log(THETA))
                turn = torch.polar(torch.ones_like(a), a)
                k, q = (torch.complex(x[..., :d // 2], x[..., d // 2:]) * turn for x in (k, q))
                k, q = (torch.cat([x.real, x.imag], -1) for x in (k, q))
            for which, x in ((0, k), (1, v)):
                if s["scales"] is None:
                    pool[page, :, which, slot] = x
                else:
                    pool[page, :, which, slot], scales[page, :, which, slot] = _code64(x)
            if case["with_q"]:
                q_out[rows] = q
        else:
            for which in range(2):
                outs[which][off + skip:off + n] = pool[page, :, which, slot]
        off += n
    if case["op"] == "attention":
        return out
    if case["op"] == "read":
        return dict(k=outs[0], v=outs[1])
    r = dict(pool=pool) if s["scales"] is None else dict(codes=pool, scales=scales)
    if case["with_q"]:
        r["q"] = q_out
    return r
