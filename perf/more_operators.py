"""The operators that serve a batch of unlike requests: block tables and slot
maps from request lengths, each request's low-rank adapter beside a shared
projection, and sampling under each request's own settings.

sample: of a row's logits z in order (value descending, index ascending) stay
the first top_k; of those the shortest run whose mass of exp(z / T) reaches
top_p of theirs; of those what has at least min_p of the largest's mass.  What
stays, divided by its sum, is the row's distribution; the token is the first
index whose running sum, in index order, is above u.  T = 0 takes the largest.

plan: a request of length n holds ceil(n / 16) pages.  Pages beyond that go
back to the free stack, request by request; then missing ones are popped,
request by request.  A request's new rows sit at its last positions.

adapters: out = base + scale_a (x A_a^T) B_a^T for the rows of each request,
a being the request's adapter (none: out = base).
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 16
VOCAB = 151936        # the bench's layer and LM head
HIDDEN, QKV, FFN = 4096, 6144, 12288


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _sample_case(name=None, **kw):
    c = dict(op="sample", rows=1, per=1, vocab=VOCAB, io="fp32", settings="mixed", tokens=True, probs=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _plan_case(name=None, **kw):
    c = dict(op="plan", batch=1, q_min=1, q_max=1, kv_min=1, kv_max=1, changing=0.0, max_len=0)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def _adapter_case(name=None, **kw):
    c = dict(op="adapters", batch=1, q_min=1, q_max=1, adapters=1, none=0.0, rank=16, k=HIDDEN, n=HIDDEN, x="bf16",
             y="fp32")
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user's next token: the smallest call
        _sample_case("sample_1_bf16", io="bf16", settings="usual"),
        # a decode step of 64 requests, each with settings of its own
        _sample_case("sample_64_mixed", rows=64),
        # the same for as many rows as 128 requests with 3 drafts bring, all under top-p alone
        _sample_case("sample_512_top_p", rows=512, per=4, settings="top_p"),
        # the target distributions that those rows' drafts are verified against
        _sample_case("distribution_512", rows=512, per=4, settings="mixed", tokens=False, probs=True),
        # a draft model's proposals and what they were proposed from: a small odd vocabulary, 16-bit logits
        _sample_case("draft_40_bf16", rows=40, vocab=20011, io="bf16", settings="warm", probs=True),
        # one request's next token
        _plan_case("plan_1", kv_min=517, kv_max=518, max_len=1024),
        # a step of a continuous batch: next tokens beside pieces of prompts, some requests end, others begin
        _plan_case("plan_64", batch=64, q_max=300, kv_min=300, kv_max=9000, changing=0.2, max_len=16384),
        # the largest batch, a quarter of it prompts
        _plan_case("plan_1024", batch=1024, q_max=120, kv_min=60, kv_max=4000, changing=0.3, max_len=8192),
        # one request's row beside the output projection
        _adapter_case("adapters_1"),
        # a decode step of 64 requests with an adapter each, beside the fused QKV projection
        _adapter_case("adapters_64", batch=64, adapters=64, n=QKV),
        # a mixed step, a third of the requests without an adapter, 16-bit values beside the gate projection
        _adapter_case("adapters_24_mixed", batch=24, q_max=300, adapters=7, none=0.34, rank=32, n=FFN, y="bf16"),
        # prompts of four requests, wide adapters
        _adapter_case("adapters_4_prompts", batch=4, q_min=300, q_max=777, adapters=3, rank=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "plan", "adapters", "adapters"])
    if op == "sample":
        vocab = _log(rng, 300, 200000)
        per = rng.choice([1, 1, 2, 4, 9])
        rows = per * _log(rng, 1, max(1, min(512, 512 * VOCAB // vocab) // per))
        tokens, probs = rng.choice([(True, False), (True, False), (False, True), (True, True)])
        return _sample_case(rows=rows, per=per, vocab=vocab, io=rng.choice(["fp32", "bf16"]), tokens=tokens, probs=probs,
                            settings=rng.choice(["usual", "mixed", "top_p", "warm", "top_k", "all", "greedy"]))
    if op == "plan":
        batch = _log(rng, 1, 1024)
        kv = _log(rng, 2, 9000)
        return _plan_case(batch=batch, q_max=_log(rng, 1, max(2, min(2000, 16000 // batch))), kv_min=max(1, kv // 5), kv_max=kv,
                          changing=round(rng.uniform(0, 0.5), 3), max_len=kv + 2000)
    batch = _log(rng, 1, 128)
    q = _log(rng, 1, max(1, 2000 // batch))
    n = rng.choice([_log(rng, 64, 12288) // 8 * 8, HIDDEN, QKV])
    return _adapter_case(batch=batch, q_min=rng.choice([1, q]), q_max=q, adapters=_log(rng, 1, 64), none=rng.choice([0.0, 0.0, 0.3]),
                         rank=rng.choice([8, 16, 16, 24, 32, 64]), k=rng.choice([_log(rng, 64, 12288) // 8 * 8, HIDDEN]), n=n,
                         x=rng.choice(["bf16", "bf16", "fp32"]), y=rng.choice(["fp32", "bf16"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

# (temperature, top_k, top_p, min_p); 0, 1 and 0 turn the last three off
USUAL = [(0.7, 50, 0.95, 0.0)]
MIXED = [(0.7, 50, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (0.0, 0, 1.0, 0.0), (0.8, 0, 1.0, 0.05), (1.3, 200, 0.98, 0.02),
         (1.0, 0, 1.0, 0.0), (0.6, 20, 1.0, 0.0), (1.1, 1000, 0.999, 0.001)]
SETTINGS = dict(usual=USUAL, mixed=MIXED, top_p=[(0.8, 0, 0.95, 0.0), (1.0, 0, 0.9, 0.0)], warm=[(1.5, 0, 0.97, 0.01), (2.0, 0, 1.0, 0.02)],
                top_k=[(1.0, 40, 1.0, 0.0), (0.9, 5, 1.0, 0.0)], all=[(1.0, 0, 1.0, 0.0)], greedy=[(0.0, 0, 1.0, 0.0)])


def _spread(batch, lo, hi, step, phase, mixed=False):
    """`batch` whole numbers between lo and hi by a fixed rule; mixed: three of four are lo."""
    out = []
    for b in range(batch):
        u = (b * step + phase) % 1.0
        if mixed:
            u = u * 4 - 3 if u > 0.75 else 0.0
        out.append(int(round(lo + (hi - lo) * u)) if batch > 1 else hi)
    return out


def _rows_of(case):
    return _spread(case["batch"], case["q_min"], case["q_max"], 0.6180339887, 0.0,
                   mixed=case["q_min"] == 1 and case["q_max"] > 16 and case["batch"] > 4)


def _steps(case):
    """(new rows, lengths) of two steps that follow each other again and again: some requests end in the second (length 0), the
    others get the first's rows once more."""
    q1 = _rows_of(case)
    kv = [max(a, b) for a, b in zip(_spread(case["batch"], case["kv_min"], case["kv_max"], 0.7548776662, 0.37), q1)]
    q2, kv2 = [], []
    for b, (n, m) in enumerate(zip(q1, kv)):
        gone = (b * 0.5698402910 + 0.11) % 1.0 < case["changing"]
        q2.append(0 if gone else n)
        kv2.append(0 if gone else min(m + n, case["max_len"]))
    return (q1, kv), (q2, kv2)


def _offsets(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return dict(sample=_prepare_sample, plan=_prepare_plan, adapters=_prepare_adapters)[case["op"]](case, g)


def _prepare_sample(case, g):
    dev, rows, V = "cuda", case["rows"], case["vocab"]
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    io = torch.bfloat16 if case["io"] == "bf16" else torch.float32
    z = torch.empty((rows, V), dtype=io, device=dev)
    n = min(V, 400)
    for r0 in range(0, rows, 64):
        # a wide bulk, and a few hundred likelier tokens up to a dozen nats above it
        x = 2.2 * rnd(min(64, rows - r0), V)
        at = torch.randint(0, V, (x.shape[0], n), generator=g, device=dev)
        x.scatter_add_(1, at, 15.0 * torch.rand(at.shape, generator=g, device=dev) ** 3)
        x += 2.0 * rnd(x.shape[0], 1)
        z[r0:r0 + 64] = x.to(io)
    z[:, V - V // 200:] = -math.inf                 # entries that pad the table
    z[::3, 7::501] = -math.inf                      # words that a request bans
    requests = -(-rows // case["per"])
    settings = [SETTINGS[case["settings"]][i % len(SETTINGS[case["settings"]])] for i in range(requests)]
    t, k, p, m = zip(*settings)
    s = dict(case=case, logits=z, status=torch.zeros(1, dtype=torch.int32, device=dev),
             temperature=torch.tensor(t, device=dev), top_k=torch.tensor(k, dtype=torch.int32, device=dev),
             top_p=torch.tensor(p, device=dev), min_p=torch.tensor(m, device=dev),
             row_request=(torch.arange(rows, device=dev) // case["per"]).to(torch.int32),
             uniforms=torch.rand(rows, generator=g, device=dev),
             tokens=torch.zeros(rows, dtype=torch.int32, device=dev) if case["tokens"] else None,
             probs=torch.zeros((rows, V), dtype=torch.float32, device=dev) if case["probs"] else None)
    return s


def _prepare_plan(case, g):
    dev, B = "cuda", case["batch"]
    i32 = dict(dtype=torch.int32, device=dev)
    steps = _steps(case)
    width = max(1, -(-case["max_len"] // PAGE))
    T = max(1, max(sum(q) for q, _ in steps))
    need = max(sum(-(-n // PAGE) for n in kv) for _, kv in steps)
    pool = need + 5
    free = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    s = dict(case=case, T=T, pool=pool, width=width, turn=0, status=torch.zeros(1, **i32),
             steps=[(torch.tensor(q, **i32), torch.tensor(kv, **i32)) for q, kv in steps])
    # before the first step each request holds what it had without its new rows
    had = [-(-max(0, m - n) // PAGE) for n, m in zip(*steps[0])]
    table = torch.full((B, width), -1, **i32)
    top = pool
    for b, n in enumerate(had):
        table[b, :n] = free[top - n:top]
        top -= n
    if own:
        from speculative_decoding_verify_ragged_gb300.cache import Tables
        s["tables"] = Tables(max_slots=B, max_rows=T, max_pages_per_seq=width, num_pages=pool)
        t = s["tables"]
        t.page_table.copy_(table)
        t.page_counts.copy_(torch.tensor(had, **i32))
        t.free_pages.copy_(free)
        t.num_free.fill_(top)
        return s
    s.update(page_table=table, page_counts=torch.tensor(had, **i32), free_pages=free, num_free=torch.tensor([top], **i32),
             row_offsets=torch.zeros(B + 1, **i32), row_request=torch.zeros(T, **i32), positions=torch.zeros(T, **i32),
             slots=torch.zeros(T, dtype=torch.int64, device=dev), last_rows=torch.zeros(B, **i32))
    return s


def _prepare_adapters(case, g):
    dev, B = "cuda", case["batch"]
    counts = _rows_of(case)
    T, K, N, r, n = sum(counts), case["k"], case["n"], case["rank"], case["adapters"]
    rnd = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    ids = [-1 if (b * 0.4142135624 + 0.05) % 1.0 < case["none"] else b % n for b in range(B)]
    s = dict(case=case, T=T, x=rnd(T, K).to(torch.bfloat16 if case["x"] == "bf16" else torch.float32),
             a=(rnd(n, r, K) / math.sqrt(K)).to(torch.bfloat16), b=(0.3 * rnd(n, N, r) / math.sqrt(r)).to(torch.bfloat16),
             scales=0.5 + torch.rand(n, generator=g, device=dev),
             base=rnd(T, N).to(torch.bfloat16 if case["y"] == "bf16" else torch.float32),
             row_offsets=torch.tensor(_offsets(counts), dtype=torch.int32, device=dev),
             ids=torch.tensor(ids, dtype=torch.int32, device=dev), status=torch.zeros(1, dtype=torch.int32, device=dev))
    s["out"] = torch.zeros_like(s["base"])
    if own:
        from speculative_decoding_verify_ragged_gb300.adapter import Adapters
        s["adapters"] = Adapters(s["a"], s["b"], s["scales"], max_rows=T, max_slots=B)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return dict(sample=_sample, plan=_plan, adapters=_adapters)[s["case"]["op"]](s)


def _sample(s):
    if own:
        from speculative_decoding_verify_ragged_gb300.sample import sample
        sample(s["logits"], s["status"], uniforms=s["uniforms"] if s["case"]["tokens"] else None, tokens=s["tokens"], probs=s["probs"],
               temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], row_request=s["row_request"])
    else:
        _sample_plain(s)
    return {k: s[k] for k in ("tokens", "probs") if s[k] is not None}


def _sample_plain(s):
    """Everything in 64 bits: which token is the last to stay, and which one a draw falls on, hang on sums over the whole row."""
    req = s["row_request"].long()
    t, k, p, m = (s[n][req][:, None] for n in ("temperature", "top_k", "top_p", "min_p"))
    V = s["logits"].shape[1]
    v, at = s["logits"].double().sort(dim=1, descending=True, stable=True)
    rank = torch.arange(V, device=v.device)
    w = torch.where(v == v[:, :1], 0.0, (v - v[:, :1]) / torch.where(t == 0, 1.0, t.double())).exp_()
    keep = rank < torch.where(t == 0, 1, torch.where(k > 0, k, V))
    w = torch.where(keep, w, 0.0)
    cum = w.cumsum(1)
    before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1)
    keep &= (before < p.double() * cum[:, -1:]) | (p >= 1)
    keep &= w >= m.double()
    f = torch.zeros_like(v).scatter_(1, at, torch.where(keep, w, 0.0))
    cum = f.cumsum(1)
    if s["tokens"] is not None:
        u = s["uniforms"].double()[:, None] * cum[:, -1:]
        s["tokens"].copy_(torch.searchsorted(cum, u, right=True)[:, 0])
    if s["probs"] is not None:
        s["probs"].copy_(f / cum[:, -1:])


PLAN_OUT = ("row_offsets", "row_request", "positions", "slots", "last_rows", "page_table", "page_counts", "free_pages", "num_free")


def _plan(s):
    new_rows, lens = s["steps"][s["turn"]]
    s["turn"] ^= 1
    if own:
        t = s["tables"]
        t.plan(new_rows, lens, s["status"])
        return {k: getattr(t, k) for k in PLAN_OUT}
    _plan_plain(s, new_rows, lens)
    return {k: s[k] for k in PLAN_OUT}


def _plan_plain(s, new_rows, lens):
    table, counts, free, B, T = s["page_table"], s["page_counts"], s["free_pages"], s["case"]["batch"], s["T"]
    dev, W, P = table.device, s["width"], s["pool"]
    need = (lens + PAGE - 1) // PAGE
    block = torch.arange(W, device=dev)
    back = ((block >= need[:, None]) & (block < counts[:, None])).reshape(-1)      # entries whose pages go back
    want = ((block >= counts[:, None]) & (block < need[:, None])).reshape(-1)      # entries that need a page
    flat = table.reshape(-1)
    top = s["num_free"].long()
    stack = torch.cat([free, free[:1]])                                            # one place more, for nothing
    stack[torch.where(back, top + back.long().cumsum(0) - 1, P)] = flat
    top = top + back.sum()
    popped = stack[torch.where(want, top - want.long().cumsum(0), P)]
    table.copy_(torch.where(want, popped, torch.where(back, -1, flat)).view(B, W))
    free.copy_(stack[:P])
    s["num_free"].copy_(top - want.sum())
    counts.copy_(need)
    ends = new_rows.cumsum(0)
    s["row_offsets"][1:] = ends
    s["last_rows"].copy_(torch.where(new_rows > 0, ends - 1, -1))
    row = torch.arange(T, device=dev)
    b = torch.searchsorted(ends, row, right=True)
    there = b < B
    b = b.clamp(max=B - 1)
    pos = lens[b] - ends[b] + row
    page = table.reshape(-1)[b * W + pos.clamp(min=0) // PAGE].long()
    s["row_request"].copy_(torch.where(there, b, -1))
    s["positions"].copy_(torch.where(there, pos, -1))
    s["slots"].copy_(torch.where(there & (pos >= 0), page * PAGE + pos % PAGE, -1))


def _adapters(s):
    if own:
        s["adapters"].apply(s["x"], s["base"], s["out"], s["row_offsets"], s["ids"], s["status"])
        return s["out"]
    n, r, K = s["a"].shape
    b = torch.searchsorted(s["row_offsets"][1:].contiguous(), torch.arange(s["T"], device="cuda"), right=True)
    mine = s["ids"][b][:, None] == torch.arange(n, device="cuda")                  # [T, n]: the row's adapter
    v = s["x"].float() @ s["a"].float().reshape(n * r, K).T                        # every adapter's, others' set to 0
    v = torch.where(mine[..., None], v.view(-1, n, r) * s["scales"][:, None], 0.0).view(-1, n * r)
    s["out"].copy_(s["base"].float() + v @ s["b"].float().transpose(1, 2).reshape(n * r, -1))
    return s["out"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "sample":
        values = case["rows"] * case["vocab"]
        return dict(bytes=values * ((2 if case["io"] == "bf16" else 4) + (4 if case["probs"] else 0)) + case["rows"] * 12, flops=4 * values)
    if case["op"] == "plan":
        steps = _steps(case)
        B, T = case["batch"], max(sum(q) for q, _ in steps)
        moved = sum(abs(-(-x // PAGE) + (-y // PAGE)) for x, y in zip(steps[0][1], steps[1][1]))
        return dict(bytes=B * 5 * 4 + T * 16 + sum(steps[0][0]) // PAGE * 4 + moved * 8, flops=0)
    counts = _rows_of(case)
    T, K, N, r, n = sum(counts), case["k"], case["n"], case["rank"], case["adapters"]
    ids = [-1 if (b * 0.4142135624 + 0.05) % 1.0 < case["none"] else b % n for b in range(case["batch"])]
    used, rows = len(set(i for i in ids if i >= 0)), sum(c for c, i in zip(counts, ids) if i >= 0)
    xb, yb = 2 if case["x"] == "bf16" else 4, 2 if case["y"] == "bf16" else 4
    return dict(bytes=used * r * (K + N) * 2 + rows * K * xb + 2 * T * N * yb, flops=2 * rows * r * (K + N))


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return dict(sample=_exact_sample, plan=_exact_plan, adapters=_exact_adapters)[case["op"]](s)


def _exact_sample(s):
    case, V = s["case"], s["case"]["vocab"]
    tokens = torch.zeros(case["rows"], dtype=torch.int64, device="cuda")
    probs = torch.zeros((case["rows"], V), dtype=torch.float64, device="cuda") if case["probs"] else None
    settings = [x.tolist() for x in (s["temperature"].double(), s["top_k"], s["top_p"].double(), s["min_p"].double())]
    for r, u in enumerate(s["uniforms"].double().tolist()):
        t, k, p, m = (x[r // case["per"]] for x in settings)
        z = s["logits"][r].double()
        order = torch.sort(-z, stable=True).indices
        if t == 0.0:
            kept, prob = order[:1], torch.ones(1, dtype=torch.float64, device="cuda")
        else:
            kept = order[:k] if k else order
            q = torch.softmax(z[kept] / t, 0)
            if p < 1.0:
                n = int((q.cumsum(0) < p).sum().item()) + 1
                kept, q = kept[:n], q[:n]
            stay = q >= m * q[0]
            kept, prob = kept[stay], q[stay] / q[stay].sum()
        if probs is not None:
            probs[r, kept] = prob
        by = torch.sort(kept).indices
        reach = prob[by].cumsum(0)
        tokens[r] = kept[by][min(int((reach <= u * reach[-1]).sum().item()), by.numel() - 1)]
    out = dict(tokens=tokens) if case["tokens"] else {}
    return dict(out, probs=probs) if case["probs"] else out


def _exact_plan(s):
    case = s["case"]
    new_rows, lens = (x.tolist() for x in s["steps"][0])
    table, counts, free = s["page_table"].tolist(), s["page_counts"].tolist(), s["free_pages"].tolist()
    stack, spare = free[:s["num_free"].item()], free
    for b, n in enumerate(lens):
        keep = -(-n // PAGE)
        for j in range(keep, counts[b]):
            stack.append(table[b][j])
            spare[len(stack) - 1] = table[b][j]
            table[b][j] = -1
    for b, n in enumerate(lens):
        for j in range(counts[b], -(-n // PAGE)):
            table[b][j] = stack.pop()
        counts[b] = -(-n // PAGE)
    offsets, request, positions, slots = _offsets(new_rows), [-1] * s["T"], [-1] * s["T"], [-1] * s["T"]
    for b in range(case["batch"]):
        for i in range(new_rows[b]):
            r, pos = offsets[b] + i, lens[b] - new_rows[b] + i
            request[r], positions[r] = b, pos
            slots[r] = table[b][pos // PAGE] * PAGE + pos % PAGE if pos >= 0 else -1
    last = [offsets[b + 1] - 1 if new_rows[b] else -1 for b in range(case["batch"])]
    i64 = lambda x: torch.tensor(x, dtype=torch.int64)  # noqa: E731
    return dict(row_offsets=i64(offsets), row_request=i64(request), positions=i64(positions), slots=i64(slots), last_rows=i64(last),
                page_table=i64(table), page_counts=i64(counts), free_pages=i64(spare), num_free=i64([len(stack)]))


def _exact_adapters(s):
    out, at = s["base"].double(), s["row_offsets"].tolist()
    for b, i in enumerate(s["ids"].tolist()):
        if i >= 0:
            rows = slice(at[b], at[b + 1])
            v = s["x"][rows].double() @ s["a"][i].double().T
            out[rows] += s["scales"][i].double() * (v @ s["b"][i].double().T)
    return out
