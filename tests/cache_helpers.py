"""Inputs of the paged cache's operators and their definition in 64 bits, for tests."""
import math

import torch

PAGE = 16
BF16_HALF = 2.0 ** -8     # half a step, relative
FP16_HALF = 2.0 ** -11
E4M3_HALF = 2.0 ** -4


def make(q_lens, kv_lens, n_q, n_kv, d, fmt, seed=0, spare=3, window=0, dev="cuda", tail=float("nan")):
    """A filled cache with shuffled pages, the chunk's queries and the cache's values in 64 bits.

    What lies behind each sequence's end in its last page is `tail` (codes 0x7F, a
    NaN, in an e4m3 cache, with a scale byte of 255)."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, T = len(q_lens), sum(q_lens)
    blocks = [-(-n // PAGE) for n in kv_lens]
    pool_pages = sum(blocks) + spare
    perm = torch.randperm(pool_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(max(blocks), 1) + 1), -1, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
    x = torch.randn((pool_pages, n_kv, 2, PAGE, d), generator=g, device=dev)
    x[:, :, 0, :, ::17] *= 3.0
    if fmt == "bf16":
        pool, scales = x.to(torch.bfloat16), None
        values = pool.double()
    else:
        e = torch.randint(-9, -4, (pool_pages, n_kv, 2, PAGE), generator=g, device=dev)
        codes = (x * torch.exp2(-e.float())[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        pool, scales = codes.view(torch.uint8), (e + 127).to(torch.uint8)
        values = codes.double() * torch.exp2(e.double())[..., None]
    for b in range(B):
        if kv_lens[b] % PAGE:
            pg = int(table[b, blocks[b] - 1])
            if fmt == "bf16":
                pool[pg, :, :, kv_lens[b] % PAGE:] = tail
            else:
                pool[pg, :, :, kv_lens[b] % PAGE:] = 0x7F
                scales[pg, :, :, kv_lens[b] % PAGE:] = 255
    off = [0]
    for n in q_lens:
        off.append(off[-1] + n)
    i32 = dict(dtype=torch.int32, device=dev)
    return dict(q_lens=list(q_lens), kv_lens=list(kv_lens), n_q=n_q, n_kv=n_kv, d=d, fmt=fmt, T=T, window=window,
                pool=pool, scales=scales, values=values, table=table, row_offsets=torch.tensor(off, **i32),
                lens=torch.tensor(kv_lens, **i32), status=torch.zeros(1, **i32),
                q=(2.0 * torch.randn((T, n_q, d), generator=g, device=dev)).to(torch.bfloat16))


def positions(s, b):
    return torch.arange(s["kv_lens"][b] - s["q_lens"][b], s["kv_lens"][b], device=s["table"].device)


def cached(s, b, h):
    """Keys and values of sequence b's head h, in 64 bits."""
    at = torch.arange(s["kv_lens"][b], device=s["table"].device)
    page = s["table"][b].long()[at // PAGE]
    return s["values"][page, h, 0, at % PAGE], s["values"][page, h, 1, at % PAGE]


def attention(s):
    """(out, how far each value of the kernel's may be off) from the definition, in 64 bits.

    The bound: the weights enter the second product in 16 bits (half a step each,
    relative to sum p |v|), the output is rounded to bf16, and a score's d products
    are summed in 32 bits (at most d 2^-23 of the sum of their magnitudes, which
    moves a weight by that much, and the sum below it too)."""
    n_q, n_kv, d = s["n_q"], s["n_kv"], s["d"]
    G = n_q // n_kv
    out = torch.zeros((s["T"], n_q, d), dtype=torch.float64, device=s["q"].device)
    tol = torch.zeros_like(out)
    r0 = 0
    half = BF16_HALF if s["fmt"] == "bf16" else FP16_HALF
    for b, n in enumerate(s["q_lens"]):
        pos = positions(s, b)
        at = torch.arange(s["kv_lens"][b], device=out.device)
        see = at[None] <= pos[:, None]
        if s["window"]:
            see &= at[None] > pos[:, None] - s["window"]
        for j in range(n_q):
            if n == 0 or s["kv_lens"][b] == 0:
                continue
            k, v = cached(s, b, j // G)
            q = s["q"][r0:r0 + n, j].double()
            z = (q @ k.T) / math.sqrt(d)
            z = z.masked_fill(~see, -math.inf)
            p = torch.nan_to_num(torch.softmax(z, -1))
            out[r0:r0 + n, j] = p @ v
            size = ((q.abs() @ k.abs().T) / math.sqrt(d)).masked_fill(~see, 0).amax(-1, keepdim=True)
            moved = 2 * (d * 2.0 ** -23 * size + 2.0 ** -20)
            tol[r0:r0 + n, j] = (p @ v.abs()) * (half + moved) + BF16_HALF * out[r0:r0 + n, j].abs()
            if s["fmt"] == "e4m3":
                # a weight below fp16's normal range is off by 2^-25 of the scale it carries
                # (at least 2^-7 of the largest code's value 448): 448 2^-25 2^-8 a key, against a sum >= 1
                tol[r0:r0 + n, j] += see.sum(-1, keepdim=True) * 448 * 2.0 ** -33
        r0 += n
    return out, tol + 1e-30


def exponent(amax):
    """The smallest e in [-15, 7] with amax <= 448 * 2^e, by trying each."""
    e = torch.full_like(amax, 7.0)
    for t in range(6, -16, -1):
        e = torch.where(amax <= 448.0 * 2.0 ** t, torch.full_like(e, float(t)), e)
    return e


def rotate(x, pos, theta, d):
    """Rotate-half rotary embedding of x [rows, heads, d] in 64 bits."""
    f = float(theta) ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d)
    a = pos.double()[:, None, None] * f
    lo, hi = x[..., :d // 2].double(), x[..., d // 2:].double()
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)
