"""What is measured of the attention operators: cases, inputs, plain forms, exact values.

Four operators over one paged key-value cache held in Q8_0 (int8 codes, one
fp16 scale per 32 values along the head), and over packed prompts:

* ``write``    new keys and values of a batch are quantised into the cache's
               pages and read back as fp32 (what the cache now stands for);
* ``read``     whole contexts are read back from the pages, packed;
* ``decode``   attention of one new token per sequence over the cache;
* ``prefill``  causal attention of packed prompts with grouped heads.

Every tensor is packed by tokens: sequence b has the rows
``cu[b] .. cu[b+1]-1``, which are its last ``cu[b+1]-cu[b]`` positions.
Lengths come from the case's own numbers, so ``work`` knows them.
"""
import math
import random

import torch

own = False

BLOCK = 32                      # values under one Q8_0 scale
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # the cache's part of one decode step: a token for each of 16 running requests, straight from fp32 projections
        dict(name="write_step", op="write", dtype="f32", batch=16, lo=1, hi=1, past=4000, kv_heads=8, dim=128, page=64, key=1),
        # a chunk of prompts admitted together, ragged, onto contexts of any length
        dict(name="write_chunk", op="write", dtype="f16", batch=6, lo=1, hi=2500, past=777, kv_heads=8, dim=128, page=16, key=2),
        # a short context fetched for a follow-up question
        dict(name="read_short", op="read", dtype="bf16", batch=3, lo=33, hi=700, kv_heads=40, dim=128, page=16, key=3),
        # long contexts fetched as the keys and values of the next prompt chunk
        dict(name="read_long", op="read", dtype="f16", batch=4, lo=9000, hi=32000, kv_heads=8, dim=128, page=128, key=4),
        # one user, a short conversation, every head with its own keys (hidden 5120 = 40 x 128): latency
        dict(name="decode_one", op="decode", dtype="f32", batch=1, lo=500, hi=500, heads=40, kv_heads=40, dim=128, page=64, key=5),
        # an ordinary serving batch of ragged lengths, grouped heads
        dict(name="decode_batch", op="decode", dtype="bf16", batch=24, lo=1, hi=6000, heads=40, kv_heads=8, dim=128, page=16, key=6),
        # one long document: few rows, so the length itself has to be shared out
        dict(name="decode_long", op="decode", dtype="f32", batch=1, lo=131072, hi=131072, heads=40, kv_heads=8, dim=128, page=64, key=7),
        # a full server: the largest step, 64 requests of up to 8192 tokens
        dict(name="decode_full", op="decode", dtype="f16", batch=64, lo=2048, hi=8192, heads=64, kv_heads=8, dim=128, page=128, key=8),
        # many short prompts at once, small heads: short ragged rows
        dict(name="prefill_short", op="prefill", dtype="f16", batch=32, lo=1, hi=190, past=0, heads=16, kv_heads=4, dim=64, key=9),
        # one prompt of the hidden-5120 stack's 2048 tokens, every head with its own keys
        dict(name="prefill_2048", op="prefill", dtype="f16", batch=1, lo=2048, hi=2048, past=0, heads=40, kv_heads=40, dim=128, key=10),
        # packed prompts of different lengths behind cached prefixes
        dict(name="prefill_packed", op="prefill", dtype="bf16", batch=5, lo=100, hi=2500, past=1000, heads=40, kv_heads=8, dim=128, key=11),
        # one long prompt
        dict(name="prefill_8192", op="prefill", dtype="bf16", batch=1, lo=8192, hi=8192, past=0, heads=40, kv_heads=8, dim=128, key=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["write", "read", "decode", "decode", "prefill", "prefill"])
        dim, group, kv = rng.choice([64, 128, 128]), rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16]), rng.choice([1, 2, 4, 5, 8, 10, 16, 40])
        c = dict(op=op, dtype=rng.choice(["f32", "f16", "bf16"]), batch=_log(rng, 1, 64), lo=1, kv_heads=kv, dim=dim, key=rng.randrange(1 << 30))
        if op == "prefill":
            c.update(dtype=rng.choice(["f16", "bf16"]), hi=_log(rng, 1, 8192), past=rng.choice([0, 0, 1, 100, 1500]), heads=kv * group)
        else:
            c.update(hi=_log(rng, 1, 131072 if op == "decode" else 32000), page=rng.choice([16, 32, 48, 64, 128, 256]))
            if op == "decode":
                c.update(heads=kv * group)
            if op == "write":
                c.update(past=rng.choice([0, 5, 300, 4000]))
        c["lo"] = rng.choice([1, max(1, c["hi"] // 2), c["hi"]])
        w, n, m = work(c), _lens(c), c["hi"] + c.get("past", 0)
        # no larger than the listed ones, the padded plain form's intermediate values among them
        pad = c["batch"] * m * (c["hi"] * c["heads"] if op == "prefill" else kv * dim)
        if w["bytes"] <= 700e6 and w["flops"] <= 0.6e12 and pad <= (2.6e9 if op == "prefill" else 4.5e8) and sum(n) <= 600000:
            return c


def _lens(c):
    """The new (write, prefill) or whole (read, decode) lengths of the case's sequences."""
    rng = random.Random(c["key"])
    n = [rng.randint(c["lo"], c["hi"]) for _ in range(c["batch"])]
    n[rng.randrange(len(n))] = c["hi"]
    return n


def _pasts(c):
    """Tokens that each sequence has in front of the new ones."""
    rng = random.Random(c["key"] + 1)
    return [rng.randint(0, c["past"]) if c.get("past") else 0 for _ in range(c["batch"])]


def work(c):
    n, past = _lens(c), _pasts(c)
    e = 4 if c["dtype"] == "f32" else 2
    kv, d = c["kv_heads"], c["dim"]
    held = 2 * kv * (d + 2 * (d // BLOCK))                     # bytes of one token's K and V in the cache
    if c["op"] == "write":                                     # rows read, quantised, and read back as fp32
        return {"bytes": sum(n) * (2 * kv * d * (e + 4) + 2 * held), "flops": sum(n) * 2 * kv * d * 4}
    if c["op"] == "read":
        return {"bytes": sum(n) * (held + 2 * kv * d * e), "flops": sum(n) * 2 * kv * d}
    h = c["heads"]
    if c["op"] == "decode":
        return {"bytes": sum(n) * held + 2 * c["batch"] * h * d * e, "flops": 4 * sum(n) * h * d}
    pairs = sum(a * p + a * (a + 1) // 2 for a, p in zip(n, past))
    keys = sum(a + p for a, p in zip(n, past))
    return {"bytes": e * d * (2 * sum(n) * h + 2 * keys * kv), "flops": 4 * pairs * h * d}


# ---------------------------------------------------------------------------
# inputs

def _cu(n):
    return torch.tensor([0] + n, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def _rows(gen, rows, heads, dim, dtype, outliers):
    """Projected rows: N(0, 1), for keys a few channels four times as large, as keys have them."""
    x = torch.randn((rows, heads, dim), generator=gen, device="cuda", dtype=torch.float32)
    if outliers:
        x[..., torch.randperm(dim, generator=gen, device="cuda")[: max(1, dim // 32)]] *= 4
    return x.to(dtype)


def _filled(gen, shape, outliers):
    """Pages that hold quantised rows."""
    codes = torch.empty(shape, dtype=torch.int8, device="cuda")
    scales = torch.empty(shape[:-1] + (shape[-1] // BLOCK,), dtype=torch.float16, device="cuda")
    step = max(1, (1 << 27) // math.prod(shape[1:]))
    for i in range(0, shape[0], step):                         # by parts: the fp32 rows are much larger than the pages
        part = (min(step, shape[0] - i),) + shape[1:]
        x = torch.randn(part, generator=gen, device="cuda")
        if outliers:
            x[..., : max(1, shape[-1] // 32)] *= 4
        q, d = _quantise(x)
        codes[i:i + step], scales[i:i + step] = q, d
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, past = _lens(case), _pasts(case)
    kv, dim, dt = case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    s = dict(op=case["op"], dtype=dt, dim=dim, kv=kv, cu=_cu(n), rows=sum(n), longest=max(n))
    if case["op"] == "prefill":
        keys = [a + p for a, p in zip(n, past)]
        s.update(q=_rows(gen, sum(n), case["heads"], dim, dt, False), k=_rows(gen, sum(keys), kv, dim, dt, True),
                 v=_rows(gen, sum(keys), kv, dim, dt, False), cu_k=_cu(keys), longest_k=max(keys))
        return s
    page = case["page"]
    total = [a + p for a, p in zip(n, past)]
    used = [-(-t // page) for t in total]
    pages = sum(used) + 3                                      # a pool with a few free pages, handed out in no order
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(n), max(used)), -1, dtype=torch.int32)
    row, col = torch.tensor([(b, j) for b, u in enumerate(used) for j in range(u)]).T
    table = table.cuda()
    table[row.cuda(), col.cuda()] = order[: sum(used)]
    s.update(table=table, lens=torch.tensor(total, dtype=torch.int32, device="cuda"), page=page)
    shape = (pages, kv, page, dim)
    s["cache"] = _filled(gen, shape, True) + _filled(gen, shape, False)
    if case["op"] == "write":
        s.update(k=_rows(gen, sum(n), kv, dim, dt, True), v=_rows(gen, sum(n), kv, dim, dt, False))
    if case["op"] == "decode":
        s.update(q=_rows(gen, len(n), case["heads"], dim, dt, False),
                 counters=torch.zeros(len(n) * case["heads"], dtype=torch.int32, device="cuda"))
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        from bit_weight_quantized_nvq_b200 import capi
        if s["op"] == "write":
            capi.kv_write(s["cache"], s["k"], s["v"], s["cu"], s["lens"], s["table"])
            return capi.kv_read(s["cache"], s["cu"], s["lens"], s["table"], s["rows"], torch.float32)
        if s["op"] == "read":
            return capi.kv_read(s["cache"], s["cu"], s["lens"], s["table"], s["rows"], s["dtype"])
        if s["op"] == "decode":
            return capi.attn_decode(s["cache"], s["q"], s["lens"], s["table"], s["counters"])
        return capi.attn_prefill(s["q"], s["k"], s["v"], s["cu"], s["cu_k"])
    if s["op"] == "write":
        return _plain_write(s)
    if s["op"] == "read":
        return _plain_read(s, s["dtype"])
    if s["op"] == "decode":
        return _plain_decode(s)
    return _plain_prefill(s)


def _quantise(x):
    """Q8_0 along the last axis: d = amax / 127, q = rint(x / d), in fp32; the scale is kept as fp16."""
    x = x.float().unflatten(-1, (-1, BLOCK))
    top = x.abs().amax(-1, keepdim=True)
    d = top / torch.full_like(top, 127)                        # a true division: by a plain number it is a product
    q = torch.where(d > 0, torch.round(x / d), 0.0).clamp(-127, 127)
    return q.flatten(-2).to(torch.int8), d.squeeze(-1).to(torch.float16)


def _values(codes, scales):
    return (codes.float().unflatten(-1, (-1, BLOCK)) * scales.float().unsqueeze(-1)).flatten(-2)


def _places(s):
    """(page, offset in the page) of each packed row."""
    row = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    pos = s["lens"].long()[b] - s["cu"].long()[b + 1] + row
    return s["table"].long()[b, pos // s["page"]], pos % s["page"]


def _plain_write(s):
    page, off = _places(s)
    kc, ks, vc, vs = s["cache"]
    kc[page, :, off], ks[page, :, off] = _quantise(s["k"])
    vc[page, :, off], vs[page, :, off] = _quantise(s["v"])
    return _plain_read(s, torch.float32)


def _plain_read(s, dtype):
    page, off = _places(s)
    kc, ks, vc, vs = s["cache"]
    return (_values(kc[page, :, off], ks[page, :, off]).to(dtype), _values(vc[page, :, off], vs[page, :, off]).to(dtype))


def _softmax(x, keep):
    """Softmax of the kept places of the last axis; a row that keeps nothing gives zeros."""
    x = x.masked_fill_(~keep, float("-inf"))
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x.sub_(torch.where(torch.isfinite(top), top, 0.0)))
    return x.div_(x.sum(-1, keepdim=True).clamp_min(1e-30))


def _plain_decode(s):
    kc, ks, vc, vs = s["cache"]
    table, page = s["table"].long().clamp_min(0), s["page"]
    b, h = s["q"].shape[:2]
    q = s["q"].float().unflatten(1, (s["kv"], -1))                                   # [b, kv, g, d]
    k = _values(kc[table], ks[table]).permute(0, 2, 1, 3, 4).flatten(2, 3)           # [b, kv, positions, d]
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(s["dim"])
    del k
    keep = torch.arange(table.shape[1] * page, device="cuda") < s["lens"].view(-1, 1, 1, 1)
    p = _softmax(x, keep)
    v = _values(vc[table], vs[table]).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return torch.matmul(p, v).flatten(1, 2).to(s["dtype"])


def _padded(x, cu, longest):
    """Packed rows [rows, h, d] as [batch, h, longest, d] in fp32, zeros behind each sequence's end."""
    at = cu[:-1].long().view(-1, 1) + torch.arange(longest, device="cuda")
    inside = at < cu[1:].long().view(-1, 1)
    return (x[at.clamp_max(x.shape[0] - 1)].float() * inside[..., None, None]).transpose(1, 2), inside


def _plain_prefill(s):
    q, inside = _padded(s["q"], s["cu"], s["longest"])
    k, _ = _padded(s["k"], s["cu_k"], s["longest_k"])
    v, _ = _padded(s["v"], s["cu_k"], s["longest_k"])
    b, h, n, d = q.shape
    q = q.unflatten(1, (s["kv"], -1)).flatten(2, 3)                                  # [b, kv, g * n, d]
    x = torch.matmul(q, k.transpose(-1, -2)).div_(math.sqrt(d))
    behind = (s["cu_k"][1:] - s["cu_k"][:-1] - s["cu"][1:] + s["cu"][:-1]).view(-1, 1, 1)
    keep = torch.arange(s["longest_k"], device="cuda") <= torch.arange(n, device="cuda").view(-1, 1) + behind
    p = _softmax(x.unflatten(2, (-1, n)), keep[:, None, None])
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, n)).flatten(1, 2)         # [b, h, n, d]
    return o.transpose(1, 2)[inside].to(s["dtype"])


# ---------------------------------------------------------------------------
# the definition in 64 bits, sequence by sequence

def _attend64(q, k, v, first):
    """q [n, h, d], k and v [m, kv, d] in 64 bits; query i sees the keys 0 .. first + i."""
    g = q.shape[1] // k.shape[1]
    out = torch.empty_like(q)
    last = torch.arange(q.shape[0], device="cuda") + first
    hide = torch.arange(k.shape[0], device="cuda")[None, :] > last[:, None]
    for h in range(q.shape[1]):
        x = q[:, h] @ k[:, h // g].T * (q.shape[2] ** -0.5)
        x[hide] = float("-inf")
        out[:, h] = torch.softmax(x, 1) @ v[:, h // g]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    n, past = _lens(case), _pasts(case)
    if case["op"] == "write":
        outs = []
        for x in (s["k"], s["v"]):
            x = x.double().reshape(s["rows"], s["kv"], -1, BLOCK)
            # the format says where its quotients are rounded to fp32, which decides between two codes at a border
            top = x.abs().amax(-1, keepdim=True)
            unit = (top / torch.full_like(top, 127.0)).float().double()
            q = torch.round((x / torch.where(unit == 0, 1.0, unit)).float().double())
            outs.append((q * unit.half().double()).reshape(s["rows"], s["kv"], -1))
        return tuple(outs)
    if case["op"] == "prefill":
        outs, i, j = [], 0, 0
        for a, p in zip(n, past):
            outs.append(_attend64(s["q"][i:i + a].double(), s["k"][j:j + a + p].double(), s["v"][j:j + a + p].double(), p))
            i, j = i + a, j + a + p
        return torch.cat(outs)
    kc, ks, vc, vs = s["cache"]
    outs = []
    for b, length in enumerate(n):
        used = s["table"][b, : -(-length // s["page"])].long()
        both = []
        for codes, scales in ((kc, ks), (vc, vs)):
            x = codes[used].double() * scales[used].double().repeat_interleave(BLOCK, -1)     # [pages, kv, page, d]
            both.append(x.transpose(1, 2).reshape(-1, s["kv"], s["dim"])[:length])
        outs.append(both if case["op"] == "read" else _attend64(s["q"][b:b + 1].double(), *both, length - 1))
    if case["op"] == "read":
        return tuple(torch.cat(x) for x in zip(*outs))
    return torch.cat(outs)
