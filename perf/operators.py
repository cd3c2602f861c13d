"""Cases of the 4-bit memory cache's operators: page plan, store, read back, attention.

A cache is one byte buffer of pages.  Page p, head h, 16-token block j of the page is one
contiguous piece of 1152 bytes per 64 values of the head size: the key codes, the value
codes (512 bytes each per 64 values), then, per token and 64 values, four bf16 numbers: key
scale, key minimum, value scale, value minimum.  A byte holds the codes of values d (low
four bits) and d + 8 (high four bits) of one token, d the lower half of a run of 16.  In
key codes, token 8 hi + g and byte 8 ks + 2 t + e sit at byte 64 g + 16 t + 4 ks + 2 e + hi;
in value codes, token 8 hi + 2 t + e and byte 8 ks + g sit at the same place.
A code c stands for scale * c + minimum.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
GROUP = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoding step of a serving batch: a token more for each of 64 requests
        dict(name="plan_step_b64", op="plan", kind="step", requests=64, page=64, max_len=16384, layout=1),
        # 256 short prompts arrive, in small pages: 60 to 130 thousand slots
        dict(name="plan_prompts_b256", op="plan", kind="prompts", requests=256, page=16, max_len=512, layout=2),
        # a batch turns over: some requests end, some start, some grow by a chunk
        dict(name="plan_turnover_b1000", op="plan", kind="turnover", requests=1000, page=32, max_len=2048, layout=3),
        # the new tokens of a decoding step, one a request, each in another page
        dict(name="store_step_t64", op="store", tokens=64, runs=64, heads=16, dim=64, page=64, dtype="bf16", layout=4),
        # the memory of 8 records of 16384 rows, as the K/V projection leaves it: strided columns of one matrix
        dict(name="store_memory_8x16k", op="store", tokens=131072, runs=8, heads=16, dim=64, page=64, dtype="bf16", layout=5),
        # ragged prompts with wide heads in fp16, in small pages
        dict(name="store_ragged_d128", op="store", tokens=20011, runs=37, heads=8, dim=128, page=16, dtype="fp16", layout=6),
        # one record's memory back in bf16
        dict(name="read_record_16k", op="read", tokens=16384, runs=1, heads=16, dim=64, page=64, dtype="bf16", layout=7),
        # short pieces of many records in fp32
        dict(name="read_pieces_d128", op="read", tokens=5003, runs=61, heads=8, dim=128, page=32, dtype="fp32", layout=8),
        # the smallest: one token of one request against a short memory
        dict(name="attend_one_l512", op="attend", requests=1, law="fixed", max_len=512, new=1, heads=16, share=1, dim=64,
             page=64, dtype="bf16", causal=True, layout=9),
        # a decoding step of a serving batch with shared key heads
        dict(name="attend_step_b64_d128", op="attend", requests=64, law="lognormal", max_len=16384, new=1, heads=8,
             share=4, dim=128, page=64, dtype="bf16", causal=True, layout=10),
        # the options of 8 records of 16384 rows against their whole memory
        dict(name="attend_options_8x16k", op="attend", requests=8, law="fixed", max_len=16384, new=64, heads=16, share=1,
             dim=64, page=64, dtype="bf16", causal=False, layout=11),
        # one token against a very long memory, few key heads
        dict(name="attend_long_l131k", op="attend", requests=1, law="fixed", max_len=131001, new=1, heads=2, share=8,
             dim=64, page=256, dtype="fp16", causal=True, layout=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "read", "attend", "attend"])
    page, layout = rng.choice([16, 32, 64, 128, 256]), rng.randrange(1 << 30)
    if op == "plan":
        kind = rng.choice(["step", "prompts", "turnover"])
        requests = _log(rng, 1, 1000)
        return dict(op=op, kind=kind, requests=requests, page=page, max_len=_log(rng, 64, max(64, min(16384, 130000 // requests))),
                    layout=layout)
    dim = rng.choice([64, 128])
    if op in ("store", "read"):
        heads = rng.choice([1, 2, 3, 8, 16])
        tokens = _log(rng, 1, min(131072, 120_000_000 // (heads * dim)))
        dtype = rng.choice(["bf16", "fp16"] if op == "store" else ["bf16", "fp16", "fp32"])
        return dict(op=op, tokens=tokens, runs=_log(rng, 1, min(64, tokens)), heads=heads, dim=dim, page=page, dtype=dtype,
                    layout=layout)
    requests = _log(rng, 1, 64)
    heads, share = rng.choice([(16, 1), (8, 4), (2, 8), (4, 5), (3, 2), (1, 7)])
    most = max(64, min(131072, 100_000_000 // (requests * heads * dim)))
    max_len = _log(rng, 16, most)
    new = rng.choice([1, 1, rng.randint(2, 9), _log(rng, 10, 96)])
    new = max(1, min(new, max_len, 4_000_000_000 // (requests * heads * share * dim * max_len)))
    return dict(op=op, requests=requests, law=rng.choice(["fixed", "uniform", "lognormal"]), max_len=max_len, new=new,
                heads=heads, share=share, dim=dim, page=page, dtype=rng.choice(["bf16", "fp16"]),
                causal=rng.random() < 0.5, layout=layout)


def _up(a, b):
    return -(-a // b)


def _lengths(case):
    """Keys and queries of every request of an attention case, from the case alone."""
    r, n, top = random.Random(case["layout"]), case["requests"], case["max_len"]
    if case["law"] == "fixed":
        lens = [top] * n
    elif case["law"] == "uniform":
        lens = [r.randint(0, top) for _ in range(n)]
    else:
        lens = [max(1, min(top, int(r.lognormvariate(math.log(max(2, top / 8)), 0.8)))) for _ in range(n)]
    new = [case["new"] if case["new"] == 1 or case["law"] == "fixed" else r.randint(0, case["new"]) for _ in lens]
    new[0] = max(1, new[0])
    return lens, new


def _plan_lengths(case):
    """Tokens of every request before and after the step."""
    r, n, top = random.Random(case["layout"]), case["requests"], case["max_len"]
    if case["kind"] == "step":
        old = [r.randint(1, top - 1) for _ in range(n)]
        return old, [x + 1 for x in old]
    if case["kind"] == "prompts":
        return [0] * n, [r.randint(top // 2, top) for _ in range(n)]
    old = [r.choice([0, r.randint(1, top)]) for _ in range(n)]
    return old, [r.choice([0, x, min(top, x + r.randint(1, 64)), r.randint(0, x)]) for x in old]


def _run_lengths(case):
    """Tokens of every run of consecutive slots of a store or read case."""
    r, n, runs = random.Random(case["layout"]), case["tokens"], case["runs"]
    cuts = sorted(r.sample(range(1, n), runs - 1)) if runs > 1 and n % runs else [n // runs * i for i in range(1, runs)]
    return [b - a for a, b in zip([0] + cuts, cuts + [n])]


def work(case):
    op = case["op"]
    if op == "plan":
        old, new = _plan_lengths(case)
        pages = sum(abs(_up(a, case["page"]) - _up(b, case["page"])) for a, b in zip(old, new))
        slots = sum(max(0, b - a) for a, b in zip(old, new))
        return {"bytes": 4 * (len(old) * 4 + 2 * pages + slots), "flops": 0}
    if op in ("store", "read"):
        size, each = (4 if case["dtype"] == "fp32" else 2), case["tokens"] * case["heads"]
        packed = each * 72 * case["dim"] // 64
        if op == "store":  # in, stored, and what it stands for read back in bf16
            return {"bytes": each * case["dim"] * 2 * (size + 2) + 2 * packed + 4 * case["tokens"], "flops": 0}
        return {"bytes": each * case["dim"] * 2 * size + packed + 4 * case["tokens"], "flops": 0}
    lens, new = _lengths(case)
    hq = case["heads"] * case["share"]
    used = sum(x for x, n in zip(lens, new) if n)
    pairs = sum(n * x if not case["causal"] else sum(max(0, x - n + 1 + i) for i in range(n)) for x, n in zip(lens, new))
    return {"bytes": used * case["heads"] * 72 * case["dim"] // 64 + sum(new) * hq * (case["dim"] * 4 + 4),
            "flops": 4 * case["dim"] * hq * pairs}


# ------------------------------------------------------- the cache's byte layout

def _place(codes, minor):
    """Codes [..., 16 tokens, dim] to bytes [..., dim / 64 * 512]; `minor` is 0 for keys, 1 for values."""
    lead = codes.shape[:-2]
    x = codes.reshape(*lead, 16, -1, 4, 2, 8)  # token, 64 values, run of 16, half, value
    x = x[..., 0, :] | (x[..., 1, :] << 4)     # token, 64 values, run of 16, byte
    n = len(lead)
    if minor == 0:
        x = x.reshape(*lead, 2, 8, -1, 4, 4, 2)  # hi g | 64s | ks t e
        order = [n + 2, n + 1, n + 4, n + 3, n + 5, n]
    else:
        x = x.reshape(*lead, 2, 4, 2, -1, 4, 8)  # hi t e | 64s | ks g
        order = [n + 3, n + 5, n + 1, n + 4, n + 2, n]
    return x.permute(*range(n), *order).reshape(*lead, -1)


def _taken(data, minor):
    """The inverse of _place: bytes [..., dim / 64 * 512] to codes [..., 16 tokens, dim]."""
    lead, n = data.shape[:-1], data.dim() - 1
    x = data.reshape(*lead, -1, 8, 4, 4, 2, 2)  # 64s | g t ks e hi
    if minor == 0:
        x = x.permute(*range(n), n + 5, n + 1, n, n + 3, n + 2, n + 4)  # hi g | 64s | ks t e
    else:
        x = x.permute(*range(n), n + 5, n + 2, n + 4, n, n + 3, n + 1)  # hi t e | 64s | ks g
    x = x.reshape(*lead, 16, -1, 4, 1, 8)
    return torch.cat([x & 15, x >> 4], -2).reshape(*lead, 16, -1)


def _block_bytes(dim):
    return 1152 * dim // 64


def _numbers(data, dim):
    """Cache bytes [..., block] to fp32 keys and values [..., 16 tokens, dim]."""
    half = dim * 8
    sm = data[..., 2 * half:].reshape(*data.shape[:-1], 16, dim // GROUP, 4, 2).contiguous().view(torch.bfloat16)
    sm = sm.squeeze(-1).float().repeat_interleave(GROUP, -2)
    k = _taken(data[..., :half], 0).float() * sm[..., 0] + sm[..., 1]
    v = _taken(data[..., half:2 * half], 1).float() * sm[..., 2] + sm[..., 3]
    return k, v


def _codes(x):
    """fp32 [..., dim] to codes, scales and minima (bf16) by groups of 64 values."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    m = low.bfloat16().float()
    s = ((high - m).clamp(min=0) / torch.full_like(m, 15.0)).bfloat16().float()
    bad = ~(torch.isfinite(s) & torch.isfinite(m))
    c = torch.where(bad | (s == 0), torch.zeros_like(g), ((g - m) / s).round().clamp(0, 15))
    nan = torch.full_like(s, math.nan)
    s, m = torch.where(bad, nan, s), torch.where(bad, nan, m)
    return c.reshape(x.shape).to(torch.uint8), s.squeeze(-1).bfloat16(), m.squeeze(-1).bfloat16()


def _packed(k, v):
    """fp32 keys and values [..., 16 tokens, dim] to cache bytes [..., block]."""
    kc, ks, km = _codes(k)
    vc, vs, vm = _codes(v)
    sm = torch.stack([ks, km, vs, vm], -1).contiguous().view(torch.uint8).reshape(*k.shape[:-2], -1)
    return torch.cat([_place(kc, 0), _place(vc, 1), sm], -1)


# --------------------------------------------------------------------- inputs

def _memory(shape, g, heads_at, dtype=torch.float32):
    """Keys and values as a projection gives them: keys with a few strong channels, values of
    uneven size from token to token."""
    dim = shape[-1]
    strong = torch.randn(shape[heads_at], dim, generator=g, device=DEVICE) * (torch.arange(dim, device=DEVICE) % 16 == 3) * 2
    strong = strong.reshape([shape[heads_at] if i == heads_at else 1 for i in range(len(shape) - 1)] + [dim])
    k = torch.randn(shape, generator=g, device=DEVICE).add_(strong)
    v = torch.randn(shape, generator=g, device=DEVICE)
    v *= torch.exp(0.4 * torch.randn(*shape[:-1], 1, generator=g, device=DEVICE))
    return k.to(dtype), v.to(dtype)


def _filled(pages, case, g):
    """A cache of `pages` pages full of stored keys and values."""
    data = torch.empty(pages, case["heads"], case["page"] // 16, _block_bytes(case["dim"]), dtype=torch.uint8, device=DEVICE)
    step = max(1, 50_000_000 // (case["heads"] * case["page"] * case["dim"]))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        k, v = _memory((n, case["heads"], case["page"] // 16, 16, case["dim"]), g, 1)
        data[p:p + n] = _packed(k.bfloat16().float(), v.bfloat16().float())
    return data


def _slot_runs(case, g):
    """A slot for every token: runs of consecutive positions, each with pages of its own in any order."""
    page, r = case["page"], random.Random(case["layout"] + 1)
    starts = [r.randrange(page) if r.random() < 0.5 else 0 for _ in range(case["runs"])]
    lens = _run_lengths(case)
    need = [_up(a + n, page) for a, n in zip(starts, lens)]
    pages = sum(need)
    perm = torch.randperm(pages, generator=g, device=DEVICE)
    pos = torch.cat([torch.arange(a, a + n, device=DEVICE) + page * f for a, n, f in
                     zip(starts, lens, [sum(need[:i]) for i in range(len(need))])])
    return pages, (perm[pos // page] * page + pos % page).int()


def _page_state(case, g):
    """Page accounts: [free count, lengths, free pages, block table], as one int32 tensor."""
    old, new = _plan_lengths(case)
    page, width, n = case["page"], _up(case["max_len"], case["page"]), case["requests"]
    have = torch.tensor([_up(x, page) for x in old], device=DEVICE)
    total = sum(_up(max(a, b), page) for a, b in zip(old, new)) + 3
    perm = torch.randperm(total, generator=g, device=DEVICE).int()
    cols = torch.arange(width, device=DEVICE)
    first = torch.cumsum(have, 0) - have
    mine = cols < have[:, None]
    table = torch.where(mine, perm[(first[:, None] + cols).clamp(max=total - 1)], -1)
    used = int(have.sum())
    free = torch.full((total,), -1, dtype=torch.int32, device=DEVICE)
    free[:total - used] = perm[used:]
    head = torch.tensor([total - used], dtype=torch.int32, device=DEVICE)
    lens = torch.tensor(old, dtype=torch.int32, device=DEVICE)
    return torch.cat([head, lens, free, table.int().reshape(-1)]), total, width


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "plan":
        s["state"], s["pages"], s["width"] = _page_state(case, g)
        s["scratch"] = torch.empty_like(s["state"])
        s["want"] = torch.tensor(_plan_lengths(case)[1], dtype=torch.int32, device=DEVICE)
        # a step's slot buffer has a place for every token that may come
        s["slots"] = max(1, sum(max(0, b - a) for a, b in zip(*_plan_lengths(case)))) + 5
        return s
    if case["op"] in ("store", "read"):
        s["pages"], s["slots"] = _slot_runs(case, g)
        shape = (case["tokens"], case["heads"], case["dim"])
        if case["op"] == "store":
            # K and V are column blocks of one matrix, as a joint projection leaves them
            kv = torch.empty(shape[0], 2, *shape[1:], dtype=TYPES[case["dtype"]], device=DEVICE)
            k, v = _memory(shape, g, 1)
            kv[:, 0], kv[:, 1] = k, v
            s["k"], s["v"] = kv[:, 0], kv[:, 1]
            s["data"] = torch.zeros(s["pages"], case["heads"], case["page"] // 16, _block_bytes(case["dim"]),
                                    dtype=torch.uint8, device=DEVICE)
        else:
            s["data"] = _filled(s["pages"], case, g)
        return s
    lens, new = _lengths(case)
    width = _up(case["max_len"], case["page"])
    need = [_up(x, case["page"]) for x in lens]
    s["pages"] = max(1, sum(need))
    perm = torch.randperm(s["pages"], generator=g, device=DEVICE).int()
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEVICE)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    s["table"] = table
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    s["cu"] = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device=DEVICE)
    s["most"] = max(new)
    s["data"] = _filled(s["pages"], case, g)
    s["scale"] = case["dim"] ** -0.5
    q = 1.5 * torch.randn(sum(new), case["heads"] * case["share"], case["dim"], generator=g, device=DEVICE)
    s["q"] = q.to(TYPES[case["dtype"]])
    return s


# ------------------------------------------------------------------ plain forms

def _plain_plan(s):
    """Pages given back by descending request and page, then granted by ascending request from the end of the free list."""
    case, page = s["case"], s["case"]["page"]
    n, pages, width = case["requests"], s["pages"], s["width"]
    state = s["state"].clone()
    count, lens, free, table = state[0], state[1:1 + n], state[1 + n:1 + n + pages], state[1 + n + pages:].view(n, width)
    old, want = lens.clone(), s["want"]
    have, need = (old + page - 1) // page, (want + page - 1) // page
    cols = torch.arange(width, device=DEVICE)
    back = (cols >= need[:, None]) & (cols < have[:, None])
    flipped = back.flatten().flip(0)
    place = torch.where(flipped, count + torch.cumsum(flipped, 0) - 1, pages)
    stack = torch.cat([free, free.new_full((1,), -1)])
    stack = stack.scatter(0, place, table.flatten().flip(0))
    top = count + back.sum()
    more = (need - have).clamp(min=0)
    ends = torch.cumsum(more, 0)
    fits = (ends <= top) | (more == 0)
    grant = (cols >= have[:, None]) & (cols < need[:, None]) & fits[:, None]
    turn = (ends - more)[:, None] + cols - have[:, None]
    taken = stack[(top - 1 - turn).clamp(0, pages)]
    table.copy_(torch.where(grant, taken, torch.where(back, -1, table)))
    top = top - (more * fits).sum()
    free.copy_(torch.where(torch.arange(pages, device=DEVICE) < top, stack[:pages], -1))
    state[0] = top
    lens.copy_(torch.where(fits, want, old))
    cu = torch.zeros(n + 1, dtype=torch.int32, device=DEVICE)
    cu[1:] = torch.cumsum((lens - old).clamp(min=0), 0)
    t = torch.arange(s["slots"], device=DEVICE, dtype=torch.int32)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=n - 1)
    pos = old[b] + t - cu[b]
    slot = table[b, (pos // page).clamp(0, width - 1)] * page + pos % page
    return {"state": state, "slots": torch.where(t < cu[n], slot, -1), "cu": cu}


def _plain_store(s):
    case, dim = s["case"], s["case"]["dim"]
    slots = s["slots"].long()
    data = s["data"].view(-1, _block_bytes(dim))
    # a token alone in its 16-token block gives the bytes that are its own
    blocks = slots // case["page"] * case["heads"] * (case["page"] // 16) + slots % case["page"] // 16
    blocks = blocks[:, None] + torch.arange(case["heads"], device=DEVICE) * (case["page"] // 16)
    half = dim * 8
    for x, minor in ((s["k"], 0), (s["v"], 1)):
        c, sc, m = _codes(x.float())
        c = c.reshape(*c.shape[:-1], -1, 2, 8)
        c = (c[..., 0, :] | (c[..., 1, :] << 4)).reshape(*c.shape[:2], -1)
        j = torch.arange(dim // 2, device=DEVICE)
        r = (slots % 16)[:, None]
        if minor == 0:
            off = j // 32 * 512 + r % 8 * 64 + j % 8 // 2 * 16 + j % 32 // 8 * 4 + j % 2 * 2 + r // 8
        else:
            off = j // 32 * 512 + j % 8 * 64 + r % 8 // 2 * 16 + j % 32 // 8 * 4 + r % 2 * 2 + r // 8
        at = blocks[:, :, None] * _block_bytes(dim) + minor * half + off[:, None, :]
        data.view(-1).index_put_((at,), c)
        n = torch.arange(dim // GROUP, device=DEVICE)
        at = blocks[:, :, None] * (_block_bytes(dim) // 4) + (2 * half + r[:, :, None] * dim // 8 + n * 8 + minor * 4) // 4
        data.view(-1).view(torch.int32).index_put_((at,), torch.stack([sc, m], -1).contiguous().view(torch.int32).squeeze(-1))
    return _plain_read(s, torch.bfloat16)


def _plain_read(s, dtype):
    case = s["case"]
    slots = s["slots"].long()
    k, v = _numbers(s["data"], case["dim"])
    at, r = (slots // case["page"], slots % case["page"] // 16), slots % 16
    return {"k": k.permute(0, 2, 3, 1, 4)[at[0], at[1], r].to(dtype), "v": v.permute(0, 2, 3, 1, 4)[at[0], at[1], r].to(dtype)}


def _plain_attend(s):
    case, dim, share = s["case"], s["case"]["dim"], s["case"]["share"]
    n, most = case["requests"], s["most"]
    blocks = s["data"][s["table"].clamp(min=0).long()]  # request, page, head, block, bytes
    k, v = _numbers(blocks, dim)
    k, v = (x.permute(0, 2, 1, 3, 4, 5).reshape(n, case["heads"], -1, dim) for x in (k, v))
    cu = s["cu"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(most, device=DEVICE)
    real = i < count[:, None]
    q = s["q"][(cu[:-1, None] + i).clamp(max=len(s["q"]) - 1)].float()  # request, query, head, dim
    q = q.reshape(n, most, case["heads"], share, dim).permute(0, 2, 1, 3, 4).reshape(n, case["heads"], most * share, dim)
    scores = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    j = torch.arange(k.shape[2], device=DEVICE)
    last = s["lens"].long()[:, None] - 1
    if case["causal"]:
        last = last - (count[:, None] - 1 - i)
    seen = (j <= last.expand(n, most)[:, :, None]) & (j < s["lens"].long()[:, None, None])
    seen = seen[:, None, :, None].expand(n, case["heads"], most, share, -1).reshape(scores.shape)
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top)).masked_fill(~seen, 0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v * (j < s["lens"].long()[:, None])[:, None, :, None]) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    out = out.reshape(n, case["heads"], most, share, dim).permute(0, 2, 1, 3, 4).reshape(n, most, -1, dim)
    lse = lse.reshape(n, case["heads"], most, share).permute(0, 2, 1, 3).reshape(n, most, -1)
    row = torch.arange(len(s["q"]), device=DEVICE)
    b = torch.searchsorted(cu[1:], row, right=True)
    return {"out": out[b, row - cu[b]].to(s["q"].dtype), "lse": lse[b, row - cu[b]]}


def run(state):
    case = state["case"]
    if own:
        cache = _handle(state)
        if case["op"] == "plan":
            state["scratch"].copy_(state["state"])
            slots, cu = cache.plan(state["want"], state["slots"])
            return {"state": state["scratch"], "slots": slots, "cu": cu}
        if case["op"] == "store":
            cache.append(state["k"], state["v"], state["slots"])
            k, v = cache.read(state["slots"], torch.bfloat16)
            return {"k": k, "v": v}
        if case["op"] == "read":
            k, v = cache.read(state["slots"], TYPES[case["dtype"]])
            return {"k": k, "v": v}
        out, lse = cache.attend(state["q"], state["cu"], state["most"], scale=state["scale"], causal=case["causal"],
                                block_table=state["table"], lengths=state["lens"])
        return {"out": out, "lse": lse}
    if case["op"] == "plan":
        return _plain_plan(state)
    if case["op"] == "store":
        return _plain_store(state)
    if case["op"] == "read":
        return _plain_read(state, TYPES[case["dtype"]])
    return _plain_attend(state)


def _handle(state):
    """The cache object over the state's buffers, which a program makes once and keeps."""
    if "cache" not in state:
        from structured_decision_model_gb300.memory import MemoryCache
        case = state["case"]
        state["cache"] = MemoryCache(state["pages"], page=case["page"], heads=case.get("heads", 1), head_dim=case.get("dim", 64),
                                     requests=case.get("requests", 1), max_len=case.get("max_len", case["page"]),
                                     device=DEVICE, data=state.get("data"), state=state.get("scratch"))
    return state["cache"]


# ------------------------------------------------- the definition, in 64 bits

def _exact_quantised(x):
    """What fp64 [tokens, heads, dim] stands for once stored."""
    t, h, dim = x.shape
    y = torch.empty_like(x)
    for a in range(0, dim, GROUP):
        part = x[:, :, a:a + GROUP]
        m = part.min(2, keepdim=True).values.to(torch.bfloat16).double()
        s = ((part.max(2, keepdim=True).values - m).clamp(min=0) / 15).to(torch.bfloat16).double()
        step = torch.where(s > 0, s, torch.ones_like(s))
        y[:, :, a:a + GROUP] = m + s * torch.round((part - m) / step).clamp(0, 15)
    return y


def _exact_numbers(data, dim, page, slots):
    """fp64 keys and values [tokens, heads, dim] of slots, byte by byte from the layout's description."""
    heads, size = data.shape[1], _block_bytes(dim)
    d = torch.arange(dim, device=data.device)
    slots = slots.long()
    r = (slots % 16)[:, None]
    block = (slots // page)[:, None] * heads + torch.arange(heads, device=data.device)
    base = (block * (page // 16) + (slots % page // 16)[:, None]) * size
    byte = d % 64 // 16 * 8 + d % 8
    ks, low = byte // 8, byte % 8
    at_k = d // 64 * 512 + 64 * (r % 8) + 16 * (low // 2) + 4 * ks + 2 * (low % 2) + r // 8
    at_v = d // 64 * 512 + 64 * low + 16 * (r % 8 // 2) + 4 * ks + 2 * (r % 2) + r // 8
    flat, halves = data.reshape(-1), []
    words = flat.view(torch.bfloat16)
    shift = (d % 16 // 8 * 4).to(torch.uint8)
    for minor, at in ((0, at_k), (1, at_v)):
        code = (flat[base[:, :, None] + minor * dim * 8 + at[:, None, :]] >> shift) & 15
        n = (base + 16 * dim)[:, :, None] // 2 + (r * (dim // 64) * 4 + d // 64 * 4)[:, None, :] + 2 * minor
        halves.append(code.double() * words[n].double() + words[n + 1].double())
    return halves


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "store":
        return {"k": _exact_quantised(s["k"].double()), "v": _exact_quantised(s["v"].double())}
    if case["op"] == "read":
        k, v = _exact_numbers(s["data"], case["dim"], case["page"], s["slots"])
        return {"k": k, "v": v}
    cu, lens, share, page = s["cu"].tolist(), s["lens"].tolist(), case["share"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEVICE)
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if n == 0 or length == 0:
            continue
        pos = torch.arange(length, device=DEVICE)
        k, v = _exact_numbers(s["data"], case["dim"], page, s["table"][b, pos // page] * page + pos % page)
        visible = torch.ones(n, length, dtype=torch.bool, device=DEVICE)
        if case["causal"]:
            visible = visible.tril(length - n)
        for h in range(case["heads"] * share):
            x = s["q"][cu[b]:cu[b + 1], h].double() @ k[:, h // share].T * s["scale"]
            x = torch.where(visible, x, -math.inf)
            total = torch.logsumexp(x, 1)
            lse[cu[b]:cu[b + 1], h] = total
            p = torch.exp(x - torch.where(torch.isinf(total), torch.zeros_like(total), total)[:, None])
            out[cu[b]:cu[b + 1], h] = p @ v[:, h // share]
    return {"out": out, "lse": lse}
