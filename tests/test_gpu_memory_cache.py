"""The 4-bit memory cache's kernels against their plain fp64 forms (cache_support.py)."""
import math
import random

import pytest
import torch

from cache_support import STEP, Pages, attention, attention_tolerance, quantised
from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300.build import build_library
from structured_decision_model_gb300.memory import MemoryCache

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_library()
    B.load()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ plan

@pytest.mark.parametrize("requests,page,max_len,n_pages,steps", [
    (1, 16, 1, 1, 3), (1, 256, 70000, 300, 4), (3, 16, 100, 21, 8), (64, 64, 4096, 3000, 6), (257, 32, 300, 1500, 5),
    (1000, 16, 600, 20000, 3), (1024, 128, 1024, 4096, 3)])
def test_plan_walk(requests, page, max_len, n_pages, steps):
    """Random growth, shrinking and ends, pages running out on the way: tables, stack and slots as
    the request-by-request form keeps them."""
    r = random.Random(requests * 7 + page)
    c = MemoryCache(n_pages, page=page, heads=1, requests=requests, max_len=max_len, device=DEV)
    plain = Pages(n_pages, page, requests, c.width)
    for step in range(steps):
        want = [r.choice([0, n, min(n + 1, max_len), r.randint(0, max_len), r.randint(n, max_len)]) for n in plain.lengths]
        slots, cu, ran_out = plain.plan(want)
        n_slots = len(slots) + r.choice([0, 3])
        got, got_cu = c.plan(ints(want), n_slots)
        assert c.device_status() == (7 if ran_out else 0)
        assert c.lengths.tolist() == plain.lengths
        assert c.free_count.item() == len(plain.free)
        assert c.free_pages.tolist() == plain.free + [-1] * (n_pages - len(plain.free))
        assert c.block_table.tolist() == plain.table()
        assert got_cu.tolist() == cu
        assert got.tolist() == slots + [-1] * (n_slots - len(slots))
    c.plan(ints([0] * requests), 0)  # everything ends
    assert c.device_status() == 0 and c.free_count.item() == n_pages
    assert sorted(c.free_pages.tolist()) == list(range(n_pages))


def test_a_step_taken_back_leaves_the_stack_as_it_was():
    c = MemoryCache(50, page=16, heads=1, requests=5, max_len=200, device=DEV)
    c.plan(ints([30, 0, 100, 17, 64]), 300)
    before = c.state.clone()
    c.plan(ints([40, 90, 100, 200, 65]), 300)
    assert not torch.equal(before, c.state)
    c.plan(ints([30, 0, 100, 17, 64]), 300)
    assert torch.equal(before, c.state) and c.device_status() == 0


def test_plan_reports_what_is_out_of_range():
    c = MemoryCache(20, page=16, heads=1, requests=3, max_len=64, device=DEV)
    slots, cu = c.plan(ints([10, 65, 20]), 40)      # request 1 past the table
    assert c.device_status() == 5 and c.lengths.tolist() == [10, 0, 20] and cu.tolist() == [0, 10, 10, 30]
    slots, cu = c.plan(ints([11, -1, 20]), 4)
    assert c.device_status() == 5 and c.lengths.tolist() == [11, 0, 20]
    slots, cu = c.plan(ints([11, 7, 20]), 4)        # 7 gained, room for 4
    assert c.device_status() == 5 and cu.tolist() == [0, 0, 7, 7] and (slots >= 0).all() and slots.numel() == 4
    c.free_count.fill_(-5)                          # accounts that someone overwrote
    c.plan(ints([11, 64, 20]), 4)
    assert c.device_status() == 5
    c.free_count.fill_(20)                          # more pages than there are come back
    c.plan(ints([0, 0, 0]), 4)
    assert c.device_status() == 5 and c.free_count.item() == 20


# ------------------------------------------------------- store and read back

def rows_of(shape, dtype, g, layout):
    """Key and value rows in one of the layouts a caller may hold them in."""
    t, h, d = shape
    if layout == "columns":      # column blocks of one matrix, as a joint projection leaves them
        x = torch.randn(t, 2, h, d, generator=g, device=DEV).to(dtype)
        return x[:, 0], x[:, 1]
    if layout == "heads first":
        x = torch.randn(2, h, t, d, generator=g, device=DEV).to(dtype).transpose(1, 2)
        return x[0], x[1]
    if layout == "odd":          # rows and heads that start at any element
        x = torch.randn(2, t, h, d + 3, generator=g, device=DEV).to(dtype)[..., 1:d + 1]
        return x[0], x[1]
    x = torch.randn(2, t, h, d, generator=g, device=DEV).to(dtype)
    return x[0], x[1]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,heads,dim,page,layout,order", [
    (1, 1, 64, 16, "plain", "runs"), (15, 3, 64, 32, "odd", "runs"), (16, 16, 64, 64, "columns", "aligned"),
    (17, 2, 128, 16, "plain", "aligned"), (100, 9, 64, 256, "heads first", "runs"), (333, 8, 128, 64, "columns", "shuffled"),
    (1000, 5, 64, 64, "odd", "shuffled"), (2050, 16, 64, 128, "columns", "runs"), (700, 4, 128, 32, "odd", "runs")])
def test_store_and_read_back(tokens, heads, dim, page, layout, order, dtype):
    """Stored rows read back as the formula's values, exactly; other slots keep their bits."""
    r, g = random.Random(tokens), gen(tokens)
    n_pages = -(-tokens // page) * 2 + 3
    c = MemoryCache(n_pages, page=page, heads=heads, head_dim=dim, device=DEV)
    every = torch.arange(n_pages * page, dtype=torch.int32, device=DEV)
    k0, v0 = rows_of((n_pages * page, heads, dim), dtype, g, "plain")
    c.append(k0, v0, every)
    if order == "aligned":
        slots = every[page:page + tokens].clone()
    elif order == "runs":        # runs that start and end anywhere
        slots, at = [], r.randrange(page)
        while len(slots) < tokens:
            n = r.choice([1, 2, 7, 16, 31, 64, 200])
            slots += range(at, min(at + n, n_pages * page))
            at += n + r.choice([0, 0, 1, 5])
            at = at if at < n_pages * page else len(slots) * 10 ** 6
        slots = ints(slots[:tokens]) if max(slots[:tokens]) < n_pages * page else every[3:3 + tokens].clone()
    else:
        slots = every[torch.randperm(len(every), generator=g, device=DEV)[:tokens]].contiguous()
    k, v = rows_of((tokens, heads, dim), dtype, g, layout)
    skipped = torch.rand(tokens, generator=g, device=DEV) < 0.05
    given = torch.where(skipped, -1 - slots, slots)
    c.append(k, v, given)
    assert c.device_status() == 0
    wk, wv = quantised(k0), quantised(v0)
    live = slots[~skipped].long()
    wk[live], wv[live] = quantised(k[~skipped]), quantised(v[~skipped])
    for t in (torch.float32, torch.bfloat16, torch.float16):
        gk, gv = c.read(every, t)
        assert torch.equal(gk, wk.float().to(t)) and torch.equal(gv, wv.float().to(t))
    back = torch.randperm(len(every), generator=g, device=DEV)[:tokens].int()
    back[::7] = -3
    gk, gv = c.read(back, torch.float32)
    at = back.long().clamp(min=0)
    keep = (back >= 0)[:, None, None]
    assert torch.equal(gk, torch.where(keep, wk[at].float(), 0)) and torch.equal(gv, torch.where(keep, wv[at].float(), 0))
    assert c.device_status() == 0


def test_store_error_is_half_a_step():
    """|stored - x| <= s / 2 + the rounding of m, s (bf16): s (1 + 2^-8) / 2 + 15 s 2^-8 + |m| 2^-8 at most."""
    k = torch.randn(500, 4, 64, generator=gen(1), device=DEV).bfloat16()
    c = MemoryCache(8, page=64, heads=4, device=DEV)
    slots = torch.arange(500, dtype=torch.int32, device=DEV)
    c.append(k, k, slots)
    gk, gv = c.read(slots, torch.float32)
    x = k.float()
    s = (x.amax(-1, keepdim=True) - x.amin(-1, keepdim=True)) / 15
    bound = s * (0.5 * (1 + 2 ** -8) + 15 * 2 ** -8) + x.amin(-1, keepdim=True).abs() * 2 ** -8
    assert ((gk - x).abs() <= bound).all() and torch.equal(gk, gv)


@pytest.mark.parametrize("dtype", TYPES)
def test_store_of_uncommon_groups(dtype):
    """Constant, zero, tiny, huge and non-finite groups; a bad group stays alone."""
    big = torch.finfo(dtype).max
    x = torch.randn(12, 2, 128, generator=gen(2), device=DEV).to(dtype)
    x[0] = 0
    x[1] = 3.25
    x[2] = -0.0
    x[3] *= torch.finfo(dtype).tiny
    x[4, :, :64] = big
    x[5, :, 5] = big
    x[5, :, 6] = -big            # bf16: the range itself overflows fp32
    x[6, 0, 70] = math.nan
    x[7, 1, 3] = math.inf
    x[8, 1, 100] = -math.inf
    x[9, 0, :64] = math.nan
    x[10, :, ::2] = 1
    x[10, :, 1::2] = 0
    c = MemoryCache(1, page=16, heads=2, head_dim=128, device=DEV)
    slots = torch.arange(12, dtype=torch.int32, device=DEV)
    c.append(x, -x, slots)
    k, v = c.read(slots, torch.float32)
    for got, want in ((k, quantised(x)), (v, quantised(-x))):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(nan=0.0), want.float().nan_to_num(nan=0.0))
    assert torch.isnan(k[6, 0, 64:]).all() and not torch.isnan(k[6, 0, :64]).any() and not torch.isnan(k[6, 1]).any()
    assert (k[1] == 3.25).all() and (k[0] == 0).all()


def test_heads_of_layers_side_by_side():
    g = gen(3)
    c = MemoryCache(4, page=16, heads=7, head_dim=64, device=DEV)
    slots = torch.randperm(64, generator=g, device=DEV)[:40].int()
    parts = [rows_of((40, n, 64), torch.bfloat16, g, "plain") for n in (3, 4)]
    c.append(*parts[1], slots, head0=3)
    c.append(*parts[0], slots, head0=0)
    k, v = c.read(slots, torch.float32)
    assert torch.equal(k, quantised(torch.cat([p[0] for p in parts], 1)).float())
    k, v = c.read(slots, torch.float32, head0=2, heads=3)
    assert torch.equal(v, quantised(torch.cat([p[1] for p in parts], 1)).float()[:, 2:5])


def test_slots_past_the_cache_are_reported_and_skipped():
    c = MemoryCache(2, page=16, heads=2, device=DEV)
    k = torch.randn(3, 2, 64, generator=gen(4), device=DEV).bfloat16()
    c.append(k, k, ints([31, 32, 2 ** 31 - 1]))
    assert c.device_status() == 5
    got, _ = c.read(ints([31, 32, 5]), torch.float32)
    assert c.device_status() == 5
    assert torch.equal(got[0], quantised(k[0]).float()) and (got[1:] == 0).all()


# ------------------------------------------------------------------ attention

def filled(lens, heads, dim, page, g, dtype=torch.bfloat16, spare=2, scale=1.0):
    """A cache with the requests' memory in shuffled pages, and what each request's rows stand for."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    c = MemoryCache(n_pages, page=page, heads=heads, head_dim=dim, requests=len(lens), max_len=max(max(lens), 1), device=DEV)
    c.data.random_(0, 256, generator=g)   # whatever was there before
    order = torch.randperm(n_pages, generator=g, device=DEV).int()
    at = 0
    for b, n in enumerate(need):
        c.block_table[b, :n] = order[at:at + n]
        at += n
    c.lengths.copy_(ints(lens))
    memory = []
    for b, n in enumerate(lens):
        pos = torch.arange(n, device=DEV)
        slots = (c.block_table[b, pos // page] * page + pos % page).int()
        k = (scale * torch.randn(n, heads, dim, generator=g, device=DEV)).to(dtype)
        v = (torch.randn(n, heads, dim, generator=g, device=DEV) * torch.exp(torch.randn(n, 1, 1, generator=g, device=DEV))).to(dtype)
        c.append(k, v, slots)
        memory.append(c.read(slots, torch.float32))
    assert c.device_status() == 0
    return c, memory


def check(c, memory, q, new, out, lse, scale, causal, dtype):
    at = 0
    for (k, v), n in zip(memory, new):
        if n:
            want, want_lse = attention(q[at:at + n], k, v, scale, causal)
            tol, lse_tol = attention_tolerance(q[at:at + n], k, v, scale, dtype)
            got, got_lse = out[at:at + n].double(), lse[at:at + n].double()
            bound = tol + (1 + 2 * STEP[dtype]) * STEP[dtype] * want.abs() + torch.finfo(dtype).tiny
            assert ((got - want).abs() <= bound).all(), ((got - want).abs().max(), tol)
            empty = torch.isinf(want_lse)
            assert torch.equal(torch.isinf(got_lse) & (got_lse < 0), empty)
            assert ((got_lse - want_lse)[~empty].abs() <= lse_tol + 2 ** -22 * want_lse[~empty].abs()).all()
            assert (got[empty] == 0).all()
        at += n


CASES = [  # lens, new, kv heads, share, dim, page
    ([1], [1], 1, 1, 64, 16), ([0], [1], 2, 3, 64, 16), ([15, 16, 17, 0, 1], [1] * 5, 2, 4, 64, 16),
    ([255, 256, 257, 512, 513], [1, 1, 0, 1, 1], 3, 1, 128, 64), ([33, 700, 5], [5, 9, 7], 2, 8, 64, 32),
    ([3, 100, 0, 64], [10, 100, 4, 3], 4, 1, 64, 64), ([1000], [33], 1, 1, 64, 256), ([777, 1200], [17, 1], 2, 5, 128, 16),
    ([4096, 100], [16, 2], 1, 7, 64, 128), ([5000], [1], 16, 1, 64, 64), ([20000, 300], [2, 2], 2, 2, 128, 256),
    ([600, 600, 90], [32, 33, 90], 1, 1, 64, 32), ([2500, 100, 0, 7], [40, 64, 65, 7], 2, 1, 64, 16),
    ([300, 3000, 40], [16, 17, 1], 2, 1, 128, 64), ([5000, 64], [13, 20], 1, 8, 64, 128),
    ([2049, 130, 1], [50, 70, 2], 1, 3, 128, 16), ([70001], [1], 1, 8, 64, 64), ([2100], [100], 2, 1, 64, 64), ([40, 2000, 1, 90, 333], [25, 0, 1, 24, 9], 1, 1, 64, 16)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, causal, dtype):
    lens, new, heads, share, dim, page = CASES[case]
    g = gen(100 + case)
    c, memory = filled(lens, heads, dim, page, g)
    total = sum(new)
    q = (1.5 * torch.randn(total, heads * share, dim, generator=g, device=DEV)).to(dtype)
    cu = ints([sum(new[:i]) for i in range(len(new) + 1)])
    out, lse = c.attend(q, cu, max(new), causal=causal)
    assert c.device_status() == 0
    check(c, memory, q, new, out, lse, dim ** -0.5, causal, dtype)
    again, lse2 = c.attend(q, cu, total, causal=causal)   # a looser bound changes the blocks, not more
    check(c, memory, q, new, again, lse2, dim ** -0.5, causal, dtype)


def test_strided_queries_layers_and_given_tables():
    g = gen(7)
    c, memory = filled([300, 40], 6, 64, 16, g)
    x = torch.randn(3, 4, 9, 64, generator=g, device=DEV).bfloat16()
    q = x.transpose(1, 2)[1]                     # heads first: rows 64 apart, heads 576
    assert q.stride() == (64, 576, 1)
    cu = ints([0, 4, 9])
    swapped = c.block_table.flip(0).contiguous()
    out, lse = c.attend(q, cu, 5, scale=0.2, causal=False, head0=4, kv_heads=2, block_table=swapped,
                        lengths=c.lengths.flip(0).contiguous())
    part = [(k[:, 4:], v[:, 4:]) for k, v in memory[::-1]]
    check(c, part, q, [4, 5], out, lse, 0.2, False, torch.bfloat16)
    assert c.device_status() == 0


@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** -10, 64.0, 2.0 ** 30])
@pytest.mark.parametrize("n", [8, 50])
def test_query_sizes(size, n):
    """Scores from nearly equal to one-hot; rows of very different size side by side."""
    g = gen(8)
    c, memory = filled([600], 2, 64, 64, g)
    q = torch.randn(n, 2, 64, generator=g, device=DEV)
    q[::2] *= size
    q[3] = 0
    q = q.bfloat16()
    out, lse = c.attend(q, ints([0, n]), n, causal=False)
    for i in range(n):
        scale = 64 ** -0.5
        want, want_lse = attention(q[i:i + 1], *memory[0], scale, False)
        if size < 2.0 ** 20 or i % 2 or i == 3:
            check(c, memory, q[i:i + 1], [1], out[i:i + 1], lse[i:i + 1], scale, False, torch.bfloat16)
        else:                    # one-hot: the output is the winner's value where it wins by a margin
            s = torch.einsum("hd,lhd->hl", q[i].double(), memory[0][0].double()) * scale
            top = s.topk(2, -1).values
            _, err = attention_tolerance(q[i:i + 1], *memory[0], scale, torch.bfloat16)
            sure = top[:, 0] - top[:, 1] > 2 * err + 20
            assert sure.any()
            assert ((out[i] - want[0]).abs().amax(-1)[sure] <= 2 ** -7 * memory[0][1].abs().max()).all()


@pytest.mark.parametrize("n", [1, 40])
def test_equal_weights_give_the_mean_value(n):
    """Zero queries over 20000 keys: 1 / n weights, a mean far smaller than the values it is made of."""
    g = gen(9)
    c, memory = filled([20000], 2, 64, 64, g)
    q = torch.zeros(n, 2, 64, dtype=torch.float16, device=DEV)
    out, lse = c.attend(q, ints([0, n]), n, causal=False)
    v = memory[0][1].double()
    # every weight (many rows: and value, and its middle) is rounded by at most 2^-11 of itself,
    # independently of the sign of its value: |error| <= 3 x 2^-11 sqrt(sum v^2) / n times 6
    # deviations, and the bias of equal weights of equal scales 2^-11 |mean|; the output's own
    # rounding 2^-11 |mean|
    bound = (6 if n == 1 else 18) * 2 ** -11 * v.square().sum(0).sqrt() / 20000 + 2 ** -10 * v.mean(0).abs() + 2 ** -24
    assert ((out.double() - v.mean(0)).abs() <= bound).all()
    assert (lse.double() - math.log(20000)).abs().max() < 2 ** -20


@pytest.mark.parametrize("n0,n1", [(4, 3), (19, 18), (36, 40)])
def test_what_is_masked_may_hold_anything(n0, n1):
    """NaN and infinite values behind the last token, in tokens that a causal row does not see, and in
    another request leave a row alone; a NaN that it does see makes it NaN."""
    g = gen(10)
    lens = [37, 50]
    c, memory = filled(lens, 2, 128, 16, g)
    clean_q = torch.randn(n0 + n1, 2, 128, generator=g, device=DEV).bfloat16()
    cu, most = ints([0, n0, n0 + n1]), max(n0, n1)
    clean, clean_lse = c.attend(clean_q, cu, most)
    bad = torch.full((1, 2, 128), math.nan, device=DEV).bfloat16()
    slot = lambda b, p: ints([c.block_table[b, p // 16].item() * 16 + p % 16])
    for p in range(37, 48):                       # behind the last token of request 0, in its last page
        c.append(bad, bad, slot(0, p))
    out, lse = c.attend(clean_q, cu, most)
    assert torch.equal(out, clean) and torch.equal(lse, clean_lse)
    c.append(bad, bad, slot(0, 36))               # its last token: only the last causal row sees it
    out, lse = c.attend(clean_q, cu, most)
    assert torch.equal(out[:n0 - 1], clean[:n0 - 1]) and torch.equal(out[n0:], clean[n0:])
    assert torch.isnan(out[n0 - 1]).all() and torch.isnan(lse[n0 - 1]).all() and not torch.isnan(lse[:n0 - 1]).any()
    k, v = memory[1]
    some = v[49:50].bfloat16()
    some[:, :, 64:] = math.nan
    c.append(k[49:50].bfloat16(), some, slot(1, 49))  # half of a value alone
    out, lse = c.attend(clean_q, cu, most)
    last = n0 + n1 - 1
    assert torch.equal(out[n0:last], clean[n0:last]) and not torch.isnan(lse[n0:]).any()
    assert torch.isnan(out[last, :, 64:]).all() and not torch.isnan(out[last, :, :64]).any()


@pytest.mark.parametrize("n", [9, 30, 70])
def test_a_bad_query_row_stays_alone(n):
    g = gen(11)
    c, _ = filled([400], 1, 64, 64, g)
    q = torch.randn(n, 1, 64, generator=g, device=DEV).bfloat16()
    clean, clean_lse = c.attend(q, ints([0, n]), n, causal=False)
    q[2, 0, 5], q[4, 0, 6] = math.nan, math.inf
    out, lse = c.attend(q, ints([0, n]), n, causal=False)
    keep = [i for i in range(n) if i not in (2, 4)]
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    assert torch.isnan(out[2]).all()


def test_a_row_does_not_depend_on_the_batch():
    g = gen(12)
    lens, new = [3000, 17, 900, 0, 2048, 2500, 1100, 5000], [1, 3, 1, 1, 2, 40, 12, 7]
    c, _ = filled(lens, 2, 64, 32, g)
    q = torch.randn(sum(new), 4, 64, generator=g, device=DEV).bfloat16()
    cu = [sum(new[:i]) for i in range(9)]
    out, lse = c.attend(q, ints(cu), 40)
    for b in range(8):
        one, one_lse = c.attend(q[cu[b]:cu[b + 1]], ints([0, new[b]]), new[b], block_table=c.block_table[b:b + 1],
                                lengths=c.lengths[b:b + 1])
        assert torch.equal(one, out[cu[b]:cu[b + 1]]) and torch.equal(one_lse, lse[cu[b]:cu[b + 1]])
    again, _ = c.attend(q, ints(cu), sum(new))
    assert torch.equal(again, out)


def test_rows_behind_the_last_request_are_left():
    g = gen(13)
    c, memory = filled([500, 60], 2, 64, 64, g)
    q = torch.randn(10, 2, 64, generator=g, device=DEV).bfloat16()
    out = torch.full_like(q, 7.0)
    c.attend(q, ints([0, 2, 5]), 5, out=out)
    assert (out[5:] == 7).all() and not (out[:5] == 7).all(-1).any()


@pytest.mark.parametrize("page,n", [(16, 2), (32, 2), (16, 40), (32, 40)])
def test_missing_pages(page, n):
    """Tokens of pages that are not there are hidden, the first ones among them; a request with none is empty."""
    g = gen(18)
    c, memory = filled([2300, 100, 70], 2, 64, page, g)
    table = c.block_table.clone()
    gone = {0: [0, 1, 2, 3, 4, 5, 9, 64, 70], 1: [1], 2: list(range(5))}
    for b, cols in gone.items():
        table[b, cols] = -1
    table[0, 9] = c.n_pages
    q = torch.randn(3 * n, 2, 64, generator=g, device=DEV).bfloat16()
    cu = ints([0, n, 2 * n, 3 * n])
    out, lse = c.attend(q, cu, n, causal=False, block_table=table)
    assert c.device_status() == 5
    left = []
    for b, (k, v) in enumerate(memory):
        keep = torch.tensor([i // page not in gone[b] for i in range(k.shape[0])], device=DEV)
        left.append((k[keep], v[keep]))
    assert left[2][0].shape[0] == 0
    check(c, left, q, [n] * 3, out, lse, 0.125, False, torch.bfloat16)


@pytest.mark.parametrize("n", [1, 6, 50])
@pytest.mark.parametrize("order", [1, -1])
def test_values_of_every_size(n, order):
    """Values whose size grows or falls by 2^60 along the memory: the powers of two that keep weights
    and values in fp16's range move with them."""
    g = gen(19)
    c, _ = filled([3000], 1, 128, 64, g)
    grow = torch.exp2((torch.arange(3000, device=DEV) / 3000 * 60 - 30) * order)[:, None, None]
    k = torch.randn(3000, 1, 128, generator=g, device=DEV).bfloat16()
    v = (torch.randn(3000, 1, 128, generator=g, device=DEV) * grow).bfloat16()
    pos = torch.arange(3000, device=DEV)
    slots = (c.block_table[0, pos // 64] * 64 + pos % 64).int()
    c.append(k, v, slots)
    memory = c.read(slots, torch.float32)
    q = torch.randn(n, 1, 128, generator=g, device=DEV).bfloat16()
    out, lse = c.attend(q, ints([0, n]), n, causal=True)
    check(c, [memory], q, [n], out, lse, 128 ** -0.5, True, torch.bfloat16)


def test_bad_tables_lengths_and_query_offsets_are_reported():
    g = gen(14)
    c, memory = filled([100, 300], 1, 64, 16, g)
    q = torch.randn(4, 1, 64, generator=g, device=DEV).bfloat16()
    cu = ints([0, 2, 4])
    clean, _ = c.attend(q, cu, 2, causal=False)
    table = c.block_table.clone()
    table[0, 2], table[0, 4] = -1, c.n_pages         # 32 tokens of request 0 are not there
    out, lse = c.attend(q, cu, 2, causal=False, block_table=table)
    assert c.device_status() == 5
    keep = torch.tensor([i for i in range(100) if i // 16 not in (2, 4)], device=DEV)
    check(c, [(memory[0][0][keep], memory[0][1][keep])], q[:2], [2], out[:2], lse[:2], 0.125, False, torch.bfloat16)
    assert torch.equal(out[2:], clean[2:])
    for bad_lens in ([100, 10 ** 9], [-5, 300]):
        c.attend(q, cu, 2, lengths=ints(bad_lens))
        assert c.device_status() == 5
    for bad_cu in ([0, 2, 9], [0, 5, 2], [-3, 2, 4], [0, 4, 4]):   # the last has more rows than max_q
        c.attend(q, ints(bad_cu), 2)
        assert c.device_status() == 5
    out, _ = c.attend(q, cu, 2, causal=False)
    assert c.device_status() == 0 and torch.equal(out, clean)


@pytest.mark.parametrize("n", [4, 40])
def test_overlapping_query_ranges_stay_in_the_workspace(n):
    """cu_q that goes back makes more partial rows than there are: reported, nothing written outside."""
    g = gen(15)
    c, _ = filled([2000] * 8, 1, 64, 64, g)
    q = torch.randn(n, 1, 64, generator=g, device=DEV).bfloat16()
    c.attend(q, ints([0, n, 0, n, 0, n, 0, n, n]), n, causal=False)
    assert c.device_status() == 5


def test_offsets_past_32_bits():
    """Pages behind 4 GiB of data and slots near the end of a large cache."""
    g = gen(16)
    n_pages = 62000                                   # 64 tokens, 16 heads: 73728 bytes a page
    c = MemoryCache(n_pages, page=64, heads=16, requests=2, max_len=300, device=DEV,
                    data=torch.empty(n_pages * 73728, dtype=torch.uint8, device=DEV))
    assert c.size_bytes > 2 ** 32
    pages = [[n_pages - 1, 3, 61000, 59000, n_pages - 2], [0, 40000, 1]]
    memory = []
    for b, (n, mine) in enumerate(zip((300, 150), pages)):
        c.block_table[b, :len(mine)] = ints(mine)
        c.lengths[b] = n
        pos = torch.arange(n, device=DEV)
        slots = (c.block_table[b, pos // 64] * 64 + pos % 64).int()
        k, v = rows_of((n, 16, 64), torch.bfloat16, g, "plain")
        c.append(k, v, slots)
        memory.append(c.read(slots, torch.float32))
        assert torch.equal(memory[b][0], quantised(k).float()) and torch.equal(memory[b][1], quantised(v).float())
    q = torch.randn(2, 16, 64, generator=g, device=DEV).bfloat16()
    out, lse = c.attend(q, ints([0, 1, 2]), 1)
    check(c, memory, q, [1, 1], out, lse, 0.125, True, torch.bfloat16)


def test_no_rows():
    c, _ = filled([20], 1, 64, 16, gen(17))
    none = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    c.append(none, none, empty)
    k, v = c.read(empty)
    assert k.shape == (0, 1, 64)
    out, lse = c.attend(none, ints([0, 0]), 0)
    assert out.shape == (0, 1, 64) and c.device_status() == 0


# ------------------------------------------------------------------ together

def decode(c, steps, want, q, k, v, scale):
    """A run as a server makes it: pages, store and attention of every step."""
    outs = []
    for i in range(steps):
        slots, cu = c.plan(want[i], k[i].shape[0])
        c.append(k[i], v[i], slots)
        out, lse = c.attend(q[i], cu, min(40, q[i].shape[0]), scale=scale)
        outs.append((out, lse, cu))
    return outs


def serving_inputs(seed, requests=5, steps=6, heads=2, share=2, dim=64):
    r, g = random.Random(seed), gen(seed)
    lens, want, q, k, v, new = [0] * requests, [], [], [], [], []
    for i in range(steps):
        grown = [r.randint(1, 40) if n == 0 and r.random() < 0.7 else n + 1 if n else 0 for n in lens]
        if i == 4:
            grown[1] = 0          # a request ends and its pages go to others
        new.append([max(0, b - a) for a, b in zip(lens, grown)])
        lens = grown
        want.append(ints(grown))
        total = sum(new[-1]) + 3  # padded rows behind the last request
        q.append(torch.randn(total, heads * share, dim, generator=g, device=DEV).bfloat16())
        k.append(torch.randn(total, heads, dim, generator=g, device=DEV).bfloat16())
        v.append(torch.randn(total, heads, dim, generator=g, device=DEV).bfloat16())
    return want, new, q, k, v


def test_serving_run():
    want, new, q, k, v = serving_inputs(21)
    c = MemoryCache(40, page=16, heads=2, requests=5, max_len=120, device=DEV)
    outs = decode(c, 6, want, q, k, v, 0.125)
    assert c.device_status() == 0
    held = [[] for _ in range(5)]
    for i in range(6):
        cu = outs[i][2].tolist()
        assert cu == [sum(new[i][:b]) for b in range(6)]
        for b in range(5):
            if want[i][b] == 0:
                held[b] = []
            elif new[i][b]:
                held[b].append((quantised(k[i][cu[b]:cu[b + 1]]), quantised(v[i][cu[b]:cu[b + 1]])))
        memory = [(torch.cat([x[0] for x in h]), torch.cat([x[1] for x in h])) if h else
                  (torch.zeros(0, 2, 64, device=DEV),) * 2 for h in held]
        check(c, memory, q[i], new[i], outs[i][0], outs[i][1], 0.125, True, torch.bfloat16)


def test_captured_steps_follow_their_buffers():
    """Two steps captured in graphs of their own, replayed in turn on side streams with new lengths
    and rows, against an eager cache; graphs share nothing but the cache."""
    want, new, q, k, v = serving_inputs(22)
    rows = max(x.shape[0] for x in q)
    eager = MemoryCache(40, page=16, heads=2, requests=5, max_len=120, device=DEV)
    ref = decode(eager, 6, want, q, k, v, 0.125)
    c = MemoryCache(40, page=16, heads=2, requests=5, max_len=120, device=DEV)
    pad = lambda x: torch.cat([x, x.new_zeros(rows - x.shape[0], *x.shape[1:])])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for _ in range(2):
            buf = dict(want=want[0].clone(), q=pad(q[0]), k=pad(k[0]), v=pad(v[0]))
            start = c.state.clone()
            decode(c, 1, [buf["want"]], [buf["q"]], [buf["k"]], [buf["v"]], 0.125)  # warm-up
            c.state.copy_(start)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                buf["out"] = decode(c, 1, [buf["want"]], [buf["q"]], [buf["k"]], [buf["v"]], 0.125)[0]
            graphs.append((graph, buf))
        for i in range(6):
            graph, buf = graphs[i % 2]
            for name, src in (("want", want), ("q", q), ("k", k), ("v", v)):
                buf[name].copy_(src[i] if name == "want" else pad(src[i]))
            graph.replay()
            n = sum(new[i])
            assert torch.equal(buf["out"][0][:n], ref[i][0][:n]) and torch.equal(buf["out"][1][:n], ref[i][1][:n])
            assert torch.equal(buf["out"][2], ref[i][2])
    assert c.device_status() == 0
    assert torch.equal(c.state, eager.state)


def test_large_plan_from_a_graph():
    """A step of many slots (a cluster launch) captured and replayed: prompts in, then out again."""
    r = random.Random(5)
    lens = [r.randint(1, 400) for _ in range(60)]
    c = MemoryCache(2000, page=16, heads=1, requests=60, max_len=400, device=DEV)
    plain = Pages(2000, 16, 60, c.width)
    want, n = ints(lens), sum(lens)
    assert n > 8192
    slots, cu = c.plan(want, n)          # the ordinary first call
    c.plan(ints([0] * 60), 0)
    start = c.state.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            c.plan(want, n, slots=slots, cu=cu)
        for _ in range(3):
            c.state.copy_(start)
            slots.fill_(-7)
            graph.replay()
            stream.synchronize()
            plain = Pages(2000, 16, 60, c.width)
            plain.free = start[61:61 + 2000].tolist()
            ref, ref_cu, _ = plain.plan(lens)
            assert slots.tolist() == ref and cu.tolist() == ref_cu and c.block_table.tolist() == plain.table()
    assert c.device_status() == 0


@pytest.mark.parametrize("n", [1, 20, 50])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales_and_one_row_for_all(scale, n):
    """Any finite scale; one query row expanded over the request (a row stride of zero)."""
    g = gen(24)
    c, memory = filled([900], 2, 64, 32, g)
    q = torch.randn(1, 4, 64, generator=g, device=DEV).bfloat16().expand(n, 4, 64)
    out, lse = c.attend(q, ints([0, n]), n, scale=scale, causal=True)
    check(c, memory, q, [n], out, lse, scale, True, torch.bfloat16)


def test_one_row_stored_in_many_slots():
    g = gen(25)
    c = MemoryCache(4, page=16, heads=3, head_dim=128, device=DEV)
    k = torch.randn(1, 3, 128, generator=g, device=DEV).half()
    slots = torch.randperm(64, generator=g, device=DEV)[:40].int()
    c.append(k.expand(40, 3, 128), -k.expand(40, 3, 128), slots)
    gk, gv = c.read(slots, torch.float32)
    assert torch.equal(gk, quantised(k).float().expand(40, 3, 128)) and torch.equal(gv, quantised(-k).float().expand(40, 3, 128))


def test_two_calls_at_once():
    """Attention of two streams over one cache at the same time, each with its own workspace."""
    g = gen(23)
    c, _ = filled([6000, 3000], 2, 64, 64, g)
    q = torch.randn(2, 16, 64, generator=g, device=DEV).bfloat16()
    cu = ints([0, 1, 2])
    ref, _ = c.attend(q, cu, 1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(c.attend(q, cu, 1)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
