"""What a row of the 4-bit cache's attention may depend on: its own request, the keys that it sees and the
weights that it gives them, and nothing else.

The bounds here are per row and group of 64 values, from the tokens that the row uses:
with p the exact softmax weights, span and reach the range and the largest magnitude of a
token's stored group, and err_s, sums as in cache_support.attention_tolerance,
  |error| <= 2 (2 err_s + 2^-22 + sums) Sum p reach             scores, exponentials, sums
           + 3 2^-11 Sum p max(span, reach)                     fp16 weights on centred codes (half a step
                                                                of p span), or weights, middles and values
                                                                (half a step of p reach each)
           + len 2^-24 Sum p max(span, reach)                   weights among fp16's subnormals: a row's
                                                                largest weight is kept at 4 and more, so the
                                                                floor of 2^-25 is 2^-27 of it, for each key,
                                                                on codes of up to 8 steps of span / 15
           + the output's own rounding.
"""
import math

import pytest
import torch

from cache_support import STEP, attention, attention_tolerance
from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300.build import build_library
from structured_decision_model_gb300.memory import MemoryCache
from test_gpu_memory_cache import DEV, filled, gen, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_library()
    B.load()


def slots_of(c, b, pos):
    return (c.block_table[b, pos // c.page] * c.page + pos % c.page).int()


def stored(k, v, page, spare=1):
    """A cache that holds one request's rows in shuffled pages, and what they stand for (fp32)."""
    n, heads, dim = k.shape
    pages = -(-n // page)
    c = MemoryCache(pages + spare, page=page, heads=heads, head_dim=dim, max_len=n, device=DEV)
    c.data.random_(0, 256, generator=gen(n))
    c.block_table[0, :pages] = torch.randperm(pages + spare, generator=gen(n + 1), device=DEV)[:pages].int()
    c.lengths.fill_(n)
    slots = slots_of(c, 0, torch.arange(n, device=DEV))
    c.append(k, v, slots)
    return c, c.read(slots, torch.float32)


def check_rows(q, k, v, out, lse, scale, causal, dtype):
    """One request: every element of `out` against fp64, within the bound above."""
    n, heads, dim = q.shape
    share, length = heads // k.shape[1], k.shape[0]
    want, want_lse = attention(q, k, v, scale, causal)
    _, lse_tol = attention_tolerance(q, k, v, scale, dtype)
    groups = v.double().reshape(length, k.shape[1], dim // 64, 64).repeat_interleave(share, 1)
    size = torch.maximum(groups.amax(-1) - groups.amin(-1), groups.abs().amax(-1))      # [len, heads, groups]
    s = torch.einsum("nhd,lhd->hnl", q.double(), k.double().repeat_interleave(share, 1)) * scale
    if causal:
        seen = torch.arange(length, device=q.device) <= (length - n + torch.arange(n, device=q.device))[:, None]
        s = s.masked_fill(~seen, -math.inf)
    p = torch.exp(s - want_lse.T[..., None])
    used = torch.einsum("hnl,lhg->nhg", p, size)
    amp = q.double().abs().sum(-1).amax().item() * k.double().abs().amax().item() * 4 * abs(scale)
    rel = 2 * (2 * 160 * 2.0 ** -24 * amp + 2.0 ** -22 + 2.0 ** -24 * (length / 8 + 100)) + 3 * 2.0 ** -11 + length * 2.0 ** -24
    bound = (rel * used).repeat_interleave(64, -1)
    bound = bound * (1 + 2 * STEP[dtype]) + (1 + 2 * STEP[dtype]) * STEP[dtype] * want.abs() + torch.finfo(dtype).tiny
    error = (out.double() - want).abs()
    assert (error <= bound).all(), (error / bound).amax()
    assert ((lse.double() - want_lse).abs() <= lse_tol + 2 ** -22 * want_lse.abs()).all()


# rows of a call for each of the two kernels: up to 32 rows (head size 128: 16) in the first
ROWS = [(1, 64), (3, 64), (20, 64), (32, 64), (33, 64), (90, 64), (4, 128), (13, 128), (16, 128), (17, 128), (70, 128)]


@pytest.mark.parametrize("jump", [12, 18, 24, 40, 90])
@pytest.mark.parametrize("n,dim", ROWS)
def test_large_values_that_a_row_gives_no_weight(n, dim, jump):
    """Tokens of values 2^jump times the others', here and there along the memory, whose scores are so low
    that their weights are zero: the rows are those of the other tokens, to their own precision."""
    g = gen(jump * 100 + n)
    length, u = 700, torch.ones(dim, device=DEV)
    u[::2] = -1
    k = torch.randn(length, 2, dim, generator=g, device=DEV)
    v = torch.randn(length, 2, dim, generator=g, device=DEV)
    far = torch.rand(length, generator=g, device=DEV) < 0.1
    far[:3] = True
    far[length - n - 2:] = False
    k[far] = -8 * u
    v[far] *= 2.0 ** jump
    q = 4 * u + torch.randn(n, 2, dim, generator=g, device=DEV)
    q, k, v = q.bfloat16(), k.bfloat16(), v.bfloat16()
    c, (gk, gv) = stored(k, v, 32)
    for causal in (False, True):
        out, lse = c.attend(q, ints([0, n]), n, causal=causal)
        check_rows(q, gk, gv, out, lse, dim ** -0.5, causal, torch.bfloat16)
    assert c.device_status() == 0


@pytest.mark.parametrize("jump", [14, 24, 40, 90])
@pytest.mark.parametrize("n,dim", [r for r in ROWS if r[0] > 1])
def test_large_values_that_a_row_does_not_see(n, dim, jump):
    """The last tokens of a causal request, of large finite values: rows that do not see them keep their
    bits, and every row is right to its own precision."""
    g = gen(jump * 100 + n + 1)
    for length in (300, n + 5):
        k = torch.randn(length, 2, dim, generator=g, device=DEV).bfloat16()
        v = torch.randn(length, 2, dim, generator=g, device=DEV).bfloat16()
        q = torch.randn(n, 2, dim, generator=g, device=DEV).bfloat16()
        clean, clean_lse = stored(k, v, 16)[0].attend(q, ints([0, n]), n)
        hidden = max(1, n // 2)
        v[length - hidden:] *= 2.0 ** jump
        c, (gk, gv) = stored(k, v, 16)
        out, lse = c.attend(q, ints([0, n]), n)
        assert torch.equal(lse, clean_lse) and torch.equal(out[:n - hidden], clean[:n - hidden])
        check_rows(q, gk, gv, out, lse, dim ** -0.5, True, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,dim", ROWS)
def test_values_of_every_size_in_any_order(n, dim, dtype):
    """Token and group sizes of 2^-40 to 2^40 (fp16: 2^-8 to 2^8) side by side, weights from even to sharp."""
    g = gen(n * 3 + dim)
    reach = 40 if dtype == torch.bfloat16 else 8
    for length, sharp in ((900, 1.0), (2600, 3.0), (n, 0.2)):
        size = torch.exp2((torch.rand(length, 2, dim // 64, 1, generator=g, device=DEV) * 2 - 1) * reach)
        k = torch.randn(length, 2, dim, generator=g, device=DEV).to(dtype)
        v = (torch.randn(length, 2, dim // 64, 64, generator=g, device=DEV) * size).reshape(length, 2, dim).to(dtype)
        q = (sharp * torch.randn(n, 4, dim, generator=g, device=DEV)).to(dtype)
        c, (gk, gv) = stored(k, v, 64)
        out, lse = c.attend(q, ints([0, n]), n)
        check_rows(q, gk, gv, out, lse, dim ** -0.5, True, dtype)
        assert c.device_status() == 0


@pytest.mark.parametrize("n,dim", ROWS)
def test_scores_that_grow_along_the_memory(n, dim):
    """Scores that rise by hundreds while the values' size falls by 2^40, and the other way round: what a row's
    weights are scaled by has to follow both."""
    g = gen(n * 5 + dim)
    length, u = 1500, torch.ones(dim, device=DEV)
    way = torch.linspace(-1, 1, length, device=DEV)[:, None, None]
    for up, values in ((1, -1), (1, 1), (-1, -1), (-1, 1)):
        k = (up * way * 6 * u + 0.3 * torch.randn(length, 1, dim, generator=g, device=DEV)).bfloat16()
        v = (torch.randn(length, 1, dim, generator=g, device=DEV) * torch.exp2(values * way * 20)).bfloat16()
        q = (4 * u + torch.randn(n, 1, dim, generator=g, device=DEV)).bfloat16()
        c, (gk, gv) = stored(k, v, 64)
        out, lse = c.attend(q, ints([0, n]), n, causal=False)
        check_rows(q, gk, gv, out, lse, dim ** -0.5, False, torch.bfloat16)


@pytest.mark.parametrize("n,dim", [(3, 64), (40, 64), (3, 128), (40, 128)])
def test_values_near_the_ends_of_the_range(n, dim):
    """Values of 2^-120 and of 2^108, constant groups and zeros among them."""
    g = gen(n + dim)
    for size in (2.0 ** -120, 2.0 ** 108):
        k = torch.randn(200, 1, dim, generator=g, device=DEV).bfloat16()
        v = torch.randn(200, 1, dim, generator=g, device=DEV) * size
        v[5], v[17], v[90:120] = 0, size, 0.5 * size
        v = v.bfloat16()
        q = torch.randn(n, 1, dim, generator=g, device=DEV).bfloat16()
        c, (gk, gv) = stored(k, v, 16)
        out, lse = c.attend(q, ints([0, n]), n)
        check_rows(q, gk, gv, out, lse, dim ** -0.5, True, torch.bfloat16)


@pytest.mark.parametrize("heads,length", [(2, 8300), (2, 12000), (2, 16384), (8, 20000), (2, 5000), (2, 17500), (1, 70000)])
@pytest.mark.parametrize("n,dim", [(1, 64), (2, 128), (40, 64), (20, 128)])
def test_a_row_does_not_depend_on_the_width_of_the_table(heads, length, n, dim):
    """The same request under tables of different widths, and beside a longer one: bit for bit the same."""
    g = gen(length + n)
    c, _ = filled([length, 300], heads, dim, 64, g)
    q = torch.randn(n + 1, heads, dim, generator=g, device=DEV).bfloat16()
    out, lse = c.attend(q, ints([0, n, n + 1]), n)
    for pages in (c.width + 1, 20 * 1024 // 64, 64 * 1024 // 64, 200 * 1024 // 64):
        if pages > c.width:
            wide = torch.cat([c.block_table, c.block_table.new_full((2, pages - c.width), -1)], 1)
            again, again_lse = c.attend(q, ints([0, n, n + 1]), n, block_table=wide)
            assert torch.equal(again, out) and torch.equal(again_lse, lse)
    assert c.device_status() == 0


@pytest.mark.parametrize("n,dim", ROWS)
def test_zero_values_that_take_the_reference(n, dim):
    """A run of zero values (no size at all) outweighs what came before; what comes after has its weight and is
    2^30 times smaller than the first tokens: it is all that the rows are made of."""
    g = gen(n * 7 + dim)
    length, u = 900, torch.ones(dim, device=DEV)
    for score in (30.0, 80.0):
        k = 0.1 * torch.randn(length, 2, dim, generator=g, device=DEV)
        k[300:] += score * dim ** 0.5 / (4 * dim) * u
        v = torch.randn(length, 2, dim, generator=g, device=DEV)
        v[300:600] = 0
        v[600:] *= 2.0 ** -30
        q = (4 * u + 0.1 * torch.randn(n, 2, dim, generator=g, device=DEV)).bfloat16()
        c, (gk, gv) = stored(k.bfloat16(), v.bfloat16(), 32)
        out, lse = c.attend(q, ints([0, n]), n, causal=False)
        check_rows(q, gk, gv, out, lse, dim ** -0.5, False, torch.bfloat16)


# ---- fp16: the output keeps 11 bits, so what comes before it is held to more

FINE = [(1, 64), (8, 64), (20, 64), (32, 64), (33, 64), (90, 64), (4, 128), (8, 128), (16, 128), (17, 128), (70, 128)]


@pytest.mark.parametrize("n,dim", FINE)
@pytest.mark.parametrize("length", [2, 7, 40, 300, 2500])
def test_fp16_rows_are_exact_up_to_their_rounding(n, dim, length):
    """Nearly even weights (small queries, so that the scores' own error is small: 160 x 2^-24 of their size).
    Before the output's rounding: weights in two fp16 parts (2^-22 of p span, the second part's floor
    len 2^-27), scores, exponentials and sums as at the top of this file."""
    g = gen(n * 11 + dim + length)
    k = torch.randn(length, 2, dim, generator=g, device=DEV).half()
    v = (torch.randn(length, 2, dim, generator=g, device=DEV) * torch.exp(torch.randn(length, 1, 1, generator=g, device=DEV))).half()
    q = (0.002 * torch.randn(n, 4, dim, generator=g, device=DEV)).half()
    c, (gk, gv) = stored(k, v, 16)
    scale = dim ** -0.5
    out, _ = c.attend(q, ints([0, n]), n, causal=False)
    want, want_lse = attention(q, gk, gv, scale, False)
    groups = gv.double().reshape(length, 2, dim // 64, 64).repeat_interleave(2, 1)
    size = torch.maximum(groups.amax(-1) - groups.amin(-1), groups.abs().amax(-1))
    s = torch.einsum("nhd,lhd->hnl", q.double(), gk.double().repeat_interleave(2, 1)) * scale
    used = torch.einsum("hnl,lhg->nhg", torch.exp(s - want_lse.T[..., None]), size).repeat_interleave(64, -1)
    amp = q.double().abs().sum(-1).amax().item() * gk.double().abs().amax().item() * 4 * scale
    rel = 2 * (2 * 160 * 2.0 ** -24 * amp + 2.0 ** -22 + 2.0 ** -24 * (length / 8 + 100)) + 2.0 ** -22 + length * 2.0 ** -27
    bound = rel * used * (1 + 2.0 ** -10) + 2.0 ** -11 * want.abs() * (1 + 2.0 ** -10) + 2.0 ** -25
    error = (out.double() - want).abs()
    assert (error <= bound).all(), (error / bound).amax()


@pytest.mark.parametrize("n,dim", FINE)
def test_fp16_rows_have_the_error_of_their_rounding(n, dim):
    """Ordinary scores: the mean square error is that of rounding the exact result once (errors in front of it
    that are a fraction r of it raise its root by r^2 / 2; 5 % allows r = 0.3, and 2^-22 is 2^-10 of it)."""
    g = gen(n * 13 + dim)
    k = torch.randn(2500, 2, dim, generator=g, device=DEV).half()
    v = (torch.randn(2500, 2, dim, generator=g, device=DEV) * torch.exp(0.4 * torch.randn(2500, 1, 1, generator=g, device=DEV))).half()
    q = torch.randn(n, 4, dim, generator=g, device=DEV).half()
    c, (gk, gv) = stored(k, v, 64)
    out, _ = c.attend(q, ints([0, n]), n)
    want, _ = attention(q, gk, gv, dim ** -0.5, True)
    rms = lambda x: x.square().mean().sqrt().item()
    assert rms(out.double() - want) <= 1.05 * rms(want.half().double() - want)


@pytest.mark.parametrize("n,share", [(1, 8), (1, 1), (2, 8), (8, 8)])
def test_fp16_rows_of_a_long_memory_have_the_error_of_their_rounding(n, share):
    """The mean of 100000 values is far smaller than they are: errors of one sign would show."""
    g = gen(n * 17 + share)
    k = torch.randn(100003, 2, 64, generator=g, device=DEV).half()
    v = torch.randn(100003, 2, 64, generator=g, device=DEV).half()
    q = torch.randn(n, 2 * share, 64, generator=g, device=DEV).half()
    c, (gk, gv) = stored(k, v, 64)
    out, _ = c.attend(q, ints([0, n]), n)
    want, _ = attention(q, gk, gv, 0.125, True)
    rms = lambda x: x.square().mean().sqrt().item()
    assert rms(out.double() - want) <= 1.05 * rms(want.half().double() - want)


@pytest.mark.parametrize("jump", [18, 40, 120])
@pytest.mark.parametrize("n,dim", ROWS)
def test_fp16_rows_beside_large_values(n, dim, jump):
    """fp16 queries over a memory stored in bf16: tokens of no weight and tokens that a row does not see are 2^jump
    times larger than the others (past fp16), or no numbers."""
    g = gen(jump * 10 + n + dim)
    length, u = 700, torch.ones(dim, device=DEV)
    u[::2] = -1
    k = torch.randn(length, 2, dim, generator=g, device=DEV)
    v = torch.randn(length, 2, dim, generator=g, device=DEV)
    far = torch.rand(length, generator=g, device=DEV) < 0.1
    far[:3] = True
    far[length - n - 2:] = False
    k[far] = -8 * u
    v[far] *= 2.0 ** jump
    q = (4 * u + torch.randn(n, 2, dim, generator=g, device=DEV)).half()
    k, v = k.bfloat16(), v.bfloat16()
    c, (gk, gv) = stored(k, v, 32)
    out, lse = c.attend(q, ints([0, n]), n)
    check_rows(q, gk, gv, out, lse, dim ** -0.5, True, torch.float16)
    hidden = n // 2                               # the last tokens: rows before them keep their bits
    for value in (2.0 ** jump, math.nan):
        if hidden:
            v[length - hidden:] = value * torch.randn(hidden, 2, dim, generator=g, device=DEV).bfloat16()
            c.append(k[length - hidden:], v[length - hidden:], slots_of(c, 0, torch.arange(length - hidden, length, device=DEV)))
            again, again_lse = c.attend(q, ints([0, n]), n)
            assert torch.equal(again[:n - hidden], out[:n - hidden]) and torch.equal(again_lse, lse)
    if hidden:
        assert torch.isnan(again[n - hidden:]).all()
    assert c.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,dim", [(2, 64), (40, 64), (2, 128), (40, 128)])
def test_half_of_a_value_that_is_no_number(n, dim, dtype):
    """A group of 64 values that is no number stays alone, and missing pages hide their tokens, in both types."""
    g = gen(n + dim)
    k = torch.randn(2100, 1, dim, generator=g, device=DEV).to(dtype)
    v = torch.randn(2100, 1, dim, generator=g, device=DEV).to(dtype)
    q = torch.randn(n, 1, dim, generator=g, device=DEV).to(dtype)
    c, (gk, gv) = stored(k, v, 32)
    clean, _ = c.attend(q, ints([0, n]), n, causal=False)
    check_rows(q, gk, gv, clean, _, dim ** -0.5, False, dtype)
    v[7, :, :64] = math.nan
    c.append(k[7:8], v[7:8], slots_of(c, 0, torch.tensor([7], device=DEV)))
    out, lse = c.attend(q, ints([0, n]), n, causal=False)
    assert torch.isnan(out[..., :64]).all() and torch.equal(out[..., 64:], clean[..., 64:]) and not torch.isnan(lse).any()
    table = c.block_table.clone()
    table[0, 0] = -1                              # the token is hidden with its page
    out, lse = c.attend(q, ints([0, n]), n, causal=False, block_table=table)
    assert c.device_status() == 5
    check_rows(q, gk[32:], gv[32:], out, lse, dim ** -0.5, False, dtype)
