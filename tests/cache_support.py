"""Plain fp64 forms of the 4-bit memory cache's operators, for the tests.

Everything here goes by the definitions in clef_cache.h: the quantiser by its formula, the
page accounts request by request in Python, attention as the textbook sum.
"""
import math

import torch

STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step


def quantised(x):
    """What rows [..., dim] stand for after a store, in fp64."""
    g = x.double().reshape(*x.shape[:-1], -1, 64)
    low, high = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    m = low.to(torch.bfloat16).double()
    s = ((high - m).clamp(min=0) / 15).to(torch.bfloat16).double()
    c = torch.where(s > 0, ((g - m) / s).round().clamp(0, 15), 0.0)
    y = s * c + m
    fine = torch.isfinite(g).all(-1, keepdim=True) & torch.isfinite((high - m).float())  # the range in fp32
    return torch.where(fine, y, math.nan).reshape(x.shape)


class Pages:
    """Page accounts, one request at a time."""

    def __init__(self, n_pages, page, requests, width):
        self.page, self.width = page, width
        self.free = list(range(n_pages - 1, -1, -1))
        self.lengths = [0] * requests
        self.held = [[] for _ in range(requests)]

    def plan(self, want):
        up = lambda n: -(-n // self.page)
        cu, slots, ran_out = [0], [], False
        for b in reversed(range(len(want))):
            while len(self.held[b]) > up(want[b]):
                self.free.append(self.held[b].pop())
        for b, n in enumerate(want):
            need = up(n) - len(self.held[b])
            if need > 0 and (ran_out or need > len(self.free)):
                ran_out = True
                gained = range(0)
            else:
                for _ in range(need):
                    self.held[b].append(self.free.pop())
                gained = range(self.lengths[b], n)
                self.lengths[b] = n
            slots += [self.held[b][p // self.page] * self.page + p % self.page for p in gained]
            cu.append(len(slots))
        return slots, cu, ran_out

    def table(self):
        return [h + [-1] * (self.width - len(h)) for h in self.held]


def attention(q, k, v, scale, causal):
    """One request: q [n, heads, dim], k and v [len, kv_heads, dim]; fp64 out and lse."""
    n, heads, dim = q.shape
    share = heads // k.shape[1]
    k, v = (x.double().repeat_interleave(share, 1) for x in (k, v))
    s = torch.einsum("nhd,lhd->hnl", q.double(), k) * scale
    if causal:
        seen = torch.arange(k.shape[0], device=q.device) <= (k.shape[0] - n + torch.arange(n, device=q.device))[:, None]
        s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if k.shape[0] else torch.full(s.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    p = torch.where(torch.isinf(s) & (s < 0), 0.0, torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None]))
    # a value that a row does not see adds nothing, whatever it is
    out = torch.einsum("hnl,lhd->nhd", p, v.nan_to_num(nan=0.0))
    bad = torch.einsum("hnl,lhd->nhd", (p > 0).double(), torch.isnan(v).double()) > 0
    return torch.where(bad, math.nan, out), lse.transpose(0, 1)


def attention_tolerance(q, k, v, scale, dtype):
    """Bound on |out - exact| and |lse - exact| of clef_cache_attend, per (query, head).

    Scores: the products of the 4-bit codes with the queries are exact and summed in fp32
    over 64 values at most twice, then scaled and shifted: with A = sum |q| 16 s and the
    shift |m sum q| <= A, at most 80 roundings (64 + scaling + shift + reference) of 2^-24,
    doubled for a matrix unit that truncates: err_s <= 160 * 2^-24 * scale * A.  A score's
    error moves every weight by that relative amount, the exponential by 2^-22 more and the
    sums over keys by the count of additions, at most 2^-24 * (len / 8 + 100).
    Output: those relative errors times max |v|, the weights' fp16 rounding (half a step,
    2^-11 relative to the weight, floored at 2^-24 of the largest) on codes centred to
    |c - 8| <= 8, so on 8 s <= max - min <= 2 max |v|, and the output's own rounding.
    Requests of many query rows instead round the values themselves to fp16, their middle
    m + 8 s and the value, half a step each of at most max |v|, and the weights on them: three
    half steps of max |v|.  The larger of the two is taken for all.
    """
    dim = q.shape[-1]
    span = (v.amax() - v.amin()).item() if v.numel() else 0.0
    reach = v.abs().amax().item() if v.numel() else 0.0
    amp = (q.double().abs().sum(-1).amax() * (k.double().abs().amax() * 2 if k.numel() else 0)).item() * abs(scale) * 2
    err_s = 160 * 2.0 ** -24 * amp
    sums = 2.0 ** -24 * (k.shape[0] / 8 + 100)
    rel = 2 * err_s + 2.0 ** -22 + sums
    out = rel * 2 * reach + max((2.0 ** -11 + 2.0 ** -20) * span, (3 * 2.0 ** -11 + 2.0 ** -20) * reach)
    return out, err_s + 2.0 ** -22 + sums + 2.0 ** -20
