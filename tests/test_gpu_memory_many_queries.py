"""Attention over the 4-bit cache of more query rows than 2^24 in one request."""
import math

import pytest
import torch

from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300.build import build_library
from test_gpu_memory_cache import DEV, check, filled, gen, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_library()
    B.load()


@pytest.mark.parametrize("share,heads_first", [(1, False), (1, True), (3, False)])
def test_more_than_two_to_the_24_rows(share, heads_first):
    """Rows on both sides of 2^24 rows, and the last ones, are their own; every row is written."""
    g = gen(31 + share)
    n = (1 << 24) + 700
    c, memory = filled([50], 1, 64, 16, g)
    shape = (share, n, 64) if heads_first else (n, share, 64)
    q = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for part in q.view(-1).split(1 << 28):
        part.normal_(generator=g)
    q = q.transpose(0, 1) if heads_first else q
    out = torch.full((n, share, 64), math.nan, dtype=torch.bfloat16, device=DEV)
    _, lse = c.attend(q, ints([0, n]), n, causal=False, out=out)
    assert c.device_status() == 0
    assert not any(bool(torch.isnan(part).any()) for part in out.view(-1).split(1 << 28))
    third = (1 << 24) // 3
    for at in (0, third - 30, (1 << 23) - 30, (1 << 24) - 300, (1 << 24) - 30, n - 300):
        rows = slice(at, at + 300)
        check(c, memory, q[rows], [300], out[rows], lse[rows], 0.125, False, torch.bfloat16)
