"""Statistics of rows whose mean is large against their spread, in 64 bits: such rows are read again."""
import pytest
import torch

from structured_decision_model_gb300.microscaled import quantize

pytestmark = pytest.mark.gpu


def rows_at(kinds, rows, cols, dtype, seed):
    """Rows of all kinds of (mean, spread), in turn."""
    g = torch.Generator().manual_seed(seed)
    kinds = torch.tensor(kinds, dtype=torch.float64).repeat(-(-rows // len(kinds)), 1)[:rows]
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64) * kinds[:, 1:] + kinds[:, :1]
    return x.to(dtype).cuda()


def test_far_rows_are_the_same_shared_or_alone():
    """A row of one warp's own and one that several warps share."""
    for cols in (1000, 2048, 4096):
        x = rows_at([(20.0, 1.0), (-300.0, 0.5), (0.25, 1.0)], 2600, cols, torch.bfloat16, cols)
        many = quantize(x, stats=True)
        for n in (1, 8, 400):
            few = quantize(x[:n], stats=True)
            assert torch.equal(few.mean, many.mean[:n]) and torch.equal(few.rstd, many.rstd[:n])
