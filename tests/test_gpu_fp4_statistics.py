"""Statistics of rows whose mean is large against their spread, or whose squares pass fp32's range, in 64 bits.

Such rows are read again."""
import pytest
import torch

from structured_decision_model_gb300.microscaled import Fp4Linear, quantize

pytestmark = pytest.mark.gpu

EPS = 1e-5


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


PAST = [(1e19, 1e17), (-3e18, 1e18), (2e17, 5e16), (0.25, 1.0)]


def check_past(x, mean, rstd):
    v = x.double()
    want = v.mean(1)
    # 42 roundings of a sum, of the sizes' mean
    off = 42 * 2.0 ** -24 * v.abs().mean(1)
    assert ((mean.double() - want).abs() <= off).all()
    # the same for the squares' sum (each rounded three times), halved by the root, whose own and the last product round too;
    # the mean's error enters squared
    var = (v - want[:, None]).square().mean(1)
    assert ((rstd.double() * (var + EPS).sqrt() - 1).abs() <= 30 * 2.0 ** -24 + off.square() / var).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(8, 24), (16, 200), (9, 1000), (24, 1111), (2600, 1024), (2600, 4096), (8, 16384)])
def test_rows_whose_squares_pass_fp32(dtype, rows, cols):
    """Half a warp, one warp and several a row."""
    x = rows_at(PAST, rows, cols, dtype, rows + cols)
    for form in ("mxfp4", "nvfp4"):
        m = quantize(x, form, stats=True, sums=True)
        check_past(x, m.mean, m.rstd)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(8, 24), (8, 1000), (8, 2048)])
def test_few_rows_whose_squares_pass_fp32(dtype, rows, cols):
    """Rows that a layer quantises inside the product."""
    x = rows_at(PAST, rows, cols, dtype, cols)
    for form in ("mxfp4", "nvfp4"):
        _, mean, rstd = Fp4Linear(torch.randn(40, cols, device="cuda"), None, form).normalized(x)
        check_past(x, mean, rstd)
        m = quantize(x, form, stats=True)
        assert torch.equal(mean, m.mean) and torch.equal(rstd, m.rstd)
