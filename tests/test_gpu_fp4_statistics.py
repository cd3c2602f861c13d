"""Statistics of rows whose mean is large against their spread, or whose squares pass fp32's range, in 64 bits.

Such rows are read again: the mean of what lies behind the first mean gives the mean to its last bit, and where
that is most of the spread, they are read once more for the spread around it.
"""
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


KINDS = [(1e5, 0.0), (1.1e19, 0.0), (1e19, 1e17), (-2e18, 3e15), (-7.7e3, 0.0), (3e18, 1e18), (0.25, 1.0), (2e5, 1.0)]


def check_statistics(x, mean, rstd):
    v = x.double()
    want = v.mean(1)
    apart = (v - want[:, None]).abs().mean(1)
    # near zero (second column): the sum itself, 42 roundings of the sizes' mean; far from it the mean is corrected by what
    # it left over: its own rounding, and 44 of the distances' mean
    near = want.square() <= 2 * (v - want[:, None]).square().mean(1)
    tol = torch.where(near, 42 * 2.0 ** -24 * v.abs().mean(1), (1 + 2.0 ** -10) * 2.0 ** -24 * want.abs() + 44 * 2.0 ** -24 * apart)
    assert ((mean.double() - want).abs() <= tol).all()
    # the corrected mean lies within half a step of the true one, so that a variance is at least half of the mean
    # square that it is taken from: 42 roundings of the squares' sum, twice as many of the sum's square, four of the
    # rest, doubled by that half, halved by the root; the root's own and the last product 10
    var = (v - want[:, None]).square().mean(1)
    assert ((rstd.double() * (var + EPS).sqrt() - 1).abs() <= 140 * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(8, 24), (16, 200), (9, 1000), (24, 1111), (2600, 1024), (2600, 4096), (8, 16384)])
def test_rows_far_from_zero(dtype, rows, cols):
    """Half a warp, one warp and several a row."""
    x = rows_at(KINDS, rows, cols, dtype, rows + cols)
    for form in ("mxfp4", "nvfp4"):
        m = quantize(x, form, stats=True, sums=True)
        check_statistics(x, m.mean, m.rstd)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(8, 24), (8, 1000), (8, 2048)])
def test_few_rows_far_from_zero(dtype, rows, cols):
    """Rows that a layer quantises inside the product."""
    x = rows_at(KINDS, rows, cols, dtype, cols)
    for form in ("mxfp4", "nvfp4"):
        layer = Fp4Linear(torch.randn(40, cols, device="cuda"), None, form)
        _, mean, rstd = layer.normalized(x)
        check_statistics(x, mean, rstd)
        m = quantize(x, form, stats=True)
        assert torch.equal(mean, m.mean) and torch.equal(rstd, m.rstd)


def test_constant_rows():
    """Every size of a constant: no variance is left, whatever the mean's own rounding would have been."""
    for cols in (7, 200, 1000, 5000):
        sizes = torch.tensor([0.1, 3.3, 777.7, 6.5e4, 1.23e6, 9.9e8, 1.7e16, 1.9e19, 3e30], device="cuda")
        x = torch.cat([sizes, -sizes])[:, None].repeat(1, cols)
        m = quantize(x, "nvfp4", stats=True)
        assert torch.equal(m.mean, x[:, 0])
        assert ((m.rstd.double() * EPS ** 0.5 - 1).abs() <= 8 * 2.0 ** -24).all()
