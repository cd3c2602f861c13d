"""The microscaled 4-bit operators on the GPU against their definition in 64 bits."""
import numpy as np
import pytest
import torch

from fp4_support import BLOCK, EPS, kept, stored
from structured_decision_model_gb300.binding import ClefError
from structured_decision_model_gb300.microscaled import Fp4Linear, Fp4Matrix, product, quantize

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FORMATS = ["mxfp4", "nvfp4"]


def rows_of(rows, cols, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))
    x *= torch.exp(spread * torch.randn(rows, cols, generator=g))
    return x.to(dtype).cuda()


def check_kept(x, form, m):
    codes, byte, r, values = kept(x.double().cpu().numpy(), form)
    got, scales, row_scale = stored(m)
    cols, blocks = x.shape[1], byte.shape[1]
    np.testing.assert_array_equal(scales[:, :blocks], byte)
    assert not scales[:, blocks:].any()
    # a value of zero may carry either sign
    same = (got[:, :cols] == codes) | ((got[:, :cols] & 7) + (codes & 7) == 0)
    assert same.all(), np.argwhere(~same)[:5]
    assert not got[:, cols:].any()
    if form == "nvfp4":
        np.testing.assert_array_equal(row_scale, r.astype(np.float32))
    return values


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 33), (130, 256), (5, 300), (64, 1111), (300, 4096), (7, 8192),
                                       (2, 16384), (1, 5121)])
def test_rows_are_kept_exactly(form, dtype, rows, cols):
    x = rows_of(rows, cols, TYPES[dtype], rows * 7 + cols)
    m = quantize(x, form)
    values = check_kept(x, form, m)
    for out in TYPES.values():
        want = torch.from_numpy(values).to(torch.float32).to(out)  # fp32 holds every value
        assert torch.equal(m.dequantize(out).cpu(), want)


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_quotients_next_to_the_borders(form, dtype):
    """Every midpoint times scales of every size, and the numbers of the type next to it on both sides."""
    t = TYPES[dtype]
    n = BLOCK[form]
    out = []
    for top in (6.0, 5.25, 4.125, 6.75, 3.1875, 7.5):
        for power in (-9, -3, 0, 5):
            head = torch.tensor([top * 2.0 ** power], dtype=t)
            scale = kept(head[None].double().numpy(), form)[3][0, 0]  # what the largest stands for
            scale = scale / 6 if form == "nvfp4" else 2.0 ** np.floor(np.log2(top * 2.0 ** power)) / 4
            mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64) * scale
            mids = mids.to(t)
            inf = torch.tensor(float("inf"), dtype=t)
            near = torch.cat([mids, torch.nextafter(mids.cuda(), inf.cuda()).cpu() if t == torch.float32 else mids * (1 + 2.0 ** -7),
                              torch.nextafter(mids.cuda(), -inf.cuda()).cpu() if t == torch.float32 else mids * (1 - 2.0 ** -7)])
            for a in range(0, len(near), n - 1):
                block = torch.zeros(n, dtype=t)
                block[0] = head[0]
                part = near[a:a + n - 1].clamp(max=float(head[0]))
                block[1:1 + len(part)] = part
                out.append(block)
                out.append(-block)
    x = torch.cat(out)
    x = torch.nn.functional.pad(x, (0, -len(x) % (4 * n))).view(-1, 4 * n).cuda()
    check_kept(x, form, quantize(x, form))


@pytest.mark.parametrize("form", FORMATS)
def test_sizes_at_the_ends_of_fp32(form):
    x = torch.tensor([[1e-38, -3e-40, 0, 5e-39] * 16, [3e38, 1, 1e30, -2e38] * 16, [0.0] * 64, [1e-45, 0, -1e-44, 0] * 16,
                      [-0.0] * 64, [2.0 ** 127, 2.0 ** 115, -2.0 ** 110, 2.0 ** 100] * 16], dtype=torch.float32, device="cuda")
    check_kept(x, form, quantize(x, form))
    y = x.bfloat16()
    check_kept(y, form, quantize(y, form))


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_no_numbers_stay_in_their_block(form, dtype):
    x = rows_of(5, 200, TYPES[dtype], 3)
    x[0, 17], x[1, 40], x[1, 199], x[3, 0] = float("nan"), float("inf"), float("-inf"), float("nan")
    m = quantize(x, form)
    values = check_kept(x, form, m)
    back = m.dequantize(torch.float32).cpu().double().numpy()
    np.testing.assert_array_equal(back, values)
    assert np.isnan(back[0]).sum() == BLOCK[form] and not np.isnan(back[2]).any() and not np.isnan(back[4]).any()


def test_strided_and_unaligned_rows():
    base = rows_of(40, 700, torch.bfloat16, 4)
    for x in (base[:, 1:301], base[::3, :256], base[:, 8:264], base[:1].expand(6, 700)):
        check_kept(x, "nvfp4", quantize(x, "nvfp4"))
    m = quantize(base, "mxfp4")
    wide = torch.full((40, 801), 7.0, dtype=torch.float16, device="cuda")
    m.dequantize(torch.float16, wide[:, 3:703])
    assert torch.equal(wide[:, 3:703], m.dequantize(torch.float16))
    assert (wide[:, :3] == 7).all() and (wide[:, 703:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (9, 1000), (300, 4096), (2, 16384)])
def test_statistics_and_sums(dtype, rows, cols):
    x = rows_of(rows, cols, TYPES[dtype], 5, spread=0.3) + 2.0
    m = quantize(x, "nvfp4", stats=True, sums=True)
    v = x.double()
    mean = v.mean(1)
    var = (v - mean[:, None]).square().mean(1)
    size = v.abs().mean(1)
    # fp32 sums in a tree of at most 2^5 terms in line and 10 levels: 42 roundings of 2^-24, of the sizes' mean
    assert ((m.mean.double() - mean).abs() <= 42 * 2.0 ** -24 * size).all()
    # the same for the variance (each term rounded three times), halved by the root, the root and the quotient
    # rounded once each; the mean's own error enters squared
    assert ((m.rstd.double() * (var + EPS).sqrt() - 1).abs() <= 30 * 2.0 ** -24).all()
    kept_rows = m.dequantize(torch.float32).double()
    assert ((m.sums.double() - kept_rows.sum(1)).abs() <= 42 * 2.0 ** -24 * kept_rows.abs().sum(1)).all()


def check_product(x, w, form, out, bias=None, normalized=False, y=None):
    """The product against 64 bits of what both sides stand for."""
    a, b = (torch.from_numpy(kept(t.double().cpu().numpy(), form)[3]).cuda() for t in (x, w))
    want = a @ b.T
    room = a.abs() @ b.abs().T  # the sum of the terms' sizes
    if normalized:
        v = x.double()
        mean = v.mean(1, keepdim=True)
        rstd = ((v - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
        shift = mean * b.sum(1)
        want = rstd * (want - shift)
        room = rstd * (room + v.abs().mean(1, keepdim=True) * b.abs().sum(1))
    if bias is not None:
        want = want + bias.double()
        room = room + bias.double().abs()
    # sums in fp32 on the tensor cores, which may cut off instead of rounding: 2^-23 of the terms' sizes for each MMA
    # of 64 columns; 50 roundings of 2^-24 for statistics, sums, factors and joined parts; the output's own
    steps = -(-x.shape[1] // 64)
    tol = room * (steps * 2.0 ** -23 + 50 * 2.0 ** -24) + want.abs() * torch.finfo(out).eps / 2
    tol = tol + torch.finfo(out).tiny
    off = (y.double() - want).abs()
    assert (off <= tol).all(), (float((off / tol).max()), int((off > tol).sum()))


SHAPES = [(1, 1, 1), (1, 128, 256), (3, 40, 32), (32, 256, 512), (33, 129, 300), (64, 512, 4096), (65, 700, 1000),
          (128, 128, 64), (200, 384, 5000), (511, 1024, 1024), (1000, 777, 515)]


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(form, out, m, n, k):
    x = rows_of(m, k, torch.bfloat16, m + n, 0.5)
    w = rows_of(n, k, torch.bfloat16, m + k, 0.5)
    bias = torch.randn(n, device="cuda") * 3
    layer = Fp4Linear(w, bias, form)
    y = layer(x, TYPES[out])
    check_product(x, w, form, TYPES[out], bias, y=y)
    assert layer.device_status() == 0


# more 128 x 128 tiles than two an SM (one, where K is long): CTA pairs; odd widths, ragged K, short last tiles
PAIR_SHAPES = [(5000, 1100, 260), (4000, 1363, 1000), (1400, 1810, 4200), (40000, 24, 64)]


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("m,n,k", PAIR_SHAPES)
def test_product_by_pairs(form, out, m, n, k):
    x, w = rows_of(m, k, torch.bfloat16, m, 0.5), rows_of(n, k, torch.bfloat16, k, 0.5)
    bias = torch.randn(n, device="cuda") * 3
    layer = Fp4Linear(w, bias, form)
    check_product(x, w, form, TYPES[out], bias, y=layer(x, TYPES[out]))
    if out != "fp16":
        x = x + 0.5
        check_product(x, w, form, TYPES[out], bias, True, layer.normalized(x, TYPES[out])[0])
    assert layer.device_status() == 0


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_normalized_product(form, m, n, k):
    x = rows_of(m, k, torch.float16, m + n, 0.3) + 0.5
    w = rows_of(n, k, torch.bfloat16, m + k, 0.5)
    layer = Fp4Linear(w, None, form)
    y, mean, rstd = layer.normalized(x, torch.float32)
    check_product(x, w, form, torch.float32, None, True, y)
    m_ = quantize(x, form, stats=True)
    assert torch.equal(m_.mean, mean) and torch.equal(m_.rstd, rstd)


# ------------------------------------------------- what a serving program meets

@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("m", [3, 70, 600])
def test_rows_of_no_numbers_stay_by_themselves(form, m):
    """NaN and infinity in a row of x, or of w, make that row's (column's) outputs NaN and no others."""
    x, w = rows_of(m, 300, torch.bfloat16, 1, 0.3), rows_of(140, 300, torch.bfloat16, 2, 0.3)
    clean = Fp4Linear(w, None, form)(x, torch.float32)
    x2, w2 = x.clone(), w.clone()
    x2[1, 299], w2[139, 0], w2[5, 77] = float("nan"), float("inf"), float("-inf")
    y = Fp4Linear(w2, None, form)(x2, torch.float32)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1], bad[:, 139], bad[:, 5] = True, True, True
    assert y[bad].isnan().all()
    # the other values of a row that holds one keep their scales, so the other outputs are as they were
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m", [1, 40, 100, 700])
def test_outputs_stay_inside_their_rows(dtype, m):
    """Row strides of every alignment; what lies between the rows and behind the last is left as it was."""
    t = TYPES[dtype]
    x, w = quantize(rows_of(m, 200, torch.bfloat16, 3), "nvfp4"), quantize(rows_of(131, 200, torch.bfloat16, 4), "nvfp4")
    want = product(x, w, None, t)
    for stride, first in ((131, 0), (132, 0), (136, 0), (137, 3), (144, 8), (140, 2)):
        wide = torch.full((m + 2, stride), 9.0, dtype=t, device="cuda")
        out = wide.view(-1)[first:first + m * stride].view(m, stride)[:, :131]
        assert torch.equal(product(x, w, None, t, out=out), want)
        left = wide.clone()
        left.view(-1)[first:first + m * stride].view(m, stride)[:, :131] = 9.0
        assert (left == 9).all()


@pytest.mark.parametrize("n", [136, 24, 131])
def test_outputs_of_many_rows_stay_inside_theirs(n):
    """The same of the pair kernel, whose outputs TMA stores where rows start and end on 16 bytes."""
    m = 40100
    x, w = quantize(rows_of(m, 64, torch.bfloat16, 3)), quantize(rows_of(n, 64, torch.bfloat16, 4))
    want = x.dequantize(torch.float32) @ w.dequantize(torch.float32).T  # 64 products of 8 bits each: exact but for the sum
    for t in (torch.bfloat16, torch.float32):
        y = product(x, w, None, t)
        assert ((y.float() - want).abs() <= want.abs() * (torch.finfo(t).eps / 2) + 2.0 ** -20 * want.abs().amax(1, keepdim=True)).all()
        for stride, first in ((n, 0), (n + 8, 8), (n + 16, 0), (n + 1, 3), (n + 2, 2)):
            wide = torch.full((m + 2, stride), 9.0, dtype=t, device="cuda")
            out = wide.view(-1)[first:first + m * stride].view(m, stride)[:, :n]
            assert torch.equal(product(x, w, None, t, out=out), y)
            wide.view(-1)[first:first + m * stride].view(m, stride)[:, :n] = 9.0
            assert (wide == 9).all()


def test_a_row_depends_on_itself_alone():
    """The same row among others of any size: equal codes, and equal outputs in calls of one shape."""
    x = rows_of(300, 1000, torch.bfloat16, 5)
    layer = Fp4Linear(rows_of(256, 1000, torch.bfloat16, 6))
    y = layer(x)
    x2 = x.clone()
    x2[1:] *= 1e20
    assert torch.equal(layer(x2)[0], y[0])


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("cols", [8, 24, 32, 104, 256])
def test_many_short_rows(form, cols):
    """Two rows a warp going in, eights of any rows coming back; the last warp is part full."""
    x = rows_of(1003, cols, torch.bfloat16, cols)
    m = quantize(x, form, stats=True)
    values = check_kept(x, form, m)
    assert torch.equal(m.dequantize(torch.float32).cpu(), torch.from_numpy(values).float())
    wide = torch.full((1003, cols + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    m.dequantize(torch.bfloat16, wide[:, :cols])
    assert torch.equal(wide[:, :cols], m.dequantize()) and (wide[:, cols:] == 5).all()
    v = x.double()
    mean = v.mean(1)
    assert ((m.mean.double() - mean).abs() <= 42 * 2.0 ** -24 * v.abs().mean(1)).all()
    var = (v - mean[:, None]).square().mean(1)
    assert ((m.rstd.double() * (var + EPS).sqrt() - 1).abs() <= 30 * 2.0 ** -24).all()


@pytest.mark.parametrize("rows,cols", [(4, 100), (3, 1000), (2500, 4096), (2, 8192)])
def test_rows_far_from_zero_keep_their_spread(rows, cols):
    """Means from none to 2000 times the spread, side by side, and rows whose squares pass fp32."""
    x = rows_of(rows, cols, torch.float32, 11, 0.2)
    x += torch.tensor([0.0, 2000.0, -30.0, 1.5], device="cuda").repeat(rows)[:rows, None]
    m = quantize(x, "nvfp4", stats=True)
    v = x.double()
    mean = v.mean(1)
    var = (v - mean[:, None]).square().mean(1)
    assert ((m.mean.double() - mean).abs() <= 42 * 2.0 ** -24 * v.abs().mean(1)).all()
    # the mean's own rounding (half a step of 2000) comes in squared, against a spread of about 1
    assert ((m.rstd.double() * (var + EPS).sqrt() - 1).abs() <= 30 * 2.0 ** -24 + (42 * 2.0 ** -24 * 2000) ** 2).all()
    y = quantize(x * 1e30, "nvfp4", stats=True)
    assert (y.rstd == 0).all()


def test_statistics_do_not_depend_on_the_number_of_rows():
    """Few rows are shared among more warps than many: the same sums in the same order."""
    for cols in (1000, 4096, 16384):
        x = rows_of(2600, cols, torch.bfloat16, cols, 0.3) + 0.25
        many = quantize(x, stats=True, sums=True)
        for n in (1, 7, 400):
            few = quantize(x[:n], stats=True, sums=True)
            for a, b in ((few.mean, many.mean), (few.rstd, many.rstd), (few.sums, many.sums)):
                assert torch.equal(a, b[:n])


@pytest.mark.parametrize("form", FORMATS)
def test_statistics_and_sums_at_once_are_those_apart(form):
    for rows, cols, dtype in ((5, 200, torch.bfloat16), (300, 1111, torch.float32), (4000, 4096, torch.bfloat16), (40, 9000, torch.float16)):
        x = rows_of(rows, cols, dtype, rows, 0.5)
        x[::3] += 20  # their squares' sum tells nothing of the spread: read once more
        plain, both = quantize(x, form), quantize(x, form, stats=True, sums=True)
        stats, sums = quantize(x, form, stats=True), quantize(x, form, sums=True)
        assert torch.equal(both.mean, stats.mean) and torch.equal(both.rstd, stats.rstd)
        assert torch.equal(both.sums, sums.sums) and sums.mean is None and stats.sums is None
        for other in (both, stats, sums):
            assert torch.equal(other.dequantize(dtype), plain.dequantize(dtype))


def test_more_tiles_than_the_card_holds():
    """Pairs of CTAs walk several tiles of 256 x 256: the accumulators in turn, each output type."""
    x, w = quantize(rows_of(3000, 512, torch.bfloat16, 1, 0.3)), quantize(rows_of(4104, 512, torch.bfloat16, 2, 0.3))
    a, b = x.dequantize(torch.float32).double(), w.dequantize(torch.float32).double()
    want, room = a @ b.T, a.abs() @ b.abs().T
    for out in TYPES.values():
        off = (product(x, w, None, out).double() - want).abs()
        # as in check_product: 8 MMAs, 50 roundings, the output's own
        assert (off <= room * (8 * 2.0 ** -23 + 50 * 2.0 ** -24) + want.abs() * torch.finfo(out).eps / 2).all()


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("m,n", [(4900, 4104), (5003, 4096), (4097, 4099), (20000, 300)])
def test_last_round_of_tiles(form, m, n):
    """Tile counts that leave most pairs of CTAs, or few, without a tile in the last round, with ragged rows and columns:
    each output type, plain and with the normalisation's terms."""
    x, w = quantize(rows_of(m, 320, torch.bfloat16, 1, 0.3), form, stats=True), quantize(rows_of(n, 320, torch.bfloat16, 2, 0.3), form, sums=True)
    a, b = x.dequantize(torch.float32).double(), w.dequantize(torch.float32).double()
    want, room = a @ b.T, a.abs() @ b.abs().T
    bias = torch.randn(n, device="cuda")
    folded = x.rstd.double()[:, None] * (want - x.mean.double()[:, None] * b.sum(1)) + bias
    folded_room = x.rstd.double()[:, None] * (room + x.mean.double().abs()[:, None] * b.abs().sum(1)) + bias.abs()
    for out in TYPES.values():
        # as in check_product: 5 MMAs, 50 roundings, the output's own
        steps = 5 * 2.0 ** -23 + 50 * 2.0 ** -24
        off = (product(x, w, None, out).double() - want).abs()
        assert (off <= room * steps + want.abs() * torch.finfo(out).eps / 2).all()
        off = (product(x, w, bias, out, normalized=True).double() - folded).abs()
        assert (off <= folded_room * steps + folded.abs() * torch.finfo(out).eps / 2).all()


def test_long_rows_and_many_tiles():
    for m, n, k in ((1, 300, 16384), (300, 260, 8200), (2100, 1100, 260)):
        x, w = rows_of(m, k, torch.bfloat16, m, 0.5), rows_of(n, k, torch.bfloat16, n, 0.5)
        check_product(x, w, "nvfp4", torch.bfloat16, y=Fp4Linear(w)(x))
        check_product(x, w, "mxfp4", torch.float32, y=Fp4Linear(w, None, "mxfp4")(x, torch.float32))


def test_values_of_any_size():
    """Rows and weights far from 1: the row scales keep both inside e4m3's range."""
    for power in (-100, -30, 60):
        x = rows_of(40, 512, torch.float32, 8, 0.5) * 2.0 ** power
        w = rows_of(200, 512, torch.float32, 9, 0.5) * 2.0 ** -power
        for form in FORMATS:
            check_product(x, w, form, torch.float32, y=Fp4Linear(w, None, form)(x))


def test_the_smallest_scales():
    """Values around 2^-126: mxfp4's least scale is 2^-127 (a byte of 0), nvfp4's rows are held by their row scale."""
    x = torch.tensor([1.5 * 2.0 ** -126, -2.0 ** -126, 2.0 ** -125, 0.0] * 64, device="cuda").repeat(20, 1)
    w = rows_of(130, 256, torch.float32, 9, 0.5) * 2.0 ** 100
    for form in FORMATS:
        y = Fp4Linear(w, None, form)(x)
        # 256 products and their sum lie near 2^-24: compared at 1
        a, b = (torch.from_numpy(kept(t.double().cpu().numpy(), form)[3]).cuda() for t in (x, w))
        want, room = a @ b.T, a.abs() @ b.abs().T
        assert ((y.double() - want).abs() <= room * (4 * 2.0 ** -23 + 50 * 2.0 ** -24)).all()


def test_leading_dimensions_and_empty_batches():
    layer = Fp4Linear(rows_of(96, 160, torch.bfloat16, 1), torch.randn(96, device="cuda"))
    x = rows_of(24, 160, torch.bfloat16, 2)
    y = layer(x)
    assert torch.equal(layer(x.view(2, 3, 4, 160)), y.view(2, 3, 4, 96))
    assert torch.equal(layer(x[0]), layer(x[:1])[0])
    assert torch.equal(layer(x.t().contiguous().t()), y)
    assert torch.equal(layer(torch.cat([x, x], 1)[:, :160]), y)
    a, mean, rstd = layer.normalized(x.view(2, 12, 160))
    assert a.shape == (2, 12, 96) and mean.shape == rstd.shape == (2, 12)
    assert layer(x[:0]).shape == (0, 96)
    a, mean, rstd = layer.normalized(x[:0])
    assert a.shape == (0, 96) and mean.shape == rstd.shape == (0,)


def test_one_row_for_all_and_a_matrix_with_itself():
    layer = Fp4Linear(rows_of(96, 160, torch.bfloat16, 1))
    x = rows_of(1, 160, torch.bfloat16, 2)
    for n in (5, 40, 900):
        assert torch.equal(layer(x.expand(n, 160)), layer(x.expand(n, 160).contiguous()))
    check_product(x.expand(5, 160), x.expand(5, 160), "nvfp4", torch.float32, y=product(*[quantize(x.expand(5, 160))] * 2, None, torch.float32))


def test_the_layer_is_its_steps():
    w, bias = rows_of(520, 640, torch.bfloat16, 1), torch.randn(520, device="cuda")
    for m in (1, 64, 300):
        x = rows_of(m, 640, torch.float16, m)
        layer = Fp4Linear(w, bias, "mxfp4")
        q = quantize(x, "mxfp4", stats=True)
        assert torch.equal(layer(x), product(q, layer.weight, layer.bias, torch.float16))
        y, mean, rstd = layer.normalized(x)
        assert torch.equal(y, product(q, layer.weight, layer.bias, torch.float16, normalized=True))
        assert torch.equal(mean, q.mean) and torch.equal(rstd, q.rstd)
    kept_data = Fp4Matrix(520, 640, "mxfp4", data=layer.weight.data.clone())
    assert torch.equal(Fp4Linear(kept_data, bias, "mxfp4")(x), layer(x))


@pytest.mark.parametrize("form", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 1, 8), (1, 100, 4096), (2, 300, 264), (5, 128, 1000), (7, 520, 16384), (8, 17000, 1032),
                                   (8, 777, 5120), (3, 4096, 8192), (9, 300, 2048), (16, 1000, 1288), (16, 520, 4096)])
def test_few_rows_are_quantised_inside_the_product(form, dtype, m, n, k):
    """One launch gives what the steps give, bit for bit, statistics too; every type in and out."""
    x = rows_of(m, k, TYPES[dtype], m + k, 0.5) + 0.25
    if m > 2:
        x[1] += 500.0                        # far from zero
        x[2, :k // 2] = 0.0
        x[m - 1, k - 1] = float("inf")
    layer = Fp4Linear(rows_of(n, k, torch.bfloat16, n, 0.5), torch.randn(n, device="cuda"), form)
    q = quantize(x, form, stats=True)
    for out in TYPES.values():
        same = lambda a, b: torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
        assert same(layer(x, out), product(q, layer.weight, layer.bias, out))
        y, mean, rstd = layer.normalized(x, out)
        assert same(y, product(q, layer.weight, layer.bias, out, normalized=True))
        assert same(mean, q.mean) and same(rstd, q.rstd)
    wide = torch.zeros(m, k + 24, dtype=x.dtype, device="cuda")
    for first in (0, 8, 3):                  # the last starts off 16 bytes: the steps again
        wide[:, first:first + k] = x
        assert same(layer(wide[:, first:first + k]), layer(x))
    assert layer.device_status() == 0


def test_streams_and_graphs():
    """Calls on two streams at once, and two captured graphs of one layer replayed in turn on new inputs."""
    layer = Fp4Linear(rows_of(1024, 512, torch.bfloat16, 1), torch.randn(1024, device="cuda"))
    xs = [rows_of(m, 512, torch.bfloat16, m) for m in (1, 64, 600)]
    want = [layer(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append([layer(x) for x in xs])
    torch.cuda.synchronize()
    for ys in got:
        for y, v in zip(ys, want):
            assert torch.equal(y, v)
    graphs, feeds, outs = [], [x.clone() for x in xs], []
    for f in feeds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer.normalized(f))
        graphs.append(g)
    for turn in range(3):
        for f, x in zip(feeds, xs):
            f.copy_(x * (1 + turn))
        torch.cuda.synchronize()
        for s, g in zip(streams + streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for f, o in zip(feeds, outs):
            for a, b in zip(o, layer.normalized(f)):
                assert torch.equal(a, b)
    assert layer.device_status() == 0


def test_weights_quantised_right_before_their_product():
    """The product waits for both sides, also when they come from the kernels directly before it."""
    x, w = rows_of(40, 4096, torch.bfloat16, 1), rows_of(4096, 4096, torch.bfloat16, 2)
    want = product(quantize(x), quantize(w))
    torch.cuda.synchronize()
    for _ in range(10):
        qx = quantize(x)
        assert torch.equal(product(qx, quantize(w)), want)
        layer = Fp4Linear(w)
        assert torch.equal(layer(x), want)


def test_gradients_and_wrong_tensors_are_refused():
    x = rows_of(4, 64, torch.bfloat16, 1)
    layer = Fp4Linear(rows_of(32, 64, torch.bfloat16, 2))
    wanted = x.clone().requires_grad_()
    with pytest.raises(ClefError):
        layer(wanted)
    with pytest.raises(ClefError):
        quantize(wanted)
    with torch.no_grad():
        layer(wanted)
    for bad in (x[:, :32], x.cpu(), x.double(), x.t()):
        with pytest.raises(ClefError):
            layer(bad)
    q, w = quantize(x), layer.weight
    with pytest.raises(ClefError):
        product(q, quantize(x, "mxfp4"))
    with pytest.raises(ClefError):
        product(q, w, normalized=True)                      # no statistics
    with pytest.raises(ClefError):
        product(q, w, torch.zeros(31, device="cuda"))
    with pytest.raises(ClefError):
        product(q, w, out=torch.empty(4, 32, device="cuda", dtype=torch.float16))
    with pytest.raises(ClefError):
        product(q, w, out=q.data.view(torch.bfloat16)[:128].view(4, 32))
    with pytest.raises(ClefError):
        quantize(x, "fp4")
    with pytest.raises(ClefError):
        quantize(x, out=Fp4Matrix(5, 64))
    with pytest.raises(ClefError):
        Fp4Matrix(4, 64, data=torch.empty(7, dtype=torch.uint8, device="cuda"))
