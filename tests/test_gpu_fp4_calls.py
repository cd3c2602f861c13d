"""Calls of the 4-bit operators as programs make them: reports, captures, streams, arguments that change or are refused."""
import pytest
import torch
from torch.autograd import forward_ad

from fp4_support import kept
from structured_decision_model_gb300 import binding as B, microscaled
from structured_decision_model_gb300.binding import ClefError
from structured_decision_model_gb300.microscaled import Fp4Linear, Fp4Matrix, product, quantize

pytestmark = pytest.mark.gpu

BOUNDS, TIMEOUT = 1, 2  # bits that kernels set


def rows_of(rows, cols, seed=0, dtype=torch.bfloat16):
    return torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def captured(f):
    """The graph of one call, and what the call returned."""
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f()
    return g, out


@pytest.mark.parametrize("bits,status", [(TIMEOUT, 6), (BOUNDS, 5), (TIMEOUT | BOUNDS, 6)])
def test_a_wait_that_ran_out_is_reported(bits, status):
    """The word as a kernel leaves it: reported once, by the layer and by the matrix."""
    layer = Fp4Linear(rows_of(130, 256, 2))
    for report in (layer.device_status, layer.weight.device_status):
        layer(rows_of(20, 256, 1))
        assert report() == 0
        layer.weight.flags.fill_(bits)
        layer(rows_of(20, 256, 1))
        assert report() == status
        assert report() == 0


def test_the_first_product_of_a_matrix_in_a_graph():
    """What products report stays through replays until it is read, and is clear before the first one."""
    x, w = quantize(rows_of(20, 256, 1)), quantize(rows_of(130, 256, 2))
    junk = torch.full((1 << 16,), -1, dtype=torch.int32, device="cuda")  # memory that a new buffer may be made from
    del junk
    g, y = captured(lambda: product(x, w))
    assert w.device_status() == 0
    g.replay()
    assert torch.equal(y, product(x, w))
    w.flags.fill_(TIMEOUT)                 # as a wait that ran out leaves it
    g.replay()
    torch.cuda.synchronize()
    assert w.device_status() == 6          # CLEF_ERR_DEVICE_TIMEOUT
    assert w.device_status() == 0


def test_matrices_report_apart():
    a, b = quantize(rows_of(8, 64, 1)), quantize(rows_of(8, 64, 2))
    a.flags.fill_(TIMEOUT)
    product(a, b)
    assert b.device_status() == 0 and a.device_status() == 6


def test_the_first_product_on_another_stream():
    """Flags are clear for every stream, whatever the one that made them still has to do."""
    x, w = quantize(rows_of(20, 256, 1)), quantize(rows_of(130, 256, 2))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    at = w.flags
    with torch.cuda.stream(s):
        at.fill_(TIMEOUT)
        s.synchronize()
    torch.cuda.synchronize()
    assert w.device_status() == 6


def test_every_matrix_has_its_own_word():
    data = torch.empty(256 + 2048 + 4, dtype=torch.uint8, device="cuda")
    matrices = [Fp4Matrix(1, 32, data=data) for _ in range(5000)]  # more than are cleared at once
    assert len({m.flags.data_ptr() for m in matrices}) == 5000


def test_a_capture_without_cleared_words(monkeypatch):
    """Nothing was made on the device before: rows are captured, a product is refused until there are words."""
    monkeypatch.setattr(microscaled, "_words", {})
    x, w = rows_of(20, 256, 1), rows_of(130, 256, 2)

    def steps():
        a, b = quantize(x), quantize(w)
        with pytest.raises(ClefError):
            product(a, b)
        return a, b

    g, (a, b) = captured(steps)
    g.replay()
    want = quantize(w)                     # outside: clears words
    assert torch.equal(product(a, b), product(quantize(x), want)) and b.device_status() == 0
    g, y = captured(lambda: product(quantize(x), quantize(w)))
    g.replay()
    assert torch.equal(y, product(a, b))


@pytest.mark.parametrize("form", ["mxfp4", "nvfp4"])
def test_few_rows_in_one_launch_or_two(form):
    """By the number of outputs, and by whether a graph is being captured; the same numbers either way."""
    def launches(f):
        before = B.clef_kernel_launches()
        out = f()
        return B.clef_kernel_launches() - before, out

    x = rows_of(2, 4096, 1)
    for outs, eager, in_graph in ((256, 1, 2 if form == "nvfp4" else 1), (33000, 2, 2)):
        layer = Fp4Linear(rows_of(outs, 4096, 2), None, form)
        n, y = launches(lambda: layer(x))
        assert n == eager
        counts = []
        g, got = captured(lambda: [counts.append(launches(lambda: layer(x))) or counts[-1][1] for _ in range(2)])
        assert [n for n, _ in counts] == [in_graph] * 2
        g.replay()
        assert torch.equal(got[0], y) and torch.equal(got[1], y)
        assert launches(lambda: layer(x))[0] == eager  # behind the capture as before it
        assert torch.equal(y, product(quantize(x, form), layer.weight))
        assert layer.device_status() == 0


def test_tangents_are_refused():
    """Dual tensors of forward-mode differentiation, which require no gradient, also where grad mode is off."""
    x, w, bias = rows_of(4, 64, 1, torch.float32), rows_of(32, 64, 2), torch.randn(32, device="cuda")
    layer = Fp4Linear(w, bias)
    q, y = quantize(x), torch.empty(4, 32, device="cuda")
    want = layer(x)
    with forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                for call in (lambda: layer(dual(x)), lambda: layer.normalized(dual(x)), lambda: quantize(dual(x)),
                             lambda: product(q, layer.weight, dual(bias)), lambda: Fp4Linear(dual(w)), lambda: Fp4Linear(w, dual(bias)),
                             lambda: product(q, layer.weight, dtype=torch.float32, out=dual(y)),
                             lambda: layer(dual(x)[:2]), lambda: layer(dual(x.view(2, 2, 64)))):
                    with pytest.raises(ClefError):
                        call()
        assert torch.equal(layer(x), want)  # the others go on as ever
        assert torch.equal(layer(forward_ad.unpack_dual(dual(x)).primal), want)


def test_the_bias_may_be_set():
    x, w, bias = rows_of(40, 64, 1), rows_of(32, 64, 2), torch.randn(32, device="cuda")
    layer = Fp4Linear(w, bias)
    plain, other = Fp4Linear(w), torch.randn(32, device="cuda").bfloat16()
    assert layer.bias is not None and torch.equal(layer(x), Fp4Linear(w, bias)(x))
    layer.bias = other
    assert torch.equal(layer(x), Fp4Linear(w, other)(x)) and torch.equal(layer.bias, other.float())
    layer.bias.zero_()
    assert torch.equal(layer(x), plain(x))
    layer.bias = None
    assert layer.bias is None and torch.equal(layer(x), plain(x))
    for bad in (bias[:31], bias.cpu(), bias[None]):
        with pytest.raises(ClefError):
            layer.bias = bad
    assert torch.equal(layer(x), plain(x))
    with pytest.raises(AttributeError):
        layer.weight = plain.weight


def test_parameters_are_taken_frozen():
    """A trained layer's parameters: taken as numbers, with grad mode on too; what comes out requires no gradient."""
    trained = torch.nn.Linear(64, 32, device="cuda")
    x = rows_of(4, 64, 1, torch.float32)
    layer = Fp4Linear(trained.weight, trained.bias)
    y = layer(x)
    assert not y.requires_grad and not layer.bias.requires_grad and trained.weight.requires_grad
    assert torch.equal(y, Fp4Linear(trained.weight.detach().clone(), trained.bias.detach().clone())(x))
    with pytest.raises(ClefError):
        quantize(trained.weight)               # by itself it is an input


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_rows_at_the_end_of_their_type(dtype):
    """What a row's largest value stands for may pass the type's range: rounded once, to infinity in that type."""
    most = torch.finfo(dtype).max
    x = torch.tensor([[most, -most] + [most / 8] * 30, [most / 2, most / 4] + [1.0] * 30], dtype=dtype, device="cuda")
    for form in ("mxfp4", "nvfp4"):
        m = quantize(x, form)
        want = torch.from_numpy(kept(x.double().cpu().numpy(), form)[3])
        assert torch.equal(m.dequantize(dtype).cpu(), want.to(dtype))
        assert want.abs().max() <= most * 18 / 17 and m.dequantize(dtype)[1].isfinite().all()
        if form == "mxfp4":
            assert m.dequantize(dtype).isfinite().all()
    if dtype == torch.float16:
        assert m.dequantize(torch.float32)[0, 0] == 67584 and m.dequantize(dtype)[0, 0].isinf()


@pytest.mark.parametrize("form", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("m,n,k", [(1, 300, 4096), (8, 40, 64), (20, 300, 4096), (100, 300, 1000), (40, 40, 64), (5000, 1100, 1000)])
def test_waits_of_the_products_run_out(form, m, n, k):
    """A K tile that never comes: few rows, tiles (in parts of K, and whole) and pairs report it and return; what follows
    is as before."""
    x, layer = rows_of(m, k, 1), Fp4Linear(rows_of(n, k, 2), None, form)
    want = layer(x)
    assert layer.device_status() == 0
    few = m <= 8
    size = 0 if few else B.clef_fp4_linear_scratch(layer.weight.struct.format, B.BF16, m, k)
    space, out = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda"), torch.full((m, n), 9.0, dtype=torch.bfloat16, device="cuda")
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    B.clef_fp4_selftest_timeout(layer.weight.struct, B.BF16, x.data_ptr(), k, m, B.BF16, out.data_ptr(), n,
                                None if few else space.data_ptr(), size, 5_000_000, layer.weight.flags.data_ptr(),
                                torch.cuda.current_stream().cuda_stream)
    end.record()
    assert layer.device_status() == 6 and layer.device_status() == 0
    assert begin.elapsed_time(end) >= 5  # ms: a wait did run out
    assert (out == 9).all()              # every tile gave up
    for _ in range(3):
        assert torch.equal(layer(x), want)
    assert layer.device_status() == 0
