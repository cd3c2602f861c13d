"""The microscaled 4-bit entry points on the host (no GPU): sizes and refusals, all before any CUDA call."""
import numpy as np
import pytest

import synth
from fp4_support import E4M3, LEVELS, kept
from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300.build import build_library

P = 1 << 20  # a well-aligned address that is never read


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return B.load()


def refused(status, f, *args):
    with pytest.raises(B.ClefError) as e:
        f(*args)
    assert e.value.status == status


def changed(args, i, v):
    return [*args[:i], v, *args[i + 1:]]


def matrix(at=P, rows=10, cols=100, form=B.NVFP4, **over):
    d = dict(codes=at, scales=at + (1 << 16), row_scale=at + (2 << 16) if form == B.NVFP4 else None)
    d.update(over)
    return B.ClefFp4(d["codes"], d["scales"], d["row_scale"], rows, cols, form)


@pytest.mark.parametrize("rows,cols", [(1, 1), (128, 256), (129, 257), (1000, 16384)])
def test_sizes(rows, cols):
    for form, each in ((B.MXFP4, 1024), (B.NVFP4, 2048)):
        codes, scales = B.clef_fp4_size(form, rows, cols)
        assert codes == rows * (-(-cols // 32) * 16)
        assert scales == -(-rows // 128) * -(-cols // 256) * each
        up = lambda n: -(-n // 256) * 256
        assert B.clef_fp4_linear_scratch(form, B.BF16, rows, cols) == up(codes) + up(scales) + (4 * rows if form else 0)


@pytest.mark.parametrize("form,rows,cols", [(2, 1, 1), (-1, 1, 1), (0, 0, 1), (1, 1, 0), (1, 1, 16385), (0, 2 ** 31 - 256, 1),
                                            (1, 2 ** 31 - 300, 16384)])
def test_unsupported_sizes(form, rows, cols):
    refused(3, B.clef_fp4_size, form, rows, cols)
    refused(3, B.clef_fp4_linear_scratch, form, B.BF16, rows, cols)
    refused(1, B.clef_fp4_linear_scratch, B.MXFP4, 3, 1, 1)


def test_matrices_are_checked():
    good = [matrix(), B.BF16, 8 * P, 100, None, None, None]
    for bad in (matrix(codes=None), matrix(scales=None), matrix(row_scale=None), matrix(codes=P + 128), matrix(scales=2 * P + 16),
                matrix(row_scale=2 * P + 2)):
        refused(1, B.clef_fp4_quantize, *changed(good, 0, bad))
    refused(3, B.clef_fp4_quantize, *changed(good, 0, matrix(form=3)))
    refused(3, B.clef_fp4_quantize, *changed(good, 0, matrix(rows=0)))


def test_quantize_refusals():
    good = [matrix(), B.BF16, 8 * P, 100, 9 * P, 10 * P, 11 * P]
    for i, v in ((1, 3), (1, -1), (2, None), (2, 8 * P + 1), (3, -1), (3, 2 ** 31 + 1), (4, None), (5, None), (4, 9 * P + 2), (6, 11 * P + 1),
                 (4, 10 * P),                    # mean and rstd in one place
                 (4, P + 64), (6, 8 * P + 40),   # outputs inside the codes, inside x
                 (2, P + 16)):                   # x inside the codes
        refused(1, B.clef_fp4_quantize, *changed(good, i, v))


def test_rows_further_apart_than_memory_reaches():
    far = [matrix(rows=2 ** 20), B.BF16, 1 << 50, 2 ** 21, None, None, None]
    refused(1, B.clef_fp4_quantize, *far)
    refused(1, B.clef_fp4_dequantize, matrix(rows=2 ** 20), B.BF16, 1 << 50, 2 ** 21)


def test_dequantize_refusals():
    good = [matrix(), B.FP32, 8 * P, 100]
    for i, v in ((1, 7), (2, None), (2, 8 * P + 2), (3, 99), (2, P + 4 * 100)):
        refused(1, B.clef_fp4_dequantize, *changed(good, i, v))


def test_product_refusals():
    x, w = matrix(), matrix(at=4 * P, rows=20)
    good = [x, w, 12 * P, 13 * P, 14 * P, 15 * P, B.BF16, 8 * P, 20, 16 * P]
    for i, v in ((1, matrix(at=4 * P, rows=20, form=B.MXFP4)), (1, matrix(at=4 * P, rows=20, cols=101)), (2, 12 * P + 2),
                 (3, None), (4, None), (5, None), (6, 3), (7, None), (7, 8 * P + 1), (8, 19), (9, None), (9, 16 * P + 1),
                 (7, P), (7, 4 * P + (1 << 16)), (7, 12 * P), (7, 16 * P)):  # out over x, w's scales, bias, flags
        refused(1, B.clef_fp4_product, *changed(good, i, v))
    big = matrix(at=1 << 44, rows=2 ** 30, cols=16, scales=1 << 45, row_scale=1 << 46)
    refused(3, B.clef_fp4_product, big, matrix(at=4 * P, rows=2 ** 20, cols=16, scales=1 << 47), *changed(good[2:], 6, 2 ** 20))


def test_layer_refusals():
    w = matrix(at=4 * P, rows=20)
    size = B.clef_fp4_linear_scratch(B.NVFP4, B.BF16, 10, 100)  # ragged rows: never without scratch
    good = [w, B.BF16, 8 * P, 100, 10, 12 * P, 15 * P, B.BF16, 9 * P, 20, 13 * P, 14 * P, 20 * P, size, 16 * P]
    for i, v in ((1, 5), (2, None), (3, -1), (5, 12 * P + 1), (6, None), (7, 9), (8, None), (9, 19), (10, None), (11, None),
                 (12, None), (12, 20 * P + 8), (14, None),
                 (8, 8 * P), (8, 20 * P + 512), (10, 20 * P), (10, 14 * P), (12, 8 * P), (12, 4 * P)):
        refused(1, B.clef_fp4_linear, *changed(good, i, v))
    refused(2, B.clef_fp4_linear, *changed(good, 13, size - 1))
    refused(3, B.clef_fp4_linear, *changed(good, 4, 0))
    # few rows: without scratch only where each starts on 16 bytes and has a multiple of 8 values
    w = matrix(at=4 * P, rows=20, cols=104)
    few = [w, B.BF16, 8 * P, 104, 8, *good[5:12], None, 0, None]
    for i, v in ((2, 8 * P + 2), (3, 107), (0, matrix(at=4 * P, rows=20, cols=100)), (4, 9)):
        refused(1, B.clef_fp4_linear, *changed(changed(few, i, v), 14, 16 * P))
    refused(1, B.clef_fp4_linear, *few)  # no flags


def test_few_rows_need_no_scratch():
    need = lambda *a: B.clef_fp4_linear_scratch(*a) > 0
    for form in (B.MXFP4, B.NVFP4):
        assert not need(form, B.BF16, 8, 4096, 0, 1) and not need(form, B.BF16, 8, 4096, 1, 1)
        assert need(form, B.BF16, 8, 4096, 0, 0) and need(form, B.BF16, 1, 4092, 0, 1) and need(form, B.BF16, 17, 64, 0, 1)
    assert need(B.NVFP4, B.FP32, 8, 4096, 0, 1) and not need(B.MXFP4, B.FP32, 8, 4096, 0, 1)
    assert need(B.MXFP4, B.FP32, 8, 4096, 1, 1) and not need(B.MXFP4, B.FP16, 16, 4096, 0, 1)


def test_head_refusals():
    cfg = B.make_config()
    spec = synth.BatchSpec(name="t", B=2, H=4096, vocab=1000, lengths=[256, 300], questions=(2, 2), options=(2, 3))
    bt = synth.make_batch(spec, seed=2, with_hidden=False)
    schema = B.Schema(bt.B, bt.Lpad, bt.H, bt.lengths, bt.q_rec, bt.q_type, bt.q_span, bt.q_opt_off, bt.o_span)
    w = matrix(at=1 << 30, rows=4096, cols=4096, scales=1 << 31, row_scale=1 << 32)
    for bad in (matrix(), None):
        refused(1, B.clef_fp4_memory_weights, cfg, P, bad, P)
    refused(1, B.clef_fp4_memory_weights, cfg, None, w, P)
    refused(3, B.clef_fp4_memory_weights, B.make_config(H=100), P, w, P)
    assert B.clef_head_forward_fp4_scratch(cfg, B.NVFP4, schema) == B.clef_stream_rows_fp4_scratch(cfg, B.NVFP4, 300)
    for lengths, rows in (([300, 300], 300), ([256, 256], 512)):  # one product where no padding lies between
        even = synth.make_batch(synth.BatchSpec(name="t", B=2, H=4096, vocab=1000, lengths=lengths, questions=(2, 2),
                                                options=(2, 3)), seed=2, with_hidden=False)
        even = B.Schema(even.B, even.Lpad, even.H, even.lengths, even.q_rec, even.q_type, even.q_span, even.q_opt_off, even.o_span)
        assert B.clef_head_forward_fp4_scratch(cfg, B.MXFP4, even) == B.clef_stream_rows_fp4_scratch(cfg, B.MXFP4, rows)
    refused(3, B.clef_stream_rows_fp4_scratch, cfg, 4, 300)
    ws = B.clef_workspace_size(cfg, schema)
    rows = [cfg, P, w, P, schema, P, B.BF16, 1, 0, 300, P, ws, P, 1 << 40]
    for i, v in ((1, None), (2, matrix()), (3, None), (5, P + 8), (6, B.FP32), (7, 2), (7, -1), (8, 1), (9, 0), (9, 301), (10, P + 16),
                 (12, P + 16)):
        refused(1, B.clef_stream_rows_fp4, *changed(rows, i, v))
    refused(2, B.clef_stream_rows_fp4, *changed(rows, 11, ws - 1))
    n = B.clef_weight_count(cfg)
    forward = [cfg, [P] * n, P, w, P, schema, P, B.BF16, P, P, P, P, P, P, P, P, ws, P, 1 << 40]
    for i, v in ((1, [P + 2] * n), (6, None), (7, B.FP32), (8, None), (9, P + 2), (14, None)):
        refused(1, B.clef_head_forward_fp4, *changed(forward, i, v))
    refused(2, B.clef_head_forward_fp4, *changed(forward, 18, 16))
    refused(2, B.clef_head_forward_fp4, *changed(forward, 16, ws - 1))


def test_the_oracle_of_the_tests():
    """The 64-bit form by hand: a block of each format whose quotients are known."""
    assert len(LEVELS) == 8 and len(E4M3) == 127 and E4M3[-1] == 448 and E4M3[8] == 2.0 ** -6
    x = np.zeros((1, 32))
    x[0, :10] = [7.9, 0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5.0, 0.2501, 4.9]
    codes, byte, _, values = kept(x, "mxfp4")
    assert byte[0, 0] == 127
    np.testing.assert_array_equal(values[0, :10], [6, 0, 1, -1, 2, 2, -4, 4, 0.5, 4])
    assert codes[0, 3] == 8 + 2
    codes, byte, r, values = kept(x / 7.9 * 6, "nvfp4")
    # amax 6: r = 2^-8, quotient 1 / r = 256 = 2^8, so the scale is 1 again
    assert r[0] == 2.0 ** -8 and E4M3[byte[0, 0]] == 256 and values[0, 0] == 6


def test_few_rows_by_the_outputs_and_the_capture():
    """One launch while a call by itself is host time; in a graph where the GPU takes less, and never for a vocabulary."""
    one = lambda form, rows, cols, norm, outs, captured, t=B.BF16: \
        B.clef_fp4_linear_scratch(form, t, rows, cols, norm, 1, outs, captured) == 0
    for form in (B.MXFP4, B.NVFP4):
        for norm in (0, 1):
            for rows in (1, 8):
                assert one(form, rows, 4096, norm, 32768, 0) and not one(form, rows, 4096, norm, 32769, 0)
                assert one(form, rows, 1024, norm, 4096, 1) and not one(form, rows, 1024, norm, 131072, 1)
    assert one(B.MXFP4, 8, 4096, 0, 4096, 1) and not one(B.MXFP4, 16, 4096, 0, 4096, 1) and one(B.MXFP4, 16, 4096, 0, 4096, 0)
    for form, norm in ((B.NVFP4, 0), (B.NVFP4, 1), (B.MXFP4, 1)):
        assert not one(form, 1, 4096, norm, 4096, 1) and not one(form, 8, 4096, norm, 20000, 1) and one(form, 4, 4096, norm, 20000, 1)
    refused(1, B.clef_fp4_linear_scratch, B.MXFP4, B.BF16, 1, 8, 0, 1, 0)


def test_head_refusals_come_before_the_first_launch():
    """What only the projection's own checks know is refused as an argument, not met behind the plan's upload."""
    cfg = B.make_config()
    bt = synth.make_batch(synth.BatchSpec(name="t", B=2, H=4096, vocab=1000, lengths=[256, 300], questions=(2, 2), options=(2, 3)),
                          seed=2, with_hidden=False)
    schema = B.Schema(bt.B, bt.Lpad, bt.H, bt.lengths, bt.q_rec, bt.q_type, bt.q_span, bt.q_opt_off, bt.o_span)
    ws = B.clef_workspace_size(cfg, schema)
    at = [(i + 1) << 32 for i in range(16)]
    over = dict(rows=4096, cols=4096, at=at[0], scales=at[1], row_scale=at[2])
    good = [cfg, [P] * B.clef_weight_count(cfg), at[3], matrix(**over), at[4], schema, at[5], B.BF16, P, P, P, P, P, P, P, at[6], ws,
            at[7], 1 << 30]
    for i, v in ((3, matrix(**dict(over, codes=None))), (3, matrix(**dict(over, codes=at[0] + 16))), (3, matrix(**dict(over, scales=None))),
                 (3, matrix(**dict(over, row_scale=None))), (4, at[4] + 2), (17, at[6]), (17, at[5]), (6, at[7])):
        refused(1, B.clef_head_forward_fp4, *changed(good, i, v))
    refused(3, B.clef_head_forward_fp4, *changed(good, 3, matrix(form=2, **over)))


def test_selftest_refusals():
    w = matrix(at=4 * P, rows=20)
    size = B.clef_fp4_linear_scratch(B.NVFP4, B.BF16, 10, 100)
    good = [w, B.BF16, 8 * P, 100, 10, B.BF16, 9 * P, 20, 20 * P, size, 1_000_000, 16 * P]
    for i, v in ((2, None), (6, None), (8, None), (10, 999), (10, 100_000_001), (11, None)):
        refused(1, B.clef_fp4_selftest_timeout, *changed(good, i, v))
