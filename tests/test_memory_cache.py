"""The 4-bit memory cache on the host (no GPU): sizes and refusals.

Every call here fails validation (or only computes sizes) before the library touches CUDA.
"""
import ctypes

import pytest
import torch

import synth
from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300.build import build_library

P = 1 << 20  # a pointer that is never followed: the calls are refused before a launch


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_library()
    return B.load()


def cache(data=P, n_pages=10, page=64, heads=4, head_dim=64):
    return B.ClefCache(data, n_pages, page, heads, head_dim)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_size_is_four_and_a_half_bits_a_value(page, dim):
    n = B.clef_cache_size(cache(n_pages=7, page=page, heads=3, head_dim=dim))
    assert n * 8 == 7 * page * 3 * dim * 2 * 4.5


@pytest.mark.parametrize("bad", [dict(page=0), dict(page=8), dict(page=48), dict(page=512), dict(heads=0),
                                 dict(heads=1025), dict(head_dim=32), dict(head_dim=96), dict(n_pages=0),
                                 dict(n_pages=1 << 30)])
def test_unsupported_caches(bad):
    with pytest.raises(B.ClefError) as e:
        B.clef_cache_size(cache(**bad))
    assert e.value.status == 3


def refused(status, call, *args):
    with pytest.raises(B.ClefError) as e:
        call(*args)
    assert e.value.status == status


def changed(args, at, value):
    out = list(args)
    out[at] = value
    return out


def test_plan_refusals():
    good = [cache(), 4, P, P, P, 8, P, P, P, P, 16, P]
    for at in (2, 3, 4, 6, 7, 8, 9, 11):                       # every pointer
        refused(1, B.clef_cache_plan, *changed(good, at, 0))
    for at in (2, 3, 4, 6, 7, 8, 9, 11):                       # and each on 4 bytes
        refused(1, B.clef_cache_plan, *changed(good, at, P + 2))
    for at, value in ((1, 0), (1, -1), (5, 0), (10, -1), (10, (1 << 30) + 1), (5, 1 << 25), (5, (1 << 25) - 1)):
        refused(1, B.clef_cache_plan, *changed(good, at, value))
    refused(3, B.clef_cache_plan, *changed(good, 1, 1025))
    refused(3, B.clef_cache_plan, *changed(good, 0, cache(page=24)))


def test_append_refusals():
    good = [cache(), 5, 0, 4, B.BF16, P, 256, 64, P, 256, 64, P, P]
    for at in (5, 8, 11, 12):
        refused(1, B.clef_cache_append, *changed(good, at, 0))
    for at, value in ((0, cache(data=0)), (0, cache(data=P + 128)), (1, -1), (2, -1), (2, 1), (3, 0), (3, 5), (4, B.FP32),
                      (4, -1), (5, P + 1), (8, P + 1), (11, P + 2), (12, P + 1), (6, -256), (7, -1), (9, -1), (10, -64)):
        refused(1, B.clef_cache_append, *changed(good, at, value))
    B.clef_cache_append(*changed(good, 1, 0))                  # nothing to do: no launch


def test_read_refusals():
    good = [cache(), 5, 0, 4, B.FP32, P, P, P, P]
    for at in (5, 6, 7, 8):
        refused(1, B.clef_cache_read, *changed(good, at, 0))
    for at, value in ((0, cache(data=0)), (1, -1), (2, 4), (3, 0), (4, 3), (5, P + 2), (6, P + 8), (7, P + 8), (8, P + 2)):
        refused(1, B.clef_cache_read, *changed(good, at, value))
    B.clef_cache_read(*changed(good, 1, 0))


def test_attend_refusals():
    c = cache()
    n = B.clef_cache_attend_workspace(c, 2, 6, 8, 40 * 64)
    assert n > 0 and B.clef_cache_attend_workspace(c, 2, 6, 8, 256) == 0
    #       0  1  2  3  4  5  6  7       8  9        10  11 12 13  14 15   16 17 18 19 20 21
    good = [c, 2, 6, 4, 8, 0, 4, B.BF16, P, 8 * 64, 64, P, P, 40, P, 0.125, 1, P, P, P, P, n]
    for at in (8, 11, 12, 14, 17, 19, 20):
        refused(1, B.clef_cache_attend, *changed(good, at, 0))
    for at, value in ((0, cache(data=0)), (1, 0), (2, -1), (3, -1), (3, 7), (4, 0), (4, 6), (5, 1), (6, 0), (6, 5),
                      (7, B.FP32), (8, P + 2), (9, 511), (10, 63), (9, -512), (11, P + 2), (12, P + 1), (13, 0),
                      (13, 1 << 25), (13, (1 << 25) - 1), (14, P + 2), (18, P + 2), (19, P + 3),
                      (15, float("nan")), (15, float("inf")), (16, 2), (17, P + 2), (20, P + 16)):
        refused(1, B.clef_cache_attend, *changed(good, at, value))
    refused(2, B.clef_cache_attend, *changed(good, 21, n - 1))
    refused(3, B.clef_cache_attend, *changed(good, 1, 1025))
    B.clef_cache_attend(*changed(good, 3, 0))                  # no queries: no launch
    # a table so wide that the partial rows cannot be counted in 32 bits
    refused(3, B.clef_cache_attend, *changed(changed(changed(good, 13, (1 << 25) - 1024), 2, 1 << 20), 21, 1 << 62))


def test_status_of_nothing_is_refused():
    assert B.load().clef_cache_status(0, None) == 1 and B.load().clef_cache_status(P + 2, None) == 1
    assert B.clef_status_string(7) == "no free cache pages left"


def _head_args():
    spec = synth.BatchSpec(name="t", B=2, H=256, vocab=1000, length_law="uniform", length_range=(300, 400),
                           questions=(2, 3), options=(2, 4), instr_len=(3, 9), option_len=(2, 6))
    bt = synth.make_batch(spec, seed=3, with_hidden=False)
    cfg = B.make_config(H=256, vocab=1000)
    sch = B.Schema(bt.B, bt.Lpad, bt.H, bt.lengths, bt.q_rec, bt.q_type, bt.q_span, bt.q_opt_off, bt.o_span)
    return bt, cfg, sch


def test_memory_store_refusals():
    bt, cfg, sch = _head_args()
    ws = B.clef_workspace_size(cfg, sch)
    good = [cfg, sch, 0, 0, 10, P, ws, cache(heads=32), P, P]
    length = int(bt.lengths[0])
    for at, value in ((2, -1), (2, 2), (3, -1), (4, 0), (4, length + 1), (5, 0), (5, P + 16), (7, cache(heads=16)),
                      (7, cache(heads=32, head_dim=128)), (7, cache(data=0, heads=32)), (8, 0), (8, P + 2), (9, 0), (9, P + 1)):
        refused(1, B.clef_memory_store, *changed(good, at, value))
    refused(2, B.clef_memory_store, *changed(good, 6, ws - 1))


def test_stream_finish_memory_refusals():
    bt, cfg, sch = _head_args()
    ws = B.clef_workspace_size(cfg, sch)
    c = cache(heads=32)
    space = B.clef_cache_attend_workspace(c, 2, sch.O, 16, 40 * 64)
    weights = [P] * B.clef_weight_count(cfg)
    first = [min(int(sch.q_span.reshape(-1, 2)[sch.q_rec == b].min()), int(min(
        sch.o_span.reshape(-1, 2)[sch.q_opt_off[q]:sch.q_opt_off[q + 1]].min() for q in range(sch.Q) if sch.q_rec[q] == b)))
        for b in range(2)]
    good = [cfg, weights, P, sch, first, P, B.BF16, P, P, P, P, P, P, P, P, ws, c, P, 40, P, P, space]
    for at in (2, 5, 7, 8, 9, 10, 11, 12, 13, 14, 17, 19, 20):
        refused(1, B.clef_stream_finish_memory, *changed(good, at, 0))
    for at, value in ((4, [first[0] + 1, first[1]]), (4, [first[0], int(bt.lengths[1])]), (4, [-1, 0]), (4, [0]),
                      (6, B.FP32), (16, cache(heads=16)), (17, P + 2), (18, 0), (18, 4), (18, 1 << 25), (18, 1 << 30), (19, P + 2), (20, P + 16)):
        refused(1, B.clef_stream_finish_memory, *changed(good, at, value))
    refused(2, B.clef_stream_finish_memory, *changed(good, 21, space - 1))
    refused(2, B.clef_stream_finish_memory, *changed(good, 15, ws - 1))


def test_python_refusals_without_a_gpu():
    """The torch layer checks types, shapes and devices itself (a cache on the CPU never launches)."""
    from structured_decision_model_gb300.memory import MemoryCache
    c = MemoryCache(4, page=16, heads=2, head_dim=64, requests=3, max_len=40, device="cpu")
    assert c.width == 3 and c.block_table.tolist() == [[-1] * 3] * 3 and c.free_pages.tolist() == [3, 2, 1, 0]
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(5, dtype=torch.int32)
    cu = torch.zeros(4, dtype=torch.int32)
    calls = [lambda: c.plan(torch.zeros(3), 4), lambda: c.plan(torch.zeros(2, dtype=torch.int32), 4),
             lambda: c.append(k.float(), k.float(), slots), lambda: c.append(k, k.half(), slots),
             lambda: c.append(k, k[:4], slots), lambda: c.append(k[:, :, :32], k[:, :, :32], slots),
             lambda: c.append(k, k, slots.long()), lambda: c.append(k, k, slots[:4]),
             lambda: c.append(k.clone().requires_grad_(), k, slots),
             lambda: c.append(k.transpose(1, 2), k.transpose(1, 2), slots),
             lambda: c.read(slots, torch.float64), lambda: c.read(slots, head0=2), lambda: c.read(slots.view(5, 1)),
             lambda: c.attend(k.float(), cu, 1), lambda: c.attend(k, cu.long(), 1), lambda: c.attend(k, cu[:1], 1),
             lambda: c.attend(k, cu, 1, lengths=slots[:2]),
             lambda: c.attend(k, cu, 1, block_table=c.block_table[:2]),
             lambda: c.attend(k, cu, 1, block_table=torch.zeros(3, 6, dtype=torch.int32)[:, :3]),
             lambda: MemoryCache(4, data=torch.zeros(3, dtype=torch.uint8), device="cpu"),
             lambda: MemoryCache(4, state=torch.zeros(3, dtype=torch.int32), device="cpu"),
             lambda: MemoryCache(4, requests=2000, device="cpu"), lambda: MemoryCache(4, page=20, device="cpu")]
    for i, call in enumerate(calls):
        with pytest.raises(B.ClefError):
            call()
            pytest.fail(f"call {i} was accepted")


def test_output_in_place_of_the_queries_is_refused():
    """Rows of a request are read by several blocks: the output cannot go over them."""
    from structured_decision_model_gb300.memory import MemoryCache
    c = MemoryCache(4, page=16, heads=2, head_dim=64, requests=3, max_len=40, device="cpu")
    q = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(B.ClefError, match="apart from q"):
        c.attend(q, torch.zeros(4, dtype=torch.int32), 1, out=q)
