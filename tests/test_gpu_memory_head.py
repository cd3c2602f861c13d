"""The head over kept 4-bit memory: clef_memory_store and clef_stream_finish_memory.

The oracle's cross attention is given the keys and values that the cache's rows stand for
(read back, fp64), so the head's ordinary parity bar applies: what the 4 bits themselves
change is in both sides.
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle.clef_head as oracle_head
import synth
from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300.build import build_library

from gpu_support import compare, device_inputs, head_for, run_oracle, schema_of

pytestmark = pytest.mark.gpu

FULL = synth.HeadShape()


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_library()
    B.load()


def _outputs(out):
    return {k: getattr(out, k).cpu().numpy() for k in ("logits", "probs", "q_value", "q_conf", "q_argmax")}


def first_rows(bt):
    """The first row that any span of a record reads."""
    first = []
    for b in range(bt.B):
        qs = np.nonzero(bt.q_rec == b)[0]
        spans = [bt.q_span[q, 0] for q in qs]
        spans += [bt.o_span[j, 0] for q in qs for j in range(bt.q_opt_off[q], bt.q_opt_off[q + 1])]
        first.append(int(min(spans)))
    return first


def oracle_over_cache(monkeypatch, cache, lengths, shape):
    """Replaces the oracle's K/V projections by the cache's rows (records and layers come in order)."""
    kept = []
    for b, n in enumerate(lengths):
        pos = torch.arange(int(n), device="cuda")
        slots = (cache.block_table[b, pos // cache.page] * cache.page + pos % cache.page).int()
        k, v = cache.read(slots, torch.float32)
        kept.append((k.double().cpu().numpy(), v.double().cpu().numpy()))
    calls = []

    def attend(qx, mem, Wq, bq, Wk, bk, Wv, bv, heads):
        b, l = divmod(len(calls), shape.n_route)
        calls.append(1)
        q = oracle_head.linear(qx, Wq, bq)
        out = np.empty(q.shape)
        for h in range(heads):
            k, v = (x[:, l * heads + h] for x in kept[b])
            out[:, h * 64:(h + 1) * 64] = oracle_head.softmax(q[:, h * 64:(h + 1) * 64] @ k.T / 8.0, axis=1) @ v
        return out
    monkeypatch.setattr(oracle_head, "cross_attention", attend)


def keep_rows(head, sch, hidden, cache, lens, starts):
    """Streams rows [starts[b], lens[b]) of every record and stores them in the slots a plan gives."""
    slots, cu = cache.plan(torch.tensor([int(n) for n in lens], dtype=torch.int32, device="cuda"), int(sum(lens)))
    head.stream_begin(sch)
    at = 0
    for b, (r0, n) in enumerate(zip(starts, lens)):
        n = int(n)
        for r in range(r0, n, 700):
            head.stream_rows(sch, hidden, b, r, min(700, n - r))
        head.memory_store(sch, b, r0, n - r0, cache, slots[at:at + n - r0])
        at += n - r0
    return at


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_head_over_a_cache(monkeypatch, dtype):
    spec = synth.BatchSpec(name="kept", B=3, length_law="uniform", length_range=(300, 1800), questions=(2, 5), options=(2, 7))
    bt = synth.make_batch(spec, seed=71)
    head, w = head_for(FULL)
    hidden, ids, lex = device_inputs(bt, FULL.vocab)
    if dtype == torch.float16:
        hidden = hidden.to(dtype)
        bt = dataclasses.replace(bt, hidden=synth.f32_to_bf16(hidden.float().cpu().numpy()))
    sch = schema_of(bt)
    cache = head.memory_cache(int(sum(-(-n // 64) for n in bt.lengths)) + 1, bt.B, bt.Lpad)
    keep_rows(head, sch, hidden, cache, bt.lengths, [0] * bt.B)
    out = head.stream_finish_memory(sch, [0] * bt.B, hidden, ids, lex, cache)
    assert head.device_status() == 0 and cache.device_status() == 0
    oracle_over_cache(monkeypatch, cache, bt.lengths, FULL)
    compare(_outputs(out), run_oracle(w, FULL, bt), bt)


def test_second_schema_over_kept_state(monkeypatch):
    """The same state asked twice: the second time only the rows behind it are streamed, its old schema's
    pages are given back, and the result is that of the whole record kept anew."""
    spec = synth.BatchSpec(name="asked", B=2, lengths=[1900, 1200], questions=(2, 4), options=(2, 6))
    first = synth.make_batch(spec, seed=81)
    second = synth.make_batch(spec, seed=82)
    state = [min(a, b) for a, b in zip(first_rows(first), first_rows(second))]
    hid = second.hidden.copy()
    for b, n in enumerate(state):
        hid[b, :n] = first.hidden[b, :n]      # a causal backbone leaves the state's rows as they were
    second = dataclasses.replace(second, hidden=hid)
    head, w = head_for(FULL)
    cache = head.memory_cache(80, 2, 2048)
    h1, ids1, lex1 = device_inputs(first, FULL.vocab)
    sch1 = schema_of(first)
    keep_rows(head, sch1, h1, cache, first.lengths, [0, 0])
    head.stream_finish_memory(sch1, [0, 0], h1, ids1, lex1, cache)
    cache.plan(torch.tensor(state, dtype=torch.int32, device="cuda"), 0)   # the first schema's rows go

    h2, ids2, lex2 = device_inputs(second, FULL.vocab)
    h2[:, :min(state)] = 0                    # the kept rows' hidden states are not needed again
    sch2 = schema_of(second)
    keep_rows(head, sch2, h2, cache, second.lengths, state)
    out = head.stream_finish_memory(sch2, state, h2, ids2, lex2, cache)
    assert head.device_status() == 0 and cache.device_status() == 0
    got = _outputs(out)

    whole = head.memory_cache(80, 2, 2048)
    h2 = device_inputs(second, FULL.vocab)[0]
    keep_rows(head, sch2, h2, whole, second.lengths, [0, 0])
    ref = _outputs(head.stream_finish_memory(sch2, [0, 0], h2, ids2, lex2, whole))
    for name in ref:
        np.testing.assert_array_equal(got[name], ref[name])
    oracle_over_cache(monkeypatch, cache, second.lengths, FULL)
    compare(got, run_oracle(w, FULL, second), second)


def test_kept_memory_after_forward():
    """clef_memory_store takes the K/V that an ordinary forward pass left, and the ordinary pass is as
    it was after a cached one used the workspace."""
    spec = synth.BatchSpec(name="after", B=2, lengths=[600, 410], questions=(2, 3), options=(2, 4))
    bt = synth.make_batch(spec, seed=91)
    head, _ = head_for(FULL)
    inputs = device_inputs(bt, FULL.vocab)
    sch = schema_of(bt)
    plain = _outputs(head.forward(sch, *inputs))
    cache = head.memory_cache(40, 2, 640, page=32)
    other = head.memory_cache(40, 2, 640, page=32)
    slots, cu = cache.plan(torch.tensor(bt.lengths, dtype=torch.int32, device="cuda"), int(sum(bt.lengths)))
    for c in (cache, other):
        c.block_table.copy_(cache.block_table)
    head.memory_store(sch, 0, 0, 600, cache, slots[:600])
    head.memory_store(sch, 1, 0, 410, cache, slots[600:])
    kept = _outputs(head.stream_finish_memory(sch, [0, 0], *inputs, cache))
    assert head.device_status() == 0 and cache.device_status() == 0
    head.stream_begin(sch)
    for b, n in enumerate(bt.lengths):
        head.stream_rows(sch, inputs[0], b, 0, int(n))
        head.memory_store(sch, b, 0, int(n), other, slots[int(cu[b]):int(cu[b]) + int(n)])
    assert torch.equal(cache.read(slots, torch.float32)[0], other.read(slots, torch.float32)[0])
    streamed = _outputs(head.stream_finish_memory(sch, [0, 0], *inputs, other))
    again = _outputs(head.forward(sch, *inputs))
    for name in plain:
        np.testing.assert_array_equal(kept[name], streamed[name])
        np.testing.assert_array_equal(again[name], plain[name])


def test_head_over_a_cache_replays_from_a_graph():
    spec = synth.BatchSpec(name="kept graph", B=2, lengths=[700, 512], questions=(2, 3), options=(2, 4))
    bt = synth.make_batch(spec, seed=95)
    head, _ = head_for(FULL)
    hidden, ids, lex = device_inputs(bt, FULL.vocab)
    sch = schema_of(bt)
    cache = head.memory_cache(30, 2, 704)
    want = torch.tensor(bt.lengths, dtype=torch.int32, device="cuda")
    slots, _ = cache.plan(want, int(sum(bt.lengths)))

    def step(out=None):
        head.stream_begin(sch)
        at = 0
        for b, n in enumerate(bt.lengths):
            head.stream_rows(sch, hidden, b, 0, int(n))
            head.memory_store(sch, b, 0, int(n), cache, slots[at:at + int(n)])
            at += int(n)
        return head.stream_finish_memory(sch, [0, 0], hidden, ids, lex, cache, out=out)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        out = step()
        ref = _outputs(out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(out)
        keep = hidden.clone()
        for x in (torch.roll(keep, 1, 1), keep):
            hidden.copy_(x)
            graph.replay()
            torch.cuda.synchronize()
            got = _outputs(out)
            eager = _outputs(step())
            for name in ref:
                np.testing.assert_array_equal(got[name], eager[name])
    for name in ref:
        np.testing.assert_array_equal(got[name], ref[name])
    assert head.device_status() == 0 and cache.device_status() == 0
