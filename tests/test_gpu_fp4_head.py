"""The head with its memory K/V projection in 4 bits, against the oracle with the same 4-bit rows and weights.

The oracle's cross attention reads keys and values that follow from the definition: rows and LayerNorm-weighted
K/V weights as they stand once kept in 4 bits (bf16 first, as the head folds them), the row's own mean and rstd,
the sums of the kept weights.  Everything else of the oracle is as it is, so the acceptance is the head's own.
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle.clef_head as oracle_head
import synth
from fp4_support import EPS, kept
from gpu_support import LOGIT_TOL, PROB_TOL, compare, device_inputs, run_oracle, schema_of
from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300.head import ClefHead

pytestmark = pytest.mark.gpu

SHAPES = {"narrow": synth.HeadShape(H=320, D=128, heads=2, F=192, n_route=2, n_joint=2, vocab=3000),
          "pages": synth.HeadShape()}
_HEADS = {}


def fp4_head(name, form):
    if (name, form) not in _HEADS:
        s = SHAPES[name]
        w = synth.make_weights(s, 0)
        _HEADS[name, form] = (ClefHead(w, s.H, s.D, s.heads, s.F, s.n_route, s.n_joint, s.vocab, memory_format=form), w)
    return _HEADS[name, form]


def batch(name, lengths, seed):
    s = SHAPES[name]
    spec = synth.BatchSpec(name="fp4", B=len(lengths), H=s.H, vocab=s.vocab, lengths=lengths, questions=(2, 4), options=(2, 5))
    return synth.make_batch(spec, seed=seed)


def outputs(out):
    return {k: getattr(out, k).cpu().numpy() for k in ("logits", "probs", "q_value", "q_conf", "q_argmax")}


def forward(head, bt, hidden, ids, lex, **more):
    out = head.forward(schema_of(bt), hidden, ids, lex, **more)
    torch.cuda.synchronize()
    assert head.device_status() == 0
    return outputs(out)


@pytest.fixture
def kept_memory(monkeypatch):
    """The oracle with 4-bit keys and values; call with the format and a conversion of the hidden rows."""
    def use(form, rows=lambda x: x):
        raw = {}
        memory_rows, weights = oracle_head.memory_rows, {}

        def remember(hidden_b, L_b, p):
            mem = memory_rows(hidden_b, L_b, p)
            x = rows(oracle_head._f64(hidden_b[:L_b]))
            mean = x.mean(1, keepdims=True)
            rstd = 1 / np.sqrt(((x - mean) ** 2).mean(1, keepdims=True) + EPS)
            raw[id(mem)] = (mem, kept(x, form)[3], mean, rstd, p)
            return mem

        def project(mem, W, b):
            _, x, mean, rstd, p = raw[id(mem)]
            if id(W) not in weights:
                folded = torch.from_numpy(W * p["mem_ln.weight"]).bfloat16().double().numpy()
                weights[id(W)] = kept(folded, form)[3]
            w = weights[id(W)]
            return rstd * (x @ w.T - mean * w.sum(1)) + W @ p["mem_ln.bias"] + b

        def cross_attention(qx, mem, Wq, bq, Wk, bk, Wv, bv, heads):
            Q, K, V = oracle_head.linear(qx, Wq, bq), project(mem, Wk, bk), project(mem, Wv, bv)
            out = np.empty_like(Q)
            dh = Q.shape[1] // heads
            for h in range(heads):
                sl = slice(h * dh, (h + 1) * dh)
                out[:, sl] = oracle_head.softmax(Q[:, sl] @ K[:, sl].T / np.sqrt(dh), axis=1) @ V[:, sl]
            return out

        monkeypatch.setattr(oracle_head, "memory_rows", remember)
        monkeypatch.setattr(oracle_head, "cross_attention", cross_attention)
    return use


@pytest.mark.parametrize("form", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("name,lengths", [("narrow", [130, 127, 700]), ("pages", [300, 1100])])
def test_forward_matches_the_oracle_over_kept_rows(form, name, lengths, kept_memory):
    head, w = fp4_head(name, form)
    bt = batch(name, lengths, 71)
    got = forward(head, bt, *device_inputs(bt, SHAPES[name].vocab))
    kept_memory(form)
    compare(got, run_oracle(w, SHAPES[name], bt), bt)


def test_fp16_rows_are_quantised_as_they_are(kept_memory):
    """Pooling reads fp16 rows rounded to bf16; keys and values come from the fp16 rows."""
    head, w = fp4_head("narrow", "nvfp4")
    bt = batch("narrow", [260, 129], 72)
    hidden, ids, lex = device_inputs(bt, SHAPES["narrow"].vocab)
    g = torch.Generator(device="cuda").manual_seed(1)
    noise = 1 + 2.0 ** -9 * torch.rand(hidden.shape, generator=g, device="cuda")
    half = (hidden.float() * noise).half()
    got = forward(head, bt, half, ids, lex)
    x16, xb = half.double().cpu().numpy(), half.bfloat16()
    rounded = dataclasses.replace(bt, hidden=xb.view(torch.int16).cpu().numpy().view(np.uint16))
    at = {}
    for b in range(bt.B):
        at[xb[b, 0].double().cpu().numpy().tobytes()] = x16[b]
    kept_memory("nvfp4", lambda x: at[np.ascontiguousarray(x[0]).tobytes()][:len(x)])
    compare(got, run_oracle(w, SHAPES["narrow"], rounded), rounded)


@pytest.mark.parametrize("form", ["mxfp4", "nvfp4"])
def test_streamed_chunks_agree_with_the_forward_pass(form):
    """Chunks are other products of the same rows: equal but for the order of fp32 sums, so for single roundings of
    keys and values to bf16, which the head's acceptance has room for."""
    head, _ = fp4_head("pages", form)
    bt = batch("pages", [700, 200, 1300], 73)
    hidden, ids, lex = device_inputs(bt, SHAPES["pages"].vocab)
    whole = forward(head, bt, hidden, ids, lex)
    sch = schema_of(bt)
    head.stream_begin(sch)
    for b, n in enumerate(bt.lengths):
        for r in range(0, int(n), 90 + 300 * b):
            head.stream_rows(sch, hidden, b, r, min(90 + 300 * b, int(n) - r))
    out = head.stream_finish(sch, hidden, ids, lex)
    torch.cuda.synchronize()
    assert head.device_status() == 0
    streamed = outputs(out)
    assert np.abs(streamed["logits"] - whole["logits"]).max() <= LOGIT_TOL
    assert np.abs(streamed["probs"] - whole["probs"]).max() <= PROB_TOL


def test_full_records_are_projected_together():
    """Records without padding between them run as one product; each alone gives the same."""
    head, _ = fp4_head("pages", "nvfp4")
    bt = batch("pages", [512, 512, 512], 74)
    inputs = device_inputs(bt, SHAPES["pages"].vocab)
    sch = schema_of(bt)
    w = head.memory_weights
    assert B.clef_head_forward_fp4_scratch(head.cfg, w.struct.format, sch) == \
        B.clef_stream_rows_fp4_scratch(head.cfg, w.struct.format, 3 * 512)
    whole = forward(head, bt, *inputs)
    head.stream_begin(sch)
    for b in range(3):
        head.stream_rows(sch, inputs[0], b, 0, 512)
    single = outputs(head.stream_finish(sch, *inputs))
    for k in whole:
        np.testing.assert_array_equal(whole[k], single[k])


def test_rows_apart_in_memory():
    """A row stride wider than the rows: the same outputs."""
    head, _ = fp4_head("narrow", "mxfp4")
    bt = batch("narrow", [256, 256, 140], 78)
    vocab = SHAPES["narrow"].vocab
    want = forward(head, bt, *device_inputs(bt, vocab))
    hidden, ids, lex = device_inputs(bt, vocab, bt.H + 72)
    out = head.forward(schema_of(bt, bt.H + 72), hidden, ids, lex)
    torch.cuda.synchronize()
    assert head.device_status() == 0
    for k, v in outputs(out).items():
        np.testing.assert_array_equal(v, want[k])


def test_kept_memory_over_a_4_bit_projection():
    head, _ = fp4_head("pages", "nvfp4")
    bt = batch("pages", [400, 900], 75)
    hidden, ids, lex = device_inputs(bt, SHAPES["pages"].vocab)
    whole = forward(head, bt, hidden, ids, lex)
    sch = schema_of(bt)
    cache = head.memory_cache(32, requests=2, max_len=1024)
    slots, _ = cache.plan(torch.tensor([400, 900], dtype=torch.int32, device="cuda"), 1300)
    head.stream_begin(sch)
    at = 0
    for b, n in enumerate((400, 900)):
        head.stream_rows(sch, hidden, b, 0, n)
        head.memory_store(sch, b, 0, n, cache, slots[at:at + n])
        at += n
    out = head.stream_finish_memory(sch, [0, 0], hidden, ids, lex, cache)
    torch.cuda.synchronize()
    assert head.device_status() == 0 and cache.device_status() == 0
    got = outputs(out)
    assert np.isfinite(got["logits"]).all()
    # 4-bit keys and values move the logits of random weights by some hundredths
    assert np.abs(got["logits"] - whole["logits"]).max() <= 0.1


def test_forward_replays_from_a_graph_beside_another():
    """Two captured passes share nothing but the workspace, which they use one after the other."""
    head, _ = fp4_head("pages", "nvfp4")
    bt = batch("pages", [600, 200], 76)
    other = dataclasses.replace(bt, hidden=batch("pages", [600, 200], 77).hidden)
    hidden, ids, lex = device_inputs(bt, SHAPES["pages"].vocab)
    second = device_inputs(other, SHAPES["pages"].vocab)[0]
    sch = schema_of(bt)
    want = [forward(head, bt, h, ids, lex) for h in (hidden, second)]
    stream, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(stream):
        for h in (hidden, second):
            out = head.alloc_outputs(sch)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                head.forward(sch, h, ids, lex, out=out)
            graphs.append((g, out))
        for k in (0, 1, 1, 0):
            g, out = graphs[k]
            g.replay()
            torch.cuda.synchronize()
            assert head.device_status() == 0
            for key, v in want[k].items():
                np.testing.assert_array_equal(outputs(out)[key], v)
