"""Calls of the head over 4 bits that are refused, or that are made without a check, and the wide head."""
import pytest
import torch

import synth
from gpu_support import LOGIT_TOL, compare, device_inputs, run_oracle, schema_of
from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300.head import ClefHead
from test_gpu_fp4_head import SHAPES, batch, forward, fp4_head, kept_memory, outputs  # noqa: F401

pytestmark = pytest.mark.gpu


def test_hidden_rows_of_other_types_are_refused():
    head, _ = fp4_head("narrow", "nvfp4")
    bt = batch("narrow", [140, 200], 81)
    hidden, ids, lex = device_inputs(bt, SHAPES["narrow"].vocab)
    sch = schema_of(bt)
    for bad in (hidden.float(), hidden.double(), hidden.cpu()):
        with pytest.raises(B.ClefError):
            head.forward(sch, bad, ids, lex)
        head.stream_begin(sch)
        with pytest.raises(B.ClefError):
            head.stream_rows(sch, bad, 0, 0, 10)
    torch.cuda.synchronize()
    assert head.device_status() == 0


def test_forward_without_a_check_returns():
    """check=False: a refused call returns, as the bf16 head's does, and nothing has run."""
    head, _ = fp4_head("narrow", "nvfp4")
    bt = batch("narrow", [140, 200], 82)
    hidden, ids, lex = device_inputs(bt, SHAPES["narrow"].vocab)
    out = head.alloc_outputs(schema_of(bt))
    out.logits.fill_(9.0)
    assert head.forward(schema_of(bt), hidden.view(-1)[1:], ids, lex, out=out, check=False) is out  # rows off 16 bytes
    torch.cuda.synchronize()
    assert (out.logits == 9).all()
    with pytest.raises(B.ClefError):
        head.forward(schema_of(bt), hidden.view(-1)[1:], ids, lex, out=out)


@pytest.mark.parametrize("form", ["mxfp4", "nvfp4"])
def test_the_5120_wide_head(form, kept_memory):
    """Twenty K tiles a row, ragged records, chunks: the same acceptance."""
    shape = synth.HeadShape(H=5120)
    w = synth.make_weights(shape, 0)
    head = ClefHead(w, shape.H, shape.D, shape.heads, shape.F, shape.n_route, shape.n_joint, shape.vocab, memory_format=form)
    spec = synth.BatchSpec(name="wide", B=3, H=shape.H, vocab=shape.vocab, lengths=[260, 700, 260], questions=(2, 4), options=(2, 5))
    bt = synth.make_batch(spec, seed=83)
    hidden, ids, lex = device_inputs(bt, shape.vocab)
    got = forward(head, bt, hidden, ids, lex)
    kept_memory(form)
    compare(got, run_oracle(w, shape, bt), bt)
    sch = schema_of(bt)
    head.stream_begin(sch)
    for b, n in enumerate(bt.lengths):
        for r in range(0, int(n), 128):
            head.stream_rows(sch, hidden, b, r, min(128, int(n) - r))
    streamed = outputs(head.stream_finish(sch, hidden, ids, lex))
    assert head.device_status() == 0
    assert abs(streamed["logits"] - got["logits"]).max() <= LOGIT_TOL


@pytest.mark.parametrize("form", ["mxfp4", "nvfp4"])
def test_short_chunks_in_one_launch_or_two(form):
    """A chunk of a few rows by itself goes in one launch, in a graph in two (its rows are long); keys and values are the same."""
    head, _ = fp4_head("pages", form)
    bt = batch("pages", [160, 300], 84)
    hidden, ids, lex = device_inputs(bt, SHAPES["pages"].vocab)
    sch = schema_of(bt)

    def rows(chunk):
        before = B.clef_kernel_launches()
        for b, n in enumerate(bt.lengths):
            for r in range(0, int(n), chunk):
                head.stream_rows(sch, hidden, b, r, min(chunk, int(n) - r))
        return B.clef_kernel_launches() - before

    def finish():
        out = outputs(head.stream_finish(sch, hidden, ids, lex))
        assert head.device_status() == 0
        return out

    head.stream_begin(sch)
    assert rows(8) == 20 + 38
    eager = finish()
    head.stream_begin(sch)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert rows(8) == 2 * (20 + 38)
    g.replay()
    for k, v in finish().items():
        assert (v == eager[k]).all()


@pytest.mark.parametrize("form", [None, "nvfp4"])
def test_finishing_over_other_types_is_refused(form):
    """The finish reads rows too, and so does a head in bf16, whose forward pass takes no fp16."""
    head, _ = fp4_head("narrow", form)
    bt = batch("narrow", [140, 200], 85)
    hidden, ids, lex = device_inputs(bt, SHAPES["narrow"].vocab)
    sch = schema_of(bt)
    head.stream_begin(sch)
    for b, n in enumerate(bt.lengths):
        head.stream_rows(sch, hidden, b, 0, int(n))
    with pytest.raises(B.ClefError):
        head.stream_finish(sch, hidden.float(), ids, lex)
    if form is None:
        for bad in (hidden.float(), hidden.double(), hidden.half()):
            with pytest.raises(B.ClefError):
                head.forward(sch, bad, ids, lex)
        with pytest.raises(B.ClefError):
            head.stream_rows(sch, hidden.float(), 0, 0, 10)
        bits = outputs(head.forward(sch, hidden.view(torch.int16), ids, lex))
        for k, v in outputs(head.forward(sch, hidden, ids, lex)).items():
            assert (v == bits[k]).all()
        head.stream_begin(sch)
        for b, n in enumerate(bt.lengths):
            head.stream_rows(sch, hidden, b, 0, int(n))
    finite = outputs(head.stream_finish(sch, hidden, ids, lex))
    assert head.device_status() == 0 and abs(finite["logits"]).max() < 100
