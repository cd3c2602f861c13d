"""Calls of the head over 4 bits that are refused, or that are made without a check."""
import pytest
import torch

from gpu_support import device_inputs, schema_of
from structured_decision_model_gb300 import binding as B
from test_gpu_fp4_head import SHAPES, batch, fp4_head

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
