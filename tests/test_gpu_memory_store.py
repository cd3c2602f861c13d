"""The head's kept memory comes from the workspace that the rows were streamed into, or from nowhere."""
import pytest
import torch

import synth
from structured_decision_model_gb300 import binding as B
from structured_decision_model_gb300.build import build_library

from gpu_support import device_inputs, head_for, schema_of

pytestmark = pytest.mark.gpu

FULL = synth.HeadShape()


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_library()
    B.load()


def test_a_schema_that_was_not_streamed_stores_nothing():
    """A larger schema than the streamed one is refused, and the streamed rows are still there to be kept."""
    small = synth.make_batch(synth.BatchSpec(name="small", B=1, lengths=[300], questions=(2, 3), options=(2, 4)), seed=5)
    large = synth.make_batch(synth.BatchSpec(name="large", B=2, lengths=[4000, 4000], questions=(2, 3), options=(2, 4)), seed=6)
    head, _ = head_for(FULL)
    head._ws = None
    hidden = device_inputs(small, FULL.vocab)[0]
    sch = schema_of(small)
    cache = head.memory_cache(20, 1, 640)
    slots, _ = cache.plan(torch.tensor([300], dtype=torch.int32, device="cuda"), 300)
    with pytest.raises(B.ClefError):                             # nothing streamed at all
        head.memory_store(sch, 0, 0, 300, cache, slots)
    head.stream_begin(sch)
    head.stream_rows(sch, hidden, 0, 0, 300)
    head.memory_store(sch, 0, 0, 300, cache, slots)
    want = cache.read(slots, torch.float32)
    before = cache.data.clone()
    with pytest.raises(B.ClefError) as e:
        head.memory_store(schema_of(large), 0, 0, 300, cache, slots)
    assert e.value.status == 2
    assert torch.equal(cache.data, before)
    cache.data.zero_()
    head.memory_store(sch, 0, 0, 300, cache, slots)
    for got, ref in zip(cache.read(slots, torch.float32), want):
        assert torch.equal(got, ref) and ref.abs().max() > 0
    assert cache.device_status() == 0
