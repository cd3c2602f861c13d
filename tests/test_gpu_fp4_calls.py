"""Calls of the 4-bit operators as programs make them: reports, captures, streams, arguments that change or are refused."""
import pytest
import torch

from structured_decision_model_gb300.microscaled import Fp4Linear, quantize

pytestmark = pytest.mark.gpu

BOUNDS, TIMEOUT = 1, 2  # bits that kernels set


def rows_of(rows, cols, seed=0, dtype=torch.bfloat16):
    return torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


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
