"""Tensors of the wrong rank are refused as such by the Python layer of the
operators around the expert products, whatever their rank."""
import pytest
import torch

from fp8_fine_grained_token_amd import moe as M


def rows():
    return torch.zeros((8, 64), dtype=torch.bfloat16)


@pytest.mark.parametrize("shape", [(), (4,), (2, 2, 2)])
@pytest.mark.parametrize("call", [
    lambda s: M.fp8_moe_combine(rows(), s), lambda s: M.fp8_moe_dispatch_grad(rows(), s),
    lambda s: M.fp8_moe_combine_grad(rows(), rows(), s), lambda s: M.fp8_moe_dispatch(rows(), s),
    lambda s: M.fp8_moe_dispatch_quant_1x128(rows(), s)])
def test_plan_of_another_rank(call, shape):
    with pytest.raises(ValueError, match="slot_row must have shape"):
        call(torch.zeros(shape, dtype=torch.int32))
