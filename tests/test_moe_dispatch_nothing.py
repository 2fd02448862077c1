"""Dispatch of codes with scales where there is nothing to copy: no tokens, or no rows
because every slot was dropped (tensors without elements have no address)."""
import os

import pytest
import torch

from mxfp8_block_scaled_quantize_gb300 import binding
from tests.test_moe_refusals import B, CALLS, reaches_the_device


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from mxfp8_block_scaled_quantize_gb300 import _build
        _build.build()
    return binding.lib()


def test_dispatch_of_no_tokens_or_to_no_rows_with_scales():
    call, args = CALLS["dispatch"]
    call(**{**args, "tokens": 0, "x": 0, "scales": 0, "row": 0})
    call(**{**args, "tokens": 0, "x": 0, "scales": 0, "row": 0, "out": 0, "out_scales": 0, "total_rows": 0})
    call(**{**args, "row_bytes": 0, "scales": 0})
    for change in (dict(out_scales=0), dict(scales=0), dict(out=0)):
        with pytest.raises(binding.TemxError, match="INVALID_ARG"):
            call(**{**args, **change})


@pytest.mark.parametrize("change", [dict(total_rows=0, out=0, out_scales=0), dict(total_rows=0, out=0, out_scales=B[4])])
def test_dispatch_to_no_rows_reaches_the_device(change):
    reaches_the_device("dispatch", change)


@pytest.mark.gpu
def test_no_tokens_and_no_rows():
    q = torch.zeros(6, 64, dtype=torch.uint8, device="cuda")
    s = torch.zeros(6, 16, dtype=torch.uint8, device="cuda")
    row = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    for total in (None, 0, 5):
        d, ds = binding.moe_dispatch(q[:0], row[:0], scales=s[:0], total_rows=total)
        assert d.shape == (total or 0, 64) and ds.shape == (total or 0, 16)
    d, ds = binding.moe_dispatch(q, row, scales=s, total_rows=0)
    assert d.shape == (0, 64) and ds.shape == (0, 16)
    assert binding.moe_dispatch(q, row, total_rows=0).shape == (0, 64)
    binding.te_mx_device_status()
    # a row that is named all the same is out of range, and reported
    row[3, 1] = 0
    binding.moe_dispatch(q, row, scales=s, total_rows=0)
    with pytest.raises(binding.TemxError, match="INVALID_ARG"):
        binding.te_mx_device_status()
