"""The largest sizes that the router, sort, dispatch and combine entry points take
(no GPU needed: what is accepted reaches a check behind the sizes')."""
import os

import pytest

from mxfp8_block_scaled_quantize_gb300 import binding
from tests.test_moe_refusals import CALLS


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from mxfp8_block_scaled_quantize_gb300 import _build
        _build.build()
    return binding.lib()


@pytest.mark.parametrize("k", [1, 2, 3, 5, 6, 7, 8, 31, 32])
@pytest.mark.parametrize("op,missing", [("route", "logits"), ("route_bwd", "index"), ("dispatch", "x"), ("combine", "row"), ("combine_bwd", "row")])
def test_tokens_times_choices_up_to_the_limit(op, missing, k):
    call, args = CALLS[op]
    change = {"k": k, missing: 0}                       # an operand is missing: refused as such where the sizes pass
    if "experts" in args:
        change.update(experts=64, ld_logits=64)
    for width in ("row_bytes", "hidden"):
        if width in args:
            change[width] = 1
    most = ((1 << 31) - 1) // k                         # tokens * k < 2^31
    for tokens, error in ((most, "INVALID_ARG"), (most + 1, "UNSUPPORTED_SHAPE")):
        with pytest.raises(binding.TemxError, match=error):
            call(**{**args, **change, "tokens": tokens})
