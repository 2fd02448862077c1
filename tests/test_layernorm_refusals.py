"""Arguments that te_mx_layernorm and te_mx_layernorm_backward refuse on the
host, before any launch (no GPU needed), and the empty problems they accept."""
import os

import pytest

from mxfp8_block_scaled_quantize_gb300 import binding


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from mxfp8_block_scaled_quantize_gb300 import _build
        _build.build()
    return binding.lib()


FWD = dict(x=16, rows=4, hidden=64, ld_x=64, dtype=0, gamma=16, beta=16, param_dtype=0, eps=1e-5, y=16, ld_y=64, mu=16,
           rsigma=16, stream=0)
BWD = dict(dy=16, ld_dy=64, x=16, ld_x=64, rows=4, hidden=64, dtype=0, gamma=16, param_dtype=0, mu=16, rsigma=16, dx=16,
           ld_dx=64, dgamma=16, dbeta=16, workspace=16, workspace_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("change,error", [
    (dict(rows=-1), "INVALID_ARG"), (dict(hidden=-1), "INVALID_ARG"), (dict(dtype=3), "INVALID_ARG"),
    (dict(dtype=-1), "INVALID_ARG"), (dict(param_dtype=1), "INVALID_ARG"), (dict(dtype=2, param_dtype=0), "INVALID_ARG"),
    (dict(eps=0.0), "INVALID_ARG"), (dict(eps=-1.0), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"),
    (dict(eps=float("nan")), "INVALID_ARG"), (dict(x=0), "INVALID_ARG"), (dict(y=0), "INVALID_ARG"),
    (dict(gamma=0), "INVALID_ARG"), (dict(mu=0), "INVALID_ARG"), (dict(rsigma=0), "INVALID_ARG"),
    (dict(ld_x=63), "MISALIGNED"), (dict(ld_y=0), "MISALIGNED"), (dict(x=17), "MISALIGNED"), (dict(y=1), "MISALIGNED"),
    (dict(dtype=2, param_dtype=2, x=18), "MISALIGNED"), (dict(gamma=17), "MISALIGNED"), (dict(beta=17), "MISALIGNED"),
    (dict(param_dtype=2, gamma=18), "MISALIGNED"), (dict(mu=18), "MISALIGNED"),
    (dict(rows=1 << 31), "UNSUPPORTED_SHAPE"), (dict(hidden=(1 << 24) + 1, ld_x=1 << 25, ld_y=1 << 25), "UNSUPPORTED_SHAPE"),
])
def test_forward_refusals(change, error):
    with pytest.raises(binding.TemxError, match=error):
        binding.te_mx_layernorm(**{**FWD, **change})


@pytest.mark.parametrize("change,error", [
    (dict(rows=-1), "INVALID_ARG"), (dict(dtype=7), "INVALID_ARG"), (dict(param_dtype=1), "INVALID_ARG"),
    (dict(dgamma=0), "INVALID_ARG"), (dict(dx=0, dgamma=0, dbeta=0), "INVALID_ARG"), (dict(dy=0), "INVALID_ARG"),
    (dict(x=0), "INVALID_ARG"), (dict(gamma=0), "INVALID_ARG"), (dict(mu=0), "INVALID_ARG"),
    (dict(rsigma=0), "INVALID_ARG"), (dict(ld_dy=10), "MISALIGNED"), (dict(ld_x=10), "MISALIGNED"),
    (dict(ld_dx=10), "MISALIGNED"), (dict(dy=17), "MISALIGNED"), (dict(dx=17), "MISALIGNED"),
    (dict(dgamma=17), "MISALIGNED"), (dict(dbeta=17), "MISALIGNED"), (dict(rsigma=18), "MISALIGNED"),
    (dict(workspace=0), "WORKSPACE_TOO_SMALL"), (dict(workspace_bytes=100), "WORKSPACE_TOO_SMALL"),
    (dict(workspace=8), "MISALIGNED"), (dict(rows=1 << 31), "UNSUPPORTED_SHAPE"),
])
def test_backward_refusals(change, error):
    with pytest.raises(binding.TemxError, match=error):
        binding.te_mx_layernorm_backward(**{**BWD, **change})


def test_empty_problems_and_workspace():
    binding.te_mx_layernorm(**{**FWD, "rows": 0, "x": 0, "y": 0, "gamma": 0})
    binding.te_mx_layernorm(**{**FWD, "hidden": 0})
    binding.te_mx_layernorm_backward(**{**BWD, "hidden": 0})
    binding.te_mx_layernorm_backward(**{**BWD, "rows": 0, "dgamma": 0, "dbeta": 0})
    size = binding.te_mx_layernorm_backward_workspace_size
    assert size(0, 64) == 0 and size(64, 0) == 0 and size(-1, 64) == 0
    assert size(1, 64) >= 2 * 64 * 4 and size(100000, 64) < 1 << 20        # grows with the rows up to a limit
