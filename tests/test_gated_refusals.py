"""Arguments that the gated feed-forward entry points refuse on the host,
before any launch (no GPU needed), and the empty problems they accept."""
import os

import pytest

from mxfp8_block_scaled_quantize_gb300 import binding


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from mxfp8_block_scaled_quantize_gb300 import _build
        _build.build()
    return binding.lib()


GEMM = dict(A=16, sA=16, ld_sA=16, W=16, sW=16, ld_sW=16, M=4, F=64, K=256, bias=16, activation=0, D=16, aux=16, stream=0)
GROUPED = dict(num_groups=2, group_m=16, total_m=8, X=16, sX=16, ld_sX=16, W=16, sW=16, ld_sW=16, F=64, K=256, bias=16,
               activation=0, D=16, aux=16, stream=0)
COMMON = [
    (dict(activation=3), "INVALID_ARG"), (dict(activation=-1), "INVALID_ARG"), (dict(W=0), "INVALID_ARG"),
    (dict(sW=0), "INVALID_ARG"), (dict(D=0), "INVALID_ARG"), (dict(K=0), "UNSUPPORTED_SHAPE"),
    (dict(K=192), "UNSUPPORTED_SHAPE"), (dict(F=0), "UNSUPPORTED_SHAPE"), (dict(F=40), "UNSUPPORTED_SHAPE"),
    (dict(F=-16), "UNSUPPORTED_SHAPE"), (dict(F=1 << 30), "UNSUPPORTED_SHAPE"), (dict(ld_sW=8), "MISALIGNED"),
    (dict(K=1024), "MISALIGNED"), (dict(W=8), "MISALIGNED"), (dict(D=8), "MISALIGNED"), (dict(aux=8), "MISALIGNED"),
    (dict(bias=8), "MISALIGNED"),
]


@pytest.mark.parametrize("change,error", COMMON + [
    (dict(M=-1), "INVALID_ARG"), (dict(A=0), "INVALID_ARG"), (dict(sA=0), "INVALID_ARG"),
    (dict(M=1 << 31), "UNSUPPORTED_SHAPE"), (dict(A=8), "MISALIGNED"), (dict(ld_sA=24), "MISALIGNED")])
def test_gemm_refusals(change, error):
    with pytest.raises(binding.TemxError, match=error):
        binding.te_mx_gated_gemm(**{**GEMM, **change})


@pytest.mark.parametrize("change,error", COMMON + [
    (dict(num_groups=0), "INVALID_ARG"), (dict(num_groups=1025), "INVALID_ARG"), (dict(group_m=0), "INVALID_ARG"),
    (dict(group_m=18), "MISALIGNED"), (dict(total_m=-1), "INVALID_ARG"), (dict(total_m=1 << 31), "UNSUPPORTED_SHAPE"),
    (dict(num_groups=1024, F=1 << 20), "UNSUPPORTED_SHAPE"), (dict(X=0), "INVALID_ARG")])
def test_grouped_refusals(change, error):
    with pytest.raises(binding.TemxError, match=error):
        binding.te_mx_grouped_gated_gemm(**{**GROUPED, **change})


def test_empty_problems():
    binding.te_mx_gated_gemm(**{**GEMM, "M": 0})
    binding.te_mx_grouped_gated_gemm(**{**GROUPED, "total_m": 0})
