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


BACKWARD = dict(dh=16, ld_dh=64, gate_up=16, ld_gate_up=128, rows=40, F=64, activation=0, d_gate_up=16, ld_d=128, q_row=16,
                s_row=16, ld_s_row=16, q_col=16, ld_q_col=128, s_col=16, ld_s_col=16, stream=0)


@pytest.mark.parametrize("change,error", [
    (dict(rows=-1), "INVALID_ARG"), (dict(F=-32), "INVALID_ARG"), (dict(activation=3), "INVALID_ARG"),
    (dict(q_row=0), "INVALID_ARG"), (dict(s_row=0), "INVALID_ARG"), (dict(q_col=0), "INVALID_ARG"),
    (dict(s_col=0), "INVALID_ARG"), (dict(dh=0), "INVALID_ARG"), (dict(gate_up=0), "INVALID_ARG"),
    (dict(F=40), "UNSUPPORTED_SHAPE"), (dict(F=48), "UNSUPPORTED_SHAPE"), (dict(rows=1 << 31), "UNSUPPORTED_SHAPE"),
    (dict(F=1 << 30), "UNSUPPORTED_SHAPE"), (dict(ld_dh=56), "MISALIGNED"), (dict(ld_dh=68), "MISALIGNED"),
    (dict(ld_gate_up=120), "MISALIGNED"), (dict(ld_gate_up=132), "MISALIGNED"), (dict(ld_d=64), "MISALIGNED"),
    (dict(dh=8), "MISALIGNED"), (dict(gate_up=8), "MISALIGNED"), (dict(d_gate_up=8), "MISALIGNED"),
    (dict(q_row=8), "MISALIGNED"), (dict(q_col=8), "MISALIGNED"), (dict(s_row=8), "MISALIGNED"),
    (dict(s_col=8), "MISALIGNED"), (dict(ld_s_row=0), "MISALIGNED"), (dict(ld_s_row=24), "MISALIGNED"),
    (dict(ld_q_col=64), "MISALIGNED"), (dict(ld_q_col=136), "MISALIGNED"), (dict(ld_s_col=0), "MISALIGNED"),
    (dict(rows=4000, ld_q_col=4096), "MISALIGNED"),
])
def test_backward_refusals(change, error):
    with pytest.raises(binding.TemxError, match=error):
        binding.te_mx_gated_backward(**{**BACKWARD, **change})


def test_backward_empty_problems():
    binding.te_mx_gated_backward(**{**BACKWARD, "rows": 0})
    binding.te_mx_gated_backward(**{**BACKWARD, "F": 0})
    binding.te_mx_gated_backward(**{**BACKWARD, "d_gate_up": 0, "q_row": 0, "s_row": 0, "q_col": 0, "s_col": 0})
