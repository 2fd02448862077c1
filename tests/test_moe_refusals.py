"""Arguments that the RMSNorm, router, sorting, dispatch and combine entry points
refuse on the host, before any launch (no GPU needed), and the empty problems they
accept."""
import os

import pytest

from mxfp8_block_scaled_quantize_gb300 import binding


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from mxfp8_block_scaled_quantize_gb300 import _build
        _build.build()
    return binding.lib()


# buffers a megabyte apart
B = [(i + 1) << 20 for i in range(12)]
CALLS = {
    "rms": (binding.te_mx_rmsnorm, dict(x=B[0], rows=4, hidden=64, ld_x=64, dtype=0, residual=B[1], ld_residual=64, gamma=B[2],
                                        param_dtype=0, eps=1e-5, z=B[3], ld_z=64, y=B[4], ld_y=64, rsigma=B[5], stream=0)),
    "rmsq": (binding.te_mx_rmsnorm_quantize,
             dict(x=B[0], rows=32, hidden=64, ld_x=64, residual=B[1], ld_residual=64, gamma=B[2], param_dtype=0, eps=1e-5,
                  z=B[3], ld_z=64, y=B[4], ld_y=64, q_row=B[5], s_row=B[6], ld_s_row=16, q_col=B[7], s_col=B[8], ld_s_col=16,
                  rsigma=B[9], stream=0)),
    "rms_bwd": (binding.te_mx_rmsnorm_backward,
                dict(dy=B[0], ld_dy=64, z=B[1], ld_z=64, rows=4, hidden=64, dtype=0, gamma=B[2], param_dtype=0, rsigma=B[3],
                     dz=B[4], ld_dz=64, dx=B[5], ld_dx=64, dgamma=B[6], workspace=B[7], workspace_bytes=1 << 20, stream=0)),
    "route": (binding.te_mx_route, dict(logits=B[0], tokens=4, experts=8, ld_logits=8, dtype=0, bias=B[1], k=2, scoring=0,
                                        renormalise=1, scale=1.0, index=B[2], weight=B[3], stream=0)),
    "route_bwd": (binding.te_mx_route_backward,
                  dict(dweight=B[0], logits=B[1], ld_logits=8, index=B[2], tokens=4, experts=8, dtype=0, k=2, scoring=0,
                       renormalise=1, scale=1.0, dlogits=B[3], ld_dlogits=8, stream=0)),
    "sort": (binding.te_mx_moe_sort, dict(index=B[0], slots=100, experts=8, group_m=B[1], row=B[2], slot=B[3], stream=0)),
    "dispatch": (binding.te_mx_moe_dispatch,
                 dict(x=B[0], ld_x=64, row_bytes=64, scales=B[1], ld_scales=16, scale_bytes=2, row=B[2], tokens=4, k=2,
                      total_rows=8, out=B[3], ld_out=64, out_scales=B[4], ld_out_scales=16, stream=0)),
    "combine": (binding.te_mx_moe_combine,
                dict(y=B[0], ld_y=64, total_rows=8, hidden=64, dtype=0, row=B[1], tokens=4, k=2, weight=B[2], residual=B[3],
                     ld_residual=64, out=B[4], ld_out=64, stream=0)),
    "combine_bwd": (binding.te_mx_moe_combine_backward,
                    dict(dout=B[0], ld_dout=64, y=B[1], ld_y=64, total_rows=8, hidden=64, dtype=0, row=B[2], weight=B[3],
                         tokens=4, k=2, dy=B[4], ld_dy=64, dweight=B[5], stream=0)),
}
ARG, SHAPE, ALIGN, SPACE = "INVALID_ARG", "UNSUPPORTED_SHAPE", "MISALIGNED", "WORKSPACE_TOO_SMALL"
INF, NAN = float("inf"), float("nan")

REFUSED = [
    ("rms", dict(rows=-1), ARG), ("rms", dict(hidden=-1), ARG), ("rms", dict(dtype=3), ARG), ("rms", dict(param_dtype=1), ARG),
    ("rms", dict(dtype=2, param_dtype=0), ARG), ("rms", dict(eps=0.0), ARG), ("rms", dict(eps=INF), ARG), ("rms", dict(eps=NAN), ARG),
    ("rms", dict(x=0), ARG), ("rms", dict(y=0), ARG), ("rms", dict(gamma=0), ARG), ("rms", dict(z=0), ARG),
    ("rms", dict(residual=0), ARG), ("rms", dict(ld_x=63), ALIGN), ("rms", dict(ld_y=0), ALIGN), ("rms", dict(ld_z=63), ALIGN),
    ("rms", dict(ld_residual=63), ALIGN), ("rms", dict(x=B[0] + 1), ALIGN), ("rms", dict(gamma=B[2] + 1), ALIGN),
    ("rms", dict(param_dtype=2, gamma=B[2] + 2), ALIGN), ("rms", dict(rsigma=B[5] + 2), ALIGN), ("rms", dict(rows=1 << 31), SHAPE),
    ("rms", dict(hidden=(1 << 24) + 1), SHAPE), ("rms", dict(y=B[3]), ARG), ("rms", dict(z=B[0] + 2), ARG),
    ("rms", dict(z=B[0], ld_z=72), ARG), ("rms", dict(y=B[0] + 128 * 3), ARG), ("rms", dict(y=B[1] + 64), ARG),
    ("rmsq", dict(hidden=48), SHAPE), ("rmsq", dict(rows=48), SHAPE), ("rmsq", dict(rsigma=0), ARG), ("rmsq", dict(s_row=0), ARG),
    ("rmsq", dict(q_col=0), ARG), ("rmsq", dict(x=B[0] + 8), ALIGN), ("rmsq", dict(z=B[3] + 8), ALIGN), ("rmsq", dict(y=B[4] + 8), ALIGN),
    ("rmsq", dict(residual=B[1] + 8), ALIGN), ("rmsq", dict(gamma=B[2] + 8), ALIGN), ("rmsq", dict(ld_x=68), ALIGN),
    ("rmsq", dict(ld_z=68), ALIGN), ("rmsq", dict(ld_y=68), ALIGN), ("rmsq", dict(ld_residual=68), ALIGN), ("rmsq", dict(ld_s_row=15), ALIGN),
    ("rmsq", dict(ld_s_col=8), ALIGN), ("rmsq", dict(q_row=B[5] + 8), ALIGN), ("rmsq", dict(eps=-1.0), ARG), ("rmsq", dict(param_dtype=1), ARG),
    ("rmsq", dict(hidden=32800, ld_x=32800, ld_residual=32800, ld_z=32800, ld_y=32800, ld_s_row=2064), SHAPE),
    ("rmsq", dict(residual=0, z=0, y=B[0]), ARG), ("rmsq", dict(z=0), ARG), ("rmsq", dict(y=B[3]), ARG),
    ("rms_bwd", dict(rows=-1), ARG), ("rms_bwd", dict(dtype=7), ARG), ("rms_bwd", dict(dx=0, dgamma=0), ARG), ("rms_bwd", dict(dy=0), ARG),
    ("rms_bwd", dict(z=0), ARG), ("rms_bwd", dict(gamma=0), ARG), ("rms_bwd", dict(rsigma=0), ARG), ("rms_bwd", dict(ld_dy=10), ALIGN),
    ("rms_bwd", dict(ld_z=10), ALIGN), ("rms_bwd", dict(ld_dz=10), ALIGN), ("rms_bwd", dict(ld_dx=10), ALIGN),
    ("rms_bwd", dict(dgamma=B[6] + 1), ALIGN), ("rms_bwd", dict(workspace=0), SPACE), ("rms_bwd", dict(workspace_bytes=100), SPACE),
    ("rms_bwd", dict(workspace=B[7] + 8), ALIGN), ("rms_bwd", dict(rows=1 << 31), SHAPE), ("rms_bwd", dict(dx=B[0] + 2), ARG),
    ("rms_bwd", dict(dx=B[1], ld_dx=80), ARG), ("rms_bwd", dict(dx=B[4] + 128), ARG),
    ("rms_bwd", dict(dgamma=B[2]), ARG), ("rms_bwd", dict(dgamma=B[2] + 126, dx=0), ARG),
    ("route", dict(tokens=-1), ARG), ("route", dict(dtype=3), ARG), ("route", dict(scoring=2), ARG), ("route", dict(renormalise=2), ARG),
    ("route", dict(scale=INF), ARG), ("route", dict(scale=NAN), ARG), ("route", dict(k=0), SHAPE), ("route", dict(k=33, experts=64, ld_logits=64), SHAPE),
    ("route", dict(k=9), SHAPE), ("route", dict(experts=1025, ld_logits=1025), SHAPE), ("route", dict(tokens=1 << 30), SHAPE),
    ("route", dict(logits=0), ARG), ("route", dict(index=0), ARG), ("route", dict(weight=0), ARG), ("route", dict(ld_logits=7), ALIGN),
    ("route", dict(logits=B[0] + 1), ALIGN), ("route", dict(bias=B[1] + 2), ALIGN), ("route", dict(weight=B[3] + 2), ALIGN),
    ("route_bwd", dict(dweight=0), ARG), ("route_bwd", dict(index=0), ARG), ("route_bwd", dict(dlogits=0), ARG),
    ("route_bwd", dict(ld_dlogits=7), ALIGN), ("route_bwd", dict(dlogits=B[1]), ARG), ("route_bwd", dict(scoring=-1), ARG),
    ("sort", dict(slots=-1), ARG), ("sort", dict(slots=1 << 31), SHAPE), ("sort", dict(experts=0), SHAPE), ("sort", dict(experts=1025), SHAPE),
    ("sort", dict(group_m=0), ARG), ("sort", dict(index=0), ARG), ("sort", dict(row=0), ARG), ("sort", dict(slot=0), ARG),
    ("sort", dict(row=B[2] + 2), ALIGN), ("sort", dict(row=B[0]), ARG), ("sort", dict(slot=B[2] + 8), ARG),
    ("sort", dict(group_m=B[0] + 396), ARG), ("sort", dict(group_m=B[2] - 28), ARG), ("sort", dict(group_m=B[3]), ARG),
    ("dispatch", dict(tokens=-1), ARG), ("dispatch", dict(total_rows=-1), ARG), ("dispatch", dict(row_bytes=-1), ARG), ("dispatch", dict(k=0), SHAPE),
    ("dispatch", dict(k=33), SHAPE), ("dispatch", dict(tokens=1 << 30), SHAPE), ("dispatch", dict(total_rows=1 << 31), SHAPE),
    ("dispatch", dict(row_bytes=1 << 38, ld_x=1 << 38, ld_out=1 << 38), SHAPE), ("dispatch", dict(scales=0), ARG),
    ("dispatch", dict(out_scales=0), ARG), ("dispatch", dict(x=0), ARG), ("dispatch", dict(out=0), ARG), ("dispatch", dict(row=0), ARG),
    ("dispatch", dict(row=B[2] + 1), ALIGN), ("dispatch", dict(ld_x=63), ALIGN), ("dispatch", dict(ld_out=63), ALIGN),
    ("dispatch", dict(ld_scales=1), ALIGN), ("dispatch", dict(ld_out_scales=1), ALIGN), ("dispatch", dict(scale_bytes=-1), ARG),
    ("dispatch", dict(out=B[0]), ARG), ("dispatch", dict(out_scales=B[1]), ARG),
    ("combine", dict(tokens=-1), ARG), ("combine", dict(hidden=-1), ARG), ("combine", dict(dtype=3), ARG), ("combine", dict(k=0), SHAPE),
    ("combine", dict(k=33), SHAPE), ("combine", dict(hidden=(1 << 24) + 1), SHAPE), ("combine", dict(y=0), ARG), ("combine", dict(row=0), ARG),
    ("combine", dict(out=0), ARG), ("combine", dict(ld_y=63), ALIGN), ("combine", dict(ld_residual=63), ALIGN), ("combine", dict(ld_out=63), ALIGN),
    ("combine", dict(weight=B[2] + 2), ALIGN), ("combine", dict(out=B[0]), ARG), ("combine", dict(out=B[3] + 2), ARG),
    ("combine_bwd", dict(weight=0), ARG), ("combine_bwd", dict(dy=0, dweight=0), ARG), ("combine_bwd", dict(dout=0), ARG),
    ("combine_bwd", dict(y=0), ARG), ("combine_bwd", dict(ld_dout=63), ALIGN), ("combine_bwd", dict(ld_dy=63), ALIGN),
    ("combine_bwd", dict(dweight=B[5] + 2), ALIGN), ("combine_bwd", dict(dy=B[0]), ARG), ("combine_bwd", dict(dy=B[1] + 2), ARG),
]


@pytest.mark.parametrize("op,change,error", REFUSED)
def test_refusals(op, change, error):
    call, args = CALLS[op]
    with pytest.raises(binding.TemxError, match=error):
        call(**{**args, **change})


def reaches_the_device(op, change):
    """Accepted by every check before the device's (which fails where there is no GPU; where
    there is one the call must not be made: the addresses are not real)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    call, args = CALLS[op]
    with pytest.raises(binding.TemxError, match="TE_MX_ERR_CUDA|TE_MX_ERR_ARCH"):
        call(**{**args, **change})


@pytest.mark.parametrize("op,change", [
    ("rms", {}), ("rms", dict(z=B[0])), ("rms", dict(z=B[1])), ("rms", dict(y=B[0])), ("rms", dict(y=B[1])),
    ("rms", dict(residual=0, z=0, y=B[0])), ("rms", dict(rsigma=0)),
    # z and y beside x in one wider buffer
    ("rms", dict(ld_x=192, z=B[0] + 128, ld_z=192, y=B[0] + 256, ld_y=192)),
    ("rmsq", {}), ("rmsq", dict(y=0)), ("rmsq", dict(y=B[0])), ("rmsq", dict(residual=0, z=0, y=B[0], q_col=0, s_col=0)),
    ("rmsq", dict(q_row=0, s_row=0, q_col=0, s_col=0)), ("rms_bwd", {}), ("rms_bwd", dict(dz=0)), ("rms_bwd", dict(dx=B[0])),
    ("rms_bwd", dict(dx=B[1])), ("rms_bwd", dict(dx=B[4])), ("rms_bwd", dict(dx=0)),
    ("rms_bwd", dict(dgamma=0, workspace=0, workspace_bytes=0)), ("rms_bwd", dict(rows=0)), ("route", {}), ("route", dict(bias=0)),
    ("route_bwd", {}), ("sort", {}), ("sort", dict(slots=0)), ("dispatch", {}), ("dispatch", dict(scales=0, out_scales=0)),
    ("dispatch", dict(total_rows=0, out=0)), ("combine", {}), ("combine", dict(weight=0, residual=0)), ("combine", dict(out=B[3])),
    ("combine", dict(total_rows=0, y=0)), ("combine_bwd", {}), ("combine_bwd", dict(dy=B[1])), ("combine_bwd", dict(dy=0)),
    ("combine_bwd", dict(dweight=0, y=0)), ("combine_bwd", dict(total_rows=0, y=0, dy=0, dweight=0)),
    ("sort", dict(group_m=B[2] - 32)), ("rms_bwd", dict(dgamma=B[2] + 128)),
])
def test_accepted(op, change):
    reaches_the_device(op, change)


def test_empty_problems_and_workspace():
    for op, change in [("rms", dict(rows=0, x=0, y=0)), ("rms", dict(hidden=0)), ("rmsq", dict(rows=0)), ("rmsq", dict(hidden=0)),
                       ("rms_bwd", dict(hidden=0)), ("rms_bwd", dict(rows=0, dgamma=0)), ("route", dict(tokens=0, logits=0)),
                       ("route_bwd", dict(tokens=0)), ("dispatch", dict(tokens=0)), ("dispatch", dict(row_bytes=0)),
                       ("combine", dict(tokens=0)), ("combine", dict(hidden=0)), ("combine_bwd", dict(tokens=0)),
                       ("combine_bwd", dict(hidden=0))]:
        call, args = CALLS[op]
        call(**{**args, **change})
    size = binding.te_mx_rmsnorm_backward_workspace_size
    assert size(0, 64) == 0 and size(64, 0) == 0 and size(-1, 64) == 0
    assert size(1, 64) >= 64 * 4 and size(100000, 64) < 1 << 20        # grows with the rows up to a limit
