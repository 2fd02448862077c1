"""Outputs that lie over an operand or over each other where blocks would read what others
write: refused on the host, before any launch (no GPU needed); what lies beside is
accepted, in one buffer too."""
import os

import pytest

from mxfp8_block_scaled_quantize_gb300 import binding
from tests.test_moe_refusals import B, CALLS, reaches_the_device


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from mxfp8_block_scaled_quantize_gb300 import _build
        _build.build()
    return binding.lib()


# per entry point: the outputs that may lie over nothing of what follows them
APART = {
    "rms": {"rsigma": ("x", "residual", "gamma", "z", "y"), "z": ("gamma", "y"), "y": ("gamma",)},
    "rmsq": {"rsigma": ("x", "residual", "gamma", "z", "y"), "z": ("gamma", "y"), "y": ("gamma",),
             "q_row": ("x", "residual", "gamma", "z", "y", "rsigma"), "s_row": ("x", "residual", "gamma", "z", "y", "rsigma", "q_row"),
             "q_col": ("x", "residual", "gamma", "z", "y", "rsigma", "q_row", "s_row"),
             "s_col": ("x", "residual", "gamma", "z", "y", "rsigma", "q_row", "s_row", "q_col")},
    "rms_bwd": {"dx": ("gamma", "rsigma", "dgamma"), "dgamma": ("dy", "z", "dz", "gamma", "rsigma"),
                "workspace": ("dy", "z", "dz", "gamma", "rsigma", "dx", "dgamma")},
    "route": {"index": ("logits", "bias"), "weight": ("logits", "bias", "index")},
    "route_bwd": {"dlogits": ("logits", "dweight", "index")},
    "dispatch": {"out": ("x", "scales", "row"), "out_scales": ("x", "scales", "row", "out")},
    "combine": {"out": ("y", "row", "weight")},
    "combine_bwd": {"dy": ("dout", "row", "weight"), "dweight": ("dout", "y", "row", "dy")},
}
PAIRS = [(op, out, other) for op, outs in APART.items() for out, others in outs.items() for other in others]


@pytest.mark.parametrize("op,out,other", PAIRS)
def test_an_output_over_another_array_is_refused(op, out, other):
    call, args = CALLS[op]
    for change in ({out: args[other]}, {other: args[out]}):
        with pytest.raises(binding.TemxError, match="INVALID_ARG"):
            call(**{**args, **change})


@pytest.mark.parametrize("op,change", [
    # touching with one element at either end: four rows of 64 bf16, rsigma of 16 bytes
    ("rms", dict(rsigma=B[0] + 508)), ("rms", dict(rsigma=B[0] - 12)), ("rms", dict(rsigma=B[2] + 124)), ("rms", dict(y=B[2] - 510)),
    # over the rows of a pitched matrix
    ("rms", dict(ld_x=192, rsigma=B[0] + 384 * 3 + 124)), ("rms", dict(ld_x=192, rsigma=B[0] + 376)),
    # codes over x, the likely misuse, and scales over what the column-wise copy reads
    ("rmsq", dict(residual=0, z=0, q_row=B[0])), ("rmsq", dict(residual=0, z=0, y=0, s_row=B[0] + 4080)),
    ("rmsq", dict(rsigma=B[0] + 4092)), ("rmsq", dict(q_col=B[3] + 4080)), ("rmsq", dict(s_col=B[3] - 1008)),
    ("rms_bwd", dict(dgamma=B[3] + 12, dx=0)), ("rms_bwd", dict(workspace=B[0] + 496)),
    ("route", dict(weight=B[0] + 60)), ("route", dict(index=B[3] + 28)), ("route_bwd", dict(dlogits=B[0] + 30)),
    ("dispatch", dict(out=B[2] + 28)), ("dispatch", dict(ld_out=80, ld_out_scales=80, out_scales=B[3] + 63)),
    ("dispatch", dict(ld_out=80, ld_out_scales=80, out_scales=B[3] + 79)),
    ("combine", dict(out=B[2] + 28)), ("combine_bwd", dict(dweight=B[3] + 4)), ("combine_bwd", dict(dweight=B[3] - 28)),
    ("combine_bwd", dict(dy=B[5] + 28)),
])
def test_partial_overlaps_are_refused(op, change):
    call, args = CALLS[op]
    with pytest.raises(binding.TemxError, match="INVALID_ARG"):
        call(**{**args, **change})


@pytest.mark.parametrize("op,change", [
    ("rms", dict(rsigma=B[0] + 512)), ("rms", dict(rsigma=B[0] - 16)), ("rms", dict(rsigma=B[2] + 128)),
    ("rms", dict(ld_x=192, rsigma=B[0] + 128)),                            # behind a row of a pitched x
    ("rms", dict(rows=1, ld_x=192, ld_y=999, y=B[0])),                     # one row has no pitch
    ("rmsq", dict(q_row=B[0] + 4096, s_row=B[0] + 4096 + 2048)), ("rmsq", dict(rsigma=B[0] + 4096)),
    ("rmsq", dict(ld_s_row=32, ld_s_col=32, s_row=B[6], s_col=B[6] + 16)), # scales side by side in rows of one buffer
    ("rms_bwd", dict(dgamma=B[3] + 16)), ("rms_bwd", dict(workspace=B[0] + 512)),
    ("rms_bwd", dict(dgamma=0, workspace=B[0])),                           # not used
    ("route", dict(index=B[0] + 64)), ("route", dict(weight=B[2] + 32)), ("route", dict(ld_logits=24, weight=B[0] + 16)),
    ("route_bwd", dict(ld_logits=16, ld_dlogits=16, dlogits=B[1] + 16)),
    ("dispatch", dict(ld_out=80, ld_out_scales=80, out_scales=B[3] + 64)), # codes and scales in rows of one buffer
    ("dispatch", dict(ld_x=80, ld_scales=80, scales=B[0] + 64)), ("dispatch", dict(out_scales=B[3] + 512)),
    ("combine", dict(out=B[2] + 32)), ("combine_bwd", dict(dweight=B[3])), # each slot's weight is read by the warp that writes
    ("combine_bwd", dict(dweight=B[3] + 32)),
])
def test_what_lies_beside_is_accepted(op, change):
    reaches_the_device(op, change)
