"""Sizes at which the block-scaled calls would count past 32 bits: refused on the host, before
anything is launched."""

import pytest

from segmented_gather_gemm_lora_amd import binding as B
from test_block_cpu import ARG, E8, F32, P, host_plan, refused


@pytest.mark.parametrize("scale_type", [F32, E8])
@pytest.mark.parametrize("out", [B.LORA_BF16, B.LORA_F32])
def test_one_row_of_nearly_2_to_the_31(scale_type, out):
    """The count of its blocks of 128 leaves 32 bits (no launch: the last accepted width is not called)."""
    k = 256
    good = dict(stream=None, T=1, x=P, ldx=k, xs=P, lds=1, d_in=k, W=P, ws=P, scale_type=scale_type, d_out=1, out=out, y=P, ldy=1,
                work=None, work_bytes=0)
    refused("lora_linear_e4m3_block", good,
            [(dict(d_in=k, ldx=k), ARG) for k in ((1 << 31) - 112, (1 << 31) - 64, (1 << 31) - 16)])


def test_the_fused_layer_past_2_to_the_30():
    """Its shrink divides a row into slices, whose ends would leave 32 bits."""
    plan = host_plan([0], [8])
    k = 256
    good = dict(stream=None, x=P, ldx=k, d_in=k, W=P, ws=P, scale_type=F32, d_out=1, seg=plan.dev(), y=P, ldy=8, work=P, work_bytes=1 << 62)
    refused("lora_fused_linear_e4m3_block", good,
            [(dict(d_in=k, ldx=k), ARG) for k in ((1 << 30) + 16, (1 << 31) - 512, (1 << 31) - 144)])
