"""Sizes at which the block-scaled calls would count past 32 bits: refused on the host, before
anything is launched."""

import pytest

from segmented_gather_gemm_lora_amd import binding as B
from test_block_cpu import ARG, E8, F32, DevicePlanArgs, P, host_plan, refused


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


def test_more_workgroups_than_a_launch_has():
    """Threads of a launch are counted in 32 bits: up to 64 rows, workgroups of 512 threads have 16 columns
    (fp32 results of more than 32 rows) or 32 (bf16)."""
    good = dict(stream=None, T=33, x=P, ldx=16, xs=P, lds=33, d_in=16, W=P, ws=P, scale_type=F32, d_out=1, out=B.LORA_F32, y=P, ldy=1 << 28,
                work=None, work_bytes=0)
    refused("lora_linear_e4m3_block", good, [(dict(d_out=1 << 27), ARG), (dict(d_out=(1 << 28) - 2), ARG), (dict(T=64, lds=64, d_out=1 << 27), ARG),
                                             (dict(out=B.LORA_BF16, d_out=(1 << 28) - 2), ARG)])
    assert "tiles" in B.last_error()


def test_the_fused_layer_refuses_them_before_anything_runs():
    """Not as the failure of a first launch (here: without a GPU)."""
    plan = host_plan([0] * 40, [8])
    good = dict(stream=None, x=P, ldx=16, d_in=16, W=P, ws=P, scale_type=F32, d_out=8, seg=plan.dev(), y=P, ldy=1 << 28, work=P, work_bytes=1 << 62)
    refused("lora_fused_linear_e4m3_block", good, [(dict(d_out=(1 << 28) - 8), ARG)])
    plan = host_plan([0] * 70000, [8])
    refused("lora_fused_linear_e4m3_block", dict(good, seg=plan.dev()), [(dict(d_out=(1 << 28) - 8), ARG)])


@pytest.mark.parametrize("T", [8192, 400000])  # of the last launch; of the product
def test_the_gradients_refuse_them_before_anything_runs(T):
    plan = host_plan([0] * T, [8])
    n = 1 << 24
    good = dict(stream=None, x=P, ldx=n, d_in=n, W=P, ws=P, scale_type=F32, dy=P, lddy=16, d_out=8, seg=plan.dev(), gA=P, gB=P, n=1, flags=0,
                dx=P + (1 << 46), lddx=n, work=P, work_bytes=1 << 62)
    refused("lora_fused_linear_e4m3_block_backward", good, [(dict(), ARG)])
    assert "tiles" in B.last_error()


def test_requests_of_a_device_plan():
    """Its loop over them adds 1024 to a 32-bit count: past 2^31 - 1024 it would not have ended."""
    d = DevicePlanArgs(64)
    refused("lora_build_segments_device", d.good(64), [(dict(R=(1 << 30) + 1), ARG), (dict(R=(1 << 31) - 1), ARG)])


def test_the_binding_refuses_counts_past_32_bits(monkeypatch):
    """ctypes would cut them: 2^32 + 1 rows are not one row.  Tensors without memory stand for large ones."""
    import torch

    new = lambda *shape, dtype=torch.uint8: torch.empty(*shape, dtype=dtype, device="meta")  # noqa: E731
    monkeypatch.setattr(torch.cuda, "current_device", lambda: new(1).get_device())
    monkeypatch.setattr(B, "_stream_handle", lambda *a: None)
    n, bf16, f32 = (1 << 32) + 1, torch.bfloat16, torch.float32
    for rows, cols in ((n, 1), (1, n), ((1 << 31), 16)):
        with pytest.raises(ValueError, match=r"2\^31"):
            B.quantize_e4m3(new(rows, cols, dtype=bf16), new(rows, cols), new((cols + 127) // 128, rows, dtype=f32))
    for T, d_in, d_out in ((n, 16, 8), (1, 16, n), (1, n + 15, 1)):
        with pytest.raises(ValueError, match=r"2\^31"):
            B.linear_e4m3_block(new(T, d_in), new((d_in + 127) // 128, T, dtype=f32), new(d_out, d_in),
                                new((d_out + 127) // 128, (d_in + 127) // 128, dtype=f32), new(T, d_out, dtype=bf16), new(0))
    plan = B.DevicePlan.__new__(B.DevicePlan)  # of the constructor's work, what build() asks for first
    plan._device, plan._fn, plan._pool_args, plan.rows = new(1).get_device(), lambda *a: 0, (), 8
    with pytest.raises(ValueError, match="requests"):
        plan.build(new(n, dtype=torch.int32), new(n, dtype=torch.int32))
