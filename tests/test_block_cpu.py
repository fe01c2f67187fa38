"""Refusals of the block-scaled calls and of plans built on the device: every one on the host,
before any GPU call, with addresses that nothing looks behind."""

import ctypes

import numpy as np
import pytest

from segmented_gather_gemm_lora_amd import binding as B
from test_abi_cpu import FAKE_BASE, build

ARG, DTYPE, RANK, ALIGN, WORKSPACE, PLAN, ADAPTER = (
    {n: c for c, n in B.STATUS.items()}[k]
    for k in ("LORA_ERR_ARG", "LORA_ERR_DTYPE", "LORA_ERR_RANK", "LORA_ERR_ALIGN", "LORA_ERR_WORKSPACE", "LORA_ERR_PLAN",
              "LORA_ERR_ADAPTER_ID"))
P = FAKE_BASE
F32, E8 = B.LORA_SCALE_F32, B.LORA_SCALE_E8M0


def refused(name, good, changes):
    """Each change to the good arguments (which end in no launch) has its status and a message."""
    fn = getattr(B.load(), name)
    names = list(good)
    for change, status in changes:
        args = dict(good, **change)
        assert set(args) == set(names), change
        st = fn(*(args[k] for k in names))
        assert st == status, (change, B.lora_status_string(st), B.last_error())
        assert B.last_error(), change


def test_quantize():
    good = dict(stream=None, dtype=B.LORA_BF16, x=P, ldx=256, rows=4, cols=256, block_rows=1, scale_type=F32, codes=P, ldq=256,
                scales=P, lds=4)
    refused("lora_quantize_e4m3", good, [
        (dict(dtype=7), DTYPE), (dict(scale_type=2), DTYPE), (dict(scale_type=-1), DTYPE), (dict(block_rows=2), ARG),
        (dict(rows=-1), ARG), (dict(rows=(1 << 27) + 1, lds=1 << 28), ARG), (dict(cols=0), ARG), (dict(cols=(1 << 22) + 1, ldx=1 << 23, ldq=1 << 23), ARG),
        (dict(x=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG), (dict(ldx=255), ARG), (dict(ldq=255), ARG),
        (dict(lds=3), ARG), (dict(block_rows=128, lds=1), ARG), (dict(x=P + 1), ALIGN), (dict(x=P + 2, dtype=B.LORA_F32), ALIGN),
        (dict(scales=P + 2), ALIGN)])
    assert B.load().lora_quantize_e4m3(*dict(good, rows=0).values()) == 0


def test_linear():
    good = dict(stream=None, T=4, x=P, ldx=256, xs=P, lds=4, d_in=256, W=P, ws=P, scale_type=F32, d_out=100, out=B.LORA_BF16,
                y=P, ldy=100, work=None, work_bytes=0)
    refused("lora_linear_e4m3_block", good, [
        (dict(out=7), DTYPE), (dict(scale_type=9), DTYPE), (dict(T=-1), ARG), (dict(x=None), ARG), (dict(xs=None), ARG),
        (dict(y=None), ARG), (dict(W=None), ARG), (dict(ws=None), ARG), (dict(ldx=255), ARG), (dict(ldy=99), ARG), (dict(lds=3), ARG),
        (dict(d_in=0), ARG), (dict(d_out=0), ARG), (dict(d_in=248), ALIGN), (dict(x=P + 8), ALIGN), (dict(ldx=264), ALIGN),
        (dict(W=P + 8), ALIGN), (dict(ws=P + 2), ALIGN), (dict(xs=P + 2), ALIGN),
        (dict(y=P + 1), ALIGN), (dict(out=B.LORA_F32, y=P + 2), ALIGN),
        (dict(T=1 << 20, lds=1 << 20, ldx=4096), ARG), (dict(ldx=1 << 62), ARG),
        (dict(d_in=1 << 16, ldx=1 << 16, d_out=1 << 16, ldy=1 << 16), ARG)])
    assert B.load().lora_linear_e4m3_block(*dict(good, T=0).values()) == 0


def host_plan(ids, ranks):
    n = len(ranks)
    A = (P + 4096 * np.arange(n)).astype(np.uint64)
    st, plan = build(ids, n, A, A + np.uint64(1 << 30), np.asarray(ranks, dtype=np.int32), np.full(n, 16.0, dtype=np.float32))
    assert st == 0
    return plan


def test_fused():
    plan = host_plan([0, 1, -1, 0], [8, 16])
    need = B.lora_workspace_bytes(B.LORA_OP_FUSED_BLOCK, 4, 256, 104, 16)
    assert need > 0
    good = dict(stream=None, x=P, ldx=256, d_in=256, W=P, ws=P, scale_type=F32, d_out=104, seg=plan.dev(), y=P, ldy=104, work=P,
                work_bytes=need)
    refused("lora_fused_linear_e4m3_block", good, [
        (dict(seg=None), ARG), (dict(scale_type=3), DTYPE), (dict(x=None), ARG), (dict(y=None), ARG), (dict(W=None), ARG),
        (dict(ws=None), ARG), (dict(ldx=248), ARG), (dict(ldy=96), ARG), (dict(d_in=0), ARG), (dict(d_out=0), ARG),
        (dict(d_in=248), ALIGN), (dict(x=P + 2), ALIGN), (dict(y=P + 8), ALIGN), (dict(ldx=260), ALIGN), (dict(ldy=108), ALIGN),
        (dict(W=P + 4), ALIGN), (dict(ws=P + 1), ALIGN), (dict(work=None), WORKSPACE), (dict(work_bytes=need - 1), WORKSPACE),
        (dict(work=P + 8), ALIGN), (dict(d_in=1 << 16, ldx=1 << 16, d_out=1 << 16, ldy=1 << 16), ARG), (dict(seg=plan.dev(buf=None)), ARG)])


def test_backward():
    plan = host_plan([0, 1, -1, 0], [8, 16])
    need = B.lora_workspace_bytes(B.LORA_OP_FUSED_BLOCK_BACKWARD, 4, 256, 104, 16)
    assert need > 0
    good = dict(stream=None, x=P, ldx=256, d_in=256, W=P, ws=P, scale_type=F32, dy=P, lddy=104, d_out=104, seg=plan.dev(), gA=P,
                gB=P, n=2, flags=0, dx=P + (1 << 24), lddx=256, work=P, work_bytes=need)
    refused("lora_fused_linear_e4m3_block_backward", good, [
        (dict(seg=None), ARG), (dict(scale_type=3), DTYPE), (dict(x=None), ARG), (dict(dy=None), ARG), (dict(dx=None), ARG),
        (dict(W=None), ARG), (dict(ws=None), ARG), (dict(ldx=248), ARG), (dict(lddy=96), ARG), (dict(lddx=248), ARG), (dict(n=1), ADAPTER),
        (dict(d_in=248), ALIGN), (dict(x=P + 8), ALIGN), (dict(dy=P + 8), ALIGN), (dict(dx=P + 8 + (1 << 24)), ALIGN), (dict(dx=P), ARG), (dict(lddy=108), ALIGN),
        (dict(lddx=260), ALIGN), (dict(W=P + 4), ALIGN), (dict(ws=P + 2), ALIGN), (dict(work=None), WORKSPACE),
        (dict(work_bytes=need - 1), WORKSPACE), (dict(work=P + 8), ALIGN), (dict(flags=1 << 20), ARG), (dict(seg=plan.dev(buf=None)), ARG)])


class DevicePlanArgs:
    def __init__(self, rows):
        self.seg = B.LoraSegments()
        assert B.lora_segments_bind(P, rows, ctypes.addressof(self.seg)) == 0
        self.geometry = (ctypes.c_uint64 * (B.PLAN_HEADER_BYTES // 8))()

    def good(self, T):
        return dict(stream=None, T=T, R=4, adapters=P, lengths=P, n=2, A=P, B=P, rank=P, alpha=P, max_rank=16, multiple=8,
                    geometry=ctypes.addressof(self.geometry), dev=ctypes.addressof(self.seg))


def test_device_plan():
    d = DevicePlanArgs(64)
    empty = B.LoraSegments()
    refused("lora_build_segments_device", d.good(64), [
        (dict(geometry=None), ARG), (dict(geometry=ctypes.addressof(d.geometry) + 4), ALIGN), (dict(dev=None), ARG),
        (dict(dev=ctypes.addressof(empty)), ARG), (dict(T=-1), ARG), (dict(T=65537), ARG), (dict(T=65), WORKSPACE), (dict(R=-1), ARG),
        (dict(R=65, lengths=None), ARG), (dict(n=-1), ARG), (dict(n=7169), ARG), (dict(adapters=None), ARG), (dict(A=None), ARG),
        (dict(B=None), ARG), (dict(rank=None), ARG), (dict(alpha=None), ARG), (dict(max_rank=0), RANK), (dict(max_rank=257), RANK),
        (dict(multiple=0), RANK), (dict(multiple=17), RANK)])


def test_gradients_refuse_a_device_plan():
    d = DevicePlanArgs(64)
    # no rows: the geometry is written and nothing is launched; then its count of rows, as a build of 4 leaves it
    assert B.load().lora_build_segments_device(*dict(d.good(64), T=0).values()) == 0
    np.frombuffer(d.geometry, dtype=np.int32)[1] = 4
    need = B.lora_workspace_bytes(B.LORA_OP_FUSED_BLOCK_BACKWARD, 4, 256, 104, 16)
    args = (None, P, 256, 256, P, P, F32, P, 104, 104, ctypes.addressof(d.seg), P, P, 2, 0, P, 256, P, need)
    assert B.load().lora_fused_linear_e4m3_block_backward(*args) == PLAN
    assert "host" in B.last_error()


@pytest.mark.parametrize("op", [B.LORA_OP_LINEAR_BLOCK, B.LORA_OP_FUSED_BLOCK, B.LORA_OP_FUSED_BLOCK_BACKWARD])
def test_workspaces_grow_with_the_batch(op):
    sizes = [B.lora_workspace_bytes(op, T, 4096, 1024, 16) for T in (0, 1, 2, 3, 16, 63, 64, 65, 500, 517, 1000, 4096, 16384)]
    assert sizes == sorted(sizes)
