"""The rows' gradient of the block-scaled fused layer against differences of the layer, row by row."""

import dataclasses

import numpy as np
import pytest

from gpu_helpers import require_gpu, say
from test_gpu_block import base, fused_reference, grad_reference
from test_gpu_block_run import gradient_job, grid
from segmented_gather_gemm_lora_amd import binding as B

pytestmark = pytest.mark.gpu
torch = None


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    global torch
    import test_gpu_block
    import test_gpu_block_run

    torch = test_gpu_block.torch = test_gpu_block_run.torch = require_gpu()


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,d_in,d_out", [(24, 256, 256), (150, 256, 256), (300, 400, 264)])
def test_dx_against_differences(kind, T, d_in, d_out):
    """With x and dy of the format's own values (scales 1, so the quantization changes nothing), L[t] = sum_n dy[t, n]
    y[t, n] is linear in x[t]: L'[t] - L[t] = <dx[t], x'[t] - x[t]>.  x' has the signs of dx, so that every row's
    step is many times what the roundings of y, y' and dx (their derived bounds) allow: a wrong sign, half of
    dx or another row's dx fails in every row."""
    say(f"differences {kind} {T} {d_in}->{d_out}")
    rng = np.random.default_rng(T)
    prob, W, ws, pool, plan, x, dy, dx, work = gradient_job(T, d_in, d_out, [8, 16, 3], kind, T)
    Wh, wsh = base(np.random.default_rng(T), d_out, d_in, kind)
    assert np.array_equal(W.cpu().numpy(), Wh)
    dyh = grid(rng, (T, d_out))
    x.copy_(torch.from_numpy(grid(rng, (T, d_in))))
    dy.copy_(torch.from_numpy(dyh))
    B.fused_linear_e4m3_block_backward(x, W, ws, dy, plan, None, dx, work)
    x2 = torch.from_numpy(np.abs(grid(rng, (T, d_in)))).cuda() * torch.where(dx >= 0, 1.0, -1.0)
    x2 = x2.to(torch.bfloat16)
    fws = B.workspace(B.LORA_OP_FUSED_BLOCK, T, d_in, d_out, 16)

    def rows(x_):
        """L, and what y's bound allows it to be off."""
        y = torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda")
        B.fused_linear_e4m3_block(x_, W, ws, plan, y, fws)
        bits = x_.cpu().view(torch.int16).numpy().view(np.uint16)
        _, bound = fused_reference(dataclasses.replace(prob, x=bits), Wh, wsh, kind)
        return (dyh * y.double().cpu().numpy()).sum(1), (np.abs(dyh) * bound).sum(1)

    L0, off0 = rows(x)
    L1, off1 = rows(x2)
    step = x2.double().cpu().numpy() - x.double().cpu().numpy()
    g = dx.double().cpu().numpy()
    _, bound, *_ = grad_reference(prob, Wh, wsh, kind, x.double().cpu().numpy(), dyh)
    want, room = (g * step).sum(1), off0 + off1 + (bound * np.abs(step)).sum(1)
    print("least step / room", np.min(np.abs(want) / room), "worst miss / room", np.max(np.abs(L1 - L0 - want) / room))
    assert (np.abs(want) > 4 * room).all()
    assert (np.abs(L1 - L0 - want) <= room).all()
