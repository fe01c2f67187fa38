"""The gradient calls where byte offsets pass 32 bits, and where a batch has more
rows than one span for each sixteenth of it: against the 64-bit reference."""

import numpy as np
import pytest
import torch

from backward_ref import Problem, check
from gpu_helpers import require_gpu, say
from segmented_gather_gemm_lora_amd import binding as B
from test_gpu_backward import ids_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()  # the far rows hold gigabytes


def far(rows, pitch):
    """The rows on the device, `pitch` elements apart (what lies between is not set)."""
    T, d = rows.shape
    flat = torch.empty((T - 1) * pitch + d, dtype=rows.dtype, device="cuda")
    t = flat.as_strided((T, d), (pitch, 1))
    t.copy_(rows)
    return t


def pitch_at(T, es, above):
    """The largest pitch of whole 16-byte pieces whose T rows stay below 2^32 bytes, or the next one."""
    step = 16 // es
    most = ((2**32 // es // T) - 1) // step * step
    assert most * es * T < 2**32 <= (most + 2 * step) * es * T
    return most + (2 * step if above else 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("above", [False, True])
@pytest.mark.parametrize("which", ["x", "dy", "dx", "x dy dx"])
def test_rows_at_32_bits(dtype, above, which):
    say(f"case backward far {dtype} above={above} {which}")
    p = Problem(dtype, [1, 0, 1], [16, 40], 136, 264, seed=3)
    d = p.device()
    for k in which.split():
        setattr(d, k, far(getattr(p, k), pitch_at(3, p.x.element_size(), above)))
    B.sgmv_backward(d.x, d.dy, d.plan, d.grads, d.dx, d.ws, dtype)
    torch.cuda.synchronize()
    check(p, d, f"{which} above={above}")


@pytest.mark.parametrize("d_out", [72, 1100])  # the sum over d_out whole, and in two parts that are joined
@pytest.mark.parametrize("above", [False, True])
@pytest.mark.parametrize("which", ["x", "dy", "dx", "x dy dx"])
def test_fused_rows_at_32_bits(d_out, above, which):
    say(f"case fused backward far {d_out} above={above} {which}")
    p = Problem("bf16", [1, -1, 0], [16, 40], 264, d_out, seed=4, w0=True, pad=(0, -d_out % 8, 0))
    d = p.device()
    for k in which.split():
        setattr(d, k, far(getattr(p, k), pitch_at(3, 2, above)))
    B.fused_linear_backward(d.x, d.W0, d.dy, d.plan, d.grads, d.dx, d.ws)
    torch.cuda.synchronize()
    check(p, d, f"{which} above={above}")


@pytest.mark.parametrize("dtype,ranks,kind", [("bf16", [16, 8], "runs"), ("f32", [16, 8], "mixed"), ("bf16", [64, 8], "runs"),
                                              ("bf16", [20, 48], "mixed")])
def test_many_rows(dtype, ranks, kind):
    """More than 32768 adapted rows: spans of 2048."""
    T = 45000 if kind == "runs" else 60000
    ids = ids_of(kind, T, len(ranks), 7)
    assert (ids >= 0).sum() > 32768 + 2048
    say(f"case backward {dtype} T={T} ranks={ranks}")
    p = Problem(dtype, ids, ranks, 72, 40, seed=8)
    d = p.device()
    B.sgmv_backward(d.x, d.dy, d.plan, d.grads, d.dx, d.ws, dtype)
    torch.cuda.synchronize()
    check(p, d, f"T={T}")
    first = [t.clone() for t in (*d.grads.A, *d.grads.B)]
    B.sgmv_backward(d.x, d.dy, d.plan, d.grads, None, d.ws, dtype)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (*d.grads.A, *d.grads.B)))
    assert np.isfinite(d.dx.float().cpu().numpy()).all()
