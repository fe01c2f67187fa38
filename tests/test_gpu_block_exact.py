"""What fp32 results of the block-scaled product are for: fp32 sums, without the 8-bit instruction's
cut; and NaN codes and scales, in every form of the product (up to 64 rows, and the three tiles)."""

import numpy as np
import pytest

import block_ref as R
from block_exact_ref import exact_operands, f32_bound
from gpu_helpers import require_gpu
from segmented_gather_gemm_lora_amd import binding as B
from test_gpu_block import check

pytestmark = pytest.mark.gpu
torch = None

# rows x columns whose tiles are each of the three sizes, and up to 64 rows of 1, 2 and 4 row tiles
SHAPES = [(5, 40), (20, 304), (50, 264), (70, 200), (1030, 4104), (2049, 4104)]


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    global torch
    torch = require_gpu()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def dtype(out):
    return torch.bfloat16 if out == "bf16" else torch.float32


def linear(xq, xs, W, ws, out):
    T, d_in = xq.shape
    y = torch.full((T, len(W)), 7.0, dtype=dtype(out), device="cuda")
    B.linear_e4m3_block(dev(xq), dev(xs), dev(W), dev(ws), y, B.workspace(B.LORA_OP_LINEAR_BLOCK, T, d_in, len(W), 1))
    return y.double().cpu().numpy()


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("small", [32, 64])
@pytest.mark.parametrize("d_in", [16, 144, 272, 384])
@pytest.mark.parametrize("T,d_out", SHAPES)
def test_fp32_results_keep_what_the_8_bit_instruction_cuts_off(kind, small, d_in, T, d_out):
    """Sums that fp32 holds exactly whatever their order: every bit is right.  Scales are 2^-3 and 2^5."""
    rng = np.random.default_rng(T + d_in)
    xq, W = exact_operands(rng, T, d_in, d_out, small)
    groups = -(-d_in // 128)
    pow2 = lambda e, shape: np.full(shape, e + 127, np.uint8) if kind == "e8m0" else np.full(shape, 2.0**e, np.float32)  # noqa: E731
    xs, ws = pow2(-3, (groups, T)), pow2(5, (-(-d_out // 128), groups))
    assert np.array_equal(linear(xq, xs, W, ws, "f32"), R.linear(xq, xs, W, ws)[0])


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,d_in,d_out", [(1, 16, 1), (3, 144, 100), (17, 1008, 1531), (33, 400, 129), (65, 2048, 512), (257, 1040, 520),
                                          (517, 1008, 1531), (1030, 640, 2064)])
def test_fp32_results_within_fp32_sums(kind, T, d_in, d_out):
    """Random operands, without an allowance for the 8-bit instruction."""
    rng = np.random.default_rng(T + d_out)
    xq, xs, _ = R.quantize(rng.standard_normal((T, d_in)) * np.exp(rng.standard_normal((1, d_in))), 1, kind)
    W, ws, _ = R.quantize(rng.standard_normal((d_out, d_in)) * 0.02, 128, kind)
    ref, mag, _ = R.linear(xq, xs, W, ws)
    check(linear(xq, xs, W, ws, "f32"), ref, f32_bound(ref, mag, d_in), f"{T} {d_in}->{d_out}")


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("d_in", [144, 400])
@pytest.mark.parametrize("T,d_out", SHAPES)
def test_nan_stays_in_its_rows_and_columns(kind, out, d_in, T, d_out):
    """A NaN scale of a row, a NaN code of W in the last place, a NaN scale of a block of W."""
    rng = np.random.default_rng(T + d_in)
    xq, xs, _ = R.quantize(rng.standard_normal((T, d_in)), 1, kind)
    W, ws, _ = R.quantize(rng.standard_normal((d_out, d_in)) * 0.02, 128, kind)
    nan = 255 if kind == "e8m0" else np.nan
    clean = linear(xq, xs, W, ws, out)
    xs[1, 3] = xs[0, T - 1] = nan
    W[17, d_in - 1] = W[d_out - 1, 0] = 0x7F
    rows, cols = [3, T - 1], [17, d_out - 1]
    if d_out > 256:
        ws[1, 1] = nan
        cols = sorted(set(cols) | set(range(128, min(256, d_out))))
    got = linear(xq, xs, W, ws, out)
    keep = np.ones((T, d_out), bool)
    keep[rows], keep[:, cols] = False, False
    assert np.isnan(got[~keep]).all() and np.array_equal(got[keep], clean[keep])


@pytest.mark.parametrize("T", [1, 70])
def test_the_product_needs_no_workspace(T):
    assert B.lora_workspace_bytes(B.LORA_OP_LINEAR_BLOCK, T, 256, 100, 1) == 0
    rng = np.random.default_rng(T)
    xq, xs, _ = R.quantize(rng.standard_normal((T, 256)), 1, "f32")
    W, ws, _ = R.quantize(rng.standard_normal((100, 256)), 128, "f32")
    y = torch.zeros(T, 100, device="cuda")
    B.linear_e4m3_block(dev(xq), dev(xs), dev(W), dev(ws), y)
    assert np.array_equal(y.double().cpu().numpy(), linear(xq, xs, W, ws, "f32"))
