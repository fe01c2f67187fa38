"""The block-scaled products at the ends of their scales, in every form of the product (up to 64 rows,
and the three tiles), both types of scales and results."""

import dataclasses

import numpy as np
import pytest

import block_ref as R
from block_exact_ref import f32_bound
from gpu_helpers import require_gpu, say
from lora_workloads import bf16_bits_to_f32
from segmented_gather_gemm_lora_amd import binding as B
from test_gpu_block import bf16, check, fused_problem, fused_reference, grad_reference
from test_gpu_block_exact import SHAPES, dev, linear

pytestmark = pytest.mark.gpu
torch = None


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    global torch
    import test_gpu_block
    import test_gpu_block_exact

    torch = test_gpu_block.torch = test_gpu_block_exact.torch = require_gpu()


def stored(rng, e, kind):
    """Scales of about 2^e: fp32 with a factor, or the bytes."""
    e = np.asarray(e)
    if kind == "e8m0":
        return (e + 127).astype(np.uint8)
    return (2.0**e * rng.choice([1.0, 1.25, 1.5625, 1.96875], e.shape)).astype(np.float32)


def codes(rng, shape, low=1, high=127):
    return (rng.integers(low, high, shape) + 128 * rng.integers(0, 2, shape)).astype(np.uint8)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_out", SHAPES)
def test_factors_whose_product_leaves_fp32(kind, out, T, d_out):
    """Four blocks: of usual scales; of scales whose product is past fp32's largest over codes of W that are 0 (nothing);
    of 2^-100 and 2^100; of scales whose product is below fp32's smallest (next to nothing)."""
    say(f"factors {kind} {out} {T} x {d_out}")
    rng = np.random.default_rng(T)
    d_in = 400
    xq, W = codes(rng, (T, d_in)), codes(rng, (d_out, d_in))
    W[:, 128:256] = 0
    nb = -(-d_out // 128)
    xs = np.stack([stored(rng, np.full(T, e), kind) for e in (-3, 100, -100, -100)])
    ws = np.stack([stored(rng, np.full(nb, e), kind) for e in (-2, 90, 98, -60)], 1)
    # the second block adds 0 whatever its scales: the reference and the bounds take small ones
    ref, mag, tops = R.linear(xq, np.where(np.arange(4)[:, None] == 1, xs[3:], xs), W, np.where(np.arange(4) == 1, ws[:, 3:], ws))
    bound = R.linear_bound(ref, mag, tops, d_in, "bf16") if out == "bf16" else f32_bound(ref, mag, d_in)
    check(linear(xq, xs, W, ws, out), ref, bound, f"{T} x {d_out}")


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_out", SHAPES)
def test_factors_whose_product_is_subnormal(kind, out, T, d_out):
    """Scales of 2^-75 and 2^-72 and codes of 256 to 448, all positive: a block's sum (2^23 and more) times both
    scales is a usual number, the product of the scales has two or three bits of fp32."""
    rng = np.random.default_rng(T + 1)
    d_in = 272
    xq, W = (rng.integers(120, 127, s).astype(np.uint8) for s in ((T, d_in), (d_out, d_in)))
    xs = stored(rng, np.full((3, T), -75), kind)
    ws = stored(rng, np.full((-(-d_out // 128), 3), -72), kind)
    ref, mag, tops = R.linear(xq, xs, W, ws)
    bound = R.linear_bound(ref, mag, tops, d_in, "bf16") if out == "bf16" else f32_bound(ref, mag, d_in)
    # the last block has 16 products: its sum may be below fp32's smallest usual number, each block's is then off by
    # half of 2^-149, before a factor below 4
    check(linear(xq, xs, W, ws, out), ref, bound + 3 * 2.0**-148, f"{T} x {d_out}")


@pytest.mark.parametrize("T,d_out", SHAPES)
def test_zero_and_subnormal_scales(T, d_out):
    """fp32 scales of 0 make 0.  A subnormal one of a row meets W's in one rounding: with W's scale f 2^e, f in [1, 2), the product f sx is off by up to half of 2^-149, which is 2^-150 2^e,
    at most 2^-150 W's scale, of the block's sum."""
    rng = np.random.default_rng(T + 2)
    d_in = 384
    xq, W = codes(rng, (T, d_in), 56), codes(rng, (d_out, d_in), 56)
    nb = -(-d_out // 128)
    xs, ws = stored(rng, np.full((3, T), -5), "f32"), stored(rng, np.full((nb, 3), -6), "f32")
    xs[0], ws[:, 1] = 0.0, 0.0
    xs[2, ::2] = np.float32(2.0**-149) * rng.integers(1, 1 << 20, xs[2, ::2].shape).astype(np.float32)
    ws[:, 2] = stored(rng, np.full(nb, 100), "f32")
    half = np.where((xs > 0) & (xs < 2.0**-126), 2.0**-150, 0.0)
    _, off, _ = R.linear(xq, half, W, ws)
    for out in ("bf16", "f32"):
        ref, mag, tops = R.linear(xq, xs, W, ws)
        bound = R.linear_bound(ref, mag, tops, d_in, "bf16") if out == "bf16" else f32_bound(ref, mag, d_in)
        check(linear(xq, xs, W, ws, out), ref, bound + off, f"{T} x {d_out} {out}")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 20, 50, 70, 300])
def test_subnormal_scales_of_w(out, T):
    """They count by their value, to the last bit."""
    rng = np.random.default_rng(T)
    xq, W = codes(rng, (T, 256), 56), codes(rng, (100, 256), 56)
    xs, ws = stored(rng, np.full((2, T), 100), "f32"), np.array([[1001, 3]], np.float32) * np.float32(2.0**-149)
    ref, mag, tops = R.linear(xq, xs, W, ws)
    check(linear(xq, xs, W, ws, out), ref, R.linear_bound(ref, mag, tops, 256, "bf16") if out == "bf16" else f32_bound(ref, mag, 256), f"{T}")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_out", SHAPES)
def test_an_infinite_scale_stays_in_its_row(out, T, d_out):
    rng = np.random.default_rng(T + 3)
    xq, W = codes(rng, (T, 144)), codes(rng, (d_out, 144))
    xs, ws = stored(rng, np.full((2, T), -5), "f32"), stored(rng, np.full((-(-d_out // 128), 2), -6), "f32")
    clean = linear(xq, xs, W, ws, out)
    xs[0, 2] = np.inf
    got = linear(xq, xs, W, ws, out)
    assert not np.isfinite(got[2]).any() and np.array_equal(np.delete(got, 2, 0), np.delete(clean, 2, 0))


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("ranks", [[8, 16], [5, 17]])
@pytest.mark.parametrize("T,d_out", SHAPES)
def test_fused_rows_of_the_largest_values(kind, ranks, T, d_out):
    """Rows whose values reach 2^120 and more (their scales 2^111), over blocks of zeros of W with scales of 2^20 and
    more, and rows that hold an infinity: the first have the product's value, the others are NaN, and the rest
    is what it was."""
    d_in = 400
    prob = fused_problem(T, d_in, d_out, ranks, T, none=0.3)
    rng = np.random.default_rng(T)
    W, ws, _ = R.quantize(rng.standard_normal((d_out, d_in)) * 2.0**-12, 128, kind)
    W[:, 128:256] = 0
    ws[:, 1] = 2.0**30 if kind == "f32" else 127 + 30
    ids = prob.ids.copy()
    large, bad = np.arange(T) % 7 == 1, np.arange(T) % 7 == 4
    ids[large] = -1  # their corrections may leave fp32
    xh = bf16_bits_to_f32(prob.x).reshape(T, d_in).astype(np.float64)
    xh[large] = rng.choice([-1.0, 1.0], (large.sum(), d_in)) * 2.0 ** rng.uniform(110, 121, (large.sum(), d_in))
    host, _ = bf16(xh)
    prob = dataclasses.replace(prob, ids=ids, x=host.view(torch.int16).numpy().view(np.uint16))
    small = ws.copy()
    small[:, 1] = 2.0**-100 if kind == "f32" else 27  # for the bounds: the block adds nothing
    ref, bound = fused_reference(prob, W, small, kind)
    pool = B.DevicePool.from_problem(prob)
    plan = B.Plan(T).build(ids, pool).upload()
    host[bad, 390] = float("inf")
    x = host.cuda()
    y = torch.full((T, d_out), 5.0, dtype=torch.bfloat16, device="cuda")
    B.fused_linear_e4m3_block(x, dev(W), dev(ws), plan, y, B.workspace(B.LORA_OP_FUSED_BLOCK, T, d_in, d_out, prob.max_rank))
    got = y.double().cpu().numpy()
    assert np.isnan(got[bad]).all()
    check(got[~bad], ref[~bad], bound[~bad], f"{T} x {d_out}")


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,d_in", [(5, 48), (70, 208), (1030, 4112), (2049, 4112)])
def test_gradients_of_the_largest_values(kind, T, d_in):
    """The same of dy, over the rows' gradient; no adapter's gradient is wanted."""
    d_out = 400
    prob = fused_problem(T, d_in, d_out, [8, 16], T, none=0.3)
    rng = np.random.default_rng(T)
    W, ws, _ = R.quantize(rng.standard_normal((d_out, d_in)) * 2.0**-12, 128, kind)
    W[128:256] = 0
    ws[1] = 2.0**30 if kind == "f32" else 127 + 30
    ids = prob.ids.copy()
    large, bad = np.arange(T) % 7 == 1, np.arange(T) % 7 == 4
    ids[large] = -1
    dyh = rng.standard_normal((T, d_out))
    dyh[large] = rng.choice([-1.0, 1.0], (large.sum(), d_out)) * 2.0 ** rng.uniform(110, 121, (large.sum(), d_out))
    host, dy = bf16(dyh)
    prob = dataclasses.replace(prob, ids=ids)
    small = ws.copy()
    small[1] = 2.0**-100 if kind == "f32" else 27
    x = bf16_bits_to_f32(prob.x).reshape(T, d_in).astype(np.float64)
    dx, bound, *_ = grad_reference(prob, W, small, kind, x, dy)
    pool = B.DevicePool.from_problem(prob)
    plan = B.Plan(T).build(ids, pool).upload()
    host[bad, 390] = float("inf")
    got = torch.empty(T, d_in, dtype=torch.bfloat16, device="cuda")
    B.fused_linear_e4m3_block_backward(B.to_device(prob.x, "bf16"), dev(W), dev(ws), host.cuda(), plan, None, got,
                                       B.workspace(B.LORA_OP_FUSED_BLOCK_BACKWARD, T, d_in, d_out, prob.max_rank))
    got = got.double().cpu().numpy()
    assert np.isnan(got[bad]).all()
    check(got[~bad], dx[~bad], bound[~bad], f"{T} x {d_in}")
