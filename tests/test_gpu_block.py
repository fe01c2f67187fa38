"""The block-scaled FP8 base on the GPU: quantization bit for bit, the product and the
fused layer against 64 bits."""

import numpy as np
import pytest

import block_ref as R
from gpu_helpers import require_gpu, say
from lora_workloads import bf16_bits_to_f32, make_problem
from segmented_gather_gemm_lora_amd import binding as B

pytestmark = pytest.mark.gpu
torch = None


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    global torch
    torch = require_gpu()


def np_dtype(kind):
    return torch.float32 if kind == "f32" else torch.uint8


def bf16(a):
    """The bf16 tensor (host) nearest to a, and its values in 64 bits."""
    t = torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


def pitched(rows, cols, dtype, pad, fill=0):
    """A device matrix with `pad` elements between its rows."""
    whole = torch.full((rows, cols + pad), fill, dtype=dtype, device="cuda")
    return whole, whole[:, :cols]


def hidden(rng, T, d):
    """Rows whose groups differ by orders of magnitude, with zeros and ties of the format."""
    x = rng.standard_normal((T, d)) * np.exp(rng.standard_normal((1, d)))
    x *= 10.0 ** rng.integers(-6, 6, (T, 1))
    x[rng.random((T, d)) < 0.05] = 0.0
    return x


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("T,d,pad", [(1, 1, 0), (1, 128, 0), (3, 129, 5), (16, 1024, 8), (17, 127, 0), (130, 257, 3),
                                     (300, 640, 0), (1025, 512, 0), (64, 4096, 0)])
def test_quantize_bits(kind, dtype, rows, T, d, pad):
    say(f"quantize {kind} {dtype} rows={rows} {T}x{d}+{pad}")
    rng = np.random.default_rng(T * d + rows)
    x = hidden(rng, T, d)
    if dtype == "bf16":
        host, x = bf16(x)
    else:
        host = torch.from_numpy(x.astype(np.float32))
        x = host.double().numpy()
    dev, view = pitched(T, d, host.dtype, pad)
    view.copy_(host)
    cdev, codes = pitched(T, d, torch.uint8, pad, 77)
    want_codes, want_scales, _ = R.quantize(x, rows, kind)
    sdev, s = pitched(*want_scales.shape, np_dtype(kind), pad, 99)
    B.quantize_e4m3(view, codes, s, block_rows=rows)
    got, gs = codes.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(gs, want_scales)
    # a zero may have either sign
    same = (got == want_codes) | (((got & 127) == 0) & ((want_codes & 127) == 0))
    assert same.all(), f"{(~same).sum()} of {same.size} codes, first at {np.argwhere(~same)[0]}"
    assert (cdev.cpu().numpy()[:, d:] == 77).all() and (sdev.cpu().numpy()[:, want_scales.shape[1]:] == 99).all()


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_quantize_ties_and_ends(kind):
    """Quotients next to the middle of two codes (small whole ratios to the block's largest value),
    the smallest and largest values, and blocks that are not finite."""
    rng = np.random.default_rng(5)
    T, d = 64, 1024
    top = rng.integers(128, 256, (T, d // 128)) * 2.0 ** rng.integers(-40, 40, (T, d // 128))
    x = np.repeat(top, 128, 1) * rng.integers(-64, 65, (T, d)) / 64.0
    x[:, ::128] = top
    x[0, :128] = 2.0**-133 * rng.integers(0, 3, 128)  # subnormal bf16
    x[1, :128] = 3.3e38 * rng.uniform(-1, 1, 128)
    x[2, :128] = 0.0
    x[2, 7] = 2.0**-126
    host, x = bf16(x)
    host[3, 5], host[4, 130], host[5, 300] = float("inf"), float("-inf"), float("nan")
    x = host.double().numpy()
    codes = torch.empty(T, d, dtype=torch.uint8, device="cuda")
    want_codes, want_scales, _ = R.quantize(x, 1, kind)
    s = torch.empty(want_scales.shape, dtype=np_dtype(kind), device="cuda")
    B.quantize_e4m3(host.cuda(), codes, s)
    got = codes.cpu().numpy()
    assert np.array_equal(s.cpu().numpy(), want_scales, equal_nan=True)
    same = (got == want_codes) | (((got & 127) == 0) & ((want_codes & 127) == 0))
    assert same.all(), f"{(~same).sum()} codes, first at {np.argwhere(~same)[0]}"
    assert np.isnan(R.scale_values(want_scales)[[0, 1, 2], [3, 4, 5]]).all()


def base(rng, d_out, d_in, kind):
    W, ws, _ = R.quantize(rng.standard_normal((d_out, d_in)) * 0.02 * np.exp(rng.standard_normal((d_out, 1))), 128, kind)
    return W, ws


def check(got, ref, bound, what):
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    if bad.any():
        pytest.fail(f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(err / bound):.3g}, first at {np.argwhere(bad)[0]}")


SHAPES = [(1, 16, 1), (1, 4096, 130), (2, 128, 128), (3, 144, 100), (15, 256, 272), (16, 1024, 384), (17, 1008, 1531),
          (33, 400, 129), (64, 2048, 512), (65, 2048, 512), (100, 272, 700), (128, 128, 4096), (200, 512, 300),
          (257, 1040, 520), (517, 1008, 1531), (1030, 640, 2064), (2049, 256, 4100), (2100, 144, 8300)]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_in,d_out", SHAPES)
def test_linear(kind, out, T, d_in, d_out):
    say(f"linear {kind} {out} {T} {d_in}->{d_out}")
    rng = np.random.default_rng(T + d_in + d_out)
    W, ws = base(rng, d_out, d_in, kind)
    xq, xs, _ = R.quantize(hidden(rng, T, d_in), 1, kind)
    ref, *mag = R.linear(xq, xs, W, ws)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    pad = T % 3  # y at odd pitches too
    ydev, y = pitched(T, d_out, dt, pad, 7)
    sdev, s = pitched(xs.shape[0], T, np_dtype(kind), T % 5)
    s.copy_(torch.from_numpy(xs))
    ws_dev = B.workspace(B.LORA_OP_LINEAR_BLOCK, T, d_in, d_out, 1)
    B.linear_e4m3_block(torch.from_numpy(xq).cuda(), s, torch.from_numpy(W).cuda(), torch.from_numpy(ws).cuda(), y, ws_dev)
    check(y.double().cpu().numpy(), ref, R.linear_bound(ref, *mag, d_in, out), f"{T} {d_in}->{d_out}")
    assert (ydev[:, d_out:] == 7).all()


def test_linear_nan_stays_in_its_row_and_column():
    rng = np.random.default_rng(3)
    T, d_in, d_out = 70, 384, 300
    W, ws = base(rng, d_out, d_in, "f32")
    xq, xs, _ = R.quantize(hidden(rng, T, d_in), 1, "f32")
    xs[1, 5] = np.nan
    W[17, 40] = 0x7F
    ref, *mag = R.linear(xq, xs, np.where(W == 0x7F, 0, W), ws)
    y = torch.zeros(T, d_out, device="cuda")
    B.linear_e4m3_block(*(torch.from_numpy(t).cuda() for t in (xq, xs, W, ws)), y, B.workspace(B.LORA_OP_LINEAR_BLOCK, T, d_in, d_out, 1))
    got = y.double().cpu().numpy()
    assert np.isnan(got[5]).all() and np.isnan(got[:, 17]).all()
    keep = np.ones((T, d_out), bool)
    keep[5], keep[:, 17] = False, False
    check(got[keep], ref[keep], R.linear_bound(ref, *mag, d_in, "f32")[keep], "the others")


# ---- the fused layer
def fused_problem(T, d_in, d_out, ranks, seed, none=0.1, layout="random"):
    rng = np.random.default_rng(seed)
    n = len(ranks)
    ids = rng.integers(0, n, T) if layout == "random" else np.sort(rng.integers(0, n, T))
    ids = ids.astype(np.int32)
    ids[rng.random(T) < none] = -1
    return make_problem(name="block", dtype="bf16", ids=ids, ranks=list(ranks), alphas=[32.0] * n, d_in=d_in, d_out=d_out,
                        seed=seed)


def fused_reference(prob, W, ws, kind):
    """The layer in 64 bits and a bound: the product's, and of the correction the rounding of v to
    two bf16 halves (2^-17, and as much for its fp32 sums and products)."""
    x = bf16_bits_to_f32(prob.x).reshape(prob.x.shape).astype(np.float64)
    xq, xs, _ = R.quantize(x, 1, kind)
    ref, *mag = R.linear(xq, xs, W, ws)
    bound = R.linear_bound(0.0, *mag, prob.d_in, "f32")
    for i in range(prob.n_adapters):
        rows = np.nonzero(prob.ids == i)[0]
        if not rows.size:
            continue
        A = bf16_bits_to_f32(prob.A(i)).astype(np.float64).reshape(-1, prob.d_in)
        Bm = bf16_bits_to_f32(prob.B(i)).astype(np.float64).reshape(prob.d_out, -1)
        s = float(np.float32(prob.alphas[i]) / np.float32(A.shape[0]))
        ref[rows] += s * (x[rows] @ A.T) @ Bm.T
        vmag = np.abs(x[rows]) @ np.abs(A).T
        bound[rows] += s * (vmag * (prob.d_in * 2.0**-23) + np.abs(x[rows] @ A.T) * 2.0**-16) @ np.abs(Bm).T
    return ref, bound + 2.0**-8 * 1.01 * np.abs(ref) + 2.0**-133


def run_fused(prob, W, ws, plan, T=None):
    T = T or prob.T
    y = torch.full((T, (prob.d_out + 7) // 8 * 8 + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    work = B.workspace(B.LORA_OP_FUSED_BLOCK, T, prob.d_in, prob.d_out, max(prob.max_rank, 1))
    x = torch.zeros(T, prob.d_in, dtype=torch.bfloat16, device="cuda")
    x[: prob.T] = B.to_device(prob.x, "bf16")
    B.fused_linear_e4m3_block(x, torch.from_numpy(W).cuda(), torch.from_numpy(ws).cuda(), plan, y[:, : prob.d_out], work)
    assert (y[:, prob.d_out:] == 5.0).all()
    return y[:, : prob.d_out].double().cpu().numpy()


FUSED = [(1, 128, 256, [16]), (8, 256, 264, [8, 8]), (64, 1024, 512, [16] * 8), (65, 528, 136, [3, 17]), (130, 400, 1000, [8, 64, 1]),
         (300, 512, 2048, [16, 32, 5, 100]), (1000, 1024, 2304, [16] * 20), (2100, 384, 4096, [8, 16, 256]), (2100, 144, 8304, [8, 16] * 40),
         (2100, 144, 8304, [5, 17]), (3, 32, 5, [1, 2]), (70, 32, 5, [1, 1, 2]), (40, 64, 1, [7, 9]), (90, 64, 3, [3, 33])]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,d_in,d_out,ranks", FUSED)
def test_fused(kind, T, d_in, d_out, ranks):
    say(f"fused {kind} {T} {d_in}->{d_out} {ranks[:4]}")
    prob = fused_problem(T, d_in, d_out, ranks, T, layout="random" if T < 500 else "runs")
    W, ws = base(np.random.default_rng(T), d_out, d_in, kind)
    pool = B.DevicePool.from_problem(prob)
    plan = B.Plan(T).build(prob.ids, pool).upload()
    ref, bound = fused_reference(prob, W, ws, kind)
    check(run_fused(prob, W, ws, plan), ref, bound, f"{T} {d_in}->{d_out}")


def test_fused_without_adapters():
    prob = fused_problem(40, 256, 128, [16], 1, none=1.1)
    W, ws = base(np.random.default_rng(1), 128, 256, "f32")
    pool = B.DevicePool.from_problem(prob)
    plan = B.Plan(40).build(prob.ids, pool).upload()
    ref, bound = fused_reference(prob, W, ws, "f32")
    check(run_fused(prob, W, ws, plan), ref, bound, "no adapter")


# ---- gradients
def grad_reference(prob, W, ws, kind, x, dy):
    """dx, dA, dB in 64 bits, and bounds.  dx: the product's bound with dy's codes, u's two halves (2^-16) and fp32 sums, one
    rounding.  dA, dB: fp32 sums of products with u and v, themselves fp32 sums (2^-23 for each addition, and 2^-22
    for u and v in three bf16 parts)."""
    T, d_in, d_out = prob.T, prob.d_in, prob.d_out
    q, s, _ = R.quantize(dy, 1, kind)
    w = R.dequantize(W, ws, 128)
    d = R.dequantize(q, s, 1)
    dx = d @ w
    tops = np.repeat(R._tops(q, s, 1), 8, 1)[:, : d_out]  # eights along d_out on both sides
    wt = np.abs(R.decode(W))
    with np.errstate(divide="ignore"):
        e = np.where(wt >= 2.0**-6, np.exp2(np.floor(np.log2(np.maximum(wt, 2.0**-6)))), 2.0**-6) * R.spread(R.scale_values(ws), 128, W.shape)
    e = np.pad(e, ((0, -d_out % 8), (0, 0))).reshape(-1, 8, d_in).max(1)
    bound = (d_out + -(-d_out // 128) + 20) * 2.0**-23 * (np.abs(d) @ np.abs(w)) + 8 * 2.0**-13 * tops[:, ::8] @ e
    dA, dB, bA, bB = {}, {}, {}, {}
    for i in range(prob.n_adapters):
        rows = np.nonzero(prob.ids == i)[0]
        if not rows.size:
            continue
        A = bf16_bits_to_f32(prob.A(i)).astype(np.float64).reshape(-1, d_in)
        Bm = bf16_bits_to_f32(prob.B(i)).astype(np.float64).reshape(d_out, -1)
        c = float(np.float32(prob.alphas[i]) / np.float32(A.shape[0]))
        u, um = c * dy[rows] @ Bm, c * np.abs(dy[rows]) @ np.abs(Bm)
        v, vm = c * x[rows] @ A.T, c * np.abs(x[rows]) @ np.abs(A).T
        dx[rows] += u @ A
        bound[rows] += (um * (d_out + 4) * 2.0**-23 + np.abs(u) * 2.0**-16 + um * 256 * 2.0**-23) @ np.abs(A)
        dA[i], dB[i] = u.T @ x[rows], dy[rows].T @ v
        n = rows.size
        bA[i] = (um * (d_out + n + 16) * 2.0**-23).T @ np.abs(x[rows])
        bB[i] = np.abs(dy[rows]).T @ (vm * (d_in + n + 16) * 2.0**-23)
    return dx, bound + 2.0**-8 * 1.01 * np.abs(dx) + 2.0**-133, dA, bA, dB, bB


GRADS = [(1, 128, 128, [16]), (40, 256, 264, [8, 8, 3]), (64, 1024, 512, [16] * 8), (65, 528, 136, [3, 17]), (130, 400, 1000, [8, 64, 1]),
         (300, 512, 2049, [16, 32, 5, 100]), (64, 256, 8192, [16] * 3), (2100, 4096, 384, [8, 16, 256]), (4200, 2064, 250, [16] * 4), (4200, 4368, 130, [8, 16])]


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,d_in,d_out,ranks", GRADS)
def test_gradients(kind, T, d_in, d_out, ranks):
    say(f"gradients {kind} {T} {d_in}->{d_out} {ranks[:4]}")
    rng = np.random.default_rng(T + d_in)
    prob = fused_problem(T, d_in, d_out, ranks, T, layout="random" if T < 500 else "runs")
    W, ws = base(rng, d_out, d_in, kind)
    pool = B.DevicePool.from_problem(prob)
    plan = B.Plan(T).build(prob.ids, pool).upload()
    dyh, dy = bf16(hidden(rng, T, d_out) * 1e-3)
    x = bf16_bits_to_f32(prob.x).reshape(prob.x.shape).astype(np.float64)
    dx, bound, dA, bA, dB, bB = grad_reference(prob, W, ws, kind, x, dy)
    lddy = (d_out + 7) // 8 * 8
    dyd = torch.zeros(T, lddy, dtype=torch.bfloat16, device="cuda")[:, :d_out]
    dyd.copy_(dyh)
    out = torch.full((T, d_in + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    grads = B.GradPool.like(pool)
    work = B.workspace(B.LORA_OP_FUSED_BLOCK_BACKWARD, T, d_in, d_out, prob.max_rank)
    call = lambda g, acc=False: B.fused_linear_e4m3_block_backward(  # noqa: E731
        B.to_device(prob.x, "bf16"), torch.from_numpy(W).cuda(), torch.from_numpy(ws).cuda(), dyd, plan, g, out[:, :d_in], work, accumulate=acc)
    call(grads)
    check(out[:, :d_in].double().cpu().numpy(), dx, bound, "dx")
    assert (out[:, d_in:] == 5.0).all()
    for i in dA:
        check(grads.A[i].double().cpu().numpy(), dA[i], bA[i] + 1e-30, f"dA {i}")
        check(grads.B[i].double().cpu().numpy(), dB[i], bB[i] + 1e-30, f"dB {i}")
    first = out.clone()
    call(None)  # dx alone
    assert torch.equal(out, first)
