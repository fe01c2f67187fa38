"""Gradients of the segmented correction (lora_sgmv_backward) on the GPU against
the 64-bit reference, at the sizes, ranks, pitches and row patterns where they
can go wrong."""

import numpy as np
import pytest
import torch

from backward_ref import Problem, check
from gpu_helpers import require_gpu, say
from segmented_gather_gemm_lora_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    return require_gpu()


def call(p, d, accumulate=False, stream=None, **kw):
    x, grads, dx = kw.get("x", d.x), kw.get("grads", d.grads), kw.get("dx", d.dx)
    B.sgmv_backward(x, d.dy, d.plan, grads, dx, d.ws, p.dtype, accumulate=accumulate, stream=stream)


def ids_of(kind, T, n, seed):
    r = np.random.default_rng(seed)
    if kind == "one":
        return np.zeros(T, dtype=np.int32)
    if kind == "each":  # every row its own adapter
        return np.arange(T) % n
    if kind == "runs":
        return np.sort(r.integers(0, n, T))
    return r.integers(-1, n, T)  # mixed, some rows without an adapter


CASES = [  # T, d_in, d_out, ranks, ids
    (1, 64, 64, [16], "one"),
    (1, 1, 1, [1], "one"),
    (1, 4096, 1024, [8], "one"),
    (2, 8, 8, [256], "one"),
    (15, 72, 136, [8, 16], "mixed"),
    (16, 64, 64, [16], "one"),
    (17, 64, 320, [32, 8], "runs"),
    (33, 256, 256, [64, 24, 40], "mixed"),
    (40, 264, 520, [16] * 40, "each"),
    (64, 512, 384, [1, 2, 3, 5, 7], "mixed"),
    (65, 100, 60, [17, 33, 100], "mixed"),
    (130, 129, 65, [3, 12], "mixed"),
    (128, 128, 128, [16], "one"),
    (300, 320, 192, [16, 48], "runs"),
    (515, 576, 640, [16], "one"),
    (515, 200, 264, [72, 256], "mixed"),
    (1030, 64, 128, [8, 128], "runs"),
    (2500, 136, 72, [20, 64], "mixed"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d_in,d_out,ranks,kind", CASES)
def test_against_64_bits(dtype, T, d_in, d_out, ranks, kind):
    say(f"case backward {dtype} T={T} {d_in}->{d_out} ranks={ranks[:6]} {kind}")
    p = Problem(dtype, ids_of(kind, T, len(ranks), T), ranks, d_in, d_out, seed=T)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    check(p, d, f"{dtype} T={T}")


LONG = [  # enough 64-row pieces to fill the chip: ranks of one, two and more tiles
    (8400, 72, 136, [16, 8], "runs"),
    (8600, 136, 64, [32, 8, 24], "mixed"),
    (8777, 200, 72, [64, 8, 40], "runs"),
    (8500, 64, 264, [72, 128, 256], "mixed"),
    (8448, 8, 8, [48], "one"),
    (8300, 128, 192, [20, 64], "runs"),
]


@pytest.mark.parametrize("T,d_in,d_out,ranks,kind", LONG)
def test_many_long_segments(T, d_in, d_out, ranks, kind):
    say(f"case backward long T={T} {d_in}->{d_out} ranks={ranks} {kind}")
    p = Problem("bf16", ids_of(kind, T, len(ranks), T), ranks, d_in, d_out, seed=T)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    check(p, d, f"long T={T}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d_in", [1032, 1029])
def test_dx_of_many_long_segments(dtype, d_in):
    say(f"case backward long dx {dtype} {d_in}")
    p = Problem(dtype, ids_of("mixed", 8450, 3, d_in), [64, 40, 97], d_in, 24, seed=d_in)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    check(p, d, f"long dx {dtype} {d_in}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,misalign", [((8, 16, 24), 0), ((3, 1, 2), 0), ((0, 0, 5), 0), ((0, 0, 0), 1), ((8, 8, 8), 8)])
def test_pitches_and_alignment(dtype, pad, misalign):
    say(f"case backward pitches {dtype} {pad} {misalign}")
    p = Problem(dtype, ids_of("mixed", 90, 3, 5), [16, 8, 30], 128, 192, seed=5, pad=pad)
    d = p.device(misalign=misalign)
    call(p, d)
    torch.cuda.synchronize()
    check(p, d, f"{dtype} {pad}")
    if pad[2]:  # nothing between the rows is written
        got = d.dx.as_strided((p.T - 1, pad[2]), (d.dx.stride(0), 1), d.dx.storage_offset() + 128)
        assert torch.equal(got.cpu(), p.dx_full[:-1, 128:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_integers_are_exact(dtype):
    """Entries in {-1, 0, 1}, scale 1: every sum is a small integer, so any
    order gives the same bits (T = 200 rows, sums below 2^8 for bf16's dx)."""
    p = Problem(dtype, ids_of("mixed", 200, 4, 2), [1, 4, 8, 3], 48, 8, seed=2, integer=True)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    (dx, dA, dB), _ = p.reference()
    assert np.abs(dx).max() <= 256
    assert np.array_equal(d.dx.double().cpu().numpy(), dx)
    for i in range(4):
        assert np.array_equal(d.grads.A[i].double().cpu().numpy(), dA[i])
        assert np.array_equal(d.grads.B[i].double().cpu().numpy(), dB[i])


def test_gradients_keep_fp32_accuracy():
    """One row, x = 1: dA is u itself, an fp32 of 24 significant bits.  Fed in
    three bf16 parts it comes back to 2 roundings (2 * 2^-24)."""
    p = Problem("bf16", [0], [16], 64, 8, seed=9, alpha=11.7)
    p.x_full.fill_(1.0)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    u = (p.dy.double() @ p.B[0].double()).float() * np.float32(p.scale[0])
    rel = ((d.grads.A[0].cpu() - u.t()).abs() / u.t().abs()).max().item()
    # u's own sum of 8 products rounds too: 8 * 2^-24 of the magnitudes
    mag = (p.dy.double().abs() @ p.B[0].double().abs()) * p.scale[0]
    assert rel <= float((2 + 9 * (mag / u.double().abs()).max()) * 2.0**-24)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_accumulate_and_partial_requests(dtype):
    ids = ids_of("runs", 600, 3, 7)
    p = Problem(dtype, ids, [16, 8, 33], 192, 128, seed=7)
    (_, dA, dB), (_, eA, eB) = p.reference()
    # accumulate: twice the gradient, dx twice too
    d = p.device()
    call(p, d)
    first = [t.clone() for t in (*d.grads.A, *d.grads.B)]
    call(p, d, accumulate=True)
    torch.cuda.synchronize()
    for t, f in zip((*d.grads.A, *d.grads.B), first):
        assert torch.equal(t, f + f)
    # overwrite again: the same bits as the first call
    call(p, d, dx=None)
    torch.cuda.synchronize()
    for t, f in zip((*d.grads.A, *d.grads.B), first):
        assert torch.equal(t, f)
    # entries of 0 and NULL tables leave gradients out
    e = p.device()
    e.grads = B.GradPool.from_tensors([e.grads.A[0], None, e.grads.A[2]], [None, e.grads.B[1], e.grads.B[2]])
    call(p, e, dx=None)
    torch.cuda.synchronize()
    assert torch.equal(e.grads.A[0], first[0]) and torch.equal(e.grads.A[2], first[2])
    assert torch.equal(e.grads.B[1].view(-1), first[4].view(-1)) and torch.equal(e.grads.B[2].view(-1), first[5].view(-1))
    assert torch.equal(e.dx.cpu(), p.dx)
    # dx alone, without x
    f = p.device()
    call(p, f, x=None, grads=None)
    torch.cuda.synchronize()
    f.grads = d.grads
    check(p, f, "dx alone")


def test_rows_and_adapters_left_alone():
    """Adapters without a row keep their gradients; rows without an adapter keep dx."""
    ids = np.array([-1, 2, -1, 0, 2, 2, -1, 0] * 5)
    p = Problem("bf16", ids, [16, 16, 8], 64, 64, seed=3)
    d = p.device()
    for t in (*d.grads.A, *d.grads.B):
        t.fill_(7.0)
    call(p, d)
    torch.cuda.synchronize()
    assert (d.grads.A[1] == 7).all() and (d.grads.B[1] == 7).all()
    assert torch.equal(d.dx.cpu()[ids < 0], p.dx[ids < 0])
    d.grads.A[1].zero_(), d.grads.B[1].zero_()
    check(p, d)


@pytest.mark.parametrize("T,ids", [(0, []), (5, [-1] * 5)])
def test_no_adapted_rows(T, ids):
    p = Problem("bf16", ids, [16], 64, 64)
    d = p.device()
    d.grads.A[0].fill_(3.0)
    call(p, d)
    torch.cuda.synchronize()
    assert torch.equal(d.dx.cpu(), p.dx) and (d.grads.A[0] == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_stay_with_their_adapter(dtype, value):
    """A NaN or infinity in one adapter's rows or matrices reaches no other adapter's results."""
    ids = ids_of("mixed", 150, 4, 11)
    p = Problem(dtype, ids, [16, 8, 20, 64], 136, 72, seed=11)
    rows = np.nonzero(ids == 1)[0]
    p.x_full[rows] = value
    p.dy_full[rows] = value
    p.x_full[ids < 0] = value
    p.dy_full[ids < 0] = value
    p.A[1].fill_(value)
    p.B[1].fill_(value)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    assert not torch.isfinite(d.grads.A[1]).any() and not torch.isfinite(d.grads.B[1]).any()
    keep = np.nonzero(ids != 1)[0]
    q = Problem(dtype, ids, [16, 8, 20, 64], 136, 72, seed=11)
    (dx, dA, dB), (edx, eA, eB) = q.reference()
    from backward_ref import worst

    assert worst(d.dx.double().cpu().numpy()[keep], dx[keep], edx[keep]) <= 1
    for i in (0, 2, 3):
        assert worst(d.grads.A[i].double().cpu().numpy(), dA[i], eA[i]) <= 1
        assert worst(d.grads.B[i].double().cpu().numpy(), dB[i], eB[i]) <= 1


def test_differences_of_the_loss():
    """L = sum(dy y) is linear in A, in B and in x one at a time, so a central
    difference of the forward (64 bits) equals the gradient's inner product."""
    import oracle

    p = Problem("f32", ids_of("mixed", 70, 3, 4), [8, 5, 16], 96, 80, seed=4)
    p.dx_full.zero_()
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()

    def loss(A, Bm, x):
        L = 0.0
        for i in range(3):
            rows = np.nonzero(p.ids == i)[0]
            y = p.scale[i] * (x[rows] @ A[i].T) @ Bm[i].T
            L += float((p.dy.double().numpy()[rows] * y).sum())
        return L

    del oracle
    r = np.random.default_rng(0)
    A, Bm, x = [t.double().numpy() for t in p.A], [t.double().numpy() for t in p.B], p.x.double().numpy()
    for which in range(3):
        dirs = [[r.standard_normal(t.shape) for t in A], [r.standard_normal(t.shape) for t in Bm], r.standard_normal(x.shape)]
        zero = [[t * 0 for t in dirs[0]], [t * 0 for t in dirs[1]], dirs[2] * 0]
        use = [dirs[k] if k == which else zero[k] for k in range(3)]
        up = loss([a + e for a, e in zip(A, use[0])], [b + e for b, e in zip(Bm, use[1])], x + use[2])
        dn = loss([a - e for a, e in zip(A, use[0])], [b - e for b, e in zip(Bm, use[1])], x - use[2])
        got = sum(float((g.double().cpu().numpy().reshape(e.shape) * e).sum()) for g, e in
                  zip((d.grads.A, d.grads.B, [d.dx])[which], use[which] if which < 2 else [use[2]]))
        mag = sum(float(np.abs(g.double().cpu().numpy().reshape(e.shape) * e).sum()) for g, e in
                  zip((d.grads.A, d.grads.B, [d.dx])[which], use[which] if which < 2 else [use[2]]))
        # fp32 gradients whose sums have at most 200 terms: 200 * 2^-24 of the magnitudes
        assert abs((up - dn) / 2 - got) <= 200 * 2.0**-24 * mag


def test_stream_and_repeats():
    p = Problem("bf16", ids_of("mixed", 700, 5, 6), [16, 8, 32, 64, 16], 256, 384, seed=6)
    d = p.device()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(p, d, stream=s)
    s.synchronize()
    check(p, d, "side stream")
    first = [t.clone() for t in (*d.grads.A, *d.grads.B)]
    for _ in range(3):
        call(p, d)
    torch.cuda.synchronize()
    for t, f in zip((*d.grads.A, *d.grads.B), first):
        assert torch.equal(t, f)


def test_two_streams_at_once():
    """Two batches on two streams, each with its own workspace: the same bits as one after the other."""
    ps = [Problem("bf16", ids_of("mixed", T, 4, T), [16, 64, 100, 8], 264, 520, seed=T) for T in (700, 900)]
    ds = [p.device() for p in ps]
    start = [d.dx.clone() for d in ds]
    for p, d in zip(ps, ds):
        call(p, d)
    torch.cuda.synchronize()
    want = [(d.dx.clone(), [t.clone() for t in (*d.grads.A, *d.grads.B)]) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    for k in range(4):
        for d, x in zip(ds, start):
            d.dx.copy_(x)
            for t in (*d.grads.A, *d.grads.B):
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for p, d, s in zip(ps, ds, streams):
            call(p, d, stream=s)
        torch.cuda.synchronize()
        for d, (dx, grads) in zip(ds, want):
            assert torch.equal(d.dx, dx), k
            assert all(torch.equal(a, b) for a, b in zip((*d.grads.A, *d.grads.B), grads)), k


def test_captured_and_replayed():
    """A captured call, replayed with new inputs between eager calls that share its workspace."""
    p = Problem("bf16", ids_of("runs", 600, 3, 8), [16, 8, 32], 256, 128, seed=8)
    d = p.device()
    dx0 = d.dx.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(p, d)
    for k in range(4):
        d.x.copy_(torch.randn(d.x.shape, device="cuda"))
        d.dx.copy_(dx0)
        for t in (*d.grads.A, *d.grads.B):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (d.dx, *d.grads.A, *d.grads.B)]
        d.dx.copy_(dx0)
        call(p, d)
        torch.cuda.synchronize()
        for a, b in zip(got, (d.dx, *d.grads.A, *d.grads.B)):
            assert torch.equal(a, b), f"replay {k}"


def test_larger_workspace_request_covers_smaller_batches():
    """One workspace for the largest batch serves every smaller one."""
    for T in (100, 4096, 4352, 9000):
        big = B.lora_workspace_bytes(B.LORA_OP_SGMV_BACKWARD, T + 300, 256, 256, 64)
        assert big >= B.lora_workspace_bytes(B.LORA_OP_SGMV_BACKWARD, T, 256, 256, 64)
    p = Problem("bf16", np.zeros(4096), [16], 64, 64, seed=1)
    d = p.device()
    d.ws = B.workspace(B.LORA_OP_SGMV_BACKWARD, 4352, 64, 64, 16)
    call(p, d)
    torch.cuda.synchronize()
    check(p, d)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["x", "dy", "A", "B"])
def test_one_infinity_enters_what_the_formulas_say(dtype, where):
    """A single infinity: results whose sums hold it are infinite or NaN, all others are as without it."""
    from backward_ref import worst

    ids = ids_of("mixed", 90, 3, 21)
    p, q = (Problem(dtype, ids, [16, 8, 40], 136, 72, seed=21) for _ in range(2))
    t = int(np.nonzero(ids == 1)[0][3])
    dst, at = {"x": (p.x_full, (t, 17)), "dy": (p.dy_full, (t, 33)), "A": (p.A[1], (5, 17)), "B": (p.B[1], (33, 5))}[where]
    dst[at] = float("inf")
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    (dx, dA, dB), (edx, eA, eB) = q.reference()
    # u = s dy B, v = s x A^T: rows (of the batch) and ranks that hold the infinity
    hit = ids == 1 if where in ("A", "B") else np.arange(90) == t
    in_dx, in_A, in_B = np.zeros(dx.shape, bool), np.zeros(dA[1].shape, bool), np.zeros(dB[1].shape, bool)
    if where == "x":  # v[t]: every rank; x's own column of dA
        in_A[:, 17], in_B[:] = True, True
    elif where == "dy":  # u[t]: every rank; dy's own row of dB
        in_dx[hit], in_A[:], in_B[33] = True, True, True
    elif where == "A":  # v's rank 5; u times A's column 17
        in_dx[np.ix_(hit, [17])] = True
        in_B[:, 5] = True
    else:  # u's rank 5
        in_dx[hit], in_A[5] = True, True
    for got, want, e, bad in ((d.dx, dx, edx, in_dx), (d.grads.A[1], dA[1], eA[1], in_A), (d.grads.B[1], dB[1], eB[1], in_B)):
        got = got.double().cpu().numpy().reshape(want.shape)
        assert not np.isfinite(got[bad]).any()
        assert worst(got[~bad], want[~bad], e[~bad]) <= 1
    for i in (0, 2):
        assert worst(d.grads.A[i].double().cpu().numpy(), dA[i], eA[i]) <= 1
        assert worst(d.grads.B[i].double().cpu().numpy(), dB[i], eB[i]) <= 1
