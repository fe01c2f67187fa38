"""Gradients of the fused layer (lora_fused_linear_backward) on the GPU against
the 64-bit reference."""

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
    return require_gpu()


def call(p, d, accumulate=False, stream=None, **kw):
    x, grads = kw.get("x", d.x), kw.get("grads", d.grads)
    B.fused_linear_backward(x, d.W0, d.dy, d.plan, grads, d.dx, d.ws, accumulate=accumulate, stream=stream)


CASES = [  # T, d_in, d_out, ranks, ids
    (1, 64, 64, [16], "one"),
    (1, 8, 1, [1], "one"),
    (3, 8, 7, [3, 256], "mixed"),
    (5, 264, 40, [8], "one"),
    (33, 256, 512, [16, 8], "mixed"),
    (63, 512, 1024, [16] * 63, "each"),
    (64, 136, 264, [64, 24, 40], "runs"),
    (65, 256, 100, [17, 33, 100], "mixed"),
    (200, 1000, 333, [16, 8, 4, 2], "mixed"),
    (256, 256, 256, [16], "one"),
    (257, 520, 96, [32, 8], "runs"),
    (300, 320, 32, [16] * 300, "each"),
    (700, 776, 4100, [16, 64, 128], "mixed"),
    (1100, 264, 31, [5, 20], "runs"),
]


@pytest.mark.parametrize("T,d_in,d_out,ranks,kind", CASES)
def test_against_64_bits(T, d_in, d_out, ranks, kind):
    say(f"case fused backward T={T} {d_in}->{d_out} ranks={ranks[:6]} {kind}")
    p = Problem("bf16", ids_of(kind, T, len(ranks), T), ranks, d_in, d_out, seed=T, w0=True, pad=(0, -d_out % 8, 0))
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    check(p, d, f"T={T}")


WIDE = [  # enough tiles of 256 rows: with the summed axis in parts and whole
    (300, 4104, 2050, [16, 8, 64], "mixed"),
    (513, 4096, 2048, [16] * 40, "runs"),
    (2100, 4104, 72, [33, 8, 100], "mixed"),
    (2305, 3848, 31, [16] * 300, "runs"),
]


@pytest.mark.parametrize("T,d_in,d_out,ranks,kind", WIDE)
def test_wide_layers(T, d_in, d_out, ranks, kind):
    test_against_64_bits(T, d_in, d_out, ranks, kind)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_stay_with_their_rows_in_large_tiles(value):
    ids = ids_of("runs", 2100, 4, 12)
    p, q = (Problem("bf16", ids, [16, 8, 20, 64], 4104, 69, seed=12, w0=True, pad=(0, 3, 0)) for _ in range(2))
    rows = np.nonzero(ids == 2)[0]
    p.dy_full[rows] = value
    p.A[2].fill_(value)
    p.B[2].fill_(value)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    keep = np.nonzero(ids != 2)[0]
    (dx, _, _), (edx, _, _) = q.reference()
    from backward_ref import worst

    assert worst(d.dx.double().cpu().numpy()[keep], dx[keep], edx[keep]) <= 1


@pytest.mark.parametrize("pad", [(8, 16, 24), (0, 8, 16)])
def test_pitches(pad):
    p = Problem("bf16", ids_of("mixed", 90, 3, 5), [16, 8, 30], 128, 192, seed=5, pad=pad, w0=True)
    d = p.device(misalign=8)
    call(p, d)
    torch.cuda.synchronize()
    check(p, d, f"{pad}")
    got = d.dx.as_strided((p.T - 1, pad[2]), (d.dx.stride(0), 1), d.dx.storage_offset() + 128)
    assert torch.equal(got.cpu(), p.dx_full[:-1, 128:])


@pytest.mark.parametrize("T", [40, 600])
def test_integers_are_exact(T):
    """Entries in {-1, 0, 1}, scale 1: small integer sums, exact in any order (|dx| <= 256)."""
    p = Problem("bf16", ids_of("mixed", T, 4, 2), [1, 4, 8, 3], 264, 50, seed=2, integer=True, w0=True, pad=(0, 6, 0))
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    (dx, dA, dB), _ = p.reference()
    assert np.abs(dx).max() <= 256
    assert np.array_equal(d.dx.double().cpu().numpy(), dx)
    for i in range(4):
        assert np.array_equal(d.grads.A[i].double().cpu().numpy(), dA[i])


@pytest.mark.parametrize("ids", [[-1] * 70, [-1] * 3])
def test_no_adapted_rows(ids):
    """Rows without an adapter get dy W0 alone; no gradient is touched."""
    p = Problem("bf16", ids, [16], 64, 96, w0=True)
    d = p.device()
    d.grads.A[0].zero_(), d.grads.B[0].zero_()
    call(p, d)
    torch.cuda.synchronize()
    check(p, d)


def test_base_alone_and_repeats():
    """Without gradients (x not given) dx is the same; repeats and another stream give the same bits."""
    p = Problem("bf16", ids_of("mixed", 500, 5, 6), [16, 8, 32, 64, 16], 256, 1024, seed=6, w0=True)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    check(p, d)
    first = d.dx.clone()
    s = torch.cuda.Stream()
    for k in range(3):
        d.dx.fill_(float("nan"))
        s.wait_stream(torch.cuda.current_stream())
        call(p, d, x=None, grads=None, stream=s)
        s.synchronize()
        assert torch.equal(d.dx, first), k


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [50, 150])
def test_bad_values_stay_with_their_rows(value, T):
    """A bad adapter or row reaches neither other adapters' rows nor the rows without one,
    and dy's columns past d_out are not read into a result."""
    ids = ids_of("mixed", T, 4, 11)
    p = Problem("bf16", ids, [16, 8, 20, 64], 136, 69, seed=11, w0=True, pad=(0, 3, 0))
    q = Problem("bf16", ids, [16, 8, 20, 64], 136, 69, seed=11, w0=True, pad=(0, 3, 0))
    p.dy_full[:, 69:] = value
    rows = np.nonzero(ids == 1)[0]
    p.x_full[rows] = value
    p.dy_full[rows] = value
    p.A[1].fill_(value)
    p.B[1].fill_(value)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    keep = np.nonzero(ids != 1)[0]
    (dx, dA, dB), (edx, eA, eB) = q.reference()
    from backward_ref import worst

    assert worst(d.dx.double().cpu().numpy()[keep], dx[keep], edx[keep]) <= 1
    assert not torch.isfinite(d.dx[torch.from_numpy(rows).cuda()]).any()
    for i in (0, 2, 3):
        assert worst(d.grads.A[i].double().cpu().numpy(), dA[i], eA[i]) <= 1
        assert worst(d.grads.B[i].double().cpu().numpy(), dB[i], eB[i]) <= 1


def test_captured_and_replayed():
    p = Problem("bf16", ids_of("runs", 300, 3, 8), [16, 8, 32], 256, 512, seed=8, w0=True)
    d = p.device()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        call(p, d)
    for k in range(4):
        d.dy.copy_(torch.randn(d.dy.shape, device="cuda"))
        for t in (d.dx, *d.grads.A, *d.grads.B):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (d.dx, *d.grads.A, *d.grads.B)]
        call(p, d)
        torch.cuda.synchronize()
        for a, b in zip(got, (d.dx, *d.grads.A, *d.grads.B)):
            assert torch.equal(a, b), f"replay {k}"


def test_large_layer():
    """The fused workload's sizes, 300 of its rows checked in 64 bits."""
    T, d_in, d_out = 1024, 4096, 12288
    ids = ids_of("runs", T, 20, 3)
    p = Problem("bf16", ids, [16] * 20, d_in, d_out, seed=3, w0=True)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    rows = np.arange(0, T, 4)[:300]
    dy, W = p.dy.double().numpy()[rows], p.W0.double().numpy()
    dx = dy @ W
    bound = (d_out + 2) * 2.0**-24 * (np.abs(dy) @ np.abs(W))
    for k, t in enumerate(rows):
        i = ids[t]
        A, Bm = p.A[i].double().numpy(), p.B[i].double().numpy()
        u = p.scale[i] * dy[k] @ Bm
        dx[k] += u @ A
        bound[k] += (2.0**-16 + 52 * 2.0**-24) * (np.abs(u) @ np.abs(A))
        bound[k] += p.scale[i] * (d_out + 2) * 2.0**-24 * (np.abs(dy[k]) @ np.abs(Bm)) @ np.abs(A)
    bound += 2.0**-8 * np.abs(dx)
    err = np.abs(d.dx.double().cpu().numpy()[rows] - dx)
    assert (err <= bound).all(), float((err / bound).max())


def _copies(d):
    return [t.clone() for t in (d.dx, *d.grads.A, *d.grads.B)]


# T 90: the sum over d_out in parts; 2100 rows, 4104 columns: whole
@pytest.mark.parametrize("T,d_in,d_out", [(90, 264, 2056), (2100, 4104, 72)])
def test_accumulate_and_partial_requests(T, d_in, d_out):
    p = Problem("bf16", ids_of("mixed", T, 3, 7), [16, 8, 33], d_in, d_out, seed=7, w0=True)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    check(p, d, f"T={T}")
    first = _copies(d)
    # added to the gradients, not to dx
    call(p, d, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(d.dx, first[0])
    assert all(torch.equal(t, f + f) for t, f in zip((*d.grads.A, *d.grads.B), first[1:]))
    # single gradients left out, and all of a kind
    for A, Bm in (([0, None, 2], [None, 1, 2]), ([None] * 3, [0, 1, 2]), ([0, 1, 2], [None] * 3)):
        e = p.device()
        g = B.GradPool.from_tensors([None if i is None else e.grads.A[i] for i in A],
                                    [None if i is None else e.grads.B[i] for i in Bm], device="cuda")
        for t in (*e.grads.A, *e.grads.B):
            t.fill_(7.0)
        call(p, e, grads=g)
        torch.cuda.synchronize()
        assert torch.equal(e.dx, first[0])
        for i in range(3):
            for at, got, f in ((A[i], e.grads.A[i], first[1 + i]), (Bm[i], e.grads.B[i], first[4 + i])):
                assert (got == 7).all() if at is None else torch.equal(got, f)


def test_two_streams_at_once():
    """Two batches on two streams, each with its own workspace: the same bits as one after the other."""
    ps = [Problem("bf16", ids_of("mixed", T, 4, T), [16, 64, 100, 8], 264, 2080, seed=T, w0=True) for T in (70, 900)]
    ds = [p.device() for p in ps]
    for p, d in zip(ps, ds):
        call(p, d)
    torch.cuda.synchronize()
    want = [_copies(d) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    for k in range(4):
        for d in ds:
            for t in (d.dx, *d.grads.A, *d.grads.B):
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for p, d, s in zip(ps, ds, streams):
            call(p, d, stream=s)
        torch.cuda.synchronize()
        for d, w in zip(ds, want):
            assert all(torch.equal(a, b) for a, b in zip(_copies(d), w)), k


LARGE = [  # long sums over d_out: tiles of 256 rows, the sum in parts (up to 1100 rows) and whole
    (1100, 4104, 2050, [16, 8, 64], "mixed"),
    (1061, 4096, 2048, [16] * 40, "runs"),
    (2100, 4104, 2050, [33, 8, 100], "mixed"),
    (2305, 3848, 2079, [16] * 300, "runs"),
]


@pytest.mark.parametrize("T,d_in,d_out,ranks,kind", LARGE)
def test_long_sums(T, d_in, d_out, ranks, kind):
    test_against_64_bits(T, d_in, d_out, ranks, kind)


@pytest.mark.parametrize("T", [1100, 2100])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_bad_values_stay_with_their_rows_in_long_sums(value, T):
    from backward_ref import worst

    ids = ids_of("runs", T, 4, 12)
    p, q = (Problem("bf16", ids, [16, 8, 20, 64], 4104, 2053, seed=12, w0=True, pad=(0, 3, 0)) for _ in range(2))
    p.dy_full[np.nonzero(ids == 2)[0]] = value
    p.A[2].fill_(value)
    p.B[2].fill_(value)
    d = p.device()
    call(p, d)
    torch.cuda.synchronize()
    keep = np.nonzero(ids != 2)[0]
    (dx, _, _), (edx, _, _) = q.reference()
    assert worst(d.dx.double().cpu().numpy()[keep], dx[keep], edx[keep]) <= 1
