"""The block-scaled operators as a model uses them: together, captured, on other streams, twice at
once, and at the ends of what they take."""

import dataclasses

import numpy as np
import pytest

import block_ref as R
from gpu_helpers import require_gpu, say
from segmented_gather_gemm_lora_amd import binding as B
from test_gpu_block import base, bf16, check, fused_problem, fused_reference

pytestmark = pytest.mark.gpu
torch = None


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    global torch
    import test_gpu_block

    torch = test_gpu_block.torch = require_gpu()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    """One projection: codes, scales and adapters on the device."""

    def __init__(self, d_in, d_out, ranks, kind, seed=0):
        self.prob = fused_problem(8, d_in, d_out, ranks, seed)
        self.kind = kind
        self.Wh, self.wsh = base(np.random.default_rng(seed), d_out, d_in, kind)
        self.W, self.ws = dev(self.Wh), dev(self.wsh)
        self.pool = B.DevicePool.from_problem(self.prob)


def requests(rng, R_, T, n):
    lengths = rng.integers(0, 2 * T // R_ + 1, R_).astype(np.int32)
    lengths = np.diff(np.minimum(np.cumsum(lengths), T), prepend=0).astype(np.int32)
    return lengths, rng.integers(-1, n, R_).astype(np.int32)


def owners(lengths, adapters):
    return np.repeat(adapters, lengths).astype(np.int32)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
@pytest.mark.parametrize("T,R_,d_in,d_out,ranks", [(64, 64, 256, 520, [16] * 6), (48, 10, 1024, 256, [8, 3, 17]),
                                                    (300, 20, 512, 1024, [8, 16, 64]), (1100, 40, 256, 2304, [16] * 30)])
def test_a_step_captured(kind, T, R_, d_in, d_out, ranks):
    """lengths -> plan -> fused layer -> its result quantized -> product with another base: one graph,
    replayed for other batches; every replay against the same calls made eagerly, on a plan of the
    host's, and against 64 bits.  Rows behind the last request hold NaN and are left as they were."""
    rng = np.random.default_rng(T + d_in)
    lay = Layer(d_in, d_out, ranks, kind, T)
    W2h, w2sh = base(rng, 200, (d_out + 15) // 16 * 16, kind)
    W2, w2s = dev(W2h), dev(w2sh)
    k2 = W2.shape[1]
    sdt = torch.float32 if kind == "f32" else torch.uint8

    def buffers():
        b = dict(x=torch.zeros(T, d_in, dtype=torch.bfloat16, device="cuda"), y=torch.zeros(T, k2, dtype=torch.bfloat16, device="cuda"),
                 q=torch.zeros(T, k2, dtype=torch.uint8, device="cuda"), s=torch.zeros((k2 + 127) // 128, (T + 3) // 4 * 4, dtype=sdt, device="cuda"),
                 z=torch.zeros(T, 200, device="cuda"), ws=B.workspace(B.LORA_OP_FUSED_BLOCK, T, d_in, d_out, max(ranks)),
                 ws2=B.workspace(B.LORA_OP_LINEAR_BLOCK, T, k2, 200, 1))
        return b

    lengths, adapters = torch.zeros(R_, dtype=torch.int32, device="cuda"), torch.zeros(R_, dtype=torch.int32, device="cuda")
    plan = B.DevicePlan(T, lay.pool)

    def step(b, p):
        B.fused_linear_e4m3_block(b["x"], lay.W, lay.ws, p, b["y"][:, :d_out], b["ws"])
        B.quantize_e4m3(b["y"], b["q"], b["s"][:, :T])
        B.linear_e4m3_block(b["q"], b["s"][:, :T], W2, w2s, b["z"], b["ws2"])

    g, e = buffers(), buffers()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        plan.build(adapters, lengths)
        step(g, plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        plan.build(adapters, lengths)
        step(g, plan)
    for i in range(5):
        say(f"replay {i}: {kind} T={T}")
        ln, ad = requests(rng, R_, T, len(ranks))
        if i == 2:
            ln[:] = 0  # nothing to do
        if i == 3:
            ad[:] = -1  # no adapter
        ids, n = owners(ln, ad), int(ln.sum())
        xh, x64 = bf16(rng.standard_normal((T, d_in)))
        for b in (g, e):
            b["x"].copy_(xh)
            b["x"][n:] = float("nan")
            b["y"].zero_()
            b["y"][:, :d_out] = 3.0
        lengths.copy_(torch.from_numpy(ln))
        adapters.copy_(torch.from_numpy(ad))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        if n:
            host = B.Plan(n).build(ids, lay.pool).upload()
            step(e, host)
            torch.cuda.synchronize()
            assert torch.equal(g["y"][:n], e["y"][:n]), i
            assert torch.equal(g["q"][:n], e["q"][:n]) and torch.equal(g["z"][:n], e["z"][:n]), i
            bits = xh[:n].view(torch.int16).numpy().view(np.uint16)
            ref, bound = fused_reference(dataclasses.replace(lay.prob, T=n, ids=ids, x=bits), lay.Wh, lay.wsh, kind)
            check(g["y"][:n, :d_out].double().cpu().numpy(), ref, bound, f"replay {i}")
        assert (g["y"][n:, :d_out] == 3.0).all()


def test_two_streams_at_once():
    """The same base and pool, two batches, each with its own workspace, on two streams at once."""
    lay = Layer(512, 1024, [16, 8, 32, 5], "f32", 3)
    rng = np.random.default_rng(5)
    jobs = []
    for T in (64, 700):
        ids = rng.integers(-1, 4, T).astype(np.int32)
        xh, _ = bf16(rng.standard_normal((T, 512)))
        plan = B.Plan(T).build(ids, lay.pool).upload()
        new = lambda: (torch.empty(T, 1024, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                       B.workspace(B.LORA_OP_FUSED_BLOCK, T, 512, 1024, 32))
        jobs.append((xh.cuda(), plan, new(), new(), torch.cuda.Stream()))
    for x, plan, (y, ws), _, _ in jobs:
        B.fused_linear_e4m3_block(x, lay.W, lay.ws, plan, y, ws)
    torch.cuda.synchronize()
    for _ in range(5):
        for x, plan, _, (y, ws), st in jobs:
            with torch.cuda.stream(st):
                B.fused_linear_e4m3_block(x, lay.W, lay.ws, plan, y, ws)
    torch.cuda.synchronize()
    for _, _, (y, _), (z, _), _ in jobs:
        assert torch.equal(y, z)


def test_an_adapter_that_is_not_finite_stays_with_its_rows():
    for T in (60, 300):
        for rank_set in ([8, 16, 5], [8, 16, 24]):
            prob = fused_problem(T, 256, 264, rank_set, T, none=0.1)
            W, ws = base(np.random.default_rng(1), 264, 256, "f32")
            pool = B.DevicePool.from_problem(prob)
            plan = B.Plan(T).build(prob.ids, pool).upload()
            x, work = B.to_device(prob.x, "bf16"), B.workspace(B.LORA_OP_FUSED_BLOCK, T, 256, 264, 24)
            y = torch.empty(T, 264, dtype=torch.bfloat16, device="cuda")
            B.fused_linear_e4m3_block(x, dev(W), dev(ws), plan, y, work)
            clean = y.clone()
            # adapter 1's B becomes NaN in place, through its address
            n = 264 * rank_set[1]
            store = pool.storage if pool.storage.dtype == torch.bfloat16 else pool.storage.view(torch.bfloat16)
            at = (int(pool.addr_B[1]) - store.data_ptr()) // 2
            store.view(-1)[at: at + n] = float("nan")
            B.fused_linear_e4m3_block(x, dev(W), dev(ws), plan, y, work)
            mine = torch.from_numpy(prob.ids == 1).cuda()
            assert torch.isnan(y[mine].float()).all() and torch.equal(y[~mine], clean[~mine])


@pytest.mark.parametrize("T", [30, 200, 2100])
@pytest.mark.parametrize("r", [1, 3, 4, 5, 8, 17, 20])
def test_a_column_that_is_not_finite_stays_alone(T, r):
    """One row of B (a column of y) holds NaN: its neighbours, whose ranks lie beside it, do not change."""
    d_out = 8312 if T > 1000 else 264
    prob = fused_problem(T, 128, d_out, [r], T, none=0.0)
    W, ws = base(np.random.default_rng(1), d_out, 128, "f32")
    pool = B.DevicePool.from_problem(prob)
    plan = B.Plan(T).build(prob.ids, pool).upload()
    x, work = B.to_device(prob.x, "bf16"), B.workspace(B.LORA_OP_FUSED_BLOCK, T, 128, d_out, r)
    y, z = (torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Wd, wsd = dev(W), dev(ws)
    B.fused_linear_e4m3_block(x, Wd, wsd, plan, y, work)
    store = pool.storage if pool.storage.dtype == torch.bfloat16 else pool.storage.view(torch.bfloat16)
    at = (int(pool.addr_B[0]) - store.data_ptr()) // 2
    cols = [0, 100, 257, d_out - 1]
    for c in cols:
        store.view(-1)[at + c * r: at + (c + 1) * r] = float("nan")
    B.fused_linear_e4m3_block(x, Wd, wsd, plan, z, work)
    keep = torch.ones(d_out, dtype=torch.bool, device="cuda")
    keep[cols] = False
    assert torch.isnan(z[:, ~keep].float()).all() and torch.equal(z[:, keep], y[:, keep])


def test_an_infinite_row_stays_alone():
    """Its codes have a NaN scale: the row's results are NaN and no other's change."""
    lay = Layer(384, 520, [16, 8], "f32", 9)
    for T in (40, 200):
        ids = (np.arange(T) % 3 - 1).astype(np.int32)
        xh, _ = bf16(np.random.default_rng(T).standard_normal((T, 384)))
        plan = B.Plan(T).build(ids, lay.pool).upload()
        work = B.workspace(B.LORA_OP_FUSED_BLOCK, T, 384, 520, 16)
        y, z = (torch.empty(T, 520, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        B.fused_linear_e4m3_block(xh.cuda(), lay.W, lay.ws, plan, y, work)
        xh[7, 200] = float("inf")
        B.fused_linear_e4m3_block(xh.cuda(), lay.W, lay.ws, plan, z, work)
        keep = torch.arange(T, device="cuda") != 7
        assert torch.isnan(z[7].float()).all() and torch.equal(y[keep], z[keep])


def gradient_job(T, d_in, d_out, ranks, kind, seed):
    prob = fused_problem(T, d_in, d_out, ranks, seed)
    W, ws = base(np.random.default_rng(seed), d_out, d_in, kind)
    pool = B.DevicePool.from_problem(prob)
    plan = B.Plan(T).build(prob.ids, pool).upload()
    x = B.to_device(prob.x, "bf16")
    dy = torch.randn(T, d_out, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(torch.bfloat16)
    work = B.workspace(B.LORA_OP_FUSED_BLOCK_BACKWARD, T, d_in, d_out, prob.max_rank)
    return prob, dev(W), dev(ws), pool, plan, x, dy, torch.empty_like(x), work


@pytest.mark.parametrize("T,d_in,d_out,ranks", [(64, 512, 256, [16] * 4), (700, 1024, 640, [8, 16, 64])])
def test_gradients_captured(T, d_in, d_out, ranks):
    """A captured backward pass, replayed with eager work between, while eager calls of the same leaves
    live: every replay is the eager call's bits; accumulate adds."""
    prob, W, ws, pool, plan, x, dy, dx, work = gradient_job(T, d_in, d_out, ranks, "f32", T)
    g1, g2 = B.GradPool.like(pool), B.GradPool.like(pool)
    dx2, work2 = torch.empty_like(dx), work.clone()
    call = lambda g, d, w, acc=False: B.fused_linear_e4m3_block_backward(x, W, ws, dy, plan, g, d, w, accumulate=acc)  # noqa: E731
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call(g1, dx, work)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(g1, dx, work)
    for i in range(4):
        dy.copy_(torch.randn(T, d_out, device="cuda", generator=torch.Generator("cuda").manual_seed(100 + i)))
        dx.zero_()
        torch.cuda.synchronize()
        graph.replay()
        call(g2, dx2, work2)
        torch.cuda.synchronize()
        assert torch.equal(dx, dx2)
        for a, b in zip(g1.A + g1.B, g2.A + g2.B):
            assert torch.equal(a, b)
    call(g2, dx2, work2, True)
    torch.cuda.synchronize()
    used = sorted(set(int(i) for i in prob.ids if i >= 0))
    for i in used:
        for a, b in ((g1.A[i], g2.A[i]), (g1.B[i], g2.B[i])):
            assert torch.allclose(b, 2 * a, rtol=2.0**-22, atol=0)
    assert torch.equal(dx, dx2)


def grid(rng, shape):
    """Multiples of the format with the largest code in every group: quantized exactly, with scales of 1."""
    v = R.values()
    x = v[rng.integers(40, 72, shape)] * rng.choice([-1.0, 1.0], shape)
    x[:, ::128] = 448.0
    return x


@pytest.mark.parametrize("T", [24, 150])
def test_gradients_against_differences(T):
    """L = sum(dy y) is linear in x, in every A and in every B (x, dy exact in E4M3, so the straight-through
    gradient is the gradient): L(p') - L(p) = <gradient, p' - p> up to the rounding of y to bf16."""
    d_in, d_out, ranks = 256, 256, [8, 16, 3]
    rng = np.random.default_rng(T)
    prob, W, ws, pool, plan, x, dy, dx, work = gradient_job(T, d_in, d_out, ranks, "e8m0", T)
    x.copy_(torch.from_numpy(grid(rng, (T, d_in))))
    dy.copy_(torch.from_numpy(grid(rng, (T, d_out))))
    grads = B.GradPool.like(pool)
    B.fused_linear_e4m3_block_backward(x, W, ws, dy, plan, grads, dx, work)
    fws = B.workspace(B.LORA_OP_FUSED_BLOCK, T, d_in, d_out, 16)

    def loss(x_):
        y = torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda")
        B.fused_linear_e4m3_block(x_, W, ws, plan, y, fws)
        p = dy.double() * y.double()
        return p.sum().item(), p.abs().sum().item()

    def same(L1, L0, step, what):
        # y: half a step of bf16 (2^-9) on each side, twice that for what is summed inside; the gradient: as much
        room = (L1[1] + L0[1]) * 2.0**-8 + step[1] * 2.0**-8
        assert abs((L1[0] - L0[0]) - step[0]) <= room, what
        assert abs(step[0]) > 0

    def inner(g, d):
        p = g.double() * d.double()
        return p.sum().item(), p.abs().sum().item()

    L0 = loss(x)
    x2 = x.clone()
    x2[T // 2] = torch.from_numpy(grid(rng, (1, d_in))[0]).to(torch.bfloat16).cuda()
    same(loss(x2), L0, inner(dx, x2.double() - x.double()), "dx")
    store = pool.storage if pool.storage.dtype == torch.bfloat16 else pool.storage.view(torch.bfloat16)
    for i in range(3):
        for addr, g, n in ((pool.addr_A, grads.A[i], ranks[i] * d_in), (pool.addr_B, grads.B[i], ranks[i] * d_out)):
            at = (int(addr[i]) - store.data_ptr()) // 2
            m = store.view(-1)[at: at + n]
            old = m.clone()
            m.copy_(old * 3 + 0.25)
            same(loss(x), L0, inner(g.reshape(-1), m.double() - old.double()), f"adapter {i}")
            m.copy_(old)


def test_columns_past_4_gib():
    """B of 8.6 GB and a base of 2^24 columns: offsets past 32 bits, in both forms."""
    d_in, d_out, r = 16, (1 << 24) + 8, 256
    gen = torch.Generator("cuda").manual_seed(1)
    Bm = torch.empty(d_out, r, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    A = torch.empty(r, d_in, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    W = torch.randint(0, 120, (d_out, d_in), dtype=torch.uint8, device="cuda", generator=gen)
    ws = torch.rand((d_out + 127) // 128, 1, device="cuda", generator=gen) + 0.5
    pool = B.DevicePool(storage=(A, Bm), n_adapters=1, dtype="bf16", d_in=d_in, d_out=d_out,
                        addr_A=np.array([A.data_ptr()], np.uint64), addr_B=np.array([Bm.data_ptr()], np.uint64),
                        rank=np.array([r], np.int32), alpha=np.array([1.0], np.float32))
    cols = torch.cat([torch.arange(64), torch.arange(d_out - 300, d_out), torch.randint(0, d_out, (2000,))]).cuda()
    for T in (2, 66):
        say(f"columns past 4 GiB, {T} rows")
        x = torch.empty(T, d_in, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        plan = B.Plan(T).build(np.zeros(T, np.int32), pool).upload()
        y = torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda")
        B.fused_linear_e4m3_block(x, W, ws, plan, y, B.workspace(B.LORA_OP_FUSED_BLOCK, T, d_in, d_out, r))
        xq, xs, _ = R.quantize(x.double().cpu().numpy(), 1, "f32")
        w = R.decode(W[cols].cpu().numpy()) * ws[cols // 128].double().cpu().numpy()
        v = x.double().cpu().numpy() @ A.double().cpu().numpy().T / r
        ref = R.dequantize(xq, xs, 1) @ w.T + v @ Bm[cols].double().cpu().numpy().T
        # 2^-8 for y, 2^-9 of the magnitudes for what is summed inside (products at 2^-13 of their largest)
        mag = np.abs(R.dequantize(xq, xs, 1)) @ np.abs(w).T + np.abs(v) @ np.abs(Bm[cols].double().cpu().numpy()).T
        check(y[:, cols].double().cpu().numpy(), ref, 2.0**-8 * np.abs(ref) + 2.0**-9 * mag, f"{T} rows")


def test_the_binding_refuses():
    lay = Layer(256, 264, [16], "f32", 2)
    T = 8
    x = torch.zeros(T, 256, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(T, 264, dtype=torch.bfloat16, device="cuda")
    plan = B.Plan(T).build(np.zeros(T, np.int32), lay.pool).upload()
    work = B.workspace(B.LORA_OP_FUSED_BLOCK, T, 256, 264, 16)
    f = B.fused_linear_e4m3_block
    for args in ((x.float(), lay.W, lay.ws, plan, y, work), (x, lay.W, lay.ws, plan, y.float(), work),
                 (x[:, :128], lay.W, lay.ws, plan, y, work), (x[:4], lay.W, lay.ws, plan, y, work), (x, lay.W, lay.ws, plan, y[:4], work),
                 (x, lay.W.view(torch.int8), lay.ws, plan, y, work), (x, lay.W, lay.ws[:1], plan, y, work),
                 (x, lay.W, lay.ws.half(), plan, y, work), (x.cpu(), lay.W, lay.ws, plan, y, work), (x, lay.W, lay.ws, plan, y, work.cpu()),
                 (x, lay.W.t().contiguous().t(), lay.ws, plan, y, work)):
        with pytest.raises(ValueError):
            f(*args)
    with pytest.raises(B.LoraError):
        f(x, lay.W, lay.ws, plan, y, work[:16])
    q, s = torch.zeros(T, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, T, device="cuda")
    for args in ((x.half(), q, s), (x, q[:, :100], s), (x, q, s[:1]), (x, q, s.half()), (x.cpu(), q, s), (x, q.cpu(), s), (x, q.float(), s)):
        with pytest.raises(ValueError):
            B.quantize_e4m3(*args)
    z = torch.zeros(T, 264, device="cuda")
    for args in ((q, s.to(torch.uint8), lay.W, lay.ws, z), (q, s, lay.W, lay.ws, z.half()), (q, s[:1], lay.W, lay.ws, z), (q, s, lay.W, lay.ws, z.cpu()),
                 (q.float(), s, lay.W, lay.ws, z)):
        with pytest.raises(ValueError):
            B.linear_e4m3_block(*args, work)
    dplan = B.DevicePlan(T, lay.pool)
    ad = torch.zeros(T, dtype=torch.int32, device="cuda")
    for a, ln in ((ad.long(), None), (ad.cpu(), None), (ad, ad[:4]), (ad, ad.long()), (ad, ad.cpu())):
        with pytest.raises(ValueError):
            dplan.build(a, ln)
    dplan.build(ad)
    with pytest.raises((ValueError, B.LoraError)):
        B.fused_linear_e4m3_block_backward(x, lay.W, lay.ws, y, dplan, B.GradPool.like(lay.pool), torch.zeros_like(x),
                                           B.workspace(B.LORA_OP_FUSED_BLOCK_BACKWARD, T, 256, 264, 16))


def test_single_rows_at_any_pitch():
    """One row out of a matrix whose pitch no call would take."""
    lay = Layer(256, 100, [16], "f32", 4)
    codes = torch.zeros(3, 263, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, 1, device="cuda")
    x = torch.randn(1, 256, device="cuda").to(torch.bfloat16)
    q = torch.zeros(1, 256, dtype=torch.uint8, device="cuda")
    B.quantize_e4m3(x, q, s)
    y, z = torch.zeros(1, 100, device="cuda"), torch.zeros(1, 100, device="cuda")
    B.linear_e4m3_block(q, s, lay.W, lay.ws, y, B.workspace(B.LORA_OP_LINEAR_BLOCK, 1, 256, 100, 1))
    codes[0, :256] = q[0]
    B.linear_e4m3_block(codes[:1, :256], s, lay.W, lay.ws, z, B.workspace(B.LORA_OP_LINEAR_BLOCK, 1, 256, 100, 1))
    assert torch.equal(y, z)


@pytest.mark.parametrize("kind", ["f32", "e8m0"])
def test_nothing_to_do(kind):
    lay = Layer(256, 264, [16], kind, 6)
    sdt = torch.float32 if kind == "f32" else torch.uint8
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros(0, 256, dtype=torch.uint8, device="cuda"), torch.zeros(2, 0, dtype=sdt, device="cuda")
    B.quantize_e4m3(x, q, s)
    y = torch.zeros(0, 264, dtype=torch.bfloat16, device="cuda")
    B.linear_e4m3_block(q, s, lay.W, lay.ws, y, B.workspace(B.LORA_OP_LINEAR_BLOCK, 0, 256, 264, 1))
    plan = B.DevicePlan(0, lay.pool).build(torch.zeros(0, dtype=torch.int32, device="cuda"))
    B.fused_linear_e4m3_block(x, lay.W, lay.ws, plan, y, B.workspace(B.LORA_OP_FUSED_BLOCK, 0, 256, 264, 16))
    torch.cuda.synchronize()
