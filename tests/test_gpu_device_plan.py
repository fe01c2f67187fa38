"""Plans built on the device: their tables against the host builder's, and the calls on them."""

import numpy as np
import pytest

import oracle
from gpu_helpers import assert_close, decode, require_gpu, say
from lora_workloads import make_problem
from segmented_gather_gemm_lora_amd import binding as B

pytestmark = pytest.mark.gpu
torch = None


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    global torch
    torch = require_gpu()


def fake_pool(ranks, device="cuda"):
    """A pool of tables alone: plans hold addresses and do not look behind them."""
    ranks = np.asarray(ranks, dtype=np.int32)
    n = len(ranks)
    at = 0x7F0000000000 + 4096 * np.arange(2 * n, dtype=np.uint64)
    alpha = (16.0 + np.arange(n) % 7).astype(np.float32)
    p = B.DevicePool(storage=None, n_adapters=n, dtype="bf16", d_in=64, d_out=64, addr_A=at[0::2].copy(),
                     addr_B=at[1::2].copy(), rank=ranks, alpha=alpha)
    for k, t in (("addr_A_dev", p.addr_A.view(np.int64)), ("addr_B_dev", p.addr_B.view(np.int64)), ("rank_dev", ranks),
                 ("alpha_dev", alpha)):
        setattr(p, k, torch.from_numpy(t.copy()).to(device))
    return p


def tokens(adapters, lengths, T):
    """Adapter of each row that a request owns."""
    lengths = np.ones(len(adapters), dtype=np.int64) if lengths is None else np.maximum(lengths, 0)
    return np.repeat(adapters, lengths)[:T].astype(np.int32)


def check_plan(plan, pool, ids, T):
    """The device plan against the host's of the same rows."""
    host = B.Plan(max(len(ids), 1)).build(ids, pool)
    hh, ha = host.header(), host.arrays()
    dh, da = plan.header(), plan.arrays()
    for k in ("num_tokens", "num_sorted", "num_segments", "num_blocks", "max_rank", "max_len", "num_chunks"):
        assert dh[k] == hh[k], (k, dh[k], hh[k])
    assert np.array_equal(da["perm"], ha["perm"]) and np.array_equal(da["unadapted"], ha["unadapted"])
    for k in ("desc", "blocks", "chunks", "segidx"):
        assert np.array_equal(da[k], ha[k]), k
    t = {k: v.cpu().numpy() for k, v in plan.tables().items()}
    S, nb, nc, n = hh["num_segments"], hh["num_blocks"], hh["num_chunks"], hh["num_tokens"]
    assert (t["perm"][n:] == -1).all() and (t["segidx"][hh["num_sorted"]:] == -1).all()
    assert (t["segments"][S:] == 0).all()
    for name, count, head in (("blocks", nb, 16), ("chunks", nc, 16)):
        assert (t[name][count:, :head] == 0).all() and (t[name][count:, head:] == -1).all()
    b, raw = plan.bounds(), plan.dev.cpu().numpy()
    Sb, o = b["num_segments"], b["soa_offset"]
    table = host.segment_table()
    A, o = raw[o: o + 8 * Sb].view(np.uint64), o + 8 * Sb
    Bm, o = raw[o: o + 8 * Sb].view(np.uint64), o + 8 * Sb
    ptr, o = raw[o: o + 4 * Sb + 4].view(np.int32), o + 4 * Sb + 4
    ad, o = raw[o: o + 4 * Sb].view(np.int32), o + 4 * Sb
    rk, o = raw[o: o + 4 * Sb].view(np.int32), o + 4 * Sb
    sc = raw[o: o + 4 * Sb].view(np.float32)
    assert np.array_equal(A[:S], table["seg_A"]) and np.array_equal(Bm[:S], table["seg_B"])
    assert np.array_equal(ptr[:S], table["seg_indptr"][:S]) and (ptr[S:] == hh["num_sorted"]).all()
    assert np.array_equal(ad[:S], table["seg_adapter"]) and (ad[S:] == -1).all()
    assert np.array_equal(rk[:S], table["seg_rank"]) and np.array_equal(sc[:S], table["seg_scale"])


def dev32(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


CASES = [  # rows, requests, mean length (0: one row each, no lengths), adapters, share without one
    (1, 1, 0, 1, 0.0), (1, 1, 1, 1, 1.0), (64, 64, 0, 32, 0.0), (64, 50, 0, 5, 0.2), (100, 7, 20, 3, 0.0), (255, 40, 3, 4, 0.1),
    (256, 256, 0, 1, 0.0), (257, 257, 0, 300, 0.0), (1000, 1, 1200, 3, 0.0), (1000, 30, 50, 1000, 0.3), (2304, 260, 8, 128, 0.0),
    (4096, 4096, 0, 16, 0.05), (4096, 3000, 1, 4000, 0.0), (16384, 600, 27, 2000, 0.05), (16385, 2, 5000, 7, 0.0),
    (20000, 20000, 0, 7168, 0.1), (65536, 65536, 0, 3, 0.0), (65536, 1500, 50, 1000, 0.0), (512, 5000, 1, 64, 0.0)]


@pytest.mark.parametrize("T,R,mean,N,none", CASES)
def test_tables(T, R, mean, N, none):
    say(f"plan {T} rows {R} requests mean {mean} of {N}")
    rng = np.random.default_rng(T + R + N)
    pool = fake_pool(rng.choice([8, 16, 33, 64, 256], N))
    adapters = rng.integers(0, N, R).astype(np.int32)
    adapters[rng.random(R) < none] = -1
    lengths = None if mean == 0 else rng.geometric(1.0 / mean, R).astype(np.int32)
    if lengths is not None and R > 3:
        lengths[rng.random(R) < 0.1] = 0
        lengths[1] = -5
    plan = B.DevicePlan(T, pool).build(dev32(adapters), dev32(lengths))
    check_plan(plan, pool, tokens(adapters, lengths, T), T)


def test_runs_and_one_adapter():
    """Whole waves of one adapter, of none, and of both in turn."""
    pool = fake_pool([16] * 9)
    ids = np.concatenate([np.full(700, 3), np.full(300, -1), np.full(500, 3), np.arange(500) % 9, np.full(2000, 8)]).astype(np.int32)
    check_plan(B.DevicePlan(4100, pool).build(dev32(ids)), pool, ids, 4100)


def test_adapters_outside_the_bounds_have_none():
    pool = fake_pool([16, 64, 12, 0, 16, 300])
    ids = np.tile(np.array([0, 1, 2, 3, 4, 5, 6, 1 << 30, -2, -1], dtype=np.int32), 30)
    plan = B.DevicePlan(400, pool, max_rank=32, rank_multiple=8).build(dev32(ids))
    check_plan(plan, pool, np.where((ids == 0) | (ids == 4), ids, -1).astype(np.int32), 400)


def test_huge_lengths_are_cut():
    pool = fake_pool([16] * 4)
    adapters = np.arange(2000, dtype=np.int32) % 4
    lengths = np.full(2000, 2**31 - 1, dtype=np.int32)
    lengths[0] = 10
    check_plan(B.DevicePlan(300, pool).build(dev32(adapters), dev32(lengths)), pool,
               np.concatenate([np.zeros(10), np.ones(290)]).astype(np.int32), 300)


@pytest.mark.parametrize("R", [0, 3])
def test_empty_batches(R):
    pool = fake_pool([16] * 4)
    plan = B.DevicePlan(33, pool).build(dev32(np.zeros(R)), dev32(np.zeros(R)))
    check_plan(plan, pool, np.zeros(0, dtype=np.int32), 33)
    none = B.DevicePlan(33, fake_pool([])).build(dev32(np.full(5, 2)))
    h = none.header()
    assert h["num_tokens"] == 5 and h["num_sorted"] == 0 and none.tables()["perm"].tolist() == [0, 1, 2, 3, 4] + [-1] * 28


# ---- calls on device plans
def problem(T, d_in, d_out, ranks, seed, dtype="bf16", w0=False, none=0.15):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, len(ranks), T).astype(np.int32)
    if T > 200:
        ids[: T // 2] = np.sort(ids[: T // 2])
    ids[rng.random(T) < none] = -1
    return make_problem(name="dev", dtype=dtype, ids=ids, ranks=list(ranks), alphas=[32.0] * len(ranks), d_in=d_in, d_out=d_out,
                        seed=seed, **({"w0_std": 0.02} if w0 else {}))


def reference(prob, fused=False):
    return oracle.lora_forward(prob, nthreads=4, fused=fused)[0]


def padded(prob, extra):
    """x and y with `extra` rows behind the batch, which no call may write."""
    x = torch.full((prob.T + extra, prob.d_in), float("nan"), device="cuda", dtype=B.torch_dtype(prob.dtype))
    x[: prob.T] = B.to_device(prob.x, prob.dtype)
    y = torch.full((prob.T + extra, prob.d_out), 3.0, device="cuda", dtype=B.torch_dtype(prob.dtype))
    y[: prob.T] = B.to_device(prob.y_base(), prob.dtype)
    return x, y


def out(y, prob):
    assert (y[prob.T:] == 3.0).all()
    return decode(B.to_host_bits(y[: prob.T], prob.dtype), prob.dtype)


SGMV = [(40, 256, 256, [8, 8], "bf16"), (40, 256, 256, [8, 8], "f32"), (64, 1024, 512, [16] * 32, "bf16"), (700, 512, 1024, [16] * 5, "bf16"),
        (700, 512, 4096, [8, 16, 32, 64], "bf16"), (300, 500, 333, [3, 100, 17], "bf16"), (300, 512, 512, [128, 256], "f32"),
        (1500, 512, 4096, [16] * 6, "bf16")]


@pytest.mark.parametrize("T,d_in,d_out,ranks,dtype", SGMV)
@pytest.mark.parametrize("call", ["combined", "split", "paged", "grouped"])
def test_sgmv(T, d_in, d_out, ranks, dtype, call):
    say(f"sgmv on a device plan {call} {T} {d_in}->{d_out} {ranks[:4]} {dtype}")
    prob = problem(T, d_in, d_out, ranks, T, dtype)
    pool = B.PagedPool.from_problem(prob, page_bytes=1024, shuffle_seed=1) if call == "paged" else B.DevicePool.from_problem(prob)
    extra = 37
    rows = T + extra
    x, y = padded(prob, extra)
    plan = B.DevicePlan(rows, pool).build(dev32(prob.ids))
    if call == "split":
        v = torch.full((rows, B.v_pitch(prob.max_rank)), float("nan"), device="cuda")
        B.sgmv_shrink(x, plan, v, dtype)
        B.sgmv_expand(v, plan, y, dtype)
    elif call == "grouped":
        ws = B.sgmv_grouped_workspace([plan], [x], [y])
        B.sgmv_grouped([x], [plan], [y], ws, dtype)
    else:
        ws = B.workspace(B.LORA_OP_SGMV, rows, d_in, d_out, prob.max_rank)
        if call == "paged":
            B.sgmv_paged(x, plan, pool, y, ws, dtype)
        else:
            B.sgmv(x, plan, y, ws, dtype)
    assert_close(out(y, prob), reference(prob), dtype, f"{call} {T}")


@pytest.mark.parametrize("T,d_in,d_out,ranks", [(40, 256, 256, [8, 8]), (300, 512, 400, [16] * 6), (700, 256, 512, [5, 17, 64])])
@pytest.mark.parametrize("e4m3", [False, True])
def test_fused(T, d_in, d_out, ranks, e4m3):
    say(f"fused on a device plan e4m3={e4m3} {T} {d_in}->{d_out}")
    prob = problem(T, d_in, d_out, ranks, T, w0=True)
    pool, rows = B.DevicePool.from_problem(prob), T + 19
    x, y = padded(prob, 19)
    plan = B.DevicePlan(rows, pool).build(dev32(prob.ids))
    ws = B.workspace(B.LORA_OP_FUSED, rows, d_in, d_out, prob.max_rank)
    if e4m3:
        codes = (B.to_device(prob.W0, "bf16").float() * 1024).clamp(-448, 448).to(torch.float8_e4m3fn)
        host = B.Plan(T).build(prob.ids, pool).upload()
        want = torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda")
        B.fused_linear_e4m3(x, codes.view(torch.uint8), 1 / 1024, host, want, ws)
        B.fused_linear_e4m3(x, codes.view(torch.uint8), 1 / 1024, plan, y, ws)
        assert_close(out(y, prob), want.double().cpu().numpy(), "bf16", "e4m3")
    else:
        B.fused_linear(x, B.to_device(prob.W0, "bf16"), plan, y, ws)
        assert_close(out(y, prob), reference(prob, fused=True), "bf16", "fused")
