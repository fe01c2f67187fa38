"""Plans built on the device at their ends: pools without adapters, and what lies behind the tables."""

import numpy as np
import pytest

from gpu_helpers import require_gpu, say
from segmented_gather_gemm_lora_amd import binding as B
from test_gpu_device_plan import check_plan, dev32, fake_pool, tokens

pytestmark = pytest.mark.gpu
torch = None


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    global torch
    import test_gpu_device_plan

    torch = test_gpu_device_plan.torch = require_gpu()


@pytest.mark.parametrize("T,N", [(1, 0), (33, 0), (1000, 0), (33, 1), (300, 40)])
def test_nothing_is_written_behind_the_tables(T, N):
    """The buffer from bytes_used on is as it was, with a pool of no adapters too, whose plan has
    no table of segments by row; its one word of seg_indptr is 0."""
    say(f"plan {T} rows of {N} adapters")
    plan = B.DevicePlan(T, fake_pool([16] * N))
    plan.dev.fill_(0x5A)
    rng = np.random.default_rng(T)
    plan.build(dev32(rng.integers(-1, max(N, 3), T)))
    torch.cuda.synchronize()
    b, raw = plan.bounds(), plan.dev.cpu().numpy()
    assert (raw[b["bytes_used"]:] == 0x5A).all()
    if N == 0:
        assert b["num_sorted"] == 0 and b["soa_offset"] == b["segidx_offset"]
        assert raw[b["soa_offset"]:][:4].view(np.int32)[0] == 0
        assert plan.header()["num_tokens"] == T and plan.tables()["perm"].tolist() == list(range(T))


def test_a_plan_of_no_rows_has_counts():
    """Nothing is launched for it; header() and tables() read zeros, not what the memory held."""
    pool = fake_pool([16] * 4)
    held = torch.full((B.lora_segments_bytes(0),), 0x5A, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del held
    plan = B.DevicePlan(0, pool).build(dev32(np.zeros(0)), dev32(np.zeros(0)))
    h = plan.header()
    assert all(h[k] == 0 for k in ("num_tokens", "num_sorted", "num_segments", "num_blocks", "num_chunks", "max_rank", "max_len"))
    assert plan.tables()["counts"].tolist() == [0] * 7 and len(plan.arrays()["perm"]) == 0


@pytest.mark.parametrize("N", [2457, 2458, 4000, 7168])
def test_many_adapters_captured(N):
    """Past 2457 adapters the tables need more LDS than a launch has unasked: built inside a capture, as the
    first build of that size, and replayed for other batches."""
    say(f"captured plan of {N} adapters")
    rng = np.random.default_rng(N)
    T, R = 700, 60
    pool = fake_pool(rng.choice([8, 16, 64], N))
    adapters, lengths = dev32(np.zeros(R)), dev32(np.zeros(R))
    plan = B.DevicePlan(T, pool)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        plan.build(adapters, lengths)
    for i in range(4):
        a = rng.integers(-1, N, R).astype(np.int32)
        a[0] = N - 1
        ln = rng.integers(0, 30, R).astype(np.int32)
        adapters.copy_(torch.from_numpy(a))
        lengths.copy_(torch.from_numpy(ln))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_plan(plan, pool, tokens(a, ln, T), T)


def test_the_tables_stay_while_the_plan_does():
    """Changes inside the pool's tables are seen; the tensors themselves may be let go."""
    pool, T = fake_pool([16] * 8), 40
    ids = (np.arange(T) % 8).astype(np.int32)
    plan = B.DevicePlan(T, pool)
    first = [getattr(pool, k) for k in ("addr_A_dev", "addr_B_dev", "rank_dev", "alpha_dev")]
    at = [t.data_ptr() for t in first]
    first[3].mul_(2)
    pool.alpha *= 2
    for k in ("addr_A_dev", "addr_B_dev", "rank_dev", "alpha_dev"):
        setattr(pool, k, None)
    del first
    others = [torch.full((8,), 3, dtype=dt, device="cuda") for dt in (torch.int64, torch.int64, torch.int32, torch.float32)]
    assert not set(t.data_ptr() for t in others) & set(at)
    plan.build(dev32(ids))
    check_plan(plan, pool, ids, T)
