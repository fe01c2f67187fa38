"""The backward calls on the CPU: refusals before any GPU call, workspace sizes,
and the reference's own gradients against differences."""

import ctypes

import numpy as np
import pytest

from segmented_gather_gemm_lora_amd import binding as B
from test_abi_cpu import FAKE_BASE, HostPlan, build, make_tables

FX = FAKE_BASE + 0x40000000
BIG = 1 << 40


def plan_of(ids, n, ranks):
    A, Bt, r, al = make_tables(n, np.random.default_rng(0), ranks)
    st, plan = build(ids, n, A, Bt, r, al)
    assert st == 0
    return plan


def run(plan, **kw):
    a = dict(dtype=B.LORA_BF16, x=FX, ldx=64, d_in=64, dy=FX + 0x100000, lddy=128, d_out=128, gA=FX + 0x200000,
             gB=FX + 0x300000, n=3, flags=0, dx=FX + 0x400000, lddx=64, ws=FX + 0x500000, ws_bytes=BIG, seg=None)
    a.update(kw)
    seg = plan.dev() if a["seg"] is None else a["seg"]
    return B.load().lora_sgmv_backward(None, a["dtype"], a["x"], a["ldx"], a["d_in"], a["dy"], a["lddy"], a["d_out"], seg,
                                       a["gA"], a["gB"], a["n"], a["flags"], a["dx"], a["lddx"], a["ws"], a["ws_bytes"])


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), "LORA_ERR_DTYPE"),
    (dict(x=None), "LORA_ERR_ARG"),
    (dict(dy=None), "LORA_ERR_ARG"),
    (dict(d_in=0), "LORA_ERR_ARG"),
    (dict(d_out=-1), "LORA_ERR_ARG"),
    (dict(d_in=(1 << 24) + 1, ldx=1 << 25, lddx=1 << 25), "LORA_ERR_ARG"),
    (dict(d_out=(1 << 24) + 8, lddy=1 << 25), "LORA_ERR_ARG"),
    (dict(ldx=63), "LORA_ERR_ARG"),
    (dict(lddy=127), "LORA_ERR_ARG"),
    (dict(lddx=63), "LORA_ERR_ARG"),
    (dict(flags=2), "LORA_ERR_ARG"),
    (dict(n=-1), "LORA_ERR_ARG"),
    (dict(n=2), "LORA_ERR_ADAPTER_ID"),
    (dict(x=FX + 1), "LORA_ERR_ALIGN"),
    (dict(dy=FX + 1), "LORA_ERR_ALIGN"),
    (dict(dx=FX + 0x400001), "LORA_ERR_ALIGN"),
    (dict(dtype=B.LORA_F32, x=FX + 2), "LORA_ERR_ALIGN"),
    (dict(gA=FX + 4), "LORA_ERR_ALIGN"),
    (dict(dx=FX), "LORA_ERR_ARG"),
    (dict(dx=FX + 0x100000), "LORA_ERR_ARG"),
    (dict(ws=None), "LORA_ERR_WORKSPACE"),
    (dict(ws_bytes=16), "LORA_ERR_WORKSPACE"),
    (dict(ws=FX + 0x500008), "LORA_ERR_ALIGN"),
])
def test_refusals(kw, status):
    plan = plan_of([0, 2, 2, -1], 3, [16, 8, 4])
    st = run(plan, **kw)
    assert B.STATUS[st] == status, (kw, B.STATUS[st], B.last_error())
    assert B.last_error()


def run_fused(plan, **kw):
    a = dict(dtype=B.LORA_BF16, x=FX, ldx=64, d_in=64, W0=FX + 0x80000, dy=FX + 0x100000, lddy=128, d_out=128,
             gA=FX + 0x200000, gB=FX + 0x300000, n=3, flags=0, dx=FX + 0x400000, lddx=64, ws=FX + 0x500000, ws_bytes=BIG)
    a.update(kw)
    return B.load().lora_fused_linear_backward(None, a["dtype"], a["x"], a["ldx"], a["d_in"], a["W0"], a["dy"], a["lddy"],
                                               a["d_out"], plan.dev(), a["gA"], a["gB"], a["n"], a["flags"], a["dx"],
                                               a["lddx"], a["ws"], a["ws_bytes"])


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=B.LORA_F32), "LORA_ERR_DTYPE"),
    (dict(W0=None), "LORA_ERR_ARG"),
    (dict(dx=None), "LORA_ERR_ARG"),
    (dict(x=None), "LORA_ERR_ARG"),
    (dict(dy=None), "LORA_ERR_ARG"),
    (dict(lddy=127), "LORA_ERR_ARG"),
    (dict(lddy=132), "LORA_ERR_ALIGN"),
    (dict(ldx=68), "LORA_ERR_ALIGN"),
    (dict(lddx=68), "LORA_ERR_ALIGN"),
    (dict(x=FX + 8), "LORA_ERR_ALIGN"),
    (dict(dy=FX + 0x100008), "LORA_ERR_ALIGN"),
    (dict(dx=FX + 0x400008), "LORA_ERR_ALIGN"),
    (dict(W0=FX + 0x80008), "LORA_ERR_ALIGN"),
    (dict(d_in=60), "LORA_ERR_ALIGN"),
    (dict(d_out=1 << 30, lddy=1 << 30), "LORA_ERR_ARG"),
    (dict(n=2), "LORA_ERR_ADAPTER_ID"),
    (dict(flags=4), "LORA_ERR_ARG"),
    (dict(ws_bytes=1000), "LORA_ERR_WORKSPACE"),
    (dict(ws=FX + 0x500004), "LORA_ERR_ALIGN"),
])
def test_fused_refusals(kw, status):
    st = run_fused(plan_of([0, 2, 2, -1], 3, [16, 8, 4]), **kw)
    assert B.STATUS[st] == status, (kw, B.STATUS[st], B.last_error())


def test_fused_without_tokens_is_a_no_op():
    assert run_fused(plan_of([], 3, [16, 8, 4]), x=None, dy=None, dx=None, W0=None, ws=None, ws_bytes=0) == 0


def test_fused_workspace_grows_with_every_size():
    f = lambda T, i, o, r: B.lora_workspace_bytes(B.LORA_OP_FUSED_BACKWARD, T, i, o, r)  # noqa: E731
    sizes = [f(T, 256, 512, 16) for T in range(0, 70000, 37)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert f(400, 256, 512, 16) <= f(400, 256, 512, 17) <= f(400, 512, 512, 17) <= f(400, 512, 1024, 17)


def test_refusals_of_segments():
    plan = plan_of([0, 2], 3, [16, 8, 4])
    L = B.load()
    assert B.STATUS[L.lora_sgmv_backward(None, 1, FX, 64, 64, FX, 64, 64, None, FX, FX, 3, 0, FX, 64, FX, BIG)] == "LORA_ERR_ARG"
    assert B.STATUS[run(plan, seg=plan.seg)] == "LORA_ERR_ARG"  # a host struct: never uploaded
    assert B.STATUS[run(plan, seg=plan.dev(buf=0))] == "LORA_ERR_ARG"
    blank = HostPlan(4)
    d = plan.dev(host=blank.ptr)
    assert B.STATUS[run(plan, seg=d)] == "LORA_ERR_PLAN"


def test_no_adapted_rows_is_a_no_op():
    for ids in ([], [-1, -1]):
        assert run(plan_of(ids, 3, [16, 8, 4]), x=None, dy=None, ws=None, ws_bytes=0) == 0


def test_nothing_wanted_is_a_no_op():
    assert run(plan_of([0, 1], 3, [16, 8, 4]), x=None, gA=None, gB=None, dx=None) == 0


def test_workspace_grows_with_every_size():
    f = lambda T, i, o, r: B.lora_workspace_bytes(B.LORA_OP_SGMV_BACKWARD, T, i, o, r)  # noqa: E731
    sizes = [f(T, 256, 512, 16) for T in range(0, 70000, 37)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert f(4096, 256, 512, 16) <= f(4096, 256, 512, 17) <= f(4096, 512, 512, 17) <= f(4096, 512, 1024, 17)
    assert f(-1, 0, 0, 0) == f(0, 1, 1, 1)


def test_reference_against_differences():
    """The 64-bit reference's gradients are those of L = sum(dy y): y is linear in A, B and x each."""
    import torch

    from backward_ref import Problem

    p = Problem("f32", [0, 1, -1, 1, 0, 0], [3, 2], 5, 4, seed=1)
    p.dx_full.zero_()
    (dx, dA, dB), _ = p.reference()
    x = p.x.double().clone().requires_grad_()
    A = [t.double().clone().requires_grad_() for t in p.A]
    Bm = [t.double().clone().requires_grad_() for t in p.B]

    def loss():
        L = 0.0
        for t, i in enumerate(p.ids):
            if i >= 0:
                L = L + (p.dy.double()[t] * (p.scale[i] * (x[t] @ A[i].t()) @ Bm[i].t())).sum()
        return L

    for t, g in ((x, dx), *zip(A, dA), *zip(Bm, dB)):
        flat = t.data.view(-1)
        for k in range(flat.numel()):
            old = flat[k].item()
            flat[k] = old + 0.5
            up = loss().item()
            flat[k] = old - 0.5
            dn = loss().item()
            flat[k] = old
            assert abs((up - dn) - g.reshape(-1)[k]) <= 1e-12 * (1 + abs(g.reshape(-1)[k]))


def test_gradient_pool_checks():
    import torch

    with pytest.raises(ValueError):
        B.GradPool.from_tensors([torch.zeros(4)], [torch.zeros(4)])  # not on a device
    with pytest.raises(ValueError):
        B.GradPool.from_tensors([None], [])


class _Rows:
    """What the binding looks at of a matrix on a device that is not here."""

    def __init__(self, shape, device=0, dtype=None, inner=1):
        import torch

        self.shape, self.dtype, self._d, self._inner = shape, dtype or torch.bfloat16, device, inner

    get_device = lambda self: self._d  # noqa: E731
    stride = lambda self: (self.shape[1], self._inner)  # noqa: E731
    data_ptr = lambda self: FX  # noqa: E731
    is_contiguous = lambda self: True  # noqa: E731


class _Plan:
    dev = _Rows((1, 1))

    class h:
        batch_tokens = 4


class _PlanElsewhere(_Plan):
    dev = _Rows((1, 1), device=1)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("kw", [
    dict(x=_Rows((4, 64), device=1)), dict(dy=_Rows((4, 32), device=1)), dict(dx=_Rows((4, 64), device=-1)),
    dict(dy=_Rows((4, 32), device=-1)), dict(x=_Rows((3, 64))), dict(dx=_Rows((3, 64))), dict(dy=_Rows((3, 32))),
    dict(plan=_PlanElsewhere), dict(ws=_Rows((1, 1), device=-1)), dict(ws=_Rows((1, 1), device=1)),
    dict(grads=B.GradPool([], [], [], _Rows((1, 1), device=1), _Rows((1, 1)))),
    dict(dx=_Rows((4, 65))), dict(x=_Rows((4, 64, 1))), dict(x=_Rows((4, 64), inner=2)), dict(dtype="f32"),
])
def test_binding_refuses_what_the_call_cannot_see(fused, kw, monkeypatch):
    import torch

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    a = dict(x=_Rows((4, 64)), dy=_Rows((4, 32)), dx=_Rows((4, 64)), W0=_Rows((32, 64)), dtype="bf16", plan=_Plan, grads=None,
             ws=_Rows((1, 1)))
    a.update(kw)
    with pytest.raises(ValueError):
        if fused:
            B.fused_linear_backward(a["x"], a["W0"], a["dy"], a["plan"], a["grads"], a["dx"], a["ws"], a["dtype"])
        else:
            B.sgmv_backward(a["x"], a["dy"], a["plan"], a["grads"], a["dx"], a["ws"], a["dtype"])


def test_binding_refuses_other_weights_and_missing_x(monkeypatch):
    import torch

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, dy, ws = _Rows((4, 64)), _Rows((4, 32)), _Rows((1, 1))
    for W0 in (_Rows((31, 64)), _Rows((32, 72)), _Rows((32, 64), device=1), _Rows((32, 64), dtype=torch.float32)):
        with pytest.raises(ValueError):
            B.fused_linear_backward(x, W0, dy, _Plan, None, x, ws)
    with pytest.raises(ValueError, match="x is None"):
        B.sgmv_backward(None, dy, _Plan, B.GradPool([], [], [], x, x), None, None, "bf16")
    assert B.sgmv_backward(None, dy, _Plan, None, None, None, "bf16") is None  # nothing wanted


def test_header_and_binding_agree():
    assert B.LORA_OP_SGMV_BACKWARD == 7 and B.LORA_GRAD_ACCUMULATE == 1
    assert ctypes.sizeof(ctypes.c_uint) == 4


def _host_plan(ids, pool):
    """A Plan in plain host memory whose device buffer is a fake address (nothing is launched before a refusal)."""
    import torch

    p = B.Plan.__new__(B.Plan)
    p.capacity = max(len(ids), 1)
    p.nbytes = B.lora_segments_bytes(p.capacity)
    raw = torch.zeros(p.nbytes + 16, dtype=torch.uint8)
    off = -raw.data_ptr() % 16
    p.host, p.dev = raw[off: off + p.nbytes], _Rows((1, 1))
    p.h, p.d = B.LoraSegments(), B.LoraSegments()
    assert B.lora_segments_bind(p.host.data_ptr(), p.capacity, ctypes.addressof(p.h)) == 0
    return p.build(np.asarray(ids, dtype=np.int32), pool)


def _pool(ranks=(16, 8, 4), d_in=64, d_out=32, dtype="bf16", cls=B.DevicePool, **kw):
    A, Bt, r, al = make_tables(len(ranks), np.random.default_rng(0), list(ranks))
    return cls(n_adapters=len(ranks), dtype=dtype, d_in=d_in, d_out=d_out, addr_A=A, addr_B=Bt, rank=r, alpha=al,
               **(dict(storage=None) if cls is B.DevicePool else kw))


class _Grad:
    """What the binding looks at of a gradient tensor on a device that is not here."""

    def __init__(self, n, device=0):
        self._n, self._d, self.device = n, device, f"cuda:{device}"

    numel = lambda self: self._n  # noqa: E731
    get_device = lambda self: self._d  # noqa: E731


def _grads(nA, nB, device=0):
    one = lambda n: None if n is None else _Grad(n, device)  # noqa: E731
    return B.GradPool(None, [one(n) for n in nA], [one(n) for n in nB], _Rows((1, 1)), _Rows((1, 1)))


def _call(fused, plan, grads, d_in=64, d_out=32, dtype="bf16"):
    import torch

    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    x, dy, W0 = _Rows((4, d_in), dtype=dt), _Rows((4, d_out), dtype=dt), _Rows((d_out, d_in), dtype=dt)
    ws = _Rows((1, 1))
    ws.numel, ws.element_size = lambda: 1 << 40, lambda: 1
    if fused:
        B.fused_linear_backward(x, W0, dy, plan, grads, _Rows((4, d_in), dtype=dt), ws, dtype)
    else:
        B.sgmv_backward(x, dy, plan, grads, _Rows((4, d_in), dtype=dt), ws, dtype)


@pytest.fixture
def no_device(monkeypatch):
    """A current device 0, and a library that only notes that it was reached."""
    import torch

    reached = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(B, "_stream_handle", lambda *a: 0)
    lib = B.load()

    class L:
        lora_sgmv_backward = staticmethod(lambda *a: reached.append(a) or 0)
        lora_fused_linear_backward = staticmethod(lambda *a: reached.append(a) or 0)

        def __getattr__(self, k):
            return getattr(lib, k)

    monkeypatch.setattr(B, "load", lambda: L())
    return reached


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("kw", [
    dict(d_in=72), dict(d_in=56), dict(d_out=40), dict(d_out=24),  # other widths than the adapters': A or B past its end
    dict(nA=[16 * 64, 0, 4 * 64 - 1]), dict(nB=[16 * 32, 0, 4 * 32 - 1]), dict(nA=[16 * 64 - 1, 0, 4 * 64]),
    dict(nB=[8, None, None]), dict(nA=[None, None, 0]), dict(device=1), dict(pool_dtype="f32"),
])
def test_sizes_of_the_plans_adapters(fused, kw, no_device):
    """Widths, type and gradients are those of the adapters that the plan was built from."""
    pool = _pool(dtype=kw.get("pool_dtype", "bf16"))
    plan = _host_plan([0, 2, 2, -1], pool)
    nA, nB = kw.get("nA", [16 * 64, 0, 4 * 64]), kw.get("nB", [16 * 32, 0, 4 * 32])
    with pytest.raises(ValueError):
        _call(fused, plan, _grads(nA, nB, kw.get("device", 0)), kw.get("d_in", 64), kw.get("d_out", 32))
    if {"d_in", "d_out", "pool_dtype"} & set(kw):
        with pytest.raises(ValueError):
            _call(fused, plan, None, kw.get("d_in", 64), kw.get("d_out", 32))
    assert not no_device


@pytest.mark.parametrize("fused", [False, True])
def test_sizes_that_fit(fused, no_device):
    """Gradients left out, larger buffers, adapters without a row, plans without an adapted row of any width; a
    plan that is built again looks again."""
    pool = _pool()
    plan = _host_plan([0, 2, 2, -1], pool)
    good = [_grads([16 * 64, 0, 4 * 64], [16 * 32, 0, 4 * 32]), _grads([None, 1, 999], [999, 1, None]), None]
    for g in (*good, *good):
        _call(fused, plan, g)
    assert len(no_device) == 6
    _call(fused, _host_plan([-1, -1], pool), None, 128, 8)
    plan.build(np.array([1, 1, 1, 1], dtype=np.int32), pool)
    for g in good[:2]:
        with pytest.raises(ValueError):
            _call(fused, plan, g)
    assert len(no_device) == 7


@pytest.mark.parametrize("fused", [False, True])
def test_paged_adapters_are_refused(fused, no_device):
    """A PagedPool's addresses are page tables, not matrices; a plan built again from whole matrices is taken."""
    none = {k: None for k in ("pages", "tables", "table_host", "frames_A", "frames_B", "alloc")}
    paged = _pool(cls=B.PagedPool, page_bytes=4096, **none)
    plan = _host_plan([0, 2, 2, -1], paged)
    for grads in (None, B.GradPool(None, [None] * 3, [None] * 3, _Rows((1, 1)), _Rows((1, 1)))):
        with pytest.raises(ValueError, match="paged"):
            _call(fused, plan, grads)
    assert not no_device
    plan.build(np.array([0, 2], dtype=np.int32), _pool())
    _call(fused, plan, None)
    assert len(no_device) == 1


def test_more_workgroups_than_one_launch_has():
    """The runtime counts a launch's threads in 32 bits (2^24 - 1 workgroups of 256): refused before anything runs."""
    wide = dict(d_in=1 << 24, d_out=1 << 24, ldx=1 << 24, lddy=1 << 24, lddx=1 << 24, n=200)
    plan = plan_of(range(200), 200, [1] * 200)
    assert B.STATUS[run(plan, **wide)] == "LORA_ERR_ARG" and "work items" in B.last_error()
    tall = plan_of([-1] * 70000, 1, [1])  # 64-row tiles of 256 columns: 1094 x 2^16
    assert B.STATUS[run_fused(tall, **dict(wide, d_out=64, lddy=64))] == "LORA_ERR_ARG" and "tiles" in B.last_error()
