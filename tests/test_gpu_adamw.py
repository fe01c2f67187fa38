"""AdamW over many tensors (lora_adamw) on the GPU: fp32 and 8-bit states
against numpy, the rounding's bias, bad gradients, graphs, and the whole
training step of a pool of adapters."""

import numpy as np
import pytest
import torch

import adamw_ref as R
from gpu_helpers import require_gpu, say
from segmented_gather_gemm_lora_amd import binding as B

pytestmark = pytest.mark.gpu

HYPER = [dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0, step=1, seed=3),
         dict(lr=3e-4, beta1=0.8, beta2=0.95, eps=1e-6, weight_decay=0.0, grad_scale=0.3, step=1234, seed=-5),
         dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, grad_scale=1.0, step=0, seed=9)]  # rests


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    return require_gpu()


def table_of(hs):
    return B.adamw_hyper(len(hs), **{k: [h[k] for h in hs] for k in HYPER[0]})


class Case:
    """Tensors of the given sizes, each followed by a guard that must stay."""

    GUARD = 8

    def __init__(self, sizes, state, gdt=torch.float32, copy=True, hs=HYPER, seed=0, make_g=None):
        r = np.random.default_rng(seed)
        self.sizes, self.state, self.hs = sizes, state, hs
        self.groups = [i % len(hs) for i in range(len(sizes))]
        self.dev, self.host = [], []
        for n in sizes:
            nb = (n + 255) // 256
            size = np.exp(r.standard_normal((nb, 1)) * 2) * 1e-3
            p = (r.standard_normal(n) * 0.05).astype(np.float32)
            g = ((r.standard_normal((nb, 256)) * size).reshape(-1)[:n]).astype(np.float32) if make_g is None else make_g(n)
            v = ((size * np.exp(r.standard_normal((nb, 256)))).reshape(-1)[:n] ** 2).astype(np.float32)
            m = (r.standard_normal(n) * np.sqrt(v)).astype(np.float32)
            g = torch.from_numpy(g).to(gdt)
            h = {"p": p, "g": g.float().numpy()}
            d = {"p": self.dev_of(torch.from_numpy(p)), "g": self.dev_of(g)}
            if state == "8bit":
                for k, x in (("m", m), ("v", v)):
                    c, s = R.encode(x, r.integers(0, 65536, n), k)
                    h[k], h[k + "_scale"] = c, s
                    d[k], d[k + "_scale"] = self.dev_of(torch.from_numpy(c)), self.dev_of(torch.from_numpy(s))
            else:
                h["m"], h["v"] = m, v
                d["m"], d["v"] = self.dev_of(torch.from_numpy(m)), self.dev_of(torch.from_numpy(v))
            if copy:
                h["copy"] = torch.from_numpy(p).to(torch.bfloat16)
                d["copy"] = self.dev_of(h["copy"])
            self.host.append(h)
            self.dev.append(d)
        self.hyper = table_of(hs)
        col = lambda k: [d[k] for d in self.dev]  # noqa: E731
        more = dict(m_scale=col("m_scale"), v_scale=col("v_scale")) if state == "8bit" else {}
        self.opt = B.AdamW(col("p"), col("g"), self.groups, self.hyper, state=state, copies=col("copy") if copy else None,
                           m=col("m"), v=col("v"), **more)

    def dev_of(self, t):
        full = torch.full((t.numel() + self.GUARD,), 7, dtype=t.dtype, device="cuda")
        full[: t.numel()] = t.cuda()
        return full[: t.numel()]

    def guards(self):
        return all((d[k].as_strided((self.GUARD,), (1,), d[k].storage_offset() + d[k].numel()) == 7).all() for d in self.dev
                   for k in d)

    def check(self):
        for i, (d, h, grp) in enumerate(zip(self.dev, self.host, self.groups)):
            hy = self.hs[grp]
            got = {k: t.cpu() for k, t in d.items()}
            if hy["step"] < 1:
                for k in got:
                    assert torch.equal(got[k], torch.as_tensor(h[k])), (i, k)
                continue
            eight = self.state == "8bit"
            m0 = R.decode(h["m"], h["m_scale"], "m") if eight else h["m"]
            v0 = R.decode(h["v"], h["v_scale"], "v") if eight else h["v"]
            p, bound, m, v = R.step(h["p"], h["g"], m0, v0, hy)
            err = np.abs(got["p"].double().numpy() - p)
            assert (err <= bound).all(), (i, float((err / bound).max()))
            if "copy" in d:
                assert torch.equal(got["copy"], got["p"].to(torch.bfloat16))
            if eight:
                rnd = R.noise(hy["seed"], hy["step"], i, self.sizes[i])
                for k, x, r16 in (("m", m, rnd & 0xFFFF), ("v", v, rnd >> 16)):
                    c, s = R.encode(x, r16, k)
                    assert np.array_equal(got[k + "_scale"].numpy(), s), (i, k)
                    assert np.array_equal(got[k].numpy(), c), (i, k, int((got[k].numpy() != c).sum()))
            else:
                assert np.array_equal(got["m"].numpy(), m) and np.array_equal(got["v"].numpy(), v)
        assert self.guards()


@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("gdt,copy", [(torch.float32, True), (torch.float32, False), (torch.bfloat16, True)])
def test_against_numpy(state, gdt, copy):
    sizes = [1, 2, 3, 4, 5, 255, 256, 257, 1023, 1024, 1025, 4097, 0, 70001, 7, 513]
    say(f"case adamw {state} {gdt} copy={copy}")
    c = Case(sizes, state, gdt, copy)
    c.opt.step()
    torch.cuda.synchronize()
    c.check()


def test_many_elements():
    """Above 2^22 elements 8-bit chunks hold two rows of 1024: sizes around both."""
    sizes = [1, 1023, 1025, 2047, 2048, 2049, 3000, 1 << 20, (1 << 20) + 1, 300, (1 << 21) + 77, 5]
    assert sum(sizes) > 1 << 22
    c = Case(sizes, "8bit")
    c.opt.step()
    torch.cuda.synchronize()
    c.check()


def test_zero_state_and_zero_gradient():
    """From nothing: zeroed states, gradients that are zero in places."""
    for state in ("f32", "8bit"):
        g = np.where(np.arange(1000) % 3 == 0, 0, 1e-3 * np.arange(1000)).astype(np.float32)
        p = torch.zeros(1000, device="cuda")
        o = B.AdamW([p], [torch.from_numpy(g).cuda()], [0], table_of(HYPER[:1]), state=state)
        o.step()
        torch.cuda.synchronize()
        want, bound, *_ = R.step(np.zeros(1000), g, np.zeros(1000), np.zeros(1000), HYPER[0])
        assert (np.abs(p.double().cpu().numpy() - want) <= bound).all()
        assert (o.m[0].cpu().numpy()[g == 0] == 0).all() and (o.v[0].cpu().numpy()[g == 0] == 0).all()
        if state == "8bit":  # a positive v stays positive, whatever its block holds
            assert (o.v[0].cpu().numpy()[g != 0] > 0).all()


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e-3, 1e15])
def test_extreme_magnitudes(scale):
    """Gradients near both ends of fp32 (g g underflows or nears the top): the
    codes stay those of numpy's fp32 values."""
    r = np.random.default_rng(1)
    c = Case([1500], "8bit", hs=HYPER[:1], make_g=lambda n: (r.standard_normal(n) * scale).astype(np.float32))
    c.opt.step()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_tiny_gradients_without_eps(state):
    """eps = 0 and g g below fp32's normal range: the quotient m / sqrt(v) is still of order 1."""
    r = np.random.default_rng(4)
    h = dict(HYPER[0], eps=0.0, weight_decay=0.0)
    g = ((np.sign(r.standard_normal(600)) * (1 + r.random(600))) * 2e-18).astype(np.float32)
    p = torch.zeros(600, device="cuda")
    o = B.AdamW([p], [torch.from_numpy(g).cuda()], [0], table_of([h]), state=state)
    o.step()
    torch.cuda.synchronize()
    want, bound, _, v = R.step(np.zeros(600), g, np.zeros(600), np.zeros(600), h)
    assert (v < 2.0**-126).sum() > 300 and (v > 2.0**-133).all()  # most of them subnormal
    # v itself has as few as 2^-149 / v of relative accuracy here, on both sides alike
    assert (np.abs(p.double().cpu().numpy() - want) <= bound).all()


def test_rounding_has_no_bias():
    """The mean of many stochastic roundings of one value is the value: each is
    off by less than a code's gap, so the mean of N is off by at most
    5 gap / (2 sqrt N) (5 standard deviations, each at most half a gap)."""
    n, steps = 256 * 64, 16
    value = np.float32(0.0123)
    m0 = np.zeros(n, dtype=np.float32)
    hs = [dict(HYPER[0], seed=k, step=k + 1) for k in range(steps)]
    for which in ("m", "v"):
        total, seen = 0.0, 0
        for k in range(steps):
            g = torch.full((n,), float(value), device="cuda")
            g[0::256] = float(value) * 30  # the block's scale is not the value's own
            o = B.AdamW([torch.zeros(n, device="cuda")], [g], [0], table_of([hs[k]]), state="8bit")
            o.step()
            mo, vo = torch.empty(n, dtype=torch.bfloat16, device="cuda"), torch.empty(n, dtype=torch.bfloat16, device="cuda")
            B.adamw_state_values(o.m[0], o.m_scale[0], o.v[0], o.v_scale[0], mo, vo)
            out = (mo if which == "m" else vo).double().cpu().numpy()
            keep = np.arange(n) % 256 != 0
            total, seen = total + out[keep].sum(), seen + keep.sum()
            _, _, m, v = R.step(m0, np.full(n, value), m0, m0, hs[k])
        want = float((m if which == "m" else v)[1])
        gap = want / 8  # codes are at most 2^-3 apart
        assert abs(total / seen - want) <= 5 * gap / 2 / np.sqrt(seen), which
        assert len(np.unique(out[keep])) == 2  # the two neighbours


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_bad_gradients_stay_where_they_are(state):
    bad = {3: np.nan, 300: np.inf, 301: -np.inf, 999: np.nan}

    def make(n):
        g = np.random.default_rng(2).standard_normal(n).astype(np.float32)
        for k, x in bad.items():
            g[k] = x
        return g

    c = Case([1000], state, hs=HYPER[:1], make_g=make)
    c.opt.step()
    torch.cuda.synchronize()
    d = c.dev[0]
    at = np.isin(np.arange(1000), list(bad))
    assert np.array_equal(~np.isfinite(d["p"].cpu().numpy()), at)
    if state == "8bit":
        mo, vo = torch.empty(1000, dtype=torch.bfloat16, device="cuda"), torch.empty(1000, dtype=torch.bfloat16, device="cuda")
        B.adamw_state_values(d["m"], d["m_scale"], d["v"], d["v_scale"], mo, vo)
        assert np.array_equal(np.isnan(mo.float().cpu().numpy()), at) and np.array_equal(np.isnan(vo.float().cpu().numpy()), at)
        h = c.host[0]
        _, _, m, v = R.step(h["p"], h["g"], R.decode(h["m"], h["m_scale"], "m"), R.decode(h["v"], h["v_scale"], "v"), HYPER[0])
        rnd = R.noise(3, 1, 0, 1000)
        for k, x, r16 in (("m", m, rnd & 0xFFFF), ("v", v, rnd >> 16)):
            code, _ = R.encode(x, r16, k)
            assert np.array_equal(d[k].cpu().numpy()[~at], code[~at])


def test_values_of_every_code():
    """All 256 codes of both formats at several scales, against the tables."""
    codes = torch.arange(256, dtype=torch.uint8).repeat(5).cuda()
    scales = torch.tensor([1, 100, 127, 200, 230], dtype=torch.uint8).cuda()
    mo, vo = torch.empty(1280, dtype=torch.bfloat16, device="cuda"), torch.empty(1280, dtype=torch.bfloat16, device="cuda")
    B.adamw_state_values(codes, scales, codes, scales, mo, vo)
    for out, k in ((mo, "m"), (vo, "v")):
        want = R.decode(codes.cpu().numpy(), scales.cpu().numpy(), k)
        got = out.double().cpu().numpy()
        ok = (np.abs(want) >= 2.0**-126) | (want == 0) | np.isnan(want)  # bf16's normal range
        assert np.array_equal(got[ok], want[ok], equal_nan=True)
    one = torch.empty(1279, dtype=torch.bfloat16, device="cuda")
    B.adamw_state_values(None, None, codes[:1279], scales, None, one)
    assert torch.equal(one.view(torch.int16), vo[:1279].view(torch.int16))


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_captured_steps_follow_the_table(state):
    """A captured step, replayed with the step counted on the device, equals eager steps."""
    a, b = Case([5000, 300], state, hs=HYPER[:2]), Case([5000, 300], state, hs=HYPER[:2])
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        a.opt.step()
    for k in range(4):
        graph.replay()
        b.opt.step()
        torch.cuda.synchronize()
        for x, y in zip(a.dev, b.dev):
            for key in x:
                assert torch.equal(x[key], y[key]), (k, key)
        for c in (a, b):
            c.hyper[:, 6] += 1
        for x, y in zip(a.dev, b.dev):
            y["g"].normal_()
            x["g"].copy_(y["g"])


def test_training_step_of_a_pool():
    """Forward, backward and step of a bf16 pool of adapters, as they are used
    together: the masters follow the gradients, the forward reads the copies."""
    from backward_ref import Problem, check

    p = Problem("bf16", np.arange(90) % 3, [8, 16, 4], 128, 96, seed=12)
    d = p.device()
    mats = [t for i in range(3) for t in (p.A[i], p.B[i])]
    es = 2
    views = [d.storage[(int(a) - d.storage.data_ptr()) // es:][: t.numel()]
             for t, a in zip(mats, [x for i in range(3) for x in (d.pool.addr_A[i], d.pool.addr_B[i])])]
    masters = [t.float().cuda().reshape(-1) for t in mats]
    grads = [t for i in range(3) for t in (d.grads.A[i], d.grads.B[i])]
    hs = [dict(HYPER[0], lr=1e-2), dict(HYPER[1], lr=1e-2, step=1, grad_scale=1.0), HYPER[2]]
    opt = B.AdamW(masters, grads, [0, 0, 1, 1, 2, 2], table_of(hs), state="8bit", copies=views)
    ws = B.workspace(B.LORA_OP_SGMV, p.T, p.d_in, p.d_out, 16)
    before = [t.clone() for t in views]
    B.sgmv_backward(d.x, d.dy, d.plan, d.grads, d.dx, d.ws, "bf16")
    check(p, d)
    opt.step()
    y = torch.zeros(p.T, p.d_out, dtype=torch.bfloat16, device="cuda")
    B.sgmv(d.x, d.plan, y, ws, "bf16")
    torch.cuda.synchronize()
    for i, (t, b, mst) in enumerate(zip(views, before, masters)):
        assert torch.equal(t, mst.to(torch.bfloat16))
        assert torch.equal(t, b) == (i >= 4)  # the third adapter rests
    x = d.x.double().cpu()
    for i in range(3):
        A, Bm = views[2 * i].double().cpu().view(p.A[i].shape), views[2 * i + 1].double().cpu().view(p.B[i].shape)
        rows = np.nonzero(p.ids == i)[0]
        want = p.scale[i] * (x[rows] @ A.t()) @ Bm.t()
        err = (y[rows].double().cpu() - want).abs()
        assert (err <= 2e-2 * (want.abs() + 1e-2)).all()


@pytest.mark.parametrize("where", ["side", "current", "side twice"])
@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_built_on_one_stream_stepped_on_another(state, where):
    """Built while its stream is busy, stepped at once on another: the plan and the zeroed states are there."""
    g = [torch.randn(n, device="cuda") for n in (5000, 700)]
    table = table_of(HYPER[:1])
    want = [torch.ones_like(t) for t in g]
    ref = B.AdamW(want, g, [0, 0], table, state=state)
    ref.step()
    p = [torch.ones_like(t) for t in g]
    junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in (5000, 20000, 20000, 5000, 700, 700)]
    torch.cuda.synchronize()
    del junk  # what the states and the plan are made in
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    busy, step = {"side": (a, None), "current": (torch.cuda.current_stream(), b), "side twice": (a, b)}[where]
    with torch.cuda.stream(busy):
        torch.cuda._sleep(20_000_000)
    o = B.AdamW(p, g, [0, 0], table, state=state, stream=None if where == "current" else a)
    o.step(stream=step)
    torch.cuda.synchronize()
    for t, w in zip((*p, *o.m, *o.v), (*want, *ref.m, *ref.v)):
        assert torch.equal(t, w)


def test_building_in_a_captured_region_is_refused():
    p, g = torch.zeros(64, device="cuda"), torch.ones(64, device="cuda")
    table = table_of(HYPER[:1])
    opt = B.AdamW([p], [g], [0], table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        with pytest.raises(ValueError, match="captured"):
            B.AdamW([p], [g], [0], table)
        opt.step()
    q = torch.zeros(64, device="cuda")
    eager = B.AdamW([q], [g], [0], table)
    for k in range(3):
        graph.replay()
        eager.step()
        torch.cuda.synchronize()
        assert torch.equal(p, q), k


@pytest.mark.parametrize("eps", [0.0, 1e-20])
@pytest.mark.parametrize("step", [1, 5000])
@pytest.mark.parametrize("state,size", [("f32", 1e-20), ("f32", 2e-19), ("8bit", 1e-20), ("8bit", 2e-18)])
def test_subnormal_second_moments(state, size, step, eps):
    """v / (1 - b2^t) below fp32's normal range is not taken as 0: the root keeps what v has."""
    r = np.random.default_rng(5)
    h = dict(HYPER[0], eps=eps, weight_decay=0.0, step=step)
    g = (np.sign(r.standard_normal(600)) * (1 + r.random(600)) * size).astype(np.float32)
    m0, v0 = (g, (g.astype(np.float64) ** 2).astype(np.float32)) if state == "f32" else (np.zeros_like(g),) * 2
    p = torch.zeros(600, device="cuda")
    more = {} if state == "8bit" else {k: [torch.from_numpy(x.copy()).cuda()] for k, x in (("m", m0), ("v", v0))}
    o = B.AdamW([p], [torch.from_numpy(g).cuda()], [0], table_of([h]), state=state, **more)
    o.step()
    torch.cuda.synchronize()
    want, bound, _, v = R.step(np.zeros(600), g, m0, v0, h)
    # the quotient v / bc2 is rounded to a multiple of 2^-149 (half of one off, at most), and its root
    # moves by half as much, relative to it
    vhat = v.astype(np.float64) / (1 - float(np.float32(h["beta2"])) ** step)
    bound = bound + np.abs(want) * 2.0**-150 / vhat
    assert (v > 0).all() and (np.abs(p.double().cpu().numpy() - want) <= bound).all()


def test_many_elements_of_bf16_gradients():
    """Two rows a chunk, bf16 gradients."""
    c = Case([1, 1025, 2047, 2049, (1 << 20) + 3, 300, (1 << 20) + 1029, 5], "8bit", torch.bfloat16)
    assert sum(c.sizes) > 1 << 21
    c.opt.step()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_states_of_bad_and_huge_gradients(state):
    """m and v of gradients that are not finite, and of finite ones whose square is not."""
    bad = {3: np.nan, 300: np.inf, 301: -np.inf, 500: 1.9e19, 501: -3e38, 700: 1.8e19}

    def make(n):
        g = np.random.default_rng(2).standard_normal(n).astype(np.float32)
        for k, x in bad.items():
            g[k] = x
        return g

    h = dict(HYPER[0], step=3)
    c = Case([1000], state, hs=[h], make_g=make)
    before = c.host[0]["p"].copy()
    c.opt.step()
    torch.cuda.synchronize()
    d = c.dev[0]
    p = d["p"].cpu().numpy()
    if state == "f32":
        m, v = d["m"].cpu().numpy(), d["v"].cpu().numpy()
        h0 = c.host[0]
        _, _, wm, wv = R.step(before, h0["g"], h0["m"], h0["v"], h)
        assert np.array_equal(m, wm, equal_nan=True) and np.array_equal(v, wv, equal_nan=True)
        assert np.isnan(m[3]) and m[300] == np.inf and m[301] == -np.inf and np.isfinite(m[[500, 501, 700]]).all()
        assert np.isnan(v[3]) and (v[[300, 301, 500, 501]] == np.inf).all() and np.isfinite(v[700])
    else:
        mo, vo = torch.empty(1000, dtype=torch.bfloat16, device="cuda"), torch.empty(1000, dtype=torch.bfloat16, device="cuda")
        B.adamw_state_values(d["m"], d["m_scale"], d["v"], d["v_scale"], mo, vo)
        m, v = mo.float().cpu().numpy(), vo.float().cpu().numpy()
        assert np.array_equal(np.isnan(m), np.isin(np.arange(1000), [3, 300, 301]))
        assert np.array_equal(np.isnan(v), np.isin(np.arange(1000), [3, 300, 301, 500, 501]))
    assert np.array_equal(np.isnan(p), np.isin(np.arange(1000), [3, 300, 301])) and np.isfinite(p[[500, 501, 700]]).all()
    decay = 1 - float(np.float32(h["lr"])) * float(np.float32(h["weight_decay"]))
    # m / infinity is 0: the element only decays (24 steps of the decay, half a step of p)
    want = before[[500, 501]].astype(np.float64) * decay
    assert (np.abs(p[[500, 501]] - want) <= 2.0**-24 * np.abs(want) + 24 * 2.0**-23 * (1 - decay) * np.abs(want)).all()
    # the next step, with gradients of order 1
    d["g"].normal_()
    c.hyper[:, 6] += 1
    c.opt.step()
    torch.cuda.synchronize()
    lost = [3, 300, 301] if state == "f32" else [3, 300, 301, 500, 501]
    assert np.array_equal(np.isnan(d["p"].cpu().numpy()), np.isin(np.arange(1000), lost))


def test_huge_gradients_by_the_formula():
    """The same in 64 bits: with g g finite in fp32 nothing is lost."""
    g = np.array([1.8e19, -1.8e19, 1e19, 3.0], dtype=np.float32)
    p = torch.ones(4, device="cuda")
    o = B.AdamW([p], [torch.from_numpy(g).cuda()], [0], table_of(HYPER[:1]))
    o.step()
    torch.cuda.synchronize()
    want, bound, *_ = R.step(np.ones(4), g, np.zeros(4), np.zeros(4), HYPER[0])
    assert (np.abs(p.double().cpu().numpy() - want) <= bound).all()


def test_the_tensors_live_as_long_as_the_optimizer():
    """The plan holds addresses: emptying the lists that were given frees nothing."""
    import weakref

    p = [torch.zeros(300, device="cuda")]
    copies, m, v, ms, vs = ([torch.zeros(n, dtype=dt, device="cuda")] for n, dt in (
        (300, torch.bfloat16), (300, torch.uint8), (300, torch.uint8), (2, torch.uint8), (2, torch.uint8)))
    g = [torch.ones(300, device="cuda")]
    lists = (p, g, copies, m, v, ms, vs)
    refs = [weakref.ref(t[0]) for t in lists]
    o = B.AdamW(p, g, [0], table_of(HYPER[:1]), state="8bit", copies=copies, m=m, v=v, m_scale=ms, v_scale=vs)
    for t in lists:
        t.clear()
    assert all(r() is not None for r in refs)
    o.step()
    torch.cuda.synchronize()
    assert torch.equal(o.copies[0], o.params[0].to(torch.bfloat16)) and (o.params[0] < 0).all()
