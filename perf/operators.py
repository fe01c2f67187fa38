"""What is measured of the adapter training operators: the gradients of the
segmented correction and of the fused layer, and the optimizer step over a pool
of adapters.

A case is run in one of two forms.  The plain form (own = False) computes the
operator with elementary torch operations in fp32.  The other calls the
library's kernels.  Both take the state that prepare() makes.

The operators (x [T, d_in], dy [T, d_out], adapter i = ids[t] with A_i
[r_i, d_in], B_i [d_out, r_i], s_i = alpha_i / r_i, -1 = no adapter):

  sgmv    u = s_i dy[t] B_i,  v = x[t] A_i^T;  dx[t] += u A_i,
          dA_i = sum_t u^T x[t],  dB_i = s_i sum_t dy[t]^T v
  fused   the same gradients, and dx[t] = dy[t] W0 + u A_i
  adamw   g = c grad;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g g;
          p -= lr (wd p + (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)),
          m and v held in fp32, or in 8 bits with a power-of-two scale for
          each 256 elements and stochastic rounding from a stated hash
"""

import math

import numpy as np
import torch

own = False

BLOCK = 256  # elements of an optimizer state block (one scale each)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one small request group on a narrow layer, all in fp32: the call's latency
        _sgmv("grad tiny fp32", "f32", 8, 256, 256, 2, "8", "runs"),
        # one row for each of 64 requests over 32 adapters: many segments of a token or two
        _sgmv("grad rows of 32 adapters", "bf16", 64, 4096, 4096, 32, "16", "random"),
        # a training batch of 4096 tokens over 16 adapters
        _sgmv("grad 4096 tokens", "bf16", 4096, 4096, 4096, 16, "16", "runs"),
        # single rows beside long sequences, ranks 8 to 64, a wide MLP projection
        _sgmv("grad mixed ranks", "bf16", 2304, 4096, 14336, 128, "8,16,32,64", "zipf"),
        # nothing aligned: odd widths, odd ranks, tokens without an adapter
        _sgmv("grad odd sizes", "bf16", 517, 1001, 1531, 9, "1,3,17,33,100", "random", none=0.2),
        # long sequences of few adapters of a high rank
        _sgmv("grad 16384 tokens rank 64", "bf16", 16384, 4096, 4096, 4, "64", "runs"),
        # the fused layer under a small batch: the base weight is most of what is read
        _fused("fused grad 64 tokens", 64, 4096, 4096, 32, "16", "random"),
        # the fused layer over many requests, some tokens without an adapter
        _fused("fused grad 1024 tokens", 1024, 4096, 12288, 200, "16", "runs", none=0.05),
        # one adapter of one projection: the step's latency
        _adamw("adamw one adapter", "f32", 1, "16", 4096, 4096, copy=False),
        # every adapter of a pool of rank 16, with the bf16 copies that the forward reads
        _adamw("adamw 128 adapters", "f32", 128, "16", 4096, 4096),
        # 8-bit states, odd sizes, adapters that rest this step
        _adamw("adamw 8-bit odd sizes", "8bit", 37, "1,7,16,33", 1001, 1531, idle=0.2),
        # 8-bit states over a large pool
        _adamw("adamw 8-bit 512 adapters", "8bit", 512, "16,32", 4096, 4096),
    ]


def _sgmv(name, dtype, T, d_in, d_out, adapters, ranks, layout, none=0.0):
    return {"name": name, "op": "sgmv", "dtype": dtype, "T": T, "d_in": d_in, "d_out": d_out, "adapters": adapters,
            "ranks": ranks, "layout": layout, "none": none}


def _fused(name, T, d_in, d_out, adapters, ranks, layout, none=0.0):
    return {"name": name, "op": "fused", "dtype": "bf16", "T": T, "d_in": d_in, "d_out": d_out, "adapters": adapters,
            "ranks": ranks, "layout": layout, "none": none}


def _adamw(name, state, adapters, ranks, d_in, d_out, copy=True, idle=0.0):
    return {"name": name, "op": "adamw", "state": state, "adapters": adapters, "ranks": ranks, "d_in": d_in,
            "d_out": d_out, "copy": copy, "idle": idle}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sgmv", "sgmv", "fused", "adamw"])
    ranks = rng.choice(["4", "8", "16", "32", "64", "8,16,32,64", "1,3,17,33", "5,24,100", "128", "256"])
    if op == "adamw":
        case = _adamw("", rng.choice(["f32", "8bit"]), _log(rng, 1, 256), ranks, _log(rng, 64, 8192),
                      _log(rng, 64, 14336), copy=rng.random() < 0.7, idle=rng.choice([0.0, 0.0, 0.3]))
        most = max(int(r) for r in ranks.split(","))
        while case["adapters"] * most * (case["d_in"] + case["d_out"]) > 50_000_000:
            case["adapters"] = max(1, case["adapters"] // 2)
            if case["adapters"] == 1:
                break
    else:
        d_in, d_out = _log(rng, 64, 8192), _log(rng, 64, 14336)
        if op == "fused" or rng.random() < 0.6:  # widths of a model, most of the time
            d_in, d_out = max(64, d_in // 64 * 64), max(64, d_out // 64 * 64)
        layout, none = rng.choice(["runs", "random", "zipf"]), rng.choice([0.0, 0.0, 0.1, 0.5])
        T, n = _log(rng, 1, 8192), _log(rng, 1, 64)
        if op == "fused":
            case = _fused("", T, d_in, d_out, n, ranks, layout, none)
        else:
            case = _sgmv("", rng.choice(["bf16", "bf16", "bf16", "f32"]), T, d_in, d_out, n, ranks, layout, none)
        most = max(int(r) for r in ranks.split(","))
        while case["adapters"] > 1 and T * case["adapters"] * most * (d_in + d_out) > 16384 * 256 * 8192:
            case["adapters"] = max(1, case["adapters"] // 2)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
def _structure(case, seed):
    """ids [T], from the seed, and ranks [adapters], which are the case's (the outputs' sizes go by them)."""
    n = case["adapters"]
    ranks = np.random.default_rng(n).choice(np.array([int(q) for q in case["ranks"].split(",")], dtype=np.int32), size=n)
    r = np.random.default_rng(seed)
    if case["op"] == "adamw":
        return None, ranks
    T = case["T"]
    if case["layout"] == "runs":  # each adapter's tokens in a row, Dirichlet(1) lengths
        cut = np.floor(np.cumsum(r.dirichlet(np.ones(n))) * T).astype(np.int64)
        cut[-1] = T
        ids = np.repeat(r.permutation(n), np.diff(cut, prepend=0))
    elif case["layout"] == "zipf":  # an eighth are single rows, the rest four long sequences
        p = 1.0 / np.arange(1, n + 1) ** 1.1
        p /= p.sum()
        head = T - T // 9 * 8
        ids = np.concatenate([r.choice(n, head, p=p), np.repeat(r.choice(n, 4, p=p), (T - head + 3) // 4)])[:T]
    else:
        ids = r.integers(0, n, T)
    ids = ids.astype(np.int32)
    if case["none"] > 0:
        ids[r.random(T) < case["none"]] = -1
        if (ids < 0).all():
            ids[0] = 0
    return ids, ranks


def _randn(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_adamw(case, seed, gen) if case["op"] == "adamw" else _prepare_grad(case, seed, gen)


def _prepare_grad(case, seed, gen):
    ids, ranks = _structure(case, seed)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    T, d_in, d_out, n = case["T"], case["d_in"], case["d_out"], case["adapters"]
    # every A_i, then every B_i, in one pool; each matrix starts at a multiple of 128 elements
    sizes = [int(r) * d_in for r in ranks] + [int(r) * d_out for r in ranks]
    starts = np.concatenate([[0], np.cumsum([(s + 127) // 128 * 128 for s in sizes])]).astype(np.int64)
    pool = _randn(gen, (int(starts[-1]),), 0.02, dt)
    A = [pool[o : o + s].view(int(r), d_in) for o, s, r in zip(starts[:n], sizes[:n], ranks)]
    Bm = [pool[o : o + s].view(d_out, int(r)) for o, s, r in zip(starts[n:-1], sizes[n:], ranks)]
    total = int(ranks.sum())
    s = {
        "case": case, "pool": pool, "A": A, "B": Bm, "ranks": [int(r) for r in ranks],
        "scale": [32.0 / int(r) for r in ranks],
        "x": _randn(gen, (T, d_in), 1.0, dt), "dy": _randn(gen, (T, d_out), 1.0, dt),
        "dx": _randn(gen, (T, d_in), 1.0, dt),
        "gA": torch.zeros(total * d_in, device="cuda"), "gB": torch.zeros(total * d_out, device="cuda"),
        "ids": torch.from_numpy(ids).cuda(),
        # the adapter and the scale of every column of the stacked adapters
        "column": torch.from_numpy(np.repeat(np.arange(n, dtype=np.int32), ranks)).cuda(),
        "column_scale": torch.from_numpy(np.repeat((np.float32(32.0) / ranks.astype(np.float32)), ranks)).cuda(),
    }
    if case["op"] == "fused":
        s["W0"] = _randn(gen, (d_out, d_in), 0.02, dt)
    if own:
        from segmented_gather_gemm_lora_amd import binding as L

        base, es = pool.data_ptr(), pool.element_size()
        dp = L.DevicePool(storage=pool, n_adapters=n, dtype=case["dtype"], d_in=d_in, d_out=d_out,
                          addr_A=(base + starts[:n] * es).astype(np.uint64),
                          addr_B=(base + starts[n:-1] * es).astype(np.uint64),
                          rank=ranks.astype(np.int32), alpha=np.full(n, 32.0, dtype=np.float32))
        s["plan"] = L.Plan(T).build(ids, dp).upload()
        s["grads"] = L.GradPool.from_tensors(_rows(s["gA"], ranks, d_in), _rows(s["gB"], ranks, d_out))
        op = L.LORA_OP_FUSED_BACKWARD if case["op"] == "fused" else L.LORA_OP_SGMV_BACKWARD
        s["ws"] = L.workspace(op, T, d_in, d_out, int(ranks.max()))
    return s


def _rows(flat, ranks, d):
    """Each adapter's part of a flat gradient buffer."""
    return list(flat.split([int(r) * d for r in ranks]))


def _prepare_adamw(case, seed, gen):
    ids, ranks = _structure(case, seed)
    n = case["adapters"]
    sizes = np.concatenate([[int(r) * case["d_in"], int(r) * case["d_out"]] for r in ranks]).astype(np.int64)
    blocks = (sizes + BLOCK - 1) // BLOCK
    starts = np.concatenate([[0], np.cumsum(blocks)]) * BLOCK
    total = int(starts[-1])
    # the tensor of every block of 256 elements, and the block's place in it
    tensor = torch.from_numpy(np.repeat(np.arange(len(sizes)), blocks)).cuda()
    place = torch.from_numpy(np.arange(total // BLOCK) - np.repeat(starts[:-1] // BLOCK, blocks)).cuda()
    inside = (place[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")) < torch.from_numpy(sizes).cuda()[tensor][:, None]
    keep = inside.reshape(-1).float()
    host = np.random.default_rng(seed + 1)
    hyper = {
        "lr": torch.from_numpy(host.choice([1e-4, 2e-4, 1e-3], n).astype(np.float32)).cuda(),
        "beta1": torch.full((n,), 0.9, device="cuda"), "beta2": torch.full((n,), 0.999, device="cuda"),
        "eps": torch.full((n,), 1e-8, device="cuda"), "weight_decay": torch.full((n,), 0.01, device="cuda"),
        "grad_scale": torch.from_numpy(host.choice([1.0, 0.5, 0.3], n).astype(np.float32)).cuda(),
        "step": torch.from_numpy(np.where(host.random(n) < case["idle"], 0, host.integers(1, 2000, n)).astype(np.int32)).cuda(),
        "seed": torch.from_numpy(host.integers(0, 2**31, n).astype(np.int32)).cuda(),
    }
    size = torch.exp(torch.randn(total // BLOCK, 1, generator=gen, device="cuda")) * 1e-3
    g = (torch.randn(total // BLOCK, BLOCK, generator=gen, device="cuda") * size).reshape(-1) * keep
    v = (size * torch.exp(torch.randn(total // BLOCK, BLOCK, generator=gen, device="cuda") * 0.5)).reshape(-1).square() * keep
    m = torch.randn(total, generator=gen, device="cuda") * v.sqrt() * 0.3
    s = {"case": case, "hyper": hyper, "group": tensor // 2, "tensor": tensor, "place": place,
         "p": _randn(gen, (total,), 0.02, torch.float32) * keep, "g": g}
    if case["copy"]:
        s["copy"] = s["p"].to(torch.bfloat16)
    if case["state"] == "f32":
        s["m"], s["v"] = m, v
    else:
        zero = torch.zeros((), device="cuda", dtype=torch.int64)
        s["m"], s["m_scale"] = _encode(m.view(-1, BLOCK), 7, 8, zero, signed=True)
        s["v"], s["v_scale"] = _encode(v.view(-1, BLOCK), 15, 16, zero, signed=False)
    if own:
        from segmented_gather_gemm_lora_amd import binding as L

        # the buffers hold whole blocks of 256, and the plain form steps all of them: so do the tensors given here
        cut = lambda t: [t.view(-1)[int(a) : int(a) + int(k) * BLOCK] for a, k in zip(starts[:-1], blocks)]  # noqa: E731
        per = lambda t: [t[int(a) // BLOCK : int(a) // BLOCK + int(k)] for a, k in zip(starts[:-1], blocks)]  # noqa: E731
        more = {"m_scale": per(s["m_scale"]), "v_scale": per(s["v_scale"])} if case["state"] == "8bit" else {}
        s["opt"] = L.AdamW(cut(s["p"]), cut(s["g"]), groups=[i // 2 for i in range(len(sizes))],
                           hyper=L.adamw_hyper(n, **hyper), state=case["state"],
                           copies=cut(s["copy"]) if case["copy"] else None, m=cut(s["m"]), v=cut(s["v"]), **more)
        if case["state"] == "8bit":
            s["m_value"] = torch.empty(total, dtype=torch.bfloat16, device="cuda")
            s["v_value"] = torch.empty(total, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if s["case"]["op"] == "adamw":
        return _run_adamw(s)
    if own:
        from segmented_gather_gemm_lora_amd import binding as L

        if s["case"]["op"] == "fused":
            L.fused_linear_backward(s["x"], s["W0"], s["dy"], s["plan"], s["grads"], s["dx"], s["ws"])
        else:
            L.sgmv_backward(s["x"], s["dy"], s["plan"], s["grads"], s["dx"], s["ws"], s["case"]["dtype"])
        return {"dx": s["dx"], "dA": s["gA"], "dB": s["gB"]}
    # all adapters stacked [R, d_in] and [d_out, R]; a token keeps the columns of its own adapter
    x, dy = s["x"].float(), s["dy"].float()
    A, Bm = torch.cat(s["A"], 0).float(), torch.cat(s["B"], 1).float()
    mine = (s["ids"][:, None] == s["column"][None, :]) * s["column_scale"]
    u = (dy @ Bm) * mine
    v = (x @ A.t()) * mine
    dA = u.t() @ x
    dB = dy.t() @ v
    dx = u @ A
    dx += dy @ s["W0"].float() if s["case"]["op"] == "fused" else s["dx"].float()
    s["dx"].copy_(dx)
    return {"dx": s["dx"], "dA": dA.reshape(-1), "dB": torch.cat([t.reshape(-1) for t in dB.split(s["ranks"], 1)])}


def _run_adamw(s):
    names = ("p", "copy") if s["case"]["copy"] else ("p",)
    if own:
        from segmented_gather_gemm_lora_amd import binding as L

        s["opt"].step()
        if s["case"]["state"] == "f32":
            return {k: s[k] for k in names + ("m", "v")}
        L.adamw_state_values(s["m"], s["m_scale"], s["v"], s["v_scale"], s["m_value"], s["v_value"])
        return {**{k: s[k] for k in names}, "m": s["m_value"], "v": s["v_value"]}
    eight = s["case"]["state"] == "8bit"
    h = {k: t[s["group"]][:, None] for k, t in s["hyper"].items()}
    live = h["step"] >= 1
    t = h["step"].clamp(min=1).double()
    bc1 = (1.0 - h["beta1"].double() ** t).float()
    bc2 = (1.0 - h["beta2"].double() ** t).float()
    p, g = s["p"].view(-1, BLOCK), s["g"].view(-1, BLOCK) * h["grad_scale"]
    m0 = _decode(s["m"], s["m_scale"], 7, signed=True) if eight else s["m"].view(-1, BLOCK)
    v0 = _decode(s["v"], s["v_scale"], 15, signed=False) if eight else s["v"].view(-1, BLOCK)
    m = h["beta1"] * m0 + (1.0 - h["beta1"]) * g
    v = h["beta2"] * v0 + (1.0 - h["beta2"]) * (g * g)
    new = p - h["lr"] * (h["weight_decay"] * p + (m / bc1) / ((v / bc2).sqrt() + h["eps"]))
    p.copy_(torch.where(live, new, p))
    out = {"p": s["p"]}
    if s["case"]["copy"]:
        s["copy"].copy_(torch.where(live, p, s["copy"].view(-1, BLOCK).float()).reshape(-1))
        out["copy"] = s["copy"]
    if not eight:
        s["m"].view(-1, BLOCK).copy_(torch.where(live, m, m0))
        s["v"].view(-1, BLOCK).copy_(torch.where(live, v, v0))
        return {**out, "m": s["m"], "v": s["v"]}
    h32 = _hash(s["hyper"], s["group"], s["tensor"], s["place"])
    mc, ms = _encode(m, 7, 8, h32 & 0xFFFF, signed=True)
    vc, vs = _encode(v, 15, 16, h32 >> 16, signed=False)
    for k, code, scale in (("m", mc, ms), ("v", vc, vs)):
        s[k].copy_(torch.where(live, code, s[k]))
        s[k + "_scale"].copy_(torch.where(live[:, 0], scale, s[k + "_scale"]))
    return {**out, "m": _decode(s["m"], s["m_scale"], 7, signed=True).to(torch.bfloat16).reshape(-1),
            "v": _decode(s["v"], s["v_scale"], 15, signed=False).to(torch.bfloat16).reshape(-1)}


# The 8-bit states.  A block of 256 elements has a scale 2^(e - 127), e in one byte, and a code for each
# element: m in OCP E4M3 (sign, 4 exponent bits of bias 7, 3 mantissa bits), v, which is never negative, in 5
# exponent bits of bias 15 and 3 mantissa bits.  e is the least for which the block's largest value is below
# 1.75 * 2^8 (m) or 1.75 * 2^16 (v) times the scale.  A value between two codes goes up with a
# probability that is its distance from the lower one, to 16 bits: `noise` / 2^16 is added to it in steps of the
# code before it is cut off.  A positive v never becomes 0.
def _encode(x, bias, top, noise, signed):
    a = x.double().abs()
    most = a.amax(1)
    mant, expo = torch.frexp(most)  # most = mant 2^expo, mant in [0.5, 1)
    e = (expo - 1 + (mant >= 0.875) - top + 127).clamp(1, 254)
    e = torch.where(most > 0, e, torch.ones_like(e))
    y = torch.ldexp(a, (127 - e)[:, None].double())
    # the binade's step is 2^(exponent - 3); below the least normal, 2^(1 - bias), the steps stay those of that binade
    ye = (torch.frexp(y)[1] - 1).clamp(min=1 - bias)
    step = torch.exp2((ye - 3).double())
    k = torch.floor(y / step + noise.double() / 65536.0)  # 8 .. 16 in a normal binade, 0 .. 8 below
    code = ((ye + bias - 1) * 8 + k.to(torch.int32)).clamp(max=(126 if signed else 254))
    code = torch.where((a > 0) & (code == 0), torch.ones_like(code), code) if not signed else code
    code = code + 128 * (x < 0) if signed else code
    return code.to(torch.uint8), e.to(torch.uint8)


def _decode(code, scale, bias, signed):
    c = code.to(torch.int32)
    mag = c & 127 if signed else c
    e, f = mag >> 3, (mag & 7).float()
    y = torch.ldexp(torch.where(e > 0, f + 8.0, f), e.clamp(min=1) - bias - 3)
    y = torch.ldexp(y, scale.to(torch.int32)[:, None] - 127)
    return torch.where(c >= 128, -y, y) if signed else y


def _mix(h):
    h = h ^ (h >> 16)
    h = (h * 0x6A09E667) & 0xFFFFFFFF
    h = h ^ (h >> 15)
    h = (h * 0xBB67AE85) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _hash(hyper, group, tensor, place):
    """The 32 random bits of every element: a hash of the group's seed and step, the tensor and the element."""
    key = _mix(((hyper["seed"].long() & 0xFFFFFFFF) + hyper["step"].long() * 0x9E3779B9) & 0xFFFFFFFF)
    key = _mix((key[group] + tensor * 0x510E527F) & 0xFFFFFFFF)
    at = place[:, None] * BLOCK + torch.arange(BLOCK, device=place.device)
    return _mix((at * 0x9E3779B9 + key[:, None]) & 0xFFFFFFFF)


# ------------------------------------------------------------------ sizes
def work(case):
    """Each input read once and each output written once, on the structure that seed 0 gives."""
    ids, ranks = _structure(case, 0)
    if case["op"] == "adamw":
        n = int(ranks.sum()) * (case["d_in"] + case["d_out"])
        state = 16 if case["state"] == "f32" else 4 + 4  # m and v read and written, and the values they stand for
        return {"bytes": n * (12 + state + (2 if case["copy"] else 0)), "flops": 20 * n}
    es = 2 if case["dtype"] == "bf16" else 4
    T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
    has = ids >= 0
    rows = int(has.sum())
    used = int(ranks[np.unique(ids[has])].sum())
    flops = 2 * int(ranks[ids[has]].sum()) * (2 * d_in + 2 * d_out + d_in)
    moved = es * (rows * (d_in + d_out) + used * (d_in + d_out)) + 4 * used * (d_in + d_out)
    if case["op"] == "fused":
        return {"bytes": moved + es * (T * d_in + d_in * d_out + (T - rows) * d_out), "flops": flops + 2 * T * d_in * d_out}
    return {"bytes": moved + 2 * es * rows * d_in, "flops": flops}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_adamw(s) if case["op"] == "adamw" else _exact_grad(s)


def _exact_grad(s):
    """Adapter by adapter, on the rows that use it."""
    fused = s["case"]["op"] == "fused"
    x, dy = s["x"].double(), s["dy"].double()
    dx = dy @ s["W0"].double() if fused else s["dx"].double()
    dA, dB = [], []
    for i, (A, Bm, scale) in enumerate(zip(s["A"], s["B"], s["scale"])):
        rows = torch.nonzero(s["ids"] == i)[:, 0]
        xi, yi, A, Bm = x[rows], dy[rows], A.double(), Bm.double()
        h = float(np.float32(scale)) * (yi @ Bm)
        dx[rows] += h @ A
        dA.append((h.t() @ xi).reshape(-1))
        dB.append((float(np.float32(scale)) * (yi.t() @ (xi @ A.t()))).reshape(-1))
    return {"dx": dx, "dA": torch.cat(dA), "dB": torch.cat(dB)}


def _values(bias):
    """What the codes 0 .. 255 of an unsigned format with 3 mantissa bits stand for."""
    c = np.arange(256)
    e, f = c // 8, c % 8
    return np.where(e > 0, (1.0 + f / 8.0) * 2.0 ** (e - float(bias)), f / 8.0 * 2.0 ** (1.0 - bias))


def _exact_state(value, bias, codes, random, sign):
    """Rows of 256 values as scale * code: the neighbouring codes are found by search in the table of the format."""
    table = torch.from_numpy(_values(bias)[: codes + 1]).cuda()
    a = value.abs()
    top = a.amax(1, keepdim=True)
    # the least power of two that brings the largest value below the largest code's
    e = torch.ceil(torch.log2(top / table[-1]).clamp(min=-126.0))
    e = torch.where(top >= torch.exp2(e) * table[-1], e + 1, e)
    e = torch.where(top < torch.exp2(e - 1) * table[-1], e - 1, e).clamp(-126.0, 127.0)
    scale = torch.exp2(e)
    y = a / scale
    low = (torch.searchsorted(table, y, right=True) - 1).clamp(0, codes)
    high = (low + 1).clamp(max=codes)
    gap = table[high] - table[low]
    share = torch.where(gap > 0, (y - table[low]) / torch.where(gap > 0, gap, 1.0), 0.0)
    code = torch.where(share + random / 65536.0 >= 1.0, high, low)
    if not sign:
        code = torch.where((a > 0) & (code == 0), 1, code)
    return torch.where(value < 0, -1.0, 1.0) * table[code] * scale


def _exact_adamw(s):
    eight = s["case"]["state"] == "8bit"
    h = {k: t.double()[s["group"]][:, None] for k, t in s["hyper"].items()}
    p0, g = s["p"].double().view(-1, BLOCK), s["g"].double().view(-1, BLOCK) * h["grad_scale"]
    if eight:
        c = s["m"].long()
        m0 = torch.from_numpy(_values(7)).cuda()[c & 127] * torch.where(c > 127, -1.0, 1.0)
        m0 = m0 * torch.exp2(s["m_scale"].double() - 127.0)[:, None]
        v0 = torch.from_numpy(_values(15)).cuda()[s["v"].long()] * torch.exp2(s["v_scale"].double() - 127.0)[:, None]
    else:
        m0, v0 = s["m"].double().view(-1, BLOCK), s["v"].double().view(-1, BLOCK)
    m = h["beta1"] * m0 + (1 - h["beta1"]) * g
    v = h["beta2"] * v0 + (1 - h["beta2"]) * g * g
    t = h["step"].clamp(min=1)
    top = m / -torch.expm1(t * torch.log(h["beta1"]))
    low = torch.sqrt(v / -torch.expm1(t * torch.log(h["beta2"]))) + h["eps"]
    rests = h["step"] < 1
    p = torch.where(rests, p0, p0 * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * top / low)
    if eight:
        bits = _exact_hash(s)
        m = _exact_state(m, 7, 126, bits % 65536, True)
        v = _exact_state(v, 15, 254, bits // 65536, False)
    out = {"p": p.reshape(-1), "m": torch.where(rests, m0, m).reshape(-1), "v": torch.where(rests, v0, v).reshape(-1)}
    return {**out, "copy": p.reshape(-1)} if s["case"]["copy"] else out


def _exact_hash(s):
    """_hash's definition, with 32-bit words of numpy."""
    word = np.uint32

    def mix(z):
        z = (z ^ (z >> word(16))) * word(0x6A09E667)
        z = (z ^ (z >> word(15))) * word(0xBB67AE85)
        return z ^ (z >> word(16))

    seed, step = (s["hyper"][k].cpu().numpy().astype(np.int64).astype(word) for k in ("seed", "step"))
    key = mix(seed + step * word(0x9E3779B9))
    key = mix(key[s["group"].cpu().numpy()] + s["tensor"].cpu().numpy().astype(word) * word(0x510E527F))
    at = (s["place"].cpu().numpy()[:, None] * BLOCK + np.arange(BLOCK)).astype(word)
    return torch.from_numpy(mix(at * word(0x9E3779B9) + key[:, None]).astype(np.int64)).cuda()
