"""AdamW's plan and refusals on the CPU, and the numpy reference against
differences and against the formats' definitions."""

import ctypes

import numpy as np
import pytest

import adamw_ref as R
from segmented_gather_gemm_lora_amd import binding as B

FX = 0x7F0000000000


def tensor(i=0, n=1000, group=0, **kw):
    base = FX + i * 0x100000
    f = dict(param=base, grad=base + 0x10000, copy=base + 0x20000, m=base + 0x30000, v=base + 0x40000, m_scale=base + 0x50000,
             v_scale=base + 0x51000, n=n, group=group, reserved=0)
    f.update(kw)
    return B.LoraAdamTensor(*(f[k] for k, _ in B.LoraAdamTensor._fields_))


def plan(tensors, n_groups=2, state=1, gdt=0, nbytes=None, buf=None):
    arr = (B.LoraAdamTensor * max(len(tensors), 1))(*tensors)
    need = B.load().lora_adamw_plan_bytes(arr, len(tensors))
    raw = np.zeros(need + 64, dtype=np.uint8)
    off = (-raw.ctypes.data) % 16
    ptr = raw.ctypes.data + off if buf is None else raw.ctypes.data + off + buf
    st = B.load().lora_adamw_plan(arr, len(tensors), n_groups, state, gdt, ptr, need if nbytes is None else nbytes)
    return B.STATUS[st], raw, ptr, need


def test_plan_records():
    st, raw, ptr, need = plan([tensor(0, 2500, 1), tensor(1, 0), tensor(2, 1, 0, copy=0)])
    assert st == "LORA_OK"
    assert need == 32 + 80 * 4
    rec = np.dtype([("param", "<u8"), ("grad", "<u8"), ("copy", "<u8"), ("m", "<u8"), ("v", "<u8"), ("ms", "<u8"),
                    ("vs", "<u8"), ("e0", "<u4"), ("n", "<i4"), ("group", "<i4"), ("tensor", "<u4"), ("r", "<u8")])
    off = ptr - raw.ctypes.data
    r = np.frombuffer(raw[off + 32: off + need].tobytes(), dtype=rec)
    assert r["e0"].tolist() == [0, 1024, 2048, 0] and r["n"].tolist() == [1024, 1024, 452, 1]
    assert r["tensor"].tolist() == [0, 0, 0, 2] and r["group"].tolist() == [1, 1, 1, 0]
    assert (r["param"][:3] - FX).tolist() == [0, 4096, 8192]
    assert (r["m"][:3] - FX - 0x30000).tolist() == [0, 1024, 2048]
    assert (r["ms"][:3] - FX - 0x50000).tolist() == [0, 4, 8]
    assert r["copy"].tolist() == [FX + 0x20000, FX + 0x20000 + 2048, FX + 0x20000 + 4096, 0]


@pytest.mark.parametrize("tensors,kw,status", [
    ([tensor(n=-1)], {}, "LORA_ERR_ARG"),
    ([tensor(n=2**31)], {}, "LORA_ERR_ARG"),
    ([tensor(group=2)], {}, "LORA_ERR_ARG"),
    ([tensor(group=-1)], {}, "LORA_ERR_ARG"),
    ([tensor(param=0)], {}, "LORA_ERR_ARG"),
    ([tensor(grad=0)], {}, "LORA_ERR_ARG"),
    ([tensor(m=0)], {}, "LORA_ERR_ARG"),
    ([tensor(v_scale=0)], {}, "LORA_ERR_ARG"),
    ([tensor(param=FX + 4)], {}, "LORA_ERR_ALIGN"),
    ([tensor(grad=FX + 0x10008)], {}, "LORA_ERR_ALIGN"),
    ([tensor(copy=FX + 0x20002)], {}, "LORA_ERR_ALIGN"),
    ([tensor()], dict(state=2), "LORA_ERR_DTYPE"),
    ([tensor()], dict(gdt=5), "LORA_ERR_DTYPE"),
    ([tensor()], dict(n_groups=-1), "LORA_ERR_ARG"),
    ([tensor()], dict(nbytes=111), "LORA_ERR_WORKSPACE"),
    ([tensor()], dict(buf=8), "LORA_ERR_ALIGN"),
    ([tensor(0), tensor(0)], {}, "LORA_ERR_ARG"),  # one tensor twice
    ([tensor(0), tensor(1, param=FX + 512)], {}, "LORA_ERR_ARG"),  # overlapping parameters
    ([tensor(0), tensor(1, v=FX + 0x30000 + 992)], {}, "LORA_ERR_ARG"),  # one's v in the other's m
    ([tensor(0), tensor(1, m_scale=FX + 0x51003)], {}, "LORA_ERR_ARG"),
])
def test_refusals(tensors, kw, status):
    st, *_ = plan(tensors, **kw)
    assert st == status and B.last_error()


def test_fp32_states_need_no_scales_and_shared_gradients_are_fine():
    st, *_ = plan([tensor(0, m_scale=0, v_scale=0), tensor(1, grad=FX + 0x10000, m_scale=0, v_scale=0)], state=0)
    assert st == "LORA_OK"


@pytest.mark.parametrize("tensors,gdt", [
    ([tensor(0), tensor(1, grad=FX + 3984)], 0),  # the other's gradient starts in a parameter's last 16 bytes
    ([tensor(0), tensor(1, grad=FX + 0x30000 - 16)], 0),  # ... ends in the other's m
    ([tensor(0, grad=FX)], 0),  # its own parameter
    ([tensor(0), tensor(1, n=9, grad=FX + 0x51000 - 16)], 1),  # 18 bytes of bf16, the last 2 in v's scales
])
def test_gradients_in_written_memory(tensors, gdt):
    st, *_ = plan(tensors, gdt=gdt)
    assert st == "LORA_ERR_ARG" and "gradient" in B.last_error()


def test_gradients_next_to_written_memory():
    st, *_ = plan([tensor(0), tensor(1, n=8, grad=FX + 0x51000 - 16), tensor(2, n=0, grad=FX)], gdt=1)
    assert st == "LORA_OK"


def test_binding_refuses_host_tensors():
    import torch

    host = torch.zeros(16)
    hyper = B.adamw_hyper(1, device="cpu")
    with pytest.raises(ValueError, match="device"):
        B.AdamW([host], [host], [0], hyper)
    with pytest.raises(ValueError, match="device"):
        B.AdamW([], [], [], hyper)
    codes, scale, out = torch.zeros(300, dtype=torch.uint8), torch.zeros(2, dtype=torch.uint8), torch.zeros(300).bfloat16()
    with pytest.raises(ValueError, match="device"):
        B.adamw_state_values(codes, scale, None, None, out, None)
    with pytest.raises(ValueError, match="scale"):
        B.adamw_state_values(codes, scale[:1], None, None, out, None)
    with pytest.raises(ValueError, match="scale"):
        B.adamw_state_values(None, None, codes, scale, None, out[:299])
    with pytest.raises(ValueError, match="scale"):
        B.adamw_state_values(codes, scale, None, None, out.float(), None)


def test_step_refusals():
    L = B.load()
    st, raw, ptr, need = plan([tensor()])
    ok = lambda *a: B.STATUS[L.lora_adamw(*a)]  # noqa: E731
    assert ok(None, None, FX, FX, 2) == "LORA_ERR_ARG"
    assert ok(None, ptr + 4, FX, FX, 2) == "LORA_ERR_ALIGN"
    assert ok(None, ptr, FX, FX, 1) == "LORA_ERR_ARG"  # fewer groups than the plan
    assert ok(None, ptr, None, FX, 2) == "LORA_ERR_ARG"
    assert ok(None, ptr, FX, None, 2) == "LORA_ERR_ARG"
    assert ok(None, ptr, FX, FX + 8, 2) == "LORA_ERR_ALIGN"
    blank = np.zeros(64, dtype=np.uint8)
    assert ok(None, blank.ctypes.data + (-blank.ctypes.data) % 16, FX, FX, 2) == "LORA_ERR_PLAN"
    up = lambda *a: B.STATUS[L.lora_adamw_upload(*a)]  # noqa: E731
    assert up(ptr, None, need, None) == "LORA_ERR_ARG"
    assert up(ptr, FX + 4, need, None) == "LORA_ERR_ALIGN"
    assert up(ptr, FX, need - 1, None) == "LORA_ERR_WORKSPACE"
    # a plan that failed to build is none
    bad = (B.LoraAdamTensor * 1)(tensor(group=9))
    assert L.lora_adamw_plan(bad, 1, 2, 1, 0, ptr, need) != 0
    assert ok(None, ptr, FX, FX, 2) == "LORA_ERR_PLAN"


def test_nothing_to_do():
    L = B.load()
    st, raw, ptr, need = plan([], n_groups=0)
    assert st == "LORA_OK" and need == 32
    assert L.lora_adamw(None, ptr, None, None, 0) == 0
    assert L.lora_adam_state_values(None, 0, FX, FX, FX, FX, FX, FX) == 0
    assert L.lora_adam_state_values(None, 5, None, None, None, None, None, None) == 0


def test_state_values_refusals():
    f = lambda *a: B.STATUS[B.load().lora_adam_state_values(None, *a)]  # noqa: E731
    assert f(-1, FX, FX, FX, FX, FX, FX) == "LORA_ERR_ARG"
    assert f(5, FX, None, FX, FX, FX, FX) == "LORA_ERR_ARG"
    assert f(5, FX, FX, FX, FX, FX, None) == "LORA_ERR_ARG"
    assert f(5, FX + 1, FX, FX, FX, FX, FX) == "LORA_ERR_ALIGN"
    assert f(5, None, None, FX, FX, None, FX + 2) == "LORA_ERR_ALIGN"


def test_plan_bytes_of_bad_lists():
    L = B.load()
    assert L.lora_adamw_plan_bytes(None, 1) == 0 and L.lora_adamw_plan_bytes(None, -1) == 0
    assert L.lora_adamw_plan_bytes((B.LoraAdamTensor * 1)(tensor(n=-3)), 1) == 0
    assert ctypes.sizeof(B.LoraAdamTensor) == 72


def test_formats():
    """m's codes are OCP E4M3 (torch's type), v's the same steps without a sign over 32 binades."""
    import torch

    e4m3 = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = R.decode(np.arange(256), np.array([127]), "m")
    assert np.array_equal(got, e4m3, equal_nan=True)
    v = R.decode(np.arange(255), np.array([127]), "v")
    assert v[0] == 0 and v[1] == 2.0**-17 and v[8] == 2.0**-14 and v[254] == 1.75 * 2.0**16
    assert (np.diff(v) > 0).all() and np.isnan(R.decode(np.array([255]), np.array([127]), "v"))[0]


def test_noise_is_uniform():
    """Means and pair products of the two 16-bit halves over 2^18 elements, within 5
    standard deviations; neighbours in step, tensor and seed are unrelated."""
    n = 1 << 18
    a = R.noise(1, 1, 0, n)
    for half in (a & 0xFFFF, a >> 16):
        u = half / 65536.0
        assert abs(u.mean() - 0.5) <= 5 * np.sqrt(1 / 12 / n)
        assert abs(np.mean((u[1:] - 0.5) * (u[:-1] - 0.5))) <= 5 / 12 / np.sqrt(n)
        assert np.abs(np.bincount(half >> 8, minlength=256) - n / 256).max() <= 6 * np.sqrt(n / 256)
    for b in (R.noise(1, 2, 0, n), R.noise(1, 1, 1, n), R.noise(2, 1, 0, n)):
        for s in (0, 16):
            x, y = ((t >> s) & 0xFFFF for t in (a, b))
            assert abs(np.mean((x / 65536.0 - 0.5) * (y / 65536.0 - 0.5))) <= 5 / 12 / np.sqrt(n)


def test_reference_step_against_torch():
    """The reference's update is AdamW's: torch.optim.AdamW in 64 bits, three steps."""
    import torch

    r = np.random.default_rng(0)
    p0 = r.standard_normal(50)
    q = torch.from_numpy(p0.astype(np.float32)).double().requires_grad_()
    opt = torch.optim.AdamW([q], lr=float(np.float32(1e-2)), betas=(float(np.float32(0.9)), float(np.float32(0.99))),
                            eps=float(np.float32(1e-8)), weight_decay=float(np.float32(0.1)))
    p, m, v = p0.astype(np.float32), np.zeros(50, np.float32), np.zeros(50, np.float32)
    for t in range(1, 4):
        g = r.standard_normal(50).astype(np.float32)
        q.grad = torch.from_numpy(g).double()
        opt.step()
        new, bound, m, v = R.step(p, g, m, v, dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, grad_scale=1.0,
                                                   step=t))
        p = new.astype(np.float32)
        # bound has p's rounding and 24 steps for the update; m and v in fp32 add 4 steps
        # to an update of at most lr (1 + 0.1 |p|)
        assert (np.abs(q.detach().numpy() - new) <= t * (bound + 4 * 2.0**-23 * 1e-2 * (1 + np.abs(new)))).all()


@pytest.mark.parametrize("n,state,gdt,chunk", [
    (1 << 21, 1, 0, 1024), ((1 << 21) + 1, 1, 0, 2048), ((1 << 21) + 1, 1, 1, 2048), (1 << 24, 0, 0, 1024), (1000, 1, 1, 1024),
])
def test_elements_of_a_chunk(n, state, gdt, chunk):
    """Two rows of 1024 for many 8-bit elements; the records cover the tensor once either way."""
    one = dict(param=FX, grad=FX + (1 << 32), copy=0, m=FX + (2 << 32), v=FX + (3 << 32), m_scale=FX + (4 << 32),
               v_scale=FX + (5 << 32), n=n, group=0, reserved=0)
    st, raw, ptr, need = plan([B.LoraAdamTensor(*(one[k] for k, _ in B.LoraAdamTensor._fields_))], state=state, gdt=gdt)
    assert st == "LORA_OK"
    off = ptr - raw.ctypes.data
    rows = (n + chunk - 1) // chunk
    at = raw[off + 32: off + 32 + 80 * rows].reshape(rows, 80)
    e0, k = at[:, 56:60].copy().view("<u4")[:, 0], at[:, 60:64].copy().view("<i4")[:, 0]
    assert np.array_equal(e0, chunk * np.arange(rows)) and k.sum() == n and (k[:-1] == chunk).all()
    assert not raw[off + 32 + 80 * rows: off + need].any()


def test_more_than_one_launch_has():
    """The runtime counts a launch's threads in 32 bits: 2^24 workgroups of 256 are refused, not cut off."""
    L = B.load()
    st, raw, ptr, need = plan([], n_groups=0)
    off = ptr - raw.ctypes.data
    for chunks in (1 << 24, 1 << 31):
        raw[off + 16: off + 24] = np.frombuffer(np.int64(chunks).tobytes(), dtype=np.uint8)
        assert B.STATUS[L.lora_adamw(None, ptr, FX, FX, 1)] == "LORA_ERR_ARG"
    n = 4096 * (1 << 24)
    assert B.STATUS[L.lora_adam_state_values(None, n, FX, FX, None, None, FX, None)] == "LORA_ERR_ARG"
