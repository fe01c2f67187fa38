"""The gradients of the segmented correction and of the fused layer in 64 bits
(numpy, adapter by adapter), with the error bounds that the GPU's results are
held to, and helpers that run them.

Bounds (per element).  2^-24 is half a step of fp32, relative to a value; a sum
of n fp32 terms is off by at most n 2^-24 times the sum of their magnitudes.
  u:  Eu = s (d_out + 2) 2^-24 |dy| |B|   (the products of bf16 are exact in
      fp32; the sum, the scale and alpha / r round)
  dA: |Eu|^T |x| + (L + 4 + P) 2^-24 |u|^T |x|, L rows, 4 for the parts that u is
      fed in and P = L / 128 + 1 for partial sums
  dx: Eu |A| + (3 r + 4) 2^-24 |u| |A| + part |u| |A| + half |dx|, part = 2^-16
      for bf16 (u in two bf16 parts), half = 2^-8 for bf16, 2^-24 for fp32
"""

from __future__ import annotations

import numpy as np
import torch

from segmented_gather_gemm_lora_amd import binding as B

EPS = 2.0**-24


class Problem:
    """Inputs of one backward call, on the host in the stored dtype (torch CPU)."""

    def __init__(self, dtype, ids, ranks, d_in, d_out, seed=0, alpha=32.0, pad=(0, 0, 0), w0=False, integer=False,
                 n_none=0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.d_in, self.d_out = dtype, d_in, d_out
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.ids = np.asarray(ids, dtype=np.int32)
        self.T = len(self.ids)
        self.rank = np.asarray(ranks, dtype=np.int32)
        self.alpha = self.rank.astype(np.float32) if integer else np.full(len(ranks), alpha, dtype=np.float32)

        def draw(*shape, std=1.0):
            if integer:
                return torch.randint(-1, 2, shape, generator=g).to(self.dt)
            return (torch.randn(*shape, generator=g) * std).to(self.dt)

        self.A = [draw(int(r), d_in, std=0.05) for r in self.rank]
        self.B = [draw(d_out, int(r), std=0.05) for r in self.rank]
        # row pitches of d + pad elements
        self.x_full, self.dy_full = draw(self.T, d_in + pad[0]), draw(self.T, d_out + pad[1])
        self.dx_full = draw(self.T, d_in + pad[2])
        self.x, self.dy, self.dx = self.x_full[:, :d_in], self.dy_full[:, :d_out], self.dx_full[:, :d_in]
        self.W0 = draw(d_out, d_in, std=0.05) if w0 else None
        self.scale = [float(np.float32(a) / np.float32(r)) for a, r in zip(self.alpha, self.rank)]

    @property
    def max_rank(self):
        return int(self.rank.max()) if len(self.rank) else 0

    # ------------------------------------------------------------ 64 bits
    def reference(self):
        """(dx, dA list, dB list) and bounds of the same shapes."""
        x, dy = self.x.double().numpy(), self.dy.double().numpy()
        if self.W0 is not None:
            W = self.W0.double().numpy()
            dx = dy @ W
            edx = (self.d_out + 2) * EPS * (np.abs(dy) @ np.abs(W))
        else:
            dx = self.dx.double().numpy().copy()
            edx = EPS * np.abs(dx)
        part = 2.0**-16 if self.dtype == "bf16" else 0.0
        dA, dB, eA, eB = [], [], [], []
        for i, r in enumerate(self.rank):
            rows = np.nonzero(self.ids == i)[0]
            A, Bm, s = self.A[i].double().numpy(), self.B[i].double().numpy(), self.scale[i]
            xi, yi, L = x[rows], dy[rows], len(rows)
            u, v = s * yi @ Bm, s * xi @ A.T
            eu = abs(s) * (self.d_out + 2) * EPS * (np.abs(yi) @ np.abs(Bm))
            ev = abs(s) * (self.d_in + 2) * EPS * (np.abs(xi) @ np.abs(A.T))
            n = L + 5 + L / 128
            dA.append(u.T @ xi)
            eA.append(eu.T @ np.abs(xi) + n * EPS * np.abs(u).T @ np.abs(xi))
            dB.append(yi.T @ v)
            eB.append(np.abs(yi).T @ ev + n * EPS * np.abs(yi).T @ np.abs(v))
            dx[rows] += u @ A
            edx[rows] += eu @ np.abs(A) + ((3 * int(r) + 4) * EPS + part) * (np.abs(u) @ np.abs(A))
        edx += (2.0**-8 if self.dtype == "bf16" else EPS) * np.abs(dx)
        return (dx, dA, dB), (edx, eA, eB)

    # ------------------------------------------------------------ device
    def device(self, misalign=0):
        """Device copies: a DevicePool whose matrices start at multiples of 128
        elements, x, dy and dx with their pitches (moved by `misalign` elements)."""
        p = DeviceProblem()
        n, es = len(self.rank), self.x.element_size()
        mats = [*self.A, *self.B]
        starts = np.concatenate([[0], np.cumsum([(t.numel() + 127) // 128 * 128 for t in mats])]).astype(np.int64)
        host = torch.zeros(max(int(starts[-1]), 1), dtype=self.dt)
        for t, o in zip(mats, starts):
            host[int(o): int(o) + t.numel()] = t.reshape(-1)
        p.storage = host.cuda()
        base = p.storage.data_ptr()
        p.pool = B.DevicePool(storage=p.storage, n_adapters=n, dtype=self.dtype, d_in=self.d_in, d_out=self.d_out,
                              addr_A=(base + starts[:n] * es).astype(np.uint64),
                              addr_B=(base + starts[n:-1] * es).astype(np.uint64), rank=self.rank, alpha=self.alpha)

        def moved(full, cols):
            flat = torch.empty(full.numel() + misalign, dtype=self.dt, device="cuda")
            flat[misalign:] = full.reshape(-1).cuda()
            return flat[misalign:].view(full.shape)[:, :cols]

        p.x, p.dy, p.dx = moved(self.x_full, self.d_in), moved(self.dy_full, self.d_out), moved(self.dx_full, self.d_in)
        p.W0 = None if self.W0 is None else self.W0.cuda()
        p.plan = B.Plan(max(self.T, 1)).build(self.ids, p.pool).upload()
        p.grads = B.GradPool.like(p.pool)
        op = B.LORA_OP_SGMV_BACKWARD if self.W0 is None else B.LORA_OP_FUSED_BACKWARD
        p.ws = B.workspace(op, self.T, self.d_in, self.d_out, max(self.max_rank, 1))
        p.ws.fill_(0xFF)  # whatever an earlier call left: NaN
        return p


class DeviceProblem:
    pass


def worst(got, ref, bound):
    """Largest |got - ref| / bound (0 / 0 = 0)."""
    if np.size(ref) == 0:
        return 0.0
    err = np.abs(np.asarray(got, dtype=np.float64) - ref)
    err = np.where(np.isnan(err), np.inf, err)
    return float(np.max(err / np.maximum(bound, 1e-300) * (err > 0)))


def check(p: Problem, d: DeviceProblem, what=""):
    """dx and every gradient of d against the 64-bit reference of p."""
    (dx, dA, dB), (edx, eA, eB) = p.reference()
    w = worst(d.dx.double().cpu().numpy(), dx, edx)
    assert w <= 1.0, f"{what}: dx worst |err|/bound {w:.3g}"
    for i in range(len(p.rank)):
        for name, got, ref, e in (("dA", d.grads.A[i], dA[i], eA[i]), ("dB", d.grads.B[i], dB[i], eB[i])):
            w = worst(got.double().cpu().numpy().reshape(ref.shape), ref, e)
            assert w <= 1.0, f"{what}: {name}[{i}] worst |err|/bound {w:.3g}"
