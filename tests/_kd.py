"""Cases of distillation from top logits and their comparison with the float64 reference.

Tolerances, derived for logits of at most 32 in size and T >= 1/2 (exponents c z = z log2(e) / T of at most
93, below 2^7):
  * a log-sum: an exponent's rounding (the scale's own 2^-24 of it and the multiply-add's) is below
    2 * 2^-24 * 2^7 * ln 2 < 2^-16.5; sums of positive terms add 2^-20, the result's rounding (below 64) 2^-19:
    2^-16 with all;
  * ce, kd: a difference of two log-sums and exact logits, 2^-15; kd's terms are formed in fp64, and the results are
    rounded (2^-24 of them: beyond 2^9 that is more than the rest);
  * p_r - q_r: each good to 2^-16 relatively and at most 1: 2^-15;
  * a gradient: the terms that it is the sum of, each a factor times an exponential of a difference with a rounded
    log-sum in it: 2^-15 of their sizes; at the target ce's factor, the fp32 product of three fp32 numbers (two
    roundings, 2 * 2^-24 of it: nothing else of the -g_ce there is rounded before the sum); half a step of the type (2^-8, 2^-11, 2^-24), of
    binary16's subnormals 2^-25, and 2^-125 for exponentials that are flushed.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import kd as oracle
from _parity import announce

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TOL_LOG, TOL_LOSS, TOL_OFF, TOL_GRAD = 2.0 ** -16, 2.0 ** -15, 2.0 ** -15, 2.0 ** -15
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -125, "f16": 2.0 ** -25, "f32": 2.0 ** -125}
NINF = float("-inf")
IGN = -100


def on_device(a, dt, pad=0, offset=0):
    """A (n, V) device view of row stride V + pad whose first element lies `offset` elements into its buffer, and the
    buffer; what lies around the rows is 77."""
    n, V = a.shape
    buf = torch.full((n * (V + pad) + offset + 8,), 77.0, dtype=dt, device=DEV)
    view = buf[offset:offset + n * (V + pad)].view(n, V + pad)[:, :V]
    view.copy_(torch.from_numpy(np.ascontiguousarray(a)))
    return view, buf


def around(buf, n, V, pad, offset):
    """The buffer's elements outside the rows."""
    keep = torch.ones(buf.shape[0], dtype=torch.bool, device=buf.device)
    keep[offset:offset + n * (V + pad)].view(n, V + pad)[:, :V] = False
    return buf[keep]


class Case:
    def __init__(self, seed, BT, V, K, dt="bf16", T=1.0, rest=True, pad=(0, 0), offset=(0, 0), scale=3.0, ignored=(),
                 noise=1.0, g=(0.7, 1.3), rows=False, g_scale=None, edit=None):
        rng = np.random.default_rng(seed)
        self.BT, self.V, self.K, self.dt, self.T = BT, V, K, dt, T
        self.pad, self.offset, self.g = pad, offset, g
        z = np.clip(rng.standard_normal((BT, V)) * scale, -30, 30).astype(np.float32)
        self.z = torch.from_numpy(z).to(DT[dt]).float().numpy()
        u = np.clip(self.z + rng.standard_normal((BT, V)) * noise, -30, 30).astype(np.float32)
        self.ids, self.top = np.zeros((BT, K), np.int32), np.zeros((BT, K), np.float32)
        self.rest = np.zeros(BT, np.float32)
        for r in range(BT):
            self.top[r], self.ids[r], _, self.rest[r] = oracle.top_row(u[r], K, T)
        if not rest:
            self.rest = None
        self.target = rng.integers(0, V, BT).astype(np.int64)
        for r in ignored:
            self.target[r] = IGN
        self.ce_rows = rng.uniform(0.5, 1.5, BT).astype(np.float32) if rows else None
        self.kd_rows = rng.uniform(0.5, 1.5, BT).astype(np.float32) if rows else None
        self.g_scale = g_scale
        if edit is not None:
            edit(self)

    def place(self):
        dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
        self.zd, self.zbuf = on_device(self.z, DT[self.dt], self.pad[0], self.offset[0])
        self.gd, self.gbuf = on_device(np.full((self.BT, self.V), 55.0, np.float32), DT[self.dt], self.pad[1], self.offset[1])
        self.set = (dev(self.target), IGN, dev(self.ids), dev(self.top))
        self.restd, self.factors = dev(self.rest), (dev(self.ce_rows), dev(self.kd_rows))
        self.scaled = None if self.g_scale is None else torch.tensor([self.g_scale], dtype=torch.float32, device=DEV)
        new = lambda *s: torch.full(s, 99.0, dtype=torch.float32, device=DEV)  # noqa: E731
        self.out = (new(self.BT), new(self.BT), new(self.BT), new(self.BT, 4))
        return self

    def forward(self, lx, **kw):
        lx.lx_ce_kd_forward(self.zd, *self.set, self.restd, self.T, *self.out, **kw)

    def backward(self, lx, grad, **kw):
        lx.lx_ce_kd_backward(grad, self.zd, *self.set, self.T, self.out[2], self.out[3], *self.g, *self.factors, self.scaled,
                             **kw)

    def step(self, lx, grad, **kw):
        lx.lx_ce_kd_forward_backward(self.zd, *self.set, self.restd, self.T, *self.out, grad, *self.g, *self.factors,
                                     self.scaled, **kw)

    def row(self, r):
        return oracle.Row(self.z[r], self.target[r], self.ids[r], self.top[r],
                          None if self.rest is None else self.rest[r], self.T)

    def check_loss(self, rows=None):
        ce, kd, lse, state = (o.double().cpu().numpy() for o in self.out)
        for r in range(self.BT) if rows is None else rows:
            if self.target[r] == IGN:
                assert ce[r] == kd[r] == lse[r] == 0 and not state[r].any(), r
                continue
            want = self.row(r)
            for got, name in ((ce[r], "ce"), (kd[r], "kd")):  # (the result's own rounding: half a step of it)
                exact = getattr(want, name)
                near(got, exact, TOL_LOSS + 2.0 ** -24 * abs(np.nan_to_num(exact, posinf=0)), f"{name}[{r}]")
            near(lse[r], NINF if want.empty else want.lse, TOL_LOG, f"lse[{r}]")
            for k, tol in enumerate((TOL_LOG, TOL_LOG, TOL_OFF, TOL_LOG)):
                near(state[r, k], want.state[k], tol, f"state[{r}][{k}]")

    def check_grad(self, grad, rows=None):
        got = grad.double().cpu().numpy()
        k = 1.0 if self.g_scale is None else float(np.float32(self.g_scale))
        for r in range(self.BT) if rows is None else rows:
            if self.target[r] == IGN:
                assert not got[r].any(), r
                continue
            a = k * float(np.float32(self.g[0])) * (1.0 if self.ce_rows is None else float(self.ce_rows[r]))
            b = k * float(np.float32(self.g[1])) * (1.0 if self.kd_rows is None else float(self.kd_rows[r]))
            want, size = self.row(r).grad(a, b)
            if np.isnan(want).any():
                assert np.isnan(got[r]).all(), r
                continue
            off = TOL_GRAD * size
            if 0 <= self.target[r] < self.V:
                off[self.target[r]] += 2 * 2.0 ** -24 * abs(a)
            bound = off + HALF[self.dt] * (np.abs(want) + off) + TINY[self.dt]
            off = np.abs(got[r] - want)
            worst = int(np.argmax(off / bound))
            assert (off <= bound).all(), (r, worst, got[r][worst], want[worst], bound[worst])

    def check_around(self):
        for buf, n in ((self.zbuf, 0), (self.gbuf, 1)):
            assert (around(buf, self.BT, self.V, self.pad[n], self.offset[n]) == 77).all()


def near(got, want, tol, what):
    if np.isnan(want):
        assert np.isnan(got), (what, got)
    elif np.isinf(want):
        assert got == want, (what, got, want)
    else:
        assert abs(got - want) <= tol, (what, got, want, tol)


def run_all(lx, c, rows=None):
    """Forward, backward, the one pass and the one pass in place of a case, each checked."""
    c.place()
    announce(f"ce_kd BT {c.BT} V {c.V} K {c.K} {c.dt} T {c.T}: forward")
    c.forward(lx)
    c.check_loss(rows)
    announce("backward")
    c.backward(lx, c.gd)
    c.check_grad(c.gd, rows)
    c.check_around()
    c.place()
    announce("one pass")
    c.step(lx, c.gd)
    c.check_loss(rows)
    c.check_grad(c.gd, rows)
    c.check_around()
    announce("one pass in place")
    c.step(lx, c.zd)
    c.check_loss(rows)
    c.check_grad(c.zd, rows)
    c.check_around()
