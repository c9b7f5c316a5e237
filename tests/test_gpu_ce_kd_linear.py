"""Cross entropy and distillation from top logits through the lm_head product, in pieces of the vocabulary, against
the float64 reference on the same hidden states and weight.

x and w are small multiples of powers of two, so that every product and every partial sum of z is exact in fp32
(whole multiples of 2^-m below 2^24 of them): the loss then has the tolerances of _kd.py.  A gradient is a sum of products
with G, whose elements are off by _kd.py's bound and half a step of bf16 (2^-8); the sum of n products in fp32 adds at
most n 2^-24 of the sum of their sizes, and the result is rounded to its type.
One test takes inputs of every size, with z off by at most H 2^-24 of the sum of its products' sizes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cross_entropy_tv_amd as lx  # noqa: E402
from _kd import DEV, DT, HALF, IGN, NINF, TOL_GRAD, Case, announce  # noqa: E402


class Linear(Case):
    """A Case whose logits are x w^T."""

    def __init__(self, seed, BT, V, H, K, T=1.0, grad="f32", exact=True, **kw):
        rng = np.random.default_rng(seed + 1000)
        if exact:
            self.x = rng.integers(-3, 4, (BT, H)).astype(np.float32) * 0.5
            self.w = rng.integers(-3, 4, (V, H)).astype(np.float32) * 2.0 ** -int(np.log2(max(4.0, 2 * H ** 0.5)))
        else:
            to = lambda a: torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16).float().numpy()  # noqa: E731
            self.x, self.w = to(rng.standard_normal((BT, H))), to(rng.standard_normal((V, H)) * 2 / H ** 0.5)
        self.H, self.grad_dt = H, grad
        z = self.x.astype(np.float64) @ self.w.astype(np.float64).T
        assert not exact or (np.abs(z).max() <= 32 and (z.astype(np.float32) == z).all())
        edit = kw.pop("edit", None)
        super().__init__(seed, BT, V, max(K, 1), "f32", T=T, **kw)
        rng = np.random.default_rng(seed + 2000)
        from oracle import kd as oracle
        self.z = z
        for r in range(BT):  # a teacher near these logits
            u = (z[r] + rng.standard_normal(V)).astype(np.float32)
            self.top[r], self.ids[r], _, rest = oracle.top_row(u, max(K, 1), T)
            if self.rest is not None:
                self.rest[r] = rest
        self.K = K
        if K == 0:
            self.ids[:] = -1
            self.rest = None
        if edit is not None:
            edit(self)

    def run(self, want="xw", piece=None, **kw):
        announce(f"linear BT {self.BT} V {self.V} H {self.H} K {self.K} T {self.T} {self.grad_dt} {want} piece {piece}")
        dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
        new = lambda *s: torch.full(s, 99.0, dtype=torch.float32, device=DEV)  # noqa: E731
        bf = lambda a: torch.from_numpy(a).to(DEV).to(torch.bfloat16)  # noqa: E731
        if not hasattr(self, "xd"):
            self.xd, self.wd = bf(self.x), bf(self.w)
            self.args = (dev(self.target), IGN) + ((dev(self.ids), dev(self.top), dev(self.rest)) if self.K else (None,) * 3)
            self.rows = (dev(self.ce_rows), dev(self.kd_rows))
            self.scaled = None if self.g_scale is None else torch.tensor([self.g_scale], dtype=torch.float32, device=DEV)
        self.out = (new(self.BT), new(self.BT), new(self.BT), new(self.BT, 4))
        ce, kd, lse, state = self.out
        if not self.K:
            kd = state = None
        dt = DT[self.grad_dt]
        self.gx = torch.full((self.BT, self.H), 55.0, dtype=dt, device=DEV) if "x" in want else None
        self.gw = torch.full((self.V, self.H), 55.0, dtype=dt, device=DEV) if "w" in want else None
        lx.lx_ce_kd_linear_forward_backward(self.xd, self.wd, *self.args, self.T, ce, kd, lse, state, self.gx, self.gw,
                                            *self.g, *self.rows, self.scaled, piece=piece, **kw)
        if not self.K:  # the reference's results of a row without a teacher
            self.out[1].zero_()
            self.out[3].zero_()
        return self

    def check(self):
        if self.K:
            self.check_loss()
        else:
            for r in range(self.BT):
                want = self.row(r)
                if self.target[r] == IGN:
                    assert self.out[0][r] == self.out[2][r] == 0
                    continue
                for got, exact in ((self.out[0][r], want.ce), (self.out[2][r], want.lse)):
                    assert np.isnan(float(got)) if np.isnan(exact) else abs(float(got) - exact) <= 2.0 ** -15, r
        return self.check_grads()

    def check_grads(self, z_off=0.0):
        k = 1.0 if self.g_scale is None else float(np.float32(self.g_scale))
        G, off = np.zeros((self.BT, self.V)), np.zeros((self.BT, self.V))
        for r in range(self.BT):
            if self.target[r] == IGN:
                continue
            a = k * float(np.float32(self.g[0])) * (1.0 if self.ce_rows is None else float(self.ce_rows[r]))
            b = k * float(np.float32(self.g[1])) * (1.0 if self.kd_rows is None else float(self.kd_rows[r]))
            G[r], size = self.row(r).grad(a, b)
            off[r] = (TOL_GRAD + z_off) * size + 2.0 ** -125
            if 0 <= self.target[r] < self.V:
                off[r, self.target[r]] += 2 * 2.0 ** -24 * abs(a)
        bad = np.isnan(G).any(1)
        Gf = np.where(np.isnan(G), 0, G)
        err = off + HALF["bf16"] * (np.abs(Gf) + off)
        size = np.abs(Gf) + err
        x, w = self.x.astype(np.float64), self.w.astype(np.float64)
        for got, want, e, mag, n in ((self.gx, Gf @ w, err @ np.abs(w), size @ np.abs(w), self.V),
                                     (self.gw, Gf.T @ x, err.T @ np.abs(x), size.T @ np.abs(x), self.BT)):
            if got is None:
                continue
            got = got.double().cpu().numpy()
            if bad.any():
                if got.shape[0] == self.BT and got is not None and want.shape == (self.BT, self.H) and n == self.V:
                    assert np.isnan(got[bad]).all()
                    got, want, e, mag = got[~bad], want[~bad], e[~bad], mag[~bad]
                else:
                    assert np.isnan(got).all()
                    continue
            bound = e + (n + 8) * 2.0 ** -24 * mag
            bound = bound + HALF[self.grad_dt] * (np.abs(want) + bound) + 2.0 ** -120
            assert (np.abs(got - want) <= bound).all(), np.abs((got - want) / bound).max()
        return self


@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("BT,V,H,K,piece", [(1, 1, 8, 1, None), (3, 7, 8, 3, None), (5, 300, 64, 9, 256), (4, 257, 72, 20, 256),
                                            (75, 5001, 1160, 16, 2048), (300, 2051, 72, 64, 512), (257, 1000, 64, 0, None),
                                            (2, 20003, 136, 50, 4096), (513, 515, 520, 7, 256), (33, 1500, 64, 256, 1024)])
def test_sizes(grad, BT, V, H, K, piece):
    Linear(1, BT, V, H, K, grad=grad).run(piece=piece).check()


@pytest.mark.parametrize("T", [0.5, 2.0])
@pytest.mark.parametrize("rest", [True, False])
def test_temperatures(T, rest):
    Linear(2, 60, 1501, 200, 12, T=T, rest=rest, ignored=(0, 33)).run(piece=512).check()


def test_pieces_agree():
    """The loss does not depend on the pieces, and the gradient of w only by its own rows."""
    c = Linear(3, 130, 3001, 128, 24, T=2.0)
    c.run(piece=1 << 20).check()
    first = [o.clone() for o in c.out] + [c.gw.clone()]
    for piece in (1, 256, 1000, 3001, 4096):
        c.run(piece=piece).check()
        for a, b in zip(first, list(c.out) + [c.gw]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("want", ["x", "w", ""])
def test_outputs_that_are_not_wanted(want):
    for K in (0, 10):
        Linear(4, 50, 700, 64, K, grad="bf16").run(want).check()


def test_rows_with_factors():
    Linear(5, 40, 900, 64, 11, rows=True, g_scale=0.25, ignored=(3, 39)).run(piece=512).check()
    Linear(6, 40, 900, 64, 11, g=(0.0, 1.0), T=2.0).run().check()
    Linear(7, 40, 900, 64, 0, rows=True, g_scale=0.5, ignored=(0,)).run().check()


def test_more_entries_in_a_tile_than_are_listed():
    c = Linear(8, 300, 300, 64, 200)
    c.run().check()
    Linear(9, 256, 256, 64, 256, T=2.0, rest=False).run().check()


@pytest.mark.parametrize("T", [1.0, 2.0])
def test_targets_and_ids_that_are_no_tokens(T):
    def edit(c):
        c.target[:2] = [IGN, 5]
        c.ids[1, :6] = -1
        c.ids[2, :] = -7
        c.ids[3, 3] = c.ids[3, 0]
        c.ids[4, :] = c.ids[4, 0]
        c.top[5, :] = NINF
        c.top[6, 1] = -3.4e38
        c.target[7] = c.ids[7, 2]
    Linear(10, 9, 900, 64, 12, T=T, edit=edit).run(piece=256).check()

    def wrong(c):
        c.target[:2] = [-1, c.V]
        c.ids[4, 2] = c.V
    c = Linear(11, 9, 900, 64, 12, T=T, edit=wrong).run(piece=256)
    c.check()
    assert torch.isnan(c.gx[[0, 1, 4]]).all() and not torch.isnan(c.gx[[2, 3, 5, 6, 7, 8]]).any()


def test_inputs_of_every_size():
    c = Linear(12, 90, 1200, 512, 20, exact=False)
    c.run(piece=512)
    # |x w| sums: H products; z is off by at most H 2^-24 of them, a log-sum by as much, a gradient's terms by twice that
    S = float((np.abs(c.x) @ np.abs(c.w).T).max())
    z_off = 2 * c.H * 2.0 ** -24 * S
    for r in range(c.BT):
        want = c.row(r)
        assert abs(float(c.out[0][r]) - want.ce) <= 2.0 ** -15 + z_off
        assert abs(float(c.out[1][r]) - want.kd) <= 2.0 ** -15 + z_off
        assert abs(float(c.out[2][r]) - want.lse) <= 2.0 ** -16 + z_off
    c.check_grads(z_off=2 * z_off)


def test_same_bits_on_every_call_graph_and_stream():
    for BT, V in ((100, 3000), (3, 9000)):
        c = Linear(13, BT, V, 64, 16, grad="bf16", edit=lambda c: c.ids.__setitem__((0, slice(1, 5)), c.ids[0, 0]))
        c.run(piece=1024)
        first = [t.clone() for t in (*c.out, c.gx, c.gw)]
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        c.run(piece=1024, stream=s)
        torch.cuda.synchronize()
        for a, b in zip(first, (*c.out, c.gx, c.gw)):
            assert torch.equal(a, b)
        need = lx.lx_ce_kd_linear_workspace_bytes(BT, V, 64, 16, 1024, True)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        c.run(piece=1024, workspace=ws)
        out = (*c.out, c.gx, c.gw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lx.lx_ce_kd_linear_forward_backward(c.xd, c.wd, *c.args, c.T, *c.out, c.gx, c.gw, *c.g, piece=1024, workspace=ws)
        for k in range(4):
            for t in out:
                t.fill_(k)
            ws.fill_(255 * (k % 2))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(first, out):
                assert torch.equal(a, b)


def test_agrees_with_the_loss_over_logits():
    """The logits through lx_gemm_bf16, then lx_ce_kd_forward_backward: the same sums in another order."""
    c = Linear(14, 64, 2000, 256, 20, T=2.0).run()
    z = torch.empty(64, 2000, device=DEV)
    lx.lx_gemm_bf16(c.xd, True, c.wd, True, z, 64, 2000, 256)
    out = [torch.empty(64, device=DEV) for _ in range(3)] + [torch.empty(64, 4, device=DEV)]
    G = torch.empty_like(z)
    lx.lx_ce_kd_forward_backward(z, *c.args, c.T, *out, G, *c.g)
    for a, b in zip(out, c.out):
        assert (a - b).abs().max() <= 2.0 ** -15
    gx = G.double().cpu() @ c.wd.double().cpu()
    assert (gx - c.gx.double().cpu()).norm() <= 2.0 ** -8 * gx.norm() * 2


def test_no_rows():
    e = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
    w, gw = e(50, 64, dt=torch.bfloat16), torch.full((50, 64), 7.0, device=DEV)
    lx.lx_ce_kd_linear_forward_backward(e(0, 64, dt=torch.bfloat16), w, e(0, dt=torch.int64), IGN, None, None, None, 1.0, e(0),
                                        None, e(0), None, e(0, 64), gw, 1.0, 0.0)
    torch.cuda.synchronize()
    assert (gw == 0).all()


@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("K", [0, 12])
def test_rows_whose_logits_are_not_used(T, K):
    """An ignored row of large finite values, whose logits overflow, and a row whose logits are all masked: they leave the
    gradients as they are without them."""
    if K == 0:
        T = 1.0

    def edit(c):
        c.target[3] = IGN
        c.x[:, 0] = 0.0
        c.w[:, 0] = 2.0 ** 50
        c.x[5] = 0.0
        c.x[5, 0] = -2.0 ** 60
        c.z = c.x.astype(np.float64) @ c.w.astype(np.float64).T

    c = Linear(15, 9, 700, 64, K, T=T, edit=edit)
    c.run(piece=256)
    rows = [r for r in range(9) if r not in (3, 5)]
    if K:
        c.check_loss(rows=rows)
    assert c.out[0][5] == 0 and c.out[1][5] == 0 and c.out[2][5] == NINF
    assert not c.gx[[3, 5]].any()
    first = [c.gx.clone(), c.gw.clone()]
    assert torch.isfinite(first[0]).all() and torch.isfinite(first[1]).all()
    c.xd[3] = 3e38
    c.xd[3, ::2] = -3e38
    c.run(piece=256)
    assert torch.equal(c.gx, first[0]) and torch.equal(c.gw, first[1])
