"""Documented sizes whose work makes more workgroups than one dimension of a launch holds (2^32 threads), and more than
the rows of workgroups that such launches are cut into, on the GPU, against float64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import draft_verify as dv

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cross_entropy_tv_amd as lx  # noqa: E402
from _parity import announce  # noqa: E402

DEV = "cuda:0"
U23 = 2.0 ** -23
TOL_LOGP = 2.0 ** -18  # the verification's own bound
ROW = 1 << 20          # workgroups of a row of a large grid


def i64(v):
    return torch.as_tensor(v, dtype=torch.int64, device=DEV)


class Adapters:
    """T requests of a row each."""

    def __init__(self, T, n, H, N, r):
        g = torch.Generator(device=DEV)
        g.manual_seed(T + H + N + r)
        normal = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV).normal_(generator=g)  # noqa: E731
        self.T, self.n, self.H, self.N, self.r = T, n, H, N, r
        self.x, self.dy, self.A, self.B = normal(T, H), normal(T, N), normal(n, r, H), normal(n, N, r)
        self.adapter = torch.randint(n, (T,), device=DEV, generator=g)
        self.scale = torch.empty(n, device=DEV).uniform_(0.5, 2.0, generator=g)

    def set(self):
        return dict(A=self.A, B=self.B, adapter=self.adapter, req_start=torch.arange(self.T + 1, device=DEV),
                    scale=self.scale, rank=None)

    def rows_of(self, a, lo, hi):
        return lo + (self.adapter[lo:hi] == a).nonzero()[:, 0]


def close(got, want, mag, K, label):
    assert ((got.double() - want).abs() <= (K + 8) * U23 * mag + U23 * want.abs() + 1e-30).all(), label


@pytest.mark.parametrize("T,N,r", [((1 << 21) + 40, 64, 8), ((1 << 21) + 40, 8, 40), ((1 << 21) + 40, 24, 128)])
def test_single_rows_forward(T, N, r):
    """8 T workgroups for y and T r / 16 for u, 2^24 at the most."""
    announce(f"large grids forward {T} rows, N {N}, r {r}")
    c = Adapters(T, 3, 8, N, r)
    # partial sums of u: the kernels of single rows
    assert lx.lx_lora_forward_workspace_bytes(T, T, 8, N, r) == T * r * 4
    y = torch.full((T, N), 55.0, device=DEV)
    lx.lx_lora_forward(c.x, base=None, y=y, **c.set())
    step = 1 << 19
    for lo in range(0, T, step):
        for a in range(c.n):
            rows = c.rows_of(a, lo, lo + step)
            x, A, B, s = c.x[rows].double(), c.A[a].double(), c.B[a].double(), c.scale[a].double()
            close(y[rows], s * (x @ A.T) @ B.T, s * (x.abs() @ A.abs().T) @ B.abs().T, c.H + r, f"rows from {lo}")


@pytest.mark.parametrize("T,H", [((1 << 20) + 8, 4104), (ROW // 2 + 64, 520)])
def test_single_rows_backward(T, H):
    """T ceil(H / 512) workgroups for dx (a multiple of 8 of them a row beyond 8)."""
    announce(f"large grids backward {T} rows of {H}")
    c = Adapters(T, 2, H, 8, 8)
    gx = torch.full((T, H), 55.0, device=DEV)
    gA, gB = torch.empty(2, 8, H, device=DEV), torch.empty(2, 8, 8, device=DEV)
    lx.lx_lora_backward(c.dy, c.x, base=None, grad_x=gx, grad_A=gA, grad_B=gB, **c.set())
    step = 1 << 16
    want = {k: [0.0, 0.0] for k in "AB"}
    mag = {k: [0.0, 0.0] for k in "AB"}
    for lo in range(0, T, step):
        for a in range(2):
            rows = c.rows_of(a, lo, min(lo + step, T))
            x, d, A, B = c.x[rows].double(), c.dy[rows].double(), c.A[a].double(), c.B[a].double()
            s = c.scale[a].double()
            v, u = s * (d @ B), s * (x @ A.T)
            close(gx[rows], v @ A, s * (d.abs() @ B.abs()) @ A.abs(), 16, f"dx, rows from {lo}")
            want["A"][a] += v.T @ x
            want["B"][a] += d.T @ u
            mag["A"][a] += (s * (d.abs() @ B.abs())).T @ x.abs()
            mag["B"][a] += d.abs().T @ (s * (x.abs() @ A.abs().T))
    for a in range(2):
        close(gA[a], want["A"][a], mag["A"][a], 8 + T, "dA")
        close(gB[a], want["B"][a], mag["B"][a], H + T, "dB")


@pytest.mark.parametrize("rows", ["single", "tiles"])
def test_many_adapters(rows):
    """3 * 2^19 workgroups of gradients, most of them of adapters that no row uses."""
    announce(f"large grids gradients {rows}")
    T, n, H, N, r = 4096, ROW // 2, 8, 264, 8
    c = Adapters(T, n, H, N, r)
    s = c.set()
    if rows == "tiles":
        c.adapter = torch.stack([c.adapter[0], i64(n - 1)]).repeat_interleave(T // 2)
        s.update(adapter=i64([int(c.adapter[0]), n - 1]), req_start=i64([0, T // 2, T]))
    else:
        c.adapter[T - 1] = n - 1
    gx, gA, gB = torch.empty(T, H, device=DEV), torch.empty(n, r, H, device=DEV), torch.empty(n, N, r, device=DEV)
    lx.lx_lora_backward(c.dy, c.x, base=None, grad_x=gx, grad_A=gA, grad_B=gB, **s)
    used = c.adapter.unique()
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[used] = False
    assert not gA[rest].any() and not gB[rest].any()
    for a in used[::1 if rows == "tiles" else 97].tolist() + [n - 1]:
        at = c.rows_of(a, 0, T)
        x, d, A, B = c.x[at].double(), c.dy[at].double(), c.A[a].double(), c.B[a].double()
        sc = c.scale[a].double()
        v, u = sc * (d @ B), sc * (x @ A.T)
        mv, mu = sc * (d.abs() @ B.abs()), sc * (x.abs() @ A.abs().T)
        close(gx[at], v @ A, mv @ A.abs(), N + r, "dx")
        close(gA[a], v.T @ x, mv.T @ x.abs(), N + T, "dA")
        close(gB[a], d.T @ u, d.abs().T @ mu, H + T, "dB")


def test_room_for_many_drafts():
    """4096 sequences of up to 4095 drafts, few of which there are: 33 million workgroups, position by position.  One
    greedy sequence is accepted up to its position 2600, which lies in the second half of them."""
    announce("large grids, room for many drafts")
    S, L, V, long, until = 4096, 4095, 16400, 2048, 2600
    rng = np.random.default_rng(3)
    lens = np.zeros(S, dtype=np.int64)
    lens[[0, 7, long, 4094, 4095]] = [3, 1, 2700, 2, 5]
    start = np.concatenate([[0], np.cumsum(lens)])
    N = int(start[-1])
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    z = torch.randn(N + S, V, device=DEV, generator=g) * 2
    u = torch.cat([z[start[i] + i:start[i + 1] + i] for i in range(S) if lens[i]])
    u = u + 0.5 * torch.randn(N, V, device=DEV, generator=g)
    x = (u.double().softmax(1).cumsum(1) < torch.rand(N, 1, device=DEV, generator=g)).sum(1).clamp(max=V - 1)
    first = int(start[long])
    x[first:first + until] = z[first + long:first + long + until].argmax(1)
    x[first + until] = (z[first + long + until].argmax() + 1) % V
    temps = np.ones(S, dtype=np.float32)
    temps[long] = 0.0
    ua, us = rng.random(N).astype(np.float32), rng.random(S).astype(np.float32)
    n, tok = torch.empty(S, dtype=torch.int64, device=DEV), torch.empty(S, L + 1, dtype=torch.int64, device=DEV)
    lp = torch.empty(S, L + 1, device=DEV)
    lx.lx_draft_verify(z, u, x, i64(start), L, torch.from_numpy(temps).to(DEV), torch.from_numpy(ua).to(DEV),
                       torch.from_numpy(us).to(DEV), n, tok, lp)
    assert n[long].item() == until
    assert torch.equal(tok[long, :until], x[first:first + until]) and not lp[long].any()
    assert tok[long, until].item() == z[first + long + until].argmax().item() and (tok[long, until + 1:] == -1).all()
    for i in [0, 1, 7, 8, 100, 2047, 2049, 4093, 4094, 4095]:
        s, e = int(start[i]), int(start[i + 1])
        a, out, logp = dv.verify_one(z[s + i:e + i + 1].cpu().numpy(), u[s:e].cpu().numpy(), x[s:e].cpu().numpy(), 1.0,
                                     ua[s:e], us[i])
        assert n[i].item() == a and tok[i, :a + 1].tolist() == out, i
        assert np.abs(lp[i, :a + 1].cpu().numpy() - logp).max() <= TOL_LOGP, i
        assert (tok[i, a + 1:] == -1).all() and (lp[i, a + 1:] == 0).all(), i


@pytest.mark.parametrize("L", [0, 1])
def test_many_sequences(L):
    """More sequences than a row of a large grid has workgroups; a draft for every other one."""
    announce(f"large grids, many sequences, {L} drafts")
    S, V = ROW + 3, 8
    rng = np.random.default_rng(5)
    lens = np.arange(S) % 2 * L
    start = np.concatenate([[0], np.cumsum(lens)])
    N = int(start[-1])
    z, u = rng.standard_normal((N + S, V)).astype(np.float32), rng.standard_normal((N, V)).astype(np.float32)
    x = rng.integers(0, V, N)
    ua, us = rng.random(N).astype(np.float32), rng.random(S).astype(np.float32)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    n, tok = torch.empty(S, dtype=torch.int64, device=DEV), torch.empty(S, L + 1, dtype=torch.int64, device=DEV)
    lp = torch.empty(S, L + 1, device=DEV)
    lx.lx_draft_verify(d(z), d(u) if L else None, d(x), d(start), L, None, d(ua), d(us), n, tok, lp)

    def softmax(a):
        e = np.exp(a.astype(np.float64) - a.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)

    p, q = softmax(z), softmax(u)
    row = start[:-1] + np.arange(S)                    # first target row of each sequence
    has = lens > 0
    accepted = np.zeros(S, dtype=np.int64)
    pick = np.arange(N)
    accepted[has] = ua.astype(np.float64) * q[pick, x] < p[row[has], x]
    mass = p[row + accepted]
    rejected = has & (accepted == 0)
    mass[rejected] = np.maximum(p[row[rejected]] - q[start[:-1][rejected]], 0)
    sums = mass.cumsum(1)
    drawn = (sums <= us.astype(np.float64)[:, None] * sums[:, -1:]).sum(1)
    want, logp = np.full((S, L + 1), -1, dtype=np.int64), np.zeros((S, L + 1))
    every = np.arange(S)
    if L:
        first = has & (accepted == 1)
        want[first, 0] = x[accepted[has] == 1]
        logp[first, 0] = np.log(p[row[first], want[first, 0]])
    want[every, accepted] = drawn
    logp[every, accepted] = np.log(p[row + accepted, drawn])
    assert np.array_equal(n.cpu().numpy(), accepted) and np.array_equal(tok.cpu().numpy(), want)
    assert np.abs(lp.cpu().numpy() - logp).max() <= TOL_LOGP
