"""The adapters, the loss and the verification of drafted tokens run one after another as they are used, on the GPU.

Training: the frozen head's product, the adapters beside it, the loss with its gradient over the logits, the gradient of
the head's input and of the adapters.  Every step is held to the float64 reference of that step on what the step before
it left, with that step's own tolerances, and the gradient of the whole run to differences of the whole run's loss in
float64.  The tolerance of the latter: the logits are rounded to bf16, so each is off by at most d = 2^-8 max|z| of its
row, and p by at most p (e^2d - 1); G is off by 2^-8 + 2^-10 of itself besides; both times the change of the logit
along the direction, summed, and 2^-12 of the same sum for the two products' fp32 sums and the differences.

Serving: the head's product, the adapters of each sequence, the verification; once eager, once in a graph."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import workloads as W
from oracle import draft_verify as dv
from oracle import lora

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cross_entropy_tv_amd as lx  # noqa: E402
from _parity import G_REL_P16, announce, check_forward, check_grad, grad_bits, grad_to_host  # noqa: E402

DEV = "cuda:0"
II = W.IGNORE_INDEX
U23 = 2.0 ** -23
TOL_LOGP = 2.0 ** -18  # the verification's own bound


def bf16(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16).to(DEV)


def f64(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


class Model:
    """A frozen head (V, H) with n adapters beside it."""

    def __init__(self, g, n, H, V, r):
        self.n, self.H, self.V, self.r = n, H, V, r
        self.W = bf16(g.standard_normal((V, H)) * H ** -0.5)
        self.A = bf16(g.standard_normal((n, r, H)) * H ** -0.5)
        self.B = bf16(g.standard_normal((n, V, r)) * 0.2)
        self.scale = torch.from_numpy(g.uniform(0.5, 1.5, n).astype(np.float32)).to(DEV)

    def logits(self, x, adapter, start, out):
        base = torch.empty(x.shape[0], self.V, device=DEV)
        lx.lx_gemm_bf16(x, True, self.W, True, base, x.shape[0], self.V, self.H)
        lx.lx_lora_forward(x, self.A, self.B, adapter, start, self.scale, None, base, out)

    def check_logits(self, x, adapter, start, out, label):
        base = f64(x) @ f64(self.W).T
        mag = np.abs(f64(x)) @ np.abs(f64(self.W)).T
        want, m, written = lora.forward(f64(x), f64(self.A), f64(self.B), adapter, start, f64(self.scale), None, base)
        assert written.all()
        half = 2.0 ** -8 if out.dtype == torch.bfloat16 else U23
        tol = (self.H + self.r + 8) * U23 * (mag + m) + half * np.abs(want) + 1e-30
        assert (np.abs(f64(out) - want) <= tol).all(), f"{label}: logits"


def train(m, x, teacher, target, adapter, start, g_ce, g_tvd):
    """(logits as the loss saw them, loss outputs, G, gx, gA, gB)."""
    T = x.shape[0]
    z = torch.empty(T, m.V, dtype=torch.bfloat16, device=DEV)
    m.logits(x, adapter, start, z)
    seen = z.clone()
    f = lambda: torch.full((T,), float("nan"), device=DEV)  # noqa: E731
    out = {k: f() for k in ("ce", "tvd", "lse_s", "lse_t", "sigma")}
    lx.lx_ce_tvd_forward_backward(z, teacher, target, II, *out.values(), z, g_ce, g_tvd)  # in place: z becomes G
    gx = torch.empty(T, m.H, device=DEV)
    lx.lx_gemm_bf16(z, True, m.W, False, gx, T, m.H, m.V)
    gA, gB = torch.empty(m.n, m.r, m.H, device=DEV), torch.empty(m.n, m.V, m.r, device=DEV)
    lx.lx_lora_backward(z, x, m.A, m.B, adapter, start, m.scale, None, gx, gx, gA, gB)
    return seen, out, z, gx, gA, gB


@pytest.mark.parametrize("T,H,V,r", [(33, 136, 520, 8), (300, 264, 2056, 16), (1500, 520, 1032, 40)])
def test_a_training_step(T, H, V, r):
    announce(f"training step {T} x {H} x {V}, rank {r}")
    g = np.random.default_rng(T)
    m = Model(g, 3, H, V, r)
    x, teacher = bf16(g.standard_normal((T, H))), bf16(g.standard_normal((T, V)) * 2)
    start, adapter = [0, T // 3, T // 3, T // 2, T], [1, 0, -1, 2]
    target = g.integers(0, V, T)
    target[::7] = II
    gs = 1.0 / int((target != II).sum())
    z, out, G, gx, gA, gB = train(m, x, teacher, torch.from_numpy(target).to(DEV), i64(adapter), i64(start), gs, gs)
    torch.cuda.synchronize()
    m.check_logits(x, adapter, start, z, "training step")
    out = {k: v.cpu().numpy() for k, v in out.items()}
    check_forward(out, bits(z), bits(teacher), target, II, "training step")
    check_grad(grad_to_host(G), grad_bits(G), bits(z), bits(teacher), target, II, gs, gs, "training step",
               rel=G_REL_P16, sigma_gpu=out["sigma"])
    (dx, dA, dB), (mx, mA, mB), _ = lora.backward(f64(G), f64(x), f64(m.A), f64(m.B), adapter, start, f64(m.scale), None,
                                                 f64(G) @ f64(m.W))
    mx = mx + np.abs(f64(G)) @ np.abs(f64(m.W))
    for got, want, mag, K, name in ((gx, dx, mx, V + r, "dx"), (gA, dA, mA, V + T, "dA"), (gB, dB, mB, H + T, "dB")):
        assert (np.abs(f64(got) - want) <= (K + 8) * U23 * mag + U23 * np.abs(want) + 1e-30).all(), name


def test_a_training_step_against_differences():
    """Cross-entropy alone (the distance has kinks): the loss of the whole run in float64, along random directions of
    the adapters and of x."""
    announce("training step against differences")
    T, H, V, r = 24, 72, 136, 8
    g = np.random.default_rng(5)
    m = Model(g, 2, H, V, r)
    x = bf16(g.standard_normal((T, H)))
    start, adapter, target = [0, 10, T], [1, 0], g.integers(0, V, T)
    _, _, _, gx, gA, gB = train(m, x, None, torch.from_numpy(target).to(DEV), i64(adapter), i64(start), 1.0 / T, 0.0)
    x0, A0, B0, s0, head = f64(x), f64(m.A), f64(m.B), f64(m.scale), f64(m.W)

    def logits(x, A, B):
        return lora.forward(x, A, B, adapter, start, s0, None, x @ head.T)[0]

    def loss(x, A, B):
        z = logits(x, A, B)
        top = z.max(1, keepdims=True)
        return (np.log(np.exp(z - top).sum(1)) + top[:, 0] - z[np.arange(T), target]).mean()

    z = logits(x0, A0, B0)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    G = (p - (np.arange(V) == target[:, None])) / T
    d = 2.0 ** -8 * np.abs(z).max(1, keepdims=True)
    off = p / T * np.expm1(2 * d) + np.abs(G) * (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12)
    h, told = 2.0 ** -16, 0
    for k, (grad, at) in enumerate(((gx, x0), (gA, A0), (gB, B0))):
        grad = f64(grad)
        for D in (grad / np.linalg.norm(grad), g.standard_normal(at.shape) / at.size ** 0.5):
            step = [np.zeros_like(a) for a in (x0, A0, B0)]
            step[k] = h * D
            up, down = ([a + sign * s for a, s in zip((x0, A0, B0), step)] for sign in (1, -1))
            want = (loss(*up) - loss(*down)) / (2 * h)
            tol = (off * np.abs(logits(*up) - logits(*down)) / (2 * h)).sum()
            assert abs((grad * D).sum() - want) <= tol, (k, want)
            told += abs(want) > 8 * tol
    assert told >= 3  # the gradient's own direction is told from 0 for each of the three


def serve(m, x, dx, tokens, start, max_draft, adapter, temps, ua, us, out):
    """Target and draft logits of every position, then the verification; a sequence's request holds its drafts' rows
    and one more."""
    S, N = len(us), len(tokens)
    rows = start + torch.arange(S + 1, device=DEV)
    z = torch.empty(N + S, m.V, dtype=torch.bfloat16, device=DEV)
    m.logits(x, adapter, rows, z)
    q32 = torch.empty(N, m.V, device=DEV)
    lx.lx_gemm_bf16(dx, True, m.W, True, q32, N, m.V, m.H)
    q = q32.to(torch.bfloat16)
    lx.lx_draft_verify(z, q, tokens, start, max_draft, temps, ua, us, *out)
    return z, q


def test_serving_steps():
    g = np.random.default_rng(9)
    lens = [3, 0, 1, 5, 2, 0, 4]
    S, N, H, V, longest = len(lens), sum(lens), 136, 4104, 5
    m = Model(g, 4, H, V, 16)
    start = np.concatenate([[0], np.cumsum(lens)])
    adapter = [2, -1, 0, 3, 3, 1, -1]
    temps = torch.tensor([1.0, 0.7, 0.0, 1.3, 1.0, 1.0, 0.9], device=DEV)
    x, dx = torch.empty(N + S, H, dtype=torch.bfloat16, device=DEV), torch.empty(N, H, dtype=torch.bfloat16, device=DEV)
    ua, us = torch.empty(N, device=DEV), torch.empty(S, device=DEV)
    tokens = torch.empty(N, dtype=torch.int64, device=DEV)
    out = (torch.empty(S, dtype=torch.int64, device=DEV), torch.empty(S, longest + 1, dtype=torch.int64, device=DEV),
           torch.empty(S, longest + 1, device=DEV))
    dstart, dadapter = i64(start.tolist()), i64(adapter)

    def inputs(seed):
        g = np.random.default_rng(seed)
        hidden = g.standard_normal((N + S, H)) * 2
        x.copy_(bf16(hidden))
        drafted = np.concatenate([hidden[start[i] + i:start[i + 1] + i] for i in range(S)])
        dx.copy_(bf16(drafted + 0.2 * g.standard_normal((N, H))))
        ua.copy_(torch.from_numpy(g.random(N).astype(np.float32)))
        us.copy_(torch.from_numpy(g.random(S).astype(np.float32)))
        best = torch.topk(dx.float() @ m.W.float().T, 3, dim=1).indices.cpu().numpy()
        tokens.copy_(torch.from_numpy(best[np.arange(N), g.integers(0, 3, N)]))

    def step():
        return serve(m, x, dx, tokens, dstart, longest, dadapter, temps, ua, us, out)

    def check(z, q, label):
        announce(f"serving {label}")
        m.check_logits(x, adapter, (start + np.arange(S + 1)).tolist(), z, label)
        n, tok, lp = dv.verify(f64(z), f64(q), tokens.cpu().numpy(), start, longest, temps.cpu().numpy(),
                               ua.cpu().numpy(), us.cpu().numpy())
        assert np.array_equal(out[0].cpu().numpy(), n) and np.array_equal(out[1].cpu().numpy(), tok), label
        assert np.abs(out[2].cpu().numpy() - lp).max() <= TOL_LOGP, label
        return n

    inputs(0)
    accepted = check(*step(), "eager").sum()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z, q = step()
    for k in range(1, 5):
        inputs(k)
        for o in out:
            o.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        accepted += check(z, q, f"replay {k}").sum()
        step()  # eager work between replays
        torch.cuda.synchronize()
    assert 0 < accepted < 5 * N


def test_calls_at_once():
    """Training and serving on two streams at once, each call with a workspace of its own: the results of one at a time."""
    announce("calls at once")
    g = np.random.default_rng(21)
    m = Model(g, 3, 264, 2056, 16)
    T = 400
    x, teacher = bf16(g.standard_normal((T, 264))), bf16(g.standard_normal((T, 2056)) * 2)
    start, adapter = i64([0, 90, 260, T]), i64([1, 0, 2])
    target = torch.from_numpy(g.integers(0, 2056, T)).to(DEV)
    S, L = 6, 3
    hidden, drafted = bf16(g.standard_normal((S * (L + 1), 264)) * 2), bf16(g.standard_normal((S * L, 264)) * 2)
    tokens = torch.from_numpy(g.integers(0, 2056, S * L)).to(DEV)
    dstart, who = torch.arange(S + 1, device=DEV) * L, i64([0, 1, 2, -1, 1, 0])
    ua, us = torch.rand(S * L, device=DEV), torch.rand(S, device=DEV)

    def training():
        return train(m, x, teacher, target, adapter, start, 1.0 / T, 1.0 / T)[3:]

    def serving():
        out = (torch.empty(S, dtype=torch.int64, device=DEV), torch.empty(S, L + 1, dtype=torch.int64, device=DEV),
               torch.empty(S, L + 1, device=DEV))
        serve(m, hidden, drafted, tokens, dstart, L, who, torch.ones(S, device=DEV), ua, us, out)
        return out

    want = training(), serving()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for k in range(8):
        for st, run in zip(streams, (training, serving) if k % 2 else (serving, training)):
            with torch.cuda.stream(st):
                got.append((run is serving, run()))
    torch.cuda.synchronize()
    for which, out in got:
        for a, b in zip(out, want[which]):
            assert torch.equal(a, b)
