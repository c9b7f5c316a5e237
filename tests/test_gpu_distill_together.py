"""The top logits, the loss trained from them and both of its forms run together, as a training step has them: the
teacher's logits through lx_gemm_bf16, lx_top_logits, then the student's step over stored logits (in place) and through the
lm_head's weight.

Tolerance between the two forms, element by element, of grad_x = G w (and grad_w = G^T x): the form through the weight
rounds G to bf16 (2^-8 |G|); its logits are the same 256 products added in another order (256 * 2^-24 * sum |x w| <= 2^-16 *
64 = 2^-10 each side at these sizes, 2^-9 of both, over T = 2 and through two exponentials with log-sums: 2^-8 of the
sizes of the terms that G is the sum of); sums of up to 2003 products in fp32 add 2003 * 2^-24 < 2^-13 of their sizes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cross_entropy_tv_amd as lx  # noqa: E402
from _kd import DEV, IGN, TOL_LOG, TOL_LOSS, Case, near  # noqa: E402
from oracle import kd as oracle  # noqa: E402


class Run:
    """A padded batch: the last `pad` rows are behind the last sequence."""

    def __init__(self, seed, BT=48, V=2003, H=256, K=32, T=2.0, pad=7):
        g = torch.Generator().manual_seed(seed)
        bf = lambda *s, k=1.0: (torch.randn(*s, generator=g).clamp(-3, 3) * k).to(torch.bfloat16).to(DEV)  # noqa: E731
        self.BT, self.V, self.H, self.K, self.T, self.pad, self.g = BT, V, H, K, T, pad, (0.6, 1.4)
        self.xt, self.x = bf(BT, H), bf(BT, H)
        self.wt, self.w = bf(V, H, k=0.15), bf(V, H, k=0.15)
        self.target = torch.randint(0, V, (BT,), generator=g)
        self.target[BT - pad:] = IGN
        self.target = self.target.to(DEV)
        f = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
        u8 = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)  # noqa: E731
        self.zt, self.z, self.G = f(BT, V), f(BT, V), f(BT, V)
        self.top, self.ids, self.rest = f(BT, K), torch.empty(BT, K, dtype=torch.int32, device=DEV), f(BT)
        self.a = [f(BT), f(BT), f(BT), f(BT, 4)]
        self.b = [f(BT), f(BT), f(BT), f(BT, 4)]
        self.gx, self.gw = f(BT, H), f(V, H)
        self.ws_top = u8(lx.lx_top_logits_workspace_bytes(BT, V, K))
        self.ws_step = u8(lx.lx_ce_kd_forward_backward_workspace_bytes(BT, V, lx.LX_F32))
        self.piece = 512
        self.ws_lin = u8(lx.lx_ce_kd_linear_workspace_bytes(BT, V, H, K, self.piece, True))

    def __call__(self):
        lx.lx_gemm_bf16(self.xt, True, self.wt, True, self.zt, self.BT, self.V, self.H)
        lx.lx_top_logits(self.zt, self.T, self.top, self.ids, None, self.rest, workspace=self.ws_top)
        lx.lx_gemm_bf16(self.x, True, self.w, True, self.z, self.BT, self.V, self.H)
        self.G.copy_(self.z)
        teacher = (self.target, IGN, self.ids, self.top, self.rest, self.T)
        lx.lx_ce_kd_forward_backward(self.G, *teacher, *self.a, self.G, *self.g, workspace=self.ws_step)
        lx.lx_ce_kd_linear_forward_backward(self.x, self.w, *teacher, *self.b, self.gx, self.gw, *self.g, piece=self.piece,
                                            workspace=self.ws_lin)

    def outputs(self):
        return [self.top, self.ids, self.rest, *self.a, *self.b, self.G, self.gx, self.gw]

    def check(self):
        z, zt = self.z.cpu().numpy(), self.zt.cpu().numpy()
        target = self.target.cpu().numpy()
        top, ids, rest = self.top.cpu().numpy(), self.ids.cpu().numpy(), self.rest.cpu().numpy()
        G = self.G.double().cpu().numpy()
        size = np.zeros_like(G)
        for r in range(self.BT):
            want_top, want_ids, _, want_rest = oracle.top_row(zt[r], self.K, self.T)
            assert (top[r] == want_top).all() and (ids[r] == want_ids).all(), r
            near(rest[r], want_rest, TOL_LOG, f"rest[{r}]")
            if target[r] == IGN:
                assert not G[r].any() and not self.gx[r].any()
                assert all(not o[r].any() for o in self.a + self.b)
                continue
            row = oracle.Row(z[r], target[r], ids[r], top[r], rest[r], self.T)
            near(self.a[0][r].item(), row.ce, TOL_LOSS, f"ce[{r}]")
            near(self.a[1][r].item(), row.kd, TOL_LOSS, f"kd[{r}]")
            size[r] = row.grad(*(float(np.float32(k)) for k in self.g))[1]
        for x, y in zip(self.a, self.b):  # (logits 2^-9 apart)
            assert (x - y).abs().max() <= 2.0 ** -8
        off = 2.0 ** -8 * np.abs(G) + 2.0 ** -8 * size
        w, x = self.w.double().cpu().numpy(), self.x.double().cpu().numpy()
        for got, want, bound in (
                (self.gx, G @ w, off @ np.abs(w) + 2.0 ** -13 * (np.abs(G) @ np.abs(w))),
                (self.gw, G.T @ x, off.T @ np.abs(x) + 2.0 ** -13 * (np.abs(G).T @ np.abs(x)))):
            assert (np.abs(got.double().cpu().numpy() - want) <= bound + 1e-30).all()


def test_a_training_step():
    run = Run(1)
    run()
    torch.cuda.synchronize()
    run.check()


def test_captured_steps_in_turn():
    """Two steps captured with a workspace each, replayed in turn and at once on two streams while their weights change,
    against the same steps run eagerly."""
    runs, graphs = [Run(2), Run(3, BT=21, V=1500, K=9, pad=2)], []
    for run in runs:
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in runs]
    for k in range(4):
        want = []
        for run in runs:
            run.w -= (0.05 * run.gw).to(torch.bfloat16)
            run.x.mul_(-1.0)
            run()
            want.append([o.clone() for o in run.outputs()])
            for o in run.outputs():
                o.fill_(k)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            if k % 2:
                with torch.cuda.stream(s):
                    graph.replay()
            else:
                graph.replay()
        torch.cuda.synchronize()
        for run, outs in zip(runs, want):
            for o, e in zip(run.outputs(), outs):
                assert torch.equal(o, e)


def test_a_step_learns_nothing_from_itself():
    """A student equal to its teacher: no divergence, and with cross entropy left out no gradient (2^-14: two log-sums of
    each side; a rest as one more token)."""
    run = Run(4, pad=0)
    run.wt.copy_(run.w)
    run.xt.copy_(run.x)
    run.g = (0.0, 1.0)
    run()
    torch.cuda.synchronize()
    assert run.a[1].abs().max() <= 2.0 ** -14 and run.G.abs().max() <= 2.0 ** -14


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_the_most_entries_over_long_rows(dt, T):
    c = Case(40, 3, 151936, 256, dt, T=T, scale=1.0).place()
    c.step(lx, c.gd)
    c.check_loss()
    c.check_grad(c.gd)
    c.forward(lx)
    c.backward(lx, c.gd)
    c.check_loss()
    c.check_grad(c.gd)


@pytest.mark.parametrize("V", [5003, 70001])
def test_rows_past_32_bits(V):
    """Rows that start 2^32 elements and more into their buffers: the results of the same rows side by side, bit for bit."""
    BT, K, ld = 4, 20, 3 << 29
    c = Case(41, BT, V, K, "bf16", T=2.0).place()
    c.step(lx, c.gd)
    torch.cuda.synchronize()
    want = [o.clone() for o in c.out] + [c.gd.clone()]
    buf = torch.empty((BT - 1) * ld + V, dtype=torch.bfloat16, device=DEV)
    far = buf.as_strided((BT, V), (ld, 1))
    far.copy_(c.zd)
    top = []
    for z in (c.zd, far):
        t, i, rest = torch.empty(BT, K, device=DEV), torch.empty(BT, K, dtype=torch.int32, device=DEV), torch.empty(BT, device=DEV)
        lx.lx_top_logits(z, 2.0, t, i, None, rest)
        top.append((t, i, rest))
    for a, b in zip(*top):
        assert torch.equal(a, b)
    c.zd = far
    c.forward(lx)
    for a, b in zip(c.out[:3], want[:3]):
        assert (a - b).abs().max() <= 2 * TOL_LOSS
    c.backward(lx, c.gd)
    torch.cuda.synchronize()
    c.check_grad(c.gd)
    c.step(lx, far)
    torch.cuda.synchronize()
    for a, b in zip([*c.out, far], want):
        assert torch.equal(a, b)
