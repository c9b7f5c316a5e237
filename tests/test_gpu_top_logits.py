"""The K largest logits of every row on the GPU against the float64 reference.  Values and ids are what comparisons
of exact numbers decide and must be equal.  The log-sums are held to 2^-16 as derived in _kd.py for logits of at most 32 in
size at T >= 1/2, and beyond that size to the same share of their exponents."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cross_entropy_tv_amd as lx  # noqa: E402
from _kd import DEV, DT, NINF, around, on_device  # noqa: E402
from _parity import announce  # noqa: E402
from oracle import kd as oracle  # noqa: E402

F32_MIN, BF16_MIN = -3.4028235e38, -3.3895314e38


class Top:
    def __init__(self, z, K, dt="bf16", T=1.0, pad=0, offset=0):
        self.z = torch.from_numpy(np.asarray(z, np.float32)).to(DT[dt]).float().numpy()
        self.K, self.T, self.pad, self.offset = K, T, pad, offset
        self.zd, self.buf = on_device(self.z, DT[dt], pad, offset)
        BT = len(self.z)
        self.top = torch.full((BT, K), 99.0, device=DEV)
        self.ids = torch.full((BT, K), 99, dtype=torch.int32, device=DEV)
        self.lse, self.rest = (torch.full((BT,), 99.0, device=DEV) for _ in range(2))

    def run(self, **kw):
        announce(f"top {tuple(self.z.shape)} K {self.K} {self.zd.dtype} T {self.T}")
        lx.lx_top_logits(self.zd, self.T, self.top, self.ids, self.lse, self.rest, **kw)
        return self

    def check(self, tol=2.0 ** -16, rows=None):
        top, ids = self.top.cpu().numpy(), self.ids.cpu().numpy()
        lse, rest = self.lse.double().cpu().numpy(), self.rest.double().cpu().numpy()
        for r in range(len(self.z)) if rows is None else rows:
            want = oracle.top_row(self.z[r], self.K, self.T)
            assert np.array_equal(ids[r], want[1]), (r, ids[r], want[1])
            assert np.array_equal(top[r], want[0]), r
            for got, w in ((lse[r], want[2]), (rest[r], want[3])):
                assert got == w if np.isinf(w) else abs(got - w) <= tol, (r, got, w)


def normal(seed, BT, V, scale=3.0):
    return np.clip(np.random.default_rng(seed).standard_normal((BT, V)) * scale, -30, 30).astype(np.float32)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("BT,V,K", [(1, 1, 1), (2, 1, 4), (3, 7, 3), (3, 8, 8), (4, 9, 256), (3, 300, 256), (5, 2048, 20),
                                    (5, 2049, 256), (4, 2056, 1), (3, 32768, 64), (2, 32769, 64), (2, 40000, 256),
                                    (2, 151936, 20), (1, 262144, 100), (1, 300001, 256)])
def test_sizes(dt, BT, V, K):
    Top(normal(1, BT, V), K, dt).run().check()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("BT,V,K", [(130, 70001, 50), (300, 3000, 256), (129, 151936, 256), (2050, 600, 5)])
def test_a_workgroup_a_row(dt, BT, V, K):
    Top(normal(2, BT, V), K, dt).run().check(rows=range(0, BT, 1 + BT // 40))


@pytest.mark.parametrize("T", [0.5, 2.0, 7.0])
def test_temperatures(T):
    Top(normal(3, 3, 5001), 17, "f32", T).run().check()
    Top(normal(3, 200, 5001), 17, "bf16", T).run().check(rows=range(0, 200, 9))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 3), (0, 5), (3, 7)])
def test_strides_and_alignment(dt, pad, offset):
    for BT in (3, 140):
        c = Top(normal(4, BT, 4099), 33, dt, pad=pad, offset=offset).run()
        c.check(rows=range(0, BT, 1 + BT // 20))
        assert (around(c.buf, BT, 4099, pad, offset) == 77).all()


def shapes_of_rows(V):
    """Rows that fill the list at once or again and again, and their kin."""
    i = np.arange(V)
    rng = np.random.default_rng(5)
    few = np.where(rng.random(V) < 0.5, 1.0, 2.0)
    waves = np.where((i // 32768) % 2 == 0, -20.0, 20.0) + 0.25 * (i % 5)
    return np.stack([np.zeros(V), i * (20.0 / V), -i * (20.0 / V), few, waves, np.where(i == V - 1, 5.0, 0.0),
                     np.where(i < V - 300, NINF, 1.0), np.where(i % 2 == 0, -0.0, 0.0), -20.0 + (i % 7),
                     np.full(V, -30.0), np.sort(rng.standard_normal(V) * 3)])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V,K", [(2500, 256), (9000, 64), (33000, 1), (70001, 256), (151936, 64)])
def test_ties_and_order(dt, V, K):
    z = shapes_of_rows(V).astype(np.float32)
    Top(z, K, dt).run().check()
    many = np.tile(z, (12, 1))  # a workgroup a row
    Top(many, K, dt).run().check(rows=list(range(11)) + [121, 127, 131])


@pytest.mark.parametrize("low", [NINF, BF16_MIN])
@pytest.mark.parametrize("BT", [6, 132])
def test_masked_rows(low, BT):
    z = normal(6, BT, 9000)
    z[0] = low                    # nothing
    z[1] = low
    z[1, 8888] = 1.0              # one
    z[2, :8192] = low
    z[3, 10:] = low               # fewer than K
    z[4, ::2] = low
    z[5, 40:] = low               # exactly K
    Top(z, 40, "bf16").run().check()
    z[0, 0] = F32_MIN
    Top(z, 40, "f32", 2.0).run().check()


def test_rest_that_vanishes():
    """The rest lies 2^-300 below the top: its log-sum is still good."""
    z = normal(7, 3, 6000) - 25.0
    z[:, 100:110] = 190.0
    # exponents of 280 (2^9, two powers of two above _kd.py's): 2^-14
    Top(z, 10, "f32").run().check(tol=2.0 ** -14)
    Top(z, 4, "f32").run().check(tol=2.0 ** -14)


def test_binary16_lowest_is_a_logit():
    z = np.full((2, 300), -65504.0, np.float32)
    z[0, 7] = 3.0
    c = Top(z, 5, "f16").run()
    assert c.ids.tolist() == [[7, 0, 1, 2, 3], [0, 1, 2, 3, 4]]
    # half a step of 65504 in fp32, 2^-8
    assert abs(float(c.lse[1]) - (-65504 + np.log(300))) <= 2.0 ** -7


def test_outputs_that_are_not_wanted():
    c = Top(normal(8, 3, 5000), 20)
    lx.lx_top_logits(c.zd, 1.0, c.top, c.ids)
    assert (c.lse == 99).all() and (c.rest == 99).all()
    a = c.top.clone()
    lx.lx_top_logits(c.zd, 1.0, c.top, c.ids, None, c.rest)
    c.lse.copy_(torch.from_numpy(np.array([oracle.top_row(z, 20, 1.0)[2] for z in c.z])))
    assert torch.equal(a, c.top)
    c.check()


@pytest.mark.parametrize("BT", [2, 200])
def test_deterministic_graph_and_streams(BT):
    z = np.concatenate([normal(9, BT, 33333), ])
    z[0] = np.arange(33333) / 2000.0
    c = Top(z, 100, "f32").run()
    first = [t.clone() for t in (c.top, c.ids, c.lse, c.rest)]
    ws = torch.empty(max(256, lx.lx_top_logits_workspace_bytes(BT, 33333, 100)), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.run(stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(workspace=ws)
    for k in range(5):
        for t in (c.top, c.ids, c.lse, c.rest):
            t.fill_(k)
        ws.fill_(255 * (k % 2))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(first, (c.top, c.ids, c.lse, c.rest)):
            assert torch.equal(x, y)


def test_the_loss_trains_from_it():
    """The selection's outputs as the loss's teacher: a student equal to the teacher has nothing to learn."""
    for T in (1.0, 2.0):
        z = normal(10, 40, 5003)
        c = Top(z, 30, "f32", T).run()
        BT = 40
        target = torch.zeros(BT, dtype=torch.int64, device=DEV)
        ce, kd, lse = (torch.empty(BT, device=DEV) for _ in range(3))
        state, grad = torch.empty(BT, 4, device=DEV), torch.empty_like(c.zd)
        lx.lx_ce_kd_forward_backward(c.zd, target, -100, c.ids, c.top, c.rest, T, ce, kd, lse, state, grad, 0.0, 1.0)
        # two log-sums of each side and their roundings
        assert kd.abs().max() <= 4 * 2.0 ** -16
        assert grad.abs().max() <= 4 * 2.0 ** -16
