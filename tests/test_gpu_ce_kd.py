"""Cross entropy with distillation from a teacher's top logits on the GPU against the float64 reference
(tolerances: _kd.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cross_entropy_tv_amd as lx  # noqa: E402
import _kd  # noqa: E402
from _kd import IGN, NINF, Case, oracle, run_all  # noqa: E402

F32_MIN, BF16_MIN, F16_MIN = -3.4028235e38, -3.3895314e38, -65504.0


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("BT,V,K", [(1, 1, 1), (3, 7, 3), (5, 8, 2), (4, 9, 9), (2, 300, 256), (3, 1024, 8), (7, 4097, 33),
                                    (2, 12345, 64), (3, 32768, 20), (2, 33000, 5)])
def test_sizes(dt, BT, V, K):
    run_all(lx, Case(1, BT, V, K, dt))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [0.5, 2.0, 4.0])
@pytest.mark.parametrize("BT,V,K", [(2, 61, 6), (3, 4100, 40), (2, 70001, 64)])
def test_temperatures(dt, T, BT, V, K):
    run_all(lx, Case(2, BT, V, K, dt, T=T, ignored=(1,)))


@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_top_alone(T, dt):
    run_all(lx, Case(3, 4, 5000, 20, dt, T=T, rest=False))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1.0, 3.0])
def test_many_rows(dt, T):
    """A workgroup a row."""
    run_all(lx, Case(4, 600, 777, 12, dt, T=T, ignored=(0, 17, 599), rows=True, g_scale=1 / 600))


@pytest.mark.parametrize("dt,V", [("bf16", 151936), ("f32", 262144), ("f16", 300001), ("bf16", 530000)])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_long_rows(dt, V, T):
    run_all(lx, Case(5, 2, V, 64, dt, T=T))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,offset", [((1, 3), (0, 0)), ((8, 8), (1, 1)), ((0, 5), (3, 2)), ((2, 2), (7, 7))])
def test_strides_and_alignment(dt, pad, offset):
    c = Case(6, 5, 2051, 16, dt, pad=pad, offset=offset, ignored=(2,))
    c.place()
    c.forward(lx)
    c.check_loss()
    c.backward(lx, c.gd)
    c.check_grad(c.gd)
    c.check_around()
    c.place()
    c.step(lx, c.gd)
    c.check_loss()
    c.check_grad(c.gd)
    c.check_around()


def test_rows_with_factors():
    run_all(lx, Case(7, 6, 3000, 24, "f32", rows=True, g_scale=0.25, ignored=(3,)))
    run_all(lx, Case(8, 6, 3000, 24, "f32", g=(0.0, 1.0)))
    run_all(lx, Case(9, 6, 3000, 24, "f32", g=(1.0, 0.0), T=2.0))


def test_targets_and_ids_that_are_no_tokens():
    def edit(c):
        c.target[:4] = [IGN, -1, c.V, 5]
        c.ids[3, :6] = -1            # left out
        c.ids[4, 2] = c.V            # past the vocabulary: NaN
        c.ids[5, :] = -7             # nothing named: the rest alone
        c.ids[6, 3] = c.ids[6, 0]    # twice
        c.ids[7, :] = c.ids[7, 0]
        c.top[8, :] = NINF
        c.top[9, 1] = F32_MIN
        c.ids[10] = c.ids[10][::-1].copy()  # any order
        c.top[10] = c.top[10][::-1].copy()
        c.target[11] = c.ids[11, 2]
    for rest in (True, False):
        for T in (1.0, 2.0):
            for V in (900, 9000):
                run_all(lx, Case(10, 13, V, 12, "f32", T=T, rest=rest, edit=edit))


@pytest.mark.parametrize("dt,low", [("bf16", NINF), ("bf16", BF16_MIN), ("f32", NINF), ("f32", F32_MIN), ("f16", NINF)])
@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("V", [600, 40000])
def test_masked_tokens(dt, low, T, V):
    def edit(c):
        keep = np.zeros(V, bool)
        keep[c.ids[0]] = True
        c.z[0, ~keep] = low                     # nothing outside the ids
        c.z[1, :] = low                         # nothing at all
        c.z[2, :V // 2] = low                   # the first groups of every thread
        c.target[2] = V - 1
        c.z[3, c.ids[3, 0]] = low               # named and masked: kd +inf
        c.z[4, c.target[4]] = low               # a masked target: ce +inf
        c.z[5, :] = low
        c.z[5, 11] = 2.0                        # one token left
        c.target[5] = 11
        c.ids[5, :] = -1
        c.rest[6] = F32_MIN
        c.z[7, V - V // 3:] = low
    run_all(lx, Case(11, 9, V, 10, dt, T=T, edit=edit))


def test_binary16_lowest_is_a_logit():
    def edit(c):
        c.z[0, 10:] = F16_MIN
        c.z[1, :] = F16_MIN
    c = Case(12, 3, 500, 4, "f16", edit=edit).place()
    c.forward(lx)
    c.check_loss(rows=[0, 2])
    # a row of equal logits: the log-sum is their value and log V, to half a step of the value (2^-8 of 65504)
    assert abs(float(c.out[2][1]) - (F16_MIN + np.log(500))) <= 2.0 ** -7
    c.backward(lx, c.gd)
    c.check_grad(c.gd, rows=[0, 2])


@pytest.mark.parametrize("T", [1.0, 2.0])
def test_outside_vanishes(T):
    """p_r far below the smallest fp32: its logarithm still counts, and the gradient outside is q_r's."""
    def edit(c):
        c.z[:] = -25.0
        for r in range(c.BT):
            c.z[r, c.ids[r, 0]] = 200.0
            c.target[r] = c.ids[r, 0]
    c = Case(13, 3, 5000, 8, "f32", T=T, edit=edit).place()
    c.forward(lx)
    for r in range(3):
        want = c.row(r)
        # exponents of up to 290 (2^9): two powers of two above the tolerances of _kd.py
        assert abs(float(c.out[1][r]) - want.kd) <= 2.0 ** -13
        assert want.kd > 1.0
    c.backward(lx, c.gd)
    a = c.gd.clone()
    c.place()
    c.step(lx, c.gd)
    for got in (a, c.gd):
        for r in range(3):
            want, size = c.row(r).grad(*c.g)
            assert (np.abs(got[r].double().cpu().numpy() - want) <= 2.0 ** -13 * size + 2.0 ** -125).all()


def test_a_thread_whose_first_group_is_low():
    """Sums against a first group far below the rest are redone."""
    def edit(c):
        c.z[:, :c.V // 2] = -30.0
        c.z[:, c.V // 2:] = 30.0
        c.z[1] = c.z[1][::-1].copy()
        c.z[2, ::2] = 30.0
        c.z[2, 1::2] = -30.0
    for T in (1.0, 0.5):
        for dt in ("bf16", "f32"):
            run_all(lx, Case(14, 4, 20011, 16, dt, T=T, edit=edit))


def test_gradient_against_differences():
    c = Case(15, 2, 40, 6, "f32", T=2.0).place()
    c.step(lx, c.gd)
    h = 1e-4
    got = c.gd.double().cpu().numpy()
    for r in range(2):
        for v in range(40):
            a, b = c.z[r].astype(np.float64), c.z[r].astype(np.float64)
            a[v] += h
            b[v] -= h
            args = (c.target[r], c.ids[r], c.top[r], c.rest[r], c.T, *c.g)
            d = (oracle.loss(a, *args) - oracle.loss(b, *args)) / (2 * h)
            # the kernel's own bound (sizes at most 0.7 (1 + 1) + 1.3), the differences' h^2 and their rounding
            assert abs(got[r, v] - d) <= 4 * 2.0 ** -15 + 4 * h * h + 1e-14 / h


@pytest.mark.parametrize("BT,V", [(3, 4000), (3, 151936), (700, 1500)])
def test_deterministic(BT, V):
    c = Case(16, BT, V, 40, "bf16", T=2.0, edit=lambda c: c.ids.__setitem__((0, slice(1, 9)), c.ids[0, 0])).place()
    first = None
    for _ in range(5):
        c.forward(lx)
        c.backward(lx, c.gd)
        got = [o.clone() for o in c.out] + [c.gd.clone()]
        c.step(lx, c.gd)
        got += [o.clone() for o in c.out] + [c.gd.clone()]
        if first is not None:
            for x, y in zip(first, got):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        first = got


def test_streams_and_graphs():
    """On another stream than the current one, and captured and replayed among other work."""
    for BT, V in ((4, 3000), (3, 151936)):
        c = Case(17, BT, V, 16, "bf16", g_scale=0.5).place()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        c.step(lx, c.gd, stream=s)
        s.synchronize()
        c.check_loss()
        c.check_grad(c.gd)
        eager = c.gd.clone()
        code = lx.LX_BF16
        ws = torch.empty(max(256, lx.lx_ce_kd_forward_backward_workspace_bytes(BT, V, code)), dtype=torch.uint8, device="cuda")
        wf = torch.empty(max(256, lx.lx_ce_kd_workspace_bytes(BT, V, code)), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        other = torch.empty_like(c.gd)
        with torch.cuda.graph(graph):
            c.step(lx, c.gd, workspace=ws)
            c.forward(lx, workspace=wf)
            c.backward(lx, other)
        for k in range(4):
            c.gd.fill_(k)
            other.fill_(k)
            for o in c.out:
                o.fill_(k)
            ws.fill_(255 * (k % 2))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.gd, eager)
            c.check_loss()
            c.check_grad(other)


def test_two_calls_at_once():
    a, b = Case(18, 40, 151936, 32, "bf16", scale=1.0).place(), Case(19, 40, 151936, 32, "bf16", T=2.0, scale=1.0).place()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(6):
        a.step(lx, a.gd, stream=s)
        b.step(lx, b.gd, stream=t)
    torch.cuda.synchronize()
    for c in (a, b):
        c.check_loss(rows=range(0, 40, 7))
        c.check_grad(c.gd, rows=range(0, 40, 13))


def test_no_rows():
    c = Case(20, 1, 50, 3, "f32").place()
    e = lambda t: t[:0]  # noqa: E731
    lx.lx_ce_kd_forward_backward(e(c.zd), e(c.set[0]), IGN, e(c.set[2]), e(c.set[3]), e(c.restd), 1.0,
                                 *(e(o) for o in c.out), e(c.gd), 1.0, 1.0)
    torch.cuda.synchronize()
    assert (c.out[0] == 99).all() and (c.gd == 55).all()


@pytest.mark.parametrize("V", [300, 50000])
def test_a_bad_id_in_a_masked_row(V):
    """A row without any unmasked logit has no gradient, whatever its ids: in one pass as in two."""
    def edit(c):
        c.z[1] = NINF
        c.ids[1, 2] = V + 5
    c = Case(21, 3, V, 5, "bf16", edit=edit).place()
    c.step(lx, c.gd)
    other = torch.empty_like(c.gd)
    assert not c.gd[1].any() and not torch.isnan(c.gd).any()
    assert c.out[0][1] == 0 and c.out[1][1] == 0 and c.out[2][1] == NINF
    c.forward(lx)
    c.backward(lx, other)
    assert not other[1].any() and not torch.isnan(other).any()
    assert c.out[0][1] == 0 and c.out[1][1] == 0 and c.out[2][1] == NINF
