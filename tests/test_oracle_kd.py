"""The float64 reference of distillation from top logits against its definition: closed forms, and the
gradient against central differences."""
import math

import numpy as np
import pytest

from oracle import kd


def case(seed, V=23, K=5, rest=True, T=1.0):
    rng = np.random.default_rng(seed)
    z, u = rng.normal(0, 2, V), rng.normal(0, 2, V)
    top, ids, _, r = kd.top_row(u, K, T)
    return z, int(rng.integers(V)), ids, top, (r if rest else None)


@pytest.mark.parametrize("T", [1.0, 2.0, 0.5])
@pytest.mark.parametrize("rest", [True, False])
def test_gradient_against_differences(T, rest):
    z, t, ids, top, r = case(3, T=T, rest=rest)
    g, _ = kd.Row(z, t, ids, top, r, T).grad(0.7, 1.3)
    h = 1e-5
    for v in range(len(z)):
        a, b = z.copy(), z.copy()
        a[v] += h
        b[v] -= h
        d = (kd.loss(a, t, ids, top, r, T, 0.7, 1.3) - kd.loss(b, t, ids, top, r, T, 0.7, 1.3)) / (2 * h)
        # the third derivative of a log-sum-exp is below 1 / T^3: h^2 / 6 of it, and the losses' rounding over 2 h
        assert abs(d - g[v]) <= h * h * 8 + 1e-13 / h, v


def test_repeated_id_gradient_against_differences():
    z, t, ids, top, r = case(4)
    ids = ids.copy()
    ids[3] = ids[1]
    g, _ = kd.Row(z, t, ids, top, r, 1.0).grad(0.0, 1.0)
    h = 1e-5
    for v in range(len(z)):
        a, b = z.copy(), z.copy()
        a[v] += h
        b[v] -= h
        d = (kd.loss(a, t, ids, top, r, 1.0, 0.0, 1.0) - kd.loss(b, t, ids, top, r, 1.0, 0.0, 1.0)) / (2 * h)
        assert abs(d - g[v]) <= h * h * 8 + 1e-13 / h, v


def test_whole_teacher_is_the_divergence():
    rng = np.random.default_rng(0)
    z, u = rng.normal(0, 2, 9), rng.normal(0, 2, 9)
    top, ids, lse, rest = kd.top_row(u, 9, 1.0)
    assert rest == -np.inf
    p, q = np.exp(z - np.log(np.exp(z).sum())), np.exp(u - lse)
    r = kd.Row(z, 2, ids, top, rest, 1.0)
    assert r.kd == pytest.approx(float((q * np.log(q / p)).sum()), abs=1e-12)
    assert np.allclose(r.grad(0.0, 1.0)[0], p - q, atol=1e-12)


def test_equal_student_and_teacher_have_nothing_to_learn():
    rng = np.random.default_rng(1)
    u = rng.normal(0, 2, 50)
    top, ids, _, rest = kd.top_row(u, 7, 2.0)
    r = kd.Row(u, 2, ids, top, rest, 2.0)
    assert abs(r.kd) < 1e-12
    assert np.abs(r.grad(0.0, 1.0)[0]).max() < 1e-12


def test_top_row_order_and_masks():
    z = np.array([1.0, 3.0, 3.0, -np.inf, -3.4e38, 0.0])
    top, ids, lse, rest = kd.top_row(z, 5, 1.0)
    assert ids.tolist() == [1, 2, 0, 5, -1]
    assert top.tolist() == [3.0, 3.0, 1.0, 0.0, -np.inf]
    assert rest == -np.inf
    assert lse == pytest.approx(math.log(2 * math.exp(3) + math.exp(1) + 1))
    assert kd.top_row(np.full(4, -np.inf), 2, 1.0)[1].tolist() == [-1, -1]


def test_nothing_named_and_masks():
    z = np.array([0.5, -1.0, -np.inf, 2.0])
    r = kd.Row(z, 0, [-1, -1], [0.0, 0.0], None, 1.0)
    assert r.kd == 0.0 and np.all(r.grad(0.0, 1.0)[0] == 0.0)
    r = kd.Row(z, 0, [2, 0], [1.0, 1.0], None, 1.0)   # named and masked by the student
    assert r.kd == np.inf
    assert r.grad(0.0, 1.0)[0][2] == pytest.approx(-0.5)
    r = kd.Row(np.full(3, -np.inf), 0, [0], [1.0], None, 1.0)
    assert r.ce == r.kd == 0.0 and np.all(r.grad(1.0, 1.0)[0] == 0.0)
