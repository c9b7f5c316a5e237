"""Pins of the adapters' float64 reference (CPU): its gradients against central
differences of a loss on its own forward and against torch's float64 autograd
of the same formula, shared adapters and cut ranks included."""
import numpy as np
import torch

from oracle import lora

T, H, N, r, n = 9, 16, 24, 8, 3
START = [0, 2, 2, 5, 9]
ADAPTER = [1, 0, 2, 1]     # requests 0 and 3 share adapter 1, request 1 is empty: adapter 0 has no rows
RANK = [8, 5, 0]


def data(seed=0):
    g = np.random.default_rng(seed)
    return (g.standard_normal((T, H)), g.standard_normal((n, r, H)), g.standard_normal((n, N, r)),
            g.uniform(0.5, 2, n), g.standard_normal((T, N)))


def loss(x, A, B, s, w):
    return float((lora.forward(x, A, B, ADAPTER, START, s, RANK, None)[0] * w).sum())


def test_gradients_against_differences():
    x, A, B, s, w = data()
    (dx, dA, dB), _, _ = lora.backward(w, x, A, B, ADAPTER, START, s, RANK, None)
    g = np.random.default_rng(1)
    h = 1e-6
    for arr, grad in ((x, dx), (A, dA), (B, dB)):
        for _ in range(25):
            at = tuple(g.integers(d) for d in arr.shape)
            old = arr[at]
            arr[at] = old + h
            up = loss(x, A, B, s, w)
            arr[at] = old - h
            down = loss(x, A, B, s, w)
            arr[at] = old
            # the loss is linear in every single element: what is left is the rounding of two sums of ~1e3
            assert abs((up - down) / (2 * h) - grad[at]) <= 1e-6


def test_gradients_against_autograd():
    x, A, B, s, w = data(2)
    tx, tA, tB = (torch.tensor(a, requires_grad=True) for a in (x, A, B))
    parts = []
    for i, a in enumerate(ADAPTER):
        k = RANK[a]
        rows = tx[START[i]:START[i + 1]]
        parts.append(s[a] * (rows @ tA[a, :k].T) @ tB[a, :, :k].T)
    y = torch.cat(parts)
    (y * torch.tensor(w)).sum().backward()
    ref, _, _ = lora.forward(x, A, B, ADAPTER, START, s, RANK, None)
    assert np.abs(y.detach().numpy() - ref).max() < 1e-12
    (dx, dA, dB), _, _ = lora.backward(w, x, A, B, ADAPTER, START, s, RANK, None)
    for got, want in ((dx, tx.grad), (dA, tA.grad), (dB, tB.grad)):
        assert np.abs(got - want.numpy()).max() < 1e-11
    assert (dA[0] == 0).all() and (dB[2] == 0).all() and (dA[1, 5:] == 0).all()


def test_rows_without_a_request_or_an_adapter():
    x, A, B, s, base = data(3)
    y, _, written = lora.forward(x, A, B, [-1, 0, 3], [1, 3, 4, 6], s, None, base)
    assert written.tolist() == [False, True, True, True, True, True, False, False, False]
    assert np.array_equal(y[1:3], base[1:3]) and np.isnan(y[4:6]).all() and not np.array_equal(y[3], base[3])
