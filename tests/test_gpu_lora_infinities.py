"""Infinities in what the low-rank adapters read, on the GPU: they reach the results that the formulas' sums say, with
their signs, whichever kernels a call takes.  A finite number other than 0 times an infinity is an infinity, 0 times one
and a sum of both signs are NaN; elements whose sums hold none stay within the adapters' own tolerance."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import lora

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cross_entropy_tv_amd as lx  # noqa: E402
import test_gpu_lora as plain  # noqa: E402
from _parity import announce  # noqa: E402

DEV = plain.DEV
INF = float("inf")


def same(got, want, mag, K, label, half=0.0):
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{label}: NaN in other places"
    assert np.array_equal(np.isposinf(got), np.isposinf(want)), f"{label}: +inf in other places"
    assert np.array_equal(np.isneginf(got), np.isneginf(want)), f"{label}: -inf in other places"
    fine = np.isfinite(want)
    tol = (K + 8) * plain.U23 * mag[fine] + (plain.U23 + half) * np.abs(want[fine]) + 1e-30
    assert (np.abs(got[fine] - want[fine]) <= tol).all(), f"{label}: finite elements"


def plant(c, what, g):
    """A few infinities of either sign in A, B, x or dy, within the ranks that are used."""
    sign = lambda: INF if g.random() < 0.5 else -INF  # noqa: E731
    for a in range(c.n):
        k = c.r if c.rank is None else c.rank[a]
        for _ in range(3 if k else 0):
            if what == "B":
                c.B[a, g.integers(c.N), g.integers(k)] = sign()
            elif what == "A":
                c.A[a, g.integers(k), g.integers(c.H)] = sign()
    if what in ("x", "dy"):
        t = c.x if what == "x" else c.dy
        for row in g.integers(c.start[0], c.start[-1], 2):
            t[row, g.integers(t.shape[1])] = sign()
        t[c.start[0], t.shape[1] - 3] = sign()  # among the last 8 columns, behind the last whole tile of them


def run(c, label, forward=True, backward=True):
    announce(f"lora infinities {label}")
    with np.errstate(invalid="ignore"):
        if forward:
            want, mag, written = lora.forward(plain.f64(c.x), *c.oracle_set(), None)
            y = torch.full((c.T, c.N), 55.0, device=DEV)
            lx.lx_lora_forward(c.x.to(DEV), base=None, y=y, **c.set())
            same(plain.f64(y)[written], want[written], mag[written], c.H + c.r, label)
        if backward:
            (dx, dA, dB), (mx, mA, mB), written = lora.backward(plain.f64(c.dy), plain.f64(c.x), *c.oracle_set(), None)
            gx = torch.full((c.T, c.H), 55.0, device=DEV)
            gA, gB = torch.empty(c.n, c.r, c.H, device=DEV), torch.empty(c.n, c.N, c.r, device=DEV)
            lx.lx_lora_backward(c.dy.to(DEV), c.x.to(DEV), base=None, grad_x=gx, grad_A=gA, grad_B=gB, **c.set())
            same(plain.f64(gx)[written], dx[written], mx[written], c.N + c.r, label + " dx")
            same(plain.f64(gA), dA, mA, c.N + c.T, label + " dA")
            same(plain.f64(gB), dB, mB, c.H + c.T, label + " dB")


def exact_u(c):
    """u of the first request's rows is a bf16 number itself: a row of x with one 2 in it, and a scale of 1."""
    a = c.adapter[0]
    c.scale[a] = 1.0
    lo, hi = c.start[0], c.start[1]
    c.x[lo:hi] = 0.0
    c.x[torch.arange(lo, hi), torch.arange(lo, hi) % c.H] = 2.0


@pytest.mark.parametrize("what", ["A", "B", "x", "dy"])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("rows", ["tiles", "single"])
def test_infinities(rows, r, what):
    c = plain.both_paths(rows, r + 3, r)
    if what == "B":
        exact_u(c)
    plant(c, what, np.random.default_rng(r))
    run(c, f"{what} r {r} {rows}")


@pytest.mark.parametrize("rows", ["tiles", "single"])
def test_infinities_beside_cut_ranks(rows):
    for r, rank in ((16, [9, 3, 16]), (24, [17, 24, 7]), (64, [5, 33, 62])):
        c = plain.both_paths(rows, r + 1, r, rank=rank, R=5)
        plant(c, "B", np.random.default_rng(r))
        run(c, f"rank {rank} {rows}")


@pytest.mark.parametrize("what", ["B", "x"])
@pytest.mark.parametrize("r", [8, 16, 24, 32])
def test_infinities_in_two_launches(r, what):
    """Single rows whose A is too much for every workgroup to read: T * ceil(N / 4096) workgroups * 2 r H bytes above
    2^25."""
    T, H, N = 200, 2104, 20008
    assert T * 5 * 2 * r * H > 1 << 25
    c = plain.Case(r, list(range(T + 1)), [i % 3 for i in range(T)], 3, H, N, r)
    assert plain.path_of(c) == "single"
    plant(c, what, np.random.default_rng(r))
    run(c, f"{what} r {r} two launches", backward=False)


@pytest.mark.parametrize("what", ["dy", "B", "x"])
def test_infinities_in_a_large_dy(what):
    """From 2^28 bytes of dy on v is formed in dB's pass over dy."""
    T, N, r = 4100, 32776, 16
    assert T * N * 2 >= 2 ** 28
    c = plain.Case(T, plain.ragged(T, 9, T), [i % 4 for i in range(9)], 4, 136, N, r)
    plant(c, what, np.random.default_rng(r))
    run(c, f"{what}, a large dy", forward=False)


@pytest.mark.parametrize("rows", ["tiles", "single"])
@pytest.mark.parametrize("r", [8, 24, 64])
def test_u_beyond_the_largest_bf16(rows, r):
    """u = 3.4e38 is an fp32 number above the largest bf16 one (3.39e38); y and dB are finite."""
    c = plain.both_paths(rows, r + 3, r, n=1)
    c.scale[0] = 3.4e38
    c.x[:] = 0.0
    c.x[torch.arange(c.T), torch.arange(c.T) % c.H] = 1.0
    c.A[:] = 1.0
    c.B *= 2.0 ** -40
    c.dy *= 2.0 ** -40
    c.base_x[:] = 0.0
    announce(f"lora u beyond bf16 r {r} {rows}")
    run(c, f"large u r {r} {rows}")
