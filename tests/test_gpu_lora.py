"""The low-rank adapters and their gradients on the GPU, through the package,
against the float64 reference.

Tolerance.  A result is two chained sums of bf16 products in fp32 with
everything between them unrounded (three bf16 terms hold 24 bits): K terms add
at most K 2^-23 of the sum of magnitudes each, so the bound is
(K1 + K2 + 8) 2^-23 of the magnitudes' sums, K1 and K2 the lengths of the two
sums, 2^-23 of the result for base's addition and, for a bf16 result, its
rounding, 2^-8.  That bound holds for any order; the typical error, which
shows a lost term, is held to 4e-6 of the norm (2^-23 times the square root of
the longest sum here, 1000)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import lora

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import cross_entropy_tv_amd as lx  # noqa: E402
from _parity import announce  # noqa: E402

DEV = "cuda:0"
U23 = 2.0 ** -23
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def bf16(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def strided(t, pad):
    """t on the device with `pad` columns more per row, which hold 77."""
    big = torch.full((t.shape[0], t.shape[1] + pad), 77.0, dtype=t.dtype, device=DEV)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


class Case:
    def __init__(self, seed, start, adapter, n, H, N, r, rank=None, T=None, dirty=True):
        g = np.random.default_rng(seed)
        self.T = int(start[-1]) if T is None else T
        self.start, self.adapter, self.n, self.H, self.N, self.r = list(start), list(adapter), n, H, N, r
        self.rank = None if rank is None else list(rank)
        self.x = bf16(g.standard_normal((self.T, H)))
        self.dy = bf16(g.standard_normal((self.T, N)) * 0.1)
        self.A = bf16(g.standard_normal((n, r, H)) * H ** -0.5)
        self.B = bf16(g.standard_normal((n, N, r)) * 0.3)
        self.scale = torch.from_numpy(g.uniform(-2, 2, n).astype(np.float32))
        self.base_y = torch.from_numpy(g.standard_normal((self.T, N)).astype(np.float32))
        self.base_x = torch.from_numpy(g.standard_normal((self.T, H)).astype(np.float32) * 0.01)
        if rank is not None and dirty:  # what lies beyond a rank is not used
            for a in range(n):
                self.A[a, max(self.rank[a], 0):] = float("nan")
                self.B[a, :, max(self.rank[a], 0):] = float("inf")

    def set(self):
        i64 = lambda v: torch.tensor(v, dtype=torch.int64, device=DEV)  # noqa: E731
        return dict(A=self.A.to(DEV), B=self.B.to(DEV), adapter=i64(self.adapter), req_start=i64(self.start),
                    scale=self.scale.to(DEV), rank=None if self.rank is None else i64(self.rank))

    def oracle_set(self):
        return f64(self.A), f64(self.B), self.adapter, self.start, self.scale.numpy(), self.rank


def within(got, want, mag, K, label, extra=0.0, rms=4e-6):
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{label}: NaN in other places"
    err = np.abs(got - want)[fine]
    tol = ((K + 8) * U23 * mag + (U23 + extra) * np.abs(want) + 1e-30)[fine]
    assert (err <= tol).all(), f"{label}: {np.max(err / tol)} of the tolerance"
    norm = np.linalg.norm(want[fine])
    if not extra and norm:
        assert np.linalg.norm(err) <= rms * max(norm, np.linalg.norm(mag[fine]) * 1e-2), f"{label}: typical error"


def check_forward(c, label, base=None, y="f32", pads=(0, 0, 0), in_place=False, **kw):
    announce(f"lora_forward {label}")
    b = None if base is None else c.base_y.to(DT[base])
    want, mag, written = lora.forward(f64(c.x), *c.oracle_set(), None if b is None else f64(b))
    x = strided(c.x.to(DEV), pads[0])
    bd = None if b is None else strided(b.to(DEV), pads[1])
    yd = bd if in_place else strided(torch.full((c.T, c.N), 55.0, dtype=DT[y], device=DEV), pads[2])
    lx.lx_lora_forward(x, base=bd, y=yd, **c.set(), **kw)
    torch.cuda.synchronize()
    got = f64(yd)
    within(got[written], want[written], mag[written], c.H + c.r, label, 2.0 ** -8 if y == "bf16" else 0.0)
    rest = got[~written]
    assert np.array_equal(rest, f64(b)[~written] if in_place else np.full_like(rest, 55.0)), f"{label}: other rows"
    whole = yd._base if yd._base is not None else yd
    assert (whole[:, c.N:] == 77.0).all(), f"{label}: wrote behind the row"
    return yd


def check_backward(c, label, base=False, pads=(0, 0, 0, 0), in_place=False, want_grads=(True, True, True), **kw):
    announce(f"lora_backward {label}")
    b = c.base_x if base else None
    (dx, dA, dB), (mx, mA, mB), written = lora.backward(f64(c.dy), f64(c.x), *c.oracle_set(),
                                                        None if b is None else f64(b))
    bd = None if b is None else strided(b.to(DEV), pads[2])
    gx = bd if in_place else strided(torch.full((c.T, c.H), 55.0, device=DEV), pads[3])
    gA = torch.full((c.n, c.r, c.H), 55.0, device=DEV)
    gB = torch.full((c.n, c.N, c.r), 55.0, device=DEV)
    use = [g if w else None for g, w in zip((gx, gA, gB), want_grads)]
    lx.lx_lora_backward(strided(c.dy.to(DEV), pads[0]), strided(c.x.to(DEV), pads[1]), base=bd if want_grads[0] else None,
                        grad_x=use[0], grad_A=use[1], grad_B=use[2], **c.set(), **kw)
    torch.cuda.synchronize()
    if want_grads[0]:
        within(f64(gx)[written], dx[written], mx[written], c.N + c.r, label + " dx")
        rest = f64(gx)[~written]
        assert np.array_equal(rest, f64(b)[~written] if in_place else np.full_like(rest, 55.0)), f"{label}: other rows"
        whole = gx._base if gx._base is not None else gx
        assert (whole[:, c.H:] == 77.0).all(), f"{label}: wrote behind the row"
    if want_grads[1]:
        within(f64(gA), dA, mA, c.N + c.T, label + " dA")
    if want_grads[2]:
        within(f64(gB), dB, mB, c.H + c.T, label + " dB")
    return gx, gA, gB


def ragged(seed, R, T):
    g = np.random.default_rng(seed)
    return [0] + sorted(int(v) for v in g.integers(0, T + 1, R - 1)) + [T]


def path_of(c, backward=False):
    """Which kernels a shape takes: those of tiles of 32 rows, or of single rows where the estimated time is less (what
    the library estimates by, in us)."""
    T, R, r, H, N = c.T, len(c.adapter), c.r, c.H, c.N
    shared = min(1 + 32 * R / T, 32)
    rows = 4 + 2 * T * r * (H + N + (H if backward else 0)) / 8e6
    one = lambda K: 1 + 3 * min(K, 8192) / 4096  # noqa: E731
    tiles = 13 + shared * (one(H) + (one(N) if backward else 0)) + (shared - 1) * T * (H if backward else N) * 8 / 10e6
    if r > 64:
        tiles *= 2
    return "single" if rows < tiles else "tiles"


def test_the_estimate_is_the_library_s():
    """The forward's workspace is partial sums for single rows and whole 1 KB operands for tiles of 32."""
    for r, tm in ((8, 1), (16, 2), (32, 3), (128, 12)):  # (128: 4 blocks of 32 ranks)
        for T in range(200, 9000, 97):
            c = Case.__new__(Case)
            c.T, c.adapter, c.r, c.H, c.N = T, [0] * (1 + T % 5), r, 520, 1032
            tiles = lx.lx_lora_forward_workspace_bytes(T, len(c.adapter), 520, 1032, r) == -(-T // 32) * 2 * tm * 1024
            assert tiles == (path_of(c) == "tiles"), (r, T)


def both_paths(rows, seed, r, n=3, rank=None, R=4, adapter=None):
    """A case of many rows (tiles of 32) or of a few (single rows)."""
    if rows == "tiles":
        T = (40000 if r <= 64 else 90000) // r + 190
        start = ragged(seed, R, T)
        c = Case(seed, start, adapter or [(i * 2 + 1) % n for i in range(R)], n, 520, 1032, r, rank)
    else:
        start = ragged(seed, R, 40) if seed % 2 else list(range(22))
        c = Case(seed, start, [i % n for i in range(len(start) - 1)], n, 200, 328, r, rank)
    assert path_of(c) == rows and path_of(c, True) == rows
    return c


RANKS = [8, 16, 24, 32, 40, 48, 56, 64, 72, 96, 128]


@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("rows", ["tiles", "single"])
def test_ranks(r, rows):
    c = both_paths(rows, r, r)
    check_forward(c, f"r {r} {rows}", base="f32")
    check_backward(c, f"r {r} {rows}", base=True)


@pytest.mark.parametrize("rows", ["tiles", "single"])
@pytest.mark.parametrize("r,rank", [(8, [1, 8, 0]), (16, [9, 3, 16]), (24, [17, 24, 7]), (64, [5, 33, 62]),
                                    (128, [128, 100, 1]), (16, [-4, 99, 8])])
def test_cut_ranks(r, rank, rows):
    c = both_paths(rows, r + 1, r, rank=rank, R=5)
    check_forward(c, f"rank {rank} {rows}", base="f32")
    check_backward(c, f"rank {rank} {rows}")


@pytest.mark.parametrize("H,N", [(8, 8), (8, 520), (1000, 8), (72, 2056), (2056, 72), (4096, 136), (520, 1032)])
@pytest.mark.parametrize("T,R", [(1, 1), (2, 2), (7, 1), (33, 2), (64, 64), (257, 3)])
def test_sizes(H, N, T, R):
    c = Case(H + N + T, ragged(T, R, T) if R < T else list(range(T + 1)), [i % 2 for i in range(R)], 2, H, N, 16)
    check_forward(c, f"{T} rows {R} requests {H} x {N}")
    check_backward(c, f"{T} rows {R} requests {H} x {N}")


@pytest.mark.parametrize("base", [None, "f32", "bf16"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("rows", ["tiles", "single"])
def test_types(base, y, rows):
    c = both_paths(rows, 5, 24, n=2, R=3)
    check_forward(c, f"base {base} y {y} {rows}", base=base, y=y, pads=(8, 16, 24))
    if base == y:
        check_forward(c, f"in place {y} {rows}", base=base, y=y, pads=(0, 40, 0), in_place=True)


@pytest.mark.parametrize("rows", ["tiles", "single"])
def test_backward_strides_and_in_place(rows):
    c = both_paths(rows, 9, 24, n=2, R=3)
    check_backward(c, "strides", base=True, pads=(8, 16, 24, 32))
    check_backward(c, "in place", base=True, pads=(0, 0, 8, 0), in_place=True)


@pytest.mark.parametrize("H,N,T,R,r", [(8, 4104, 5000, 2, 8), (4104, 8, 3000, 3, 16), (72, 2056, 2500, 5, 24),
                                       (2056, 72, 2500, 1, 16), (128, 136, 5000, 4, 128), (1032, 1544, 1500, 40, 40)])
def test_sizes_in_tiles(H, N, T, R, r):
    c = Case(H + N + T, ragged(T, R, T), [i % 2 for i in range(R)], 2, H, N, r)
    assert path_of(c) == "tiles"
    check_forward(c, f"tiles, {T} rows {R} requests {H} x {N}")
    check_backward(c, f"tiles, {T} rows {R} requests {H} x {N}")


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True), (True, True, False),
                                  (True, False, True), (False, True, True)])
@pytest.mark.parametrize("rows", ["tiles", "single"])
def test_some_gradients(want, rows):
    check_backward(both_paths(rows, 11, 16, n=2, R=3), f"only {want} {rows}", want_grads=want)


@pytest.mark.parametrize("rows", ["tiles", "single"])
def test_requests_of_every_kind(rows):
    """Rows in front of the first request and behind the last, empty requests, no adapter, an id that does not exist,
    adapters without rows, a tile shared by many requests."""
    scale, H, N = (25, 520, 1032) if rows == "tiles" else (1, 136, 264)
    start = [3, 3, 10, 11, 11] + [11 + scale * k for k in (29, 30, 34, 34, 66, 89)]
    adapter = [0, 2, -1, 1, 2, 0, 4, 2, -7, 0]
    c = Case(13, start, adapter, 4, H, N, 16, rank=[16, 16, 5, 16], T=start[-1] + 17)
    assert path_of(c) == rows and path_of(c, True) == rows
    check_forward(c, "every kind", base="f32")
    _, gA, gB = check_backward(c, "every kind", base=True)
    assert (gA[1] == 0).all() and (gA[3] == 0).all() and (gB[1] == 0).all() and (gB[3] == 0).all()
    # requests of one row, then a long one
    start = [2] + list(range(2, 30)) + ([30] if rows == "single" else [3000])
    c = Case(14, start, [(i * 5) % 6 - 1 for i in range(len(start) - 1)], 4, H, N, 16, rank=[16, 16, 5, 16],
             T=start[-1] + 3)
    assert path_of(c) == rows
    check_forward(c, "every kind, single", base="f32")
    check_backward(c, "every kind, single", base=True)


def test_starts_outside_the_rows():
    for T, H, N in ((64, 136, 136), (4200, 520, 1032)):
        c = Case(15, [-5, 20, T + 26], [0, 1], 2, H, N, 8, T=T)
        check_forward(c, "starts outside")
        check_backward(c, "starts outside")


@pytest.mark.parametrize("rows", ["tiles", "single"])
def test_other_requests_rows_do_not_leak(rows):
    """NaN and infinities in one request's rows, or between requests, reach no other row and no other adapter."""
    H, N, T = (520, 1032, 2400) if rows == "tiles" else (264, 264, 110)
    mid, end = T - 46, T - 10
    start, adapter = [5, 36, mid, end], [0, 1, 0]
    c = Case(17, start, adapter, 2, H, N, 16, T=T)
    assert path_of(c) == rows and path_of(c, True) == rows
    clean = check_forward(c, "clean").clone()
    gx, gA, gB = (g.clone() for g in check_backward(c, "clean"))
    bad = Case(17, start, adapter, 2, H, N, 16, T=T)
    for t in (bad.x, bad.dy):
        t[36:mid] = float("nan")
        t[40] = float("inf")
        t[:5] = float("nan")
        t[end:] = float("inf")
    y = torch.full((T, N), 55.0, device=DEV)
    lx.lx_lora_forward(bad.x.to(DEV), base=None, y=y, **bad.set())
    hx, hA, hB = torch.full((T, H), 55.0, device=DEV), torch.empty_like(gA), torch.empty_like(gB)
    lx.lx_lora_backward(bad.dy.to(DEV), bad.x.to(DEV), base=None, grad_x=hx, grad_A=hA, grad_B=hB, **bad.set())
    keep = list(range(0, 36)) + list(range(mid, T))
    assert torch.equal(y[keep], clean[keep]) and torch.equal(hx[keep], gx[keep])
    assert torch.equal(hA[0], gA[0]) and torch.equal(hB[0], gB[0])
    assert torch.isnan(hA[1]).any() and torch.isnan(hB[1]).any()


@pytest.mark.parametrize("T,R,n,H,N,r", [(3000, 5, 2, 1160, 520, 16), (1300, 40, 6, 520, 2056, 64),
                                         (2100, 1, 1, 264, 264, 128), (700, 700, 9, 264, 520, 16),
                                         (256, 256, 3, 240, 1144, 16), (256, 256, 2, 136, 488, 128)])
def test_larger(T, R, n, H, N, r):
    """Several splits of the rows and of the long axes; more than 64 requests."""
    start = ragged(T, R, T) if R < T else list(range(T + 1))
    g = np.random.default_rng(T)
    c = Case(T, start, [int(v) for v in g.integers(-1, n, R)], n, H, N, r)
    check_forward(c, f"larger {T}", base="f32", y="bf16")
    check_backward(c, f"larger {T}", base=True)


def test_long_axis_splits():
    """A vocabulary-sized N: v's sum is cut into ranges that are added in order."""
    c = Case(19, [0, 9, 40], [0, 1], 2, 72, 20008, 16)
    check_forward(c, "long N", base="f32", y="bf16")
    check_backward(c, "long N")
    c = Case(20, list(range(10)), [i % 2 for i in range(9)], 2, 72, 20008, 16)
    check_backward(c, "long N, single rows")


def test_no_rows_or_requests():
    c = Case(21, [0, 0], [0], 1, 16, 16, 8, T=4)
    y = torch.full((4, 16), 55.0, device=DEV)
    lx.lx_lora_forward(c.x.to(DEV), base=None, y=y, **c.set())
    gA, gB, gx = torch.full((1, 8, 16), 9.0, device=DEV), torch.full((1, 16, 8), 9.0, device=DEV), y.clone()
    lx.lx_lora_backward(c.dy.to(DEV), c.x.to(DEV), base=None, grad_x=gx, grad_A=gA, grad_B=gB, **c.set())
    assert (y == 55).all() and (gx == 55).all() and (gA == 0).all() and (gB == 0).all()
    s = c.set()
    s["adapter"], s["req_start"] = s["adapter"][:0], s["req_start"][:1]
    gA.fill_(9), gB.fill_(9)
    lx.lx_lora_backward(c.dy.to(DEV), c.x.to(DEV), base=None, grad_x=gx, grad_A=gA, grad_B=gB, **s)
    lx.lx_lora_forward(c.x.to(DEV), base=None, y=y, **s)
    assert (y == 55).all() and (gA == 0).all() and (gB == 0).all()
    e = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)
    gA.fill_(9)
    lx.lx_lora_backward(e, e, base=None, grad_x=None, grad_A=gA, grad_B=None, **s)
    assert (gA == 0).all()


def test_repeats_streams_and_dirty_workspaces():
    c = Case(23, ragged(23, 6, 1500), [0, 1, 0, 2, 1, 0], 3, 520, 776, 16)
    y0 = check_forward(c, "repeat", base="f32").clone()
    g0 = [g.clone() for g in check_backward(c, "repeat")]
    side = torch.cuda.Stream()
    fw = lx.lx_lora_forward_workspace_bytes(1500, 6, 520, 776, 16)
    bw = lx.lx_lora_backward_workspace_bytes(1500, 6, 3, 520, 776, 16)
    for k in range(4):
        wf = torch.full((fw,), 0xff, dtype=torch.uint8, device=DEV) if k % 2 else None
        wb = torch.full((bw,), 0xff, dtype=torch.uint8, device=DEV) if k % 2 else None
        torch.cuda.synchronize()
        st = side if k >= 2 else None
        assert torch.equal(check_forward(c, "again", base="f32", workspace=wf, stream=st), y0)
        for a, b in zip(check_backward(c, "again", workspace=wb, stream=st), g0):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    """A training step's two calls in one graph, replayed on new inputs with eager work between."""
    c = Case(29, ragged(29, 4, 300), [0, 1, 0, 1], 2, 264, 392, 16)
    s, x, dy = c.set(), c.x.to(DEV), c.dy.to(DEV)
    y, gx = torch.empty(300, 392, device=DEV), torch.empty(300, 264, device=DEV)
    gA, gB = torch.empty(2, 16, 264, device=DEV), torch.empty(2, 392, 16, device=DEV)

    def step():
        lx.lx_lora_forward(x, base=None, y=y, **s)
        lx.lx_lora_backward(dy, x, base=None, grad_x=gx, grad_A=gA, grad_B=gB, **s)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        x.copy_(torch.randn(300, 264, generator=torch.Generator().manual_seed(k)))
        for t in (y, gx, gA, gB):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, gx, gA, gB)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, gx, gA, gB)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,R,n,H,N,r", [(1300, 3, 2, 9000, 264, 16), (1300, 2, 2, 264, 20008, 40)])
def test_long_axis_splits_in_tiles(T, R, n, H, N, r):
    """Beyond 8192 terms a down product of few tiles is cut into ranges whose sums are added in order."""
    c = Case(T + H, ragged(T + H, R, T), [i % n for i in range(R)], n, H, N, r)
    assert path_of(c) == "tiles" and path_of(c, True) == "tiles"
    check_forward(c, "long H, tiles", base="f32")
    check_backward(c, "long H, tiles", base=True)


@pytest.mark.parametrize("T,R,N,r,rank", [(1100, 3, 131080, 16, None), (4100, 9, 32776, 16, [16, 3, 0]),
                                          (34000, 700, 4040, 8, [8, 8, 5])])
def test_a_large_dy(T, R, N, r, rank):
    """From 2^28 bytes of dy on: v is formed in dB's pass over dy.  Odd sizes, tiles that requests share, ranks cut."""
    assert T * N * 2 >= 2 ** 28
    c = Case(T, ragged(T, R, T), [(i * 7) % 4 - (i % 5 == 4) for i in range(R)], 4, 136, N, r,
             None if rank is None else rank + [r], T=T + 5)
    c.adapter[1] = -1
    assert path_of(c, True) == "tiles"
    gx, gA, gB = check_backward(c, "a large dy", base=True, pads=(8, 16, 8, 24))
    again = check_backward(c, "a large dy, without dx", want_grads=(False, True, True))
    assert torch.equal(again[1], gA) and torch.equal(again[2], gB)
    # NaN and infinities of one adapter's rows stay with it
    bad = int(np.argmax([c.start[i + 1] - c.start[i] if c.adapter[i] == 2 else 0 for i in range(R)]))
    lo, hi = c.start[bad], c.start[bad + 1]
    c.dy[lo:hi], c.dy[T:] = float("nan"), float("inf")
    c.x[T:] = float("nan")
    hx, hA, hB = torch.full_like(gx, 55.0), torch.empty_like(gA), torch.empty_like(gB)
    lx.lx_lora_backward(c.dy.to(DEV), c.x.to(DEV), base=c.base_x.to(DEV), grad_x=hx, grad_A=hA, grad_B=hB, **c.set())
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[lo:hi] = False
    assert torch.equal(hx[:T][keep], gx[:T][keep])
    others = [a for a in range(4) if a != 2]
    assert torch.equal(hA[others], gA[others]) and torch.equal(hB[others], gB[others])
