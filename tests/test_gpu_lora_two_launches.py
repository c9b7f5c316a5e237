"""Single rows of the low-rank adapters' forward that take two launches up to 32 ranks (u first, then y a column a lane),
on the GPU.  They do where A's part, read by every workgroup, would be too much: rows times groups of 16 * 256 columns
(or of all, where they are fewer) times 2 r H bytes above 2^25.  Tolerances: those of test_gpu_lora.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import test_gpu_lora as plain  # noqa: E402

# 100 rows: a wave takes 64 columns; 200 rows: three times 64, the last ones in part
ROWS = {100: 4208, 200: 2104}
N = 20008


def case(T, r, rank=None, adapter=None, start=None, n=3, H=None, N=N):
    H = ROWS[T] if H is None else H
    start = list(range(T + 1)) if start is None else start
    c = plain.Case(T + r, start, [i % n for i in range(len(start) - 1)] if adapter is None else adapter, n, H, N, r, rank,
                   T=T)
    units = -(-N // 256)
    assert plain.path_of(c) == "single" and r <= 32 and T * -(-units // 16) * 2 * r * H > 1 << 25
    return c


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("r", [8, 16, 24, 32])
def test_ranks(r, T):
    plain.check_forward(case(T, r), f"two launches r {r} T {T}", base="f32")


@pytest.mark.parametrize("r,rank", [(8, [1, 8, 0]), (16, [9, 3, 16]), (24, [17, 24, 7]), (32, [5, 33, 30]),
                                    (16, [-4, 99, 8])])
def test_cut_ranks(r, rank):
    plain.check_forward(case(200, r, rank=rank), f"two launches rank {rank}", base="f32")


@pytest.mark.parametrize("base", [None, "f32", "bf16"])
@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("r", [8, 16, 24, 32])
def test_types(r, base, y):
    c = case(100, r)
    plain.check_forward(c, f"two launches base {base} y {y}", base=base, y=y, pads=(8, 16, 24))
    if base == y:
        plain.check_forward(c, f"two launches in place {y}", base=base, y=y, pads=(0, 40, 0), in_place=True)


@pytest.mark.parametrize("r", [8, 24, 32])
def test_requests_of_every_kind(r):
    """Rows in front of the first request and behind the last, empty requests, no adapter, ids that do not exist."""
    g = np.random.default_rng(r)
    start = [3, 3, 10, 11, 11] + list(range(12, 150)) + [150, 150, 171]
    adapter = [int(v) for v in g.integers(-2, 6, len(start) - 1)]
    assert min(adapter) < 0 and max(adapter) >= 4
    c = case(200, r, rank=[r, 3, r, r - 1], adapter=adapter, start=start, n=4)
    plain.check_forward(c, "two launches, every kind", base="f32")
    plain.check_forward(c, "two launches, every kind, without base", y="bf16")


@pytest.mark.parametrize("T,H,N,r", [(512, 4104, 520, 16), (700, 2056, 72, 24), (300, 16392, 1032, 8)])
def test_a_few_column_ranges(T, H, N, r):
    """Fewer ranges of columns than dies."""
    c = case(T, r, H=H, N=N)
    plain.check_forward(c, f"two launches {T} rows of {N}", base="f32", y="bf16")
