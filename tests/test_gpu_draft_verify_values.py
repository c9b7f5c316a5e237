"""Verification of drafted tokens on values that its other tests leave out, on the GPU, against the float64 reference."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import test_gpu_draft_verify as plain  # noqa: E402
from _parity import announce  # noqa: E402
from test_gpu_draft_verify import room  # noqa: E402,F401  (every test on both paths)

NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("temp", [1.0, 0.0])
@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "lookup"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_nan_and_infinite_logits(dt, with_draft, temp):
    """They give an unspecified token in [-1, V) for their own sequence and change nothing in the others: one NaN, rows of
    NaN, +inf, all of it +inf; in the target, in the draft."""
    V = 3003  # (the last group of 8 is cut)
    c = plain.Case(83, [3, 0, 2, 2, 1, 0, 4, 2, 2], V, dt, with_draft, temps=np.full(9, temp, dtype=np.float32))
    want = c.reference()
    s = c.start
    for i, bad in ((0, NAN), (2, NAN), (4, INF), (5, NAN), (7, INF)):
        rows = slice(s[i] + i, s[i + 1] + i + 1)
        if i % 2 == 0:
            c.z[rows, 100::701] = bad
            c.z[rows, V - 1] = bad
        else:
            c.z[rows] = bad
    if with_draft:
        c.u[s[3]] = NAN
        c.u[s[3] + 1, 7] = INF
        c.u[s[8], V - 3:] = INF
    odd = [0, 2, 4, 5, 7] + ([3, 8] if with_draft else [])
    announce(f"draft_verify NaN {dt} {with_draft} {temp}")
    n, tok, lp = c.run()
    for i in range(9):
        if i not in odd:
            assert n[i] == want[0][i] and np.array_equal(tok[i], want[1][i]), i
            assert np.abs(lp[i] - want[2][i]).max() <= plain.TOL_LOGP, i
            continue
        a = int(n[i])
        assert 0 <= a <= c.lens[i], i
        assert np.array_equal(tok[i, :a], c.tokens[s[i]:s[i] + a]) and (tok[i, a + 1:] == -1).all(), i
        assert -1 <= tok[i, a] < V, i


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("S", [9, 200, 300])
def test_greedy_takes_the_first_of_equals(S, dt):
    """Several tokens with the largest logit, of a drafted position and of the row behind the drafts: in one group of 8,
    in two lanes, in two waves of which the lower one holds the later token (of the next 2048), in later rounds of a
    chunk, in two chunks, at the end of the row.  9, 200 and 300 sequences take chunks of 1, 8 and 4 times 2048."""
    V = 20003
    kinds = [(17, 21), (25, 322), (1900, 2053), (2047, 2048, 4096), (4000, 6150, 6151), (100, 19000), (9000, 20002),
             (1531, 3066, 5117, 8200)]
    c = plain.Case(89, [1] * S, V, dt, temps=np.zeros(S, dtype=np.float32))
    for i in range(S):
        for j in range(2):
            c.z[2 * i + j, list(kinds[(i + j) % len(kinds)])] = 50.0
        k = kinds[i % len(kinds)]
        c.tokens[i] = k[0] if i // len(kinds) % 2 == 0 else k[-1]
    n = plain.check(c, f"ties of {S} {dt}")
    assert 0 < n.sum() < S and np.array_equal(n, [i // len(kinds) % 2 == 0 for i in range(S)])
