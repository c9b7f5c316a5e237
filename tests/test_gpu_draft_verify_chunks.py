"""Verification of drafted tokens where a chunk of a row is several rounds of what a workgroup holds, on the GPU, against
the float64 reference."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import test_gpu_draft_verify as plain  # noqa: E402

UNIT = 2048  # logits of a round that a workgroup holds one group of 8 a thread of


def rejecting(c):
    """Nearly every draft is rejected, so that the residual is drawn from."""
    c.ua[:] = np.nextafter(np.float32(1), np.float32(0))
    return c


def units_of(c, chunk):
    """In which unit of its chunk each sequence's drawn token lies, after a rejection and after none."""
    n, tok, _ = c.reference()
    at = {True: set(), False: set()}
    for i, a in enumerate(n):
        at[bool(a < c.lens[i])].add(int(tok[i, a]) // UNIT % chunk)
    return at


@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "lookup"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("accept", ["some", "none"])
def test_chunks_of_four_units(accept, dt, with_draft):
    """From S ceil(V / 4096) > 1280 on the row that a token is drawn from goes in chunks of 4 units: one round of four
    groups (2-byte logits), two of two (fp32; the residual of any type)."""
    S, V = 112, 50001
    assert S * -(-V // (2 * UNIT)) > 1280
    c = plain.Case(97, [1, 2, 0, 1] * (S // 4), V, dt, with_draft)
    if accept == "none":
        rejecting(c)
    at = units_of(c, 4)
    assert at[True] == at[False] == {0, 1, 2, 3}
    plain.check(c, f"chunks of 4 {dt} {with_draft} {accept}")


@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "lookup"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_chunks_of_two_units(dt, with_draft):
    """S ceil(V / 2048) > 1280, S ceil(V / 4096) below: chunks of 2 units, and more than 2^23 logits."""
    S, V = 60, 50001
    assert S * -(-V // UNIT) > 1280 >= S * -(-V // (2 * UNIT))
    c = plain.Case(101, [2, 3, 0, 2, 4] * (S // 5), V, dt, with_draft)
    c.ua[::2] = np.float32(0.9999)
    at = units_of(c, 2)
    assert at[True] == at[False] == {0, 1}
    plain.check(c, f"chunks of 2 {dt} {with_draft}")


@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "lookup"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("S,L,V", [(59, 6, 20001), (512, 1, 8190), (36, 6, 32771)])
def test_long_chunks_of_a_few_rows(S, L, V, dt, with_draft):
    """Up to 2^23 logits, every row in fp64 at once, and more than 1024 chunks of a unit: chunks of 2 to 8."""
    assert S * (L + 1) * V <= 1 << 23 and S * (L + 1) * -(-V // UNIT) > 1024
    rng = np.random.default_rng(S)
    lens = [int(v) for v in rng.integers(0, L + 1, S)]
    c = plain.Case(103 + S, lens, V, dt, with_draft, max_draft=L)
    c.ua[::3] = np.float32(0.9999)
    plain.check(c, f"long chunks {S} {dt} {with_draft}")


def two_levels(rows, V, level):
    """bf16 logits of 0 at every eighth token and `level` elsewhere: added up in one place in fp32, their exponentials
    are rounded the same way every time."""
    t = torch.full((rows, V), level, dtype=torch.bfloat16, device=plain.DEV)
    t[:, ::8] = 0.0
    return t


def of_two_levels(V, level):
    """The sum of the exponentials."""
    return V / 8 * (1.0 + 7.0 * np.exp(level))


def call(z, u, token, r, w):
    V, dev = z.shape[1], plain.DEV
    n, tok, lp = (torch.full(s, 99, dtype=t, device=dev) for s, t in
                  (((1,), torch.int64), ((1, 2), torch.int64), ((1, 2), torch.float32)))
    plain.lx.lx_draft_verify(z, u, torch.tensor([token], device=dev), torch.tensor([0, 1], device=dev), 1, None,
                             torch.tensor([r], dtype=torch.float32, device=dev),
                             torch.tensor([w], dtype=torch.float32, device=dev), n, tok, lp)
    return n.item(), tok[0].tolist(), lp[0].tolist()


def test_log_p_of_a_very_long_row():
    plain.announce("draft_verify log p, V 2^28")
    V, level = 1 << 28, -1 / 128
    n, tok, lp = call(two_levels(2, V, level), two_levels(1, V, level), 8 * 12345, 0.5, 0.5)
    assert n == 1 and tok[0] == 8 * 12345
    assert abs(lp[0] + np.log(of_two_levels(V, level))) <= plain.TOL_LOGP
    assert abs(lp[1] + np.log(of_two_levels(V, level)) - (level if tok[1] % 8 else 0.0)) <= plain.TOL_LOGP


def test_acceptance_over_a_very_long_row():
    """r beyond p / q, and below it, by 2^-17."""
    plain.announce("draft_verify acceptance, V 2^30")
    V, zl, ul, w = (1 << 30) - 40, -1 / 64, -87 / 128, 0.3
    z, u = two_levels(2, V, zl), two_levels(1, V, ul)
    St, Sd = of_two_levels(V, zl), of_two_levels(V, ul)
    ratio = Sd / St
    n, tok, lp = call(z, u, 800, ratio * (1 - 2.0 ** -17), w)
    assert n == 1 and tok[0] == 800 and abs(lp[0] + np.log(St)) <= plain.TOL_LOGP
    n, tok, lp = call(z, u, 800, ratio * (1 + 2.0 ** -17), w)
    # max(p - q, 0) is the same at every token but the eighths: the one at w of them
    k = float(np.float32(w)) * (V // 8 * 7)
    assert 0.4 < k % 1 < 0.6
    assert n == 0 and tok == [int(k) // 7 * 8 + int(k) % 7 + 1, -1]
    assert abs(lp[0] + np.log(St) - zl) <= plain.TOL_LOGP
