"""Pins of the draft verification's float64 reference (CPU): the law of what it
emits, by integrating over its random numbers on tiny vocabularies, and the
rules at its edges."""
import numpy as np
import pytest

from oracle import draft_verify as dv


def first_token_law(z, u, temperature=1.0, grid=400):
    """The law of the first emitted token when the drafted one is drawn from q, by a
    midpoint grid over both random numbers."""
    V = len(z)
    q = dv.probabilities(u, temperature)
    law = np.zeros(V)
    mid = (np.arange(grid) + 0.5) / grid
    for x in range(V):
        for r in mid:
            # the draw's number matters after a rejection only
            n, out, _ = dv.verify_one(np.stack([z, z]), u[None], [x], temperature, [r], 0.5)
            if n == 1:
                law[x] += q[x] / grid
            else:
                p = dv.probabilities(z, temperature)
                rest = np.maximum(p - q, 0)
                law += q[x] / grid * rest / rest.sum()
    return law


@pytest.mark.parametrize("temperature", [1.0, 0.5])
def test_emitted_tokens_follow_the_target(temperature):
    rng = np.random.default_rng(3)
    z, u = rng.normal(0, 1.5, 6), rng.normal(0, 1.5, 6)
    p, q = dv.probabilities(z, temperature), dv.probabilities(u, temperature)
    # the grid over r resolves the acceptance probability to 1 / (2 grid) per token
    assert np.abs(first_token_law(z, u, temperature) - p).max() <= 6 / 800
    # the rejection probability is the total variation distance
    accept = np.minimum(p, q).sum()
    assert abs((1 - accept) - 0.5 * np.abs(p - q).sum()) < 1e-12


def test_the_draw_inverts_the_running_sum():
    mass = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    assert [dv.draw(mass, w) for w in (0.0, 0.2499, 0.25, 0.7499, 0.75, 0.9999, 1.0)] == [1, 1, 3, 3, 4, 4, 4]
    assert dv.draw(np.zeros(4), 0.3) == -1


def test_edges():
    z = np.array([[1.0, 3.0, 3.0, 0.0], [0.0, 0.0, 5.0, 0.0]])
    u = np.array([[1.0, 3.0, 3.0, 0.0]])
    # equal rows accept every r < 1
    n, out, lp = dv.verify_one(z, u, [2], 1.0, [0.999999], 0.0)
    assert n == 1 and out[0] == 2 and abs(lp[0] - np.log(dv.probabilities(z[0], 1.0)[2])) < 1e-15
    # greedy: the first of equal logits
    assert dv.verify_one(z, u, [2], 0.0, [0.0], 0.0)[:2] == (0, [1])
    assert dv.verify_one(z, u, [1], 0.0, [0.9], 0.0)[:2] == (1, [1, 2])
    # a token outside the vocabulary is not accepted
    assert dv.verify_one(z, u, [7], 1.0, [0.0], 0.0)[0] == 0
    # without draft logits the rejected token is left out of the draw
    n, out, _ = dv.verify_one(z, None, [1], 1.0, [0.9999], 0.5)
    assert n == 0 and out[0] != 1
    # a masked row accepts nothing and draws nothing
    assert dv.verify_one(np.full((2, 4), -np.inf), u, [1], 1.0, [0.0], 0.5) == (0, [-1], [0.0])
