"""Float64 reference of the verification of drafted tokens (test infrastructure only).

One sequence at a time, position by position, from the definition: a drafted
token x with random number r is accepted when r q(x) < p(x); the first
rejection draws the sequence's token from max(p - q, 0), a sequence without
one from p of the row behind its last draft, by inversion of the running sum.
It shares no code with the HIP path.
"""
from __future__ import annotations

import math

import numpy as np


def probabilities(z: np.ndarray, temperature: float) -> np.ndarray:
    """softmax(z / T) in float64 (T > 0); all 0 for a row without a finite logit;
    T <= 0: 1 at the first largest logit."""
    z = np.asarray(z, dtype=np.float64)
    m = z.max()
    if m == -np.inf:
        return np.zeros_like(z)
    if not temperature > 0:
        p = np.zeros_like(z)
        p[int(np.argmax(z))] = 1.0
        return p
    e = np.exp((z - m) / float(np.float32(temperature)))
    return e / math.fsum(e)


def draw(mass: np.ndarray, w: float) -> int:
    """The smallest v whose running sum exceeds w times the total; the last v with
    mass should none; -1 without any mass."""
    some = np.nonzero(mass > 0)[0]
    if len(some) == 0:
        return -1
    sums = np.cumsum(mass)
    v = int(np.searchsorted(sums, w * sums[-1], side="right"))
    return min(v, int(some[-1]))


def verify_one(target, draft, tokens, temperature, u_accept, u_sample):
    """(accepted count, [emitted tokens], [their log p]) of one sequence: target
    (n + 1, V), draft (n, V) or None, tokens [n]."""
    n, V = len(tokens), target.shape[1]
    out, logp = [], []
    greedy = not temperature > 0
    for j in range(n + 1):
        p = probabilities(target[j], temperature)
        mass = p
        if j < n:
            x = int(tokens[j])
            inside = 0 <= x < V
            px = float(p[x]) if inside else 0.0
            if greedy:
                ok = px > 0
            elif draft is None:
                ok = float(u_accept[j]) < px
                mass = p.copy()
                if inside:
                    mass[x] = 0.0
            else:
                q = probabilities(draft[j], temperature)
                qx = float(q[x]) if inside else 0.0
                ok = px > 0 and float(u_accept[j]) * qx < px
                mass = np.maximum(p - q, 0.0)
            if ok:
                out.append(x)
                logp.append(0.0 if greedy else math.log(px))
                continue
        if not mass.sum() > 0:
            mass = p
        v = draw(mass, float(u_sample))
        out.append(v)
        logp.append(0.0 if v < 0 or greedy else math.log(p[v]))
        return j, out, logp
    raise AssertionError


def verify(target, draft, tokens, start, max_draft, temperature, u_accept, u_sample):
    """All sequences: (n_accepted [S], tokens [S][max_draft + 1], logprobs)."""
    S = len(start) - 1
    n_acc = np.zeros(S, dtype=np.int64)
    out = np.full((S, max_draft + 1), -1, dtype=np.int64)
    logp = np.zeros((S, max_draft + 1), dtype=np.float64)
    for i in range(S):
        s, e = int(start[i]), int(start[i + 1])
        t = 1.0 if temperature is None else float(temperature[i])
        n_acc[i], o, lp = verify_one(target[s + i:e + i + 1], None if draft is None else draft[s:e], tokens[s:e], t,
                                     u_accept[s:e], u_sample[i])
        out[i, :len(o)] = o
        logp[i, :len(o)] = lp
    return n_acc, out, logp
