"""Float64 reference of the selection of top logits and of cross entropy with distillation from them
(test infrastructure only).

One row at a time, from the definitions; a logit below -1e30 is masked.  It shares no code with the
HIP path.
"""
from __future__ import annotations

import math

import numpy as np

MASKED = -1e30


def _log_sum(x) -> float:
    x = np.asarray(x, dtype=np.float64)
    m = x.max() if len(x) else -np.inf
    if m == -np.inf:
        return -np.inf
    return float(m) + math.log(math.fsum(np.exp(x - m)))


def _masked(z):
    z = np.asarray(z, dtype=np.float64)
    return np.where(z < MASKED, -np.inf, z)


def top_row(z, K: int, temperature: float):
    """(top [K], ids [K], lse, lse of the others) of one row."""
    z = _masked(z)
    order = np.argsort(-z, kind="stable")[:K]
    order = order[z[order] > -np.inf]
    top, ids = np.full(K, -np.inf), np.full(K, -1, dtype=np.int64)
    top[:len(order)], ids[:len(order)] = z[order], order
    rest = z.copy()
    rest[order] = -np.inf
    T = float(np.float32(temperature))
    return top, ids, _log_sum(z / T), _log_sum(rest / T)


class Row:
    """The loss of one row and what its gradient is made of."""

    def __init__(self, z, target, ids, top, lse_rest, temperature):
        self.z = _masked(z)
        self.T = T = float(np.float32(temperature))
        V = len(self.z)
        self.V, self.t = V, int(target)
        entries = [(int(i), float(u) / T) for i, u in zip(ids, top) if 0 <= i < V and not u < MASKED]
        self.bad = any(int(i) >= V for i in ids)
        R = -np.inf if lse_rest is None or lse_rest < MASKED else float(lse_rest)
        A = _log_sum([u for _, u in entries] + [R])
        self.empty = not np.any(self.z > -np.inf)
        self.named = sorted({i for i, _ in entries})
        self.norm = A if A > -np.inf else 0.0
        self.log_q = [(i, u - A) for i, u in entries]
        self.q = np.zeros(V)
        for i, lq in self.log_q:
            self.q[i] += math.exp(lq)
        self.log_qr = R - A if R > -np.inf else -np.inf
        self.qr = math.exp(self.log_qr) if R > -np.inf else 0.0
        self.any = A > -np.inf
        outside = self.z / T
        outside = np.where(np.isin(np.arange(V), self.named), -np.inf, outside)
        self.outside = outside
        self.lse_rest, self.lse_t, self.lse = _log_sum(outside), _log_sum(self.z / T), _log_sum(self.z)
        if self.empty:
            self.ce = self.kd = 0.0
            self.state = (-np.inf, 0.0, 0.0, 0.0)
            return
        t_ok = 0 <= self.t < V
        self.ce = self.lse - self.z[self.t] if t_ok else math.nan
        kd = 0.0
        for i, lq in self.log_q:
            if math.exp(lq) > 0:
                kd += math.exp(lq) * (lq - (self.z[i] / T - self.lse_t))
        if self.qr > 0:
            kd += self.qr * (self.log_qr - (self.lse_rest - self.lse_t))
        self.kd = math.nan if self.bad else kd
        p_rest = math.exp(self.lse_rest - self.lse_t) if self.lse_rest > -np.inf else 0.0
        self.off = p_rest - self.qr if self.any else 0.0
        self.state = (self.lse_t, self.lse_rest if self.lse_rest > -np.inf else 0.0, self.off, self.norm)

    def grad(self, g_ce: float, g_kd: float):
        """(gradient [V], sum of the sizes of the terms that it is the sum of [V])."""
        V = self.V
        if self.empty:
            return np.zeros(V), np.zeros(V)
        if self.bad or not 0 <= self.t < V:
            return np.full(V, np.nan), np.zeros(V)
        p1 = np.exp(self.z - self.lse)
        g = g_ce * p1
        size = abs(g_ce) * p1
        g[self.t] -= g_ce
        b = g_kd / self.T
        if self.any:
            p = np.exp(self.z / self.T - self.lse_t)
            e = np.exp(self.outside - self.lse_rest) if self.lse_rest > -np.inf else np.zeros(V)
            inside = np.isin(np.arange(V), self.named)
            g = g + b * np.where(inside, p - self.q, p - self.qr * e)
            size = size + abs(b) * np.where(inside, p + self.q, p + self.qr * e)
        return g, size


def loss(z, target, ids, top, lse_rest, temperature, g_ce, g_kd) -> float:
    """g_ce ce + g_kd kd of one row (for differences)."""
    r = Row(z, target, ids, top, lse_rest, temperature)
    return g_ce * r.ce + g_kd * r.kd
