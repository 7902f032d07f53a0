"""CPU oracle of the operators on logits, in float64 from the definitions:
log probabilities, entropy, the largest entries, distillation from named
tokens, and the gradients, with what the error bounds of the tests need."""
from __future__ import annotations

import numpy as np


class Rows:
    """Of logits x [M][V] (float64 values) at temperature T: p, ln p, entropy;
    `empty`: rows without an entry above -inf; `broken`: with a NaN or +inf."""

    def __init__(self, x: np.ndarray, T: float):
        self.x, self.T = x, T
        self.broken = (np.isnan(x) | (x == np.inf)).any(1)
        self.empty = (x == -np.inf).all(1)
        ok = ~(self.broken | self.empty)
        with np.errstate(all="ignore"):
            self.z = x / T
            top = np.where(ok, np.where(ok[:, None], self.z, 0).max(1), 0.0)
            self.d = self.z - top[:, None]                  # distance to the maximum, <= 0
            e = np.where(ok[:, None], np.exp(self.d), 0.0)
            S = np.where(ok, e.sum(1), 1.0)
            self.logS = np.log(S)
            self.p = e / S[:, None]
            self.lp = np.where(ok[:, None], self.d - self.logS[:, None], -np.inf)
            self.H = -np.where(self.p > 0, self.p * self.lp, 0.0).sum(1)
            # means of the distance and its square: how roundings of the exponents weigh
            dist = np.where(self.p > 0, -self.d, 0.0)
            self.mean, self.square = (self.p * dist).sum(1), (self.p * dist * dist).sum(1)
            self.far = np.where(np.isfinite(self.d), -self.d, 0.0)
        self.ok = ok


def top(x: np.ndarray, k: int) -> np.ndarray:
    """Indices [M][k] of the largest entries, equal ones by index; -1 behind the
    last entry above -inf, and all of a row with a NaN or +inf."""
    M, V = x.shape
    out = np.full((M, k), -1, np.int64)
    for m in range(M):
        if np.isnan(x[m]).any() or (x[m] == np.inf).any():
            continue
        order = np.argsort(-x[m], kind="stable")[:k]
        order = order[x[m][order] > -np.inf]
        out[m, :len(order)] = order
    return out


def logprobs_grad(r: Rows, targets, a, b):
    """Gradient of sum a logp + b H, rows not ok or without weight 0."""
    hot = np.zeros_like(r.p)
    has = (targets >= 0) & (targets < r.x.shape[1])
    hot[np.nonzero(has)[0], targets[has]] = 1.0
    a = np.where(has, a, 0.0)
    lp = np.where(r.p > 0, r.lp, 0.0)
    g = a[:, None] * (hot - r.p) - b[:, None] * r.p * (lp + r.H[:, None])
    return np.where(r.ok[:, None], g, 0.0) / r.T


def distill(r: Rows, index, t, tail: bool):
    """(loss [M], gradient of each row's loss [M][V], bound [M][V]: the sizes of
    the gradient's parts that carry the students' sums' errors)."""
    M, V = r.x.shape
    loss, grad, size = np.zeros(M), np.zeros((M, V)), np.zeros((M, V))
    for m in range(M):
        slots = [(int(i), float(v)) for i, v in zip(index[m], t[m]) if i >= 0 and v != -np.inf]
        w = np.array([v for _, v in slots])
        with np.errstate(all="ignore"):
            if tail:
                p = np.exp(w)
                rest = max(0.0, 1.0 - p.sum())
            else:
                p = np.exp(w - w.max()) / np.exp(w - w.max()).sum() if slots else w
                rest = 0.0
            named = np.zeros(V, bool)
            want = np.zeros(V)
            for (i, _), pj in zip(slots, p):
                named[i] = True
                want[i] += pj
            q_rest = r.p[m][~named].sum()
            rest = 0.0 if q_rest == 0 and rest <= 2.0 ** -15 else rest
            L = sum(pj * (np.log(pj) - r.lp[m, i]) for (i, _), pj in zip(slots, p) if pj > 0)
            if rest > 0:
                L += rest * (np.log(rest) - np.log(q_rest)) if not r.empty[m] else np.inf
            loss[m] = L
            if not r.ok[m]:
                continue
            share = np.where(named, 0.0, rest * r.p[m] / q_rest) if q_rest > 0 else 0.0
            grad[m] = ((p.sum() + rest) * r.p[m] - want - share) / r.T
            size[m] = ((p.sum() + rest) * r.p[m] + 2 * share) / r.T
    return loss, grad, size
