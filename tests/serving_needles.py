"""Rows whose softmax falls on one or two chosen tokens, and the bound of their error:
sharp enough that a kernel without the low half of the rotated query, a token that is
dropped or a token that leaks is past it."""
import math

import numpy as np

from oracle import tq_oracle as o

SCORE = 1000.0     # the needles' score (the other tokens' lie some 700 below)
SCALE = 1 / math.sqrt(128)


def rot(x):
    """Vectors [n, 128] in the rotated basis."""
    return (np.asarray(x, np.float64) * o.sign_vector(42)) @ o.hadamard() / math.sqrt(128.0)


def needle_query(K, a, b):
    """The fp16 query of least norm that gives tokens a and b the score SCORE (a alone
    where b is None)."""
    k = K[[a]] if b is None else K[[a, b]]
    s = np.full(len(k), SCORE / SCALE)
    return (k.T @ np.linalg.solve(k @ k.T, s)).astype(np.float16)


def score_errors(q, K, rotated):
    """How far the scores q . k scale of tokens K [n, 128] may be off, in a kernel that
    holds q as two fp16 halves (rotated; K then as levels and a norm) or as it is.

    The products are summed 16 at a time with the sum so far, once for each half.  An
    addend is cut 24 bits below the largest one or better, the result to 24 bits: in a step
    17 2^-24 + 2^-23 of the largest addend or result.  Rot(q)'s seven levels of fp32 sums
    each round by 2^-24 of values whose 2-norm the rest of the transform keeps (7 2^-24 |q|
    in all), its second half by 2^-22 of it.  The scale, a base that moves and the exponent
    of the merge round by 2^-24 of the score each (8 of them here)."""
    q = np.asarray(q, np.float64)
    p = (rot(q[None])[0] * rot(K)) if rotated else q * K
    sums = np.cumsum(p.reshape(-1, 8, 16).sum(-1), axis=1)
    top = np.maximum(np.maximum(np.abs(sums), np.abs(np.pad(sums, ((0, 0), (1, 0)))[:, :8])),
                     np.abs(p).reshape(-1, 8, 16).max(-1))
    err = (2 if rotated else 1) * (17 * 2.0 ** -24 + 2.0 ** -23) * top.sum(1)
    if rotated:
        size = np.linalg.norm(q) * np.linalg.norm(K, axis=1)
        err = err + (7 * 2.0 ** -24 + 2.0 ** -22) * size + 2.0 ** -25 * math.sqrt(128.0) * np.linalg.norm(K, axis=1)
    return SCALE * (err + 8 * 2.0 ** -24 * np.abs(p.sum(1)))


def needle_rows(q, K, V, seen, rotated):
    """Exact rows [R, 128] and bounds [R] of needle queries q [R, 128] under seen [R, n].

    Weights change by w D in first order where D bounds a score's error (their changes
    move the row by (V_t - out) each); a term w v is rounded to fp16 once (2^-11), its sums
    in fp32 and the exponentials below 2^-17 together, the output to fp16."""
    out, bound = np.zeros((len(q), 128)), np.zeros(len(q))
    for r in range(len(q)):
        i = np.flatnonzero(seen[r])
        if len(i) == 0:
            continue
        s = K[i] @ q[r].astype(np.float64) * SCALE
        w = np.exp(s - s.max())
        w /= w.sum()
        i, w = i[w > 1e-30], w[w > 1e-30]
        out[r] = w @ V[i]
        d = score_errors(q[r], K[i], rotated)
        mass = float(np.sum(w * np.linalg.norm(V[i], axis=1)))
        bound[r] = (float(np.sum(w * d * np.linalg.norm(V[i] - out[r], axis=1))) * math.exp(2 * d.max())
                    + (2.0 ** -11 + 2.0 ** -17) * mass + 2.0 ** -11 * np.linalg.norm(out[r])
                    + math.sqrt(128.0) * 2.0 ** -25)
    return out, bound


def pick(rng, visible, hidden, places):
    """A row's two needles: places among the visible tokens (most of them at `places`, the
    last visible and the first hidden ones), the second hidden in every third row."""
    vis = [t for t in places if t in visible] or sorted(visible)
    a = int(rng.choice(vis))
    if len(hidden) and rng.random() < 1 / 3:
        return a, int(rng.choice(sorted(hidden)))
    rest = [t for t in (vis if rng.random() < 0.7 else sorted(visible)) if t != a]
    return a, int(rng.choice(rest)) if rest else None
