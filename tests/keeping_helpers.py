"""Shared by the tests of attention weights, eviction and draft verification: the
same in 64 bits on the host, and the error bounds derived from the kernels' roundings."""
import math

import numpy as np

from oracle import tq_oracle as o
from tests import helpers as H

# A score's error as a part of |q| |k| scale: the rotated query as two fp16 halves
# (2^-22); eight tensor-core steps over 16 products, each addend cut 25 bits below the
# largest's leading bit and the sum cut to 24 bits, eight more over the low halves'
# (8 * (16 * 2^-25 + 2^-23) = 2^-17.7 of sums that Cauchy bounds by |q| |k|); the
# rotation's seven fp32 levels (7 * 2^-24) and the scale's three factors (3 * 2^-24).
SCORE = 2.0 ** -17
# exp2's own error, and that of a 32-bit logarithm or reciprocal
EXP2 = 2.0 ** -21


def scores_of(mode, records, q, b, h, n, scale, cbk=None):
    """Scores [G * Tq, n] (head, query) of unit (b, h) in 64 bits, and |q| |k| scale."""
    kb = H.MODE_BITS[mode][0]
    unit = H.oracle_unit_from_records(mode, *records, b, h, n)
    cb = cbk if cbk is not None else (o.codebook(kb) if kb != 16 else None)
    K, _ = o.unit_kv_full(mode, unit, cb, o.codebook(H.MODE_BITS[mode][1]), o.sign_vector(42))
    rows = np.asarray(q, np.float64).reshape(-1, 128)
    size = np.linalg.norm(rows, axis=1)[:, None] * np.linalg.norm(K, axis=1)[None, :] * scale
    return rows @ K.T * scale, size


def weights(mode, records, q, lengths, Hkv, scale=0.0, hint=None):
    """A [B, Hkv, cap] and its error bound: the softmax weights of q [B, Hq, Tq, 128] on
    the tokens of each KV head, summed over the rows."""
    B, Hq, T, _ = q.shape
    G, cap = Hq // Hkv, records[2].shape[2]
    scale = scale or 1.0 / math.sqrt(128.0)
    A, bound = np.zeros((B, Hkv, cap)), np.zeros((B, Hkv, cap))
    for b in range(B):
        L = lengths[b]
        n = min(L, hint or cap)
        if n <= 0:
            continue
        seen = np.tile(np.arange(n)[None, :] <= (L - T + np.arange(T))[:, None], (G, 1))
        for h in range(Hkv):
            s, size = scores_of(mode, records, q[b, h * G:(h + 1) * G], b, h, n, scale)
            live = seen.any(1)
            x = np.where(seen, s, -np.inf)[live]
            top = x.max(1, keepdims=True)
            p = np.exp(x - top)
            total = p.sum(1, keepdims=True)
            p /= total
            # exp's argument: the score's error and the row's (through its sum), the
            # rounding of score - log2(sum) of numbers below `far`; the row's sum over n
            # tokens in chains of 16, tiles and shares
            big = np.where(seen, size, 0.0)[live].max(1, keepdims=True)
            far = np.where(seen[live], np.abs(x - top), 0.0) + np.abs(top) + np.log(total)
            rel = 2 * SCORE * big + 4 * 2.0 ** -24 * 1.4427 * far + 2 * EXP2 + (32 + n / 64) * 2.0 ** -24
            A[b, h, :n] = p.sum(0)
            # (the sum over the rows: chains of 32, then tiles of rows)
            bound[b, h, :n] = (p * rel).sum(0) * 1.01 + (40 + len(p) / 64) * 2.0 ** -24 * p.sum(0) + 1e-35
    return A, bound


def evict(w, L, n, sinks, recent):
    """Places kept of a row of weights w [>= L]."""
    if L <= n:
        return np.arange(L)
    key = np.where(np.isnan(w[:L]), -np.inf, w[:L]) + 0.0
    free = np.arange(sinks, L - recent)
    order = free[np.argsort(-key[free], kind="stable")][:n - sinks - recent]
    return np.sort(np.concatenate([np.arange(sinks), order, np.arange(L - recent, L)])).astype(int)


def verify(tokens, parents, target, draft, u):
    """One sequence's (path, next token), and how near its decisions came to a border,
    as a part of the whole: tests of nodes and the draw."""
    unit = lambda x: np.clip(np.nan_to_num(np.asarray(x, np.float64), nan=0.0), 0.0, 1.0)  # noqa: E731
    n, v = target.shape
    path, rest, whole, near = [0], unit(target[0]), 1.0, np.inf
    for i in range(1, n):
        if parents[i] != path[-1] or not 0 <= tokens[i] < v:
            continue
        q = np.zeros(v) if draft is None else unit(draft[path[-1]])
        if draft is None:
            q[tokens[i]] = 1.0
        a, b = unit(u[i]) * q[tokens[i]] * whole, rest[tokens[i]]
        if max(a, b) > 0 and a != b:
            near = min(near, abs(a - b) / max(a, b))
        if a < b:
            path.append(i)
            rest, whole = unit(target[i]), 1.0
        else:
            rest = np.maximum(rest - whole * q, 0.0)
            whole = rest.sum()
    if not rest.sum() > 0:
        rest = unit(target[path[-1]])
    if not rest.sum() > 0:
        return path, 0, near
    c = np.cumsum(rest)
    at = unit(u[0]) * c[-1]
    near = min(near, float(np.min(np.abs(c - at)[rest > 0]) / c[-1]) if at > 0 else np.inf)
    return path, int(np.searchsorted(c, at, side="right")), near
