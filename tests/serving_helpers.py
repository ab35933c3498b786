"""Shared by the tests of packed prompts, drafted trees and record moves: plain
64-bit forms and the error bounds derived from the kernels' roundings."""
import math

import numpy as np

from oracle import tq_oracle as o
from tests import helpers as H

# Roundings of an attention row, as vectors of the rotated basis (the inverse
# rotation keeps 2-norms).  One token's term w v of the sum is rounded to fp16
# once (p * n_v, or p alone) or twice (also c * n_v): at most half a step,
# 2^-11 of the term each.  A score is within SCORE of its size: q as two fp16
# halves (2^-22), 128 fp32 sums of products (at most 2^-24 * 128 of the sum of
# magnitudes; 2^-17), the e4m3 residual of a codebook of other levels (2^-16).
# The exp2 and the merges stay below 2^-20.  The output is rounded to fp16.
HALF = 2.0 ** -11
SCORE = 2.0 ** -15


def row_bound(w, V, out, smax, roundings=2):
    """2-norm bound of a row's error: weights w [n], values V [n, 128] (64 bit),
    the row's exact output and the largest |q| |k| scale of its scores."""
    mass = float(np.sum(w * np.linalg.norm(V, axis=1)))
    return (roundings * HALF + 2.0 ** -18 + 2 * SCORE * smax) * mass + HALF * np.linalg.norm(out) + 2.0 ** -24


def attention_rows(q, K, V, seen, scale):
    """Plain 64-bit attention of rows q [R, 128] over K, V [n, 128] with the
    boolean mask seen [R, n]; returns (out [R, 128], bounds [R])."""
    q = np.asarray(q, np.float64)
    out, bound = np.zeros((len(q), 128)), np.zeros(len(q))
    kn = np.linalg.norm(np.where(np.isfinite(K), K, 0.0), axis=1)
    for r in range(len(q)):
        i = np.flatnonzero(seen[r])
        if len(i) == 0:
            continue
        s = K[i] @ q[r] * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        out[r] = w @ V[i]
        bound[r] = row_bound(w, V[i], out[r], float(kn[i].max() * np.linalg.norm(q[r]) * scale))
    return out, bound


def assert_rows(got, want, bound, what=""):
    got = np.asarray(got, np.float64).reshape(-1, 128)
    err = np.linalg.norm(got - want.reshape(-1, 128), axis=1)
    bound = bound.reshape(-1)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    bad = np.flatnonzero(err > bound)
    assert len(bad) == 0, (f"{what}: {len(bad)} rows past their bound, the first {bad[0]}: "
                           f"{err[bad[0]]:.3e} > {bound[bad[0]]:.3e}")


def kv_of(mode, records, b, h, n, cbk=None, cbv=None, v_rescale=1.0):
    """K and V (64 bit, original basis) of the first n tokens of a unit."""
    kb, vb = H.MODE_BITS[mode]
    cbk = cbk if cbk is not None else (o.codebook(kb) if kb != 16 else None)
    cbv = cbv if cbv is not None else o.codebook(vb)
    unit = H.oracle_unit_from_records(mode, *records, b, h, n)
    K, V = o.unit_kv_full(mode, unit, cbk, cbv, o.sign_vector(42))
    return K, V * v_rescale


def encode_exact(x, bits, cb=None):
    """Packed codes of vectors x [..., 128] decided in 64 bits (the transform of
    fp16 values is exact there) and their fp16 norms."""
    cb = np.asarray(cb if cb is not None else o.codebook(bits), np.float64)
    v = np.asarray(x, np.float16).reshape(-1, 128)
    s = o.sign_vector(42)
    y = (v.astype(np.float64) * s) @ o.hadamard()
    n = np.sqrt(np.sum(v.astype(np.float64) ** 2, axis=1))
    mids = 0.5 * (cb[:-1] + cb[1:])
    u = np.where(n[:, None] > 0, y / (math.sqrt(128.0) * np.maximum(n, 1e-300)[:, None]), 0.0)
    idx = np.searchsorted(mids, u, side="left").astype(np.uint8)   # ties to the lower index
    norms = np.array([o.fp16_norm(r) for r in v], np.float16)
    return (o.pack_codes(idx, bits).reshape(*x.shape[:-1], 16 * bits), norms.reshape(x.shape[:-1]))
