"""Attention weights of rows with infinite scores, in each of the call's forms: what scores
-inf gets nothing, a row that has no other score adds nothing (and says so), a row with
+inf is NaN on every token that it sees, those of -inf among them."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
from quantized_kv_cache_flash_gb300 import workloads as wl
from tests import helpers as H
from tests import keeping_helpers as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_kv_cache_flash_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def visible_weights(s, size, seen):
    """Sum over the rows of their softmax weights on what `seen` says, and its error bound
    (keeping_helpers.weights's)."""
    live = seen.any(1)
    x = np.where(seen, s, -np.inf)[live]
    top = x.max(1, keepdims=True)
    p = np.exp(x - top)
    total = p.sum(1, keepdims=True)
    p /= total
    big = np.where(seen, size, 0.0)[live].max(1, keepdims=True)
    far = np.where(seen[live], np.abs(s[live] - top), 0.0) + np.abs(top) + np.log(total)
    rel = 2 * K.SCORE * big + 4 * 2.0 ** -24 * 1.4427 * far + 2 * K.EXP2 + (32 + s.shape[1] / 64) * 2.0 ** -24
    return p.sum(0), (p * rel).sum(0) * 1.01 + (40 + len(p) / 64) * 2.0 ** -24 * p.sum(0) + 1e-35


def problem(mode, B, Hq, Hkv, T, L, kinds):
    """Records of which some score -inf (or +inf) for every row of their unit: the rows are
    one direction at several lengths, so that a token's score has the same sign for all."""
    G, cap = Hq // Hkv, (L + 15) // 16 * 16 + 16
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, B, Hkv, cap, 300 + T)]
    one = np.array(wl.random_fp16(301, (B, Hkv, 1, 1, 128)))
    one[..., 0] = 0.5
    length = 2.0 ** np.random.default_rng(5).integers(-1, 2, (B, Hkv, G, T, 1))
    q = (one * length).astype(np.float16).reshape(B, Hq, T, 128)
    low, high = np.zeros((B, Hkv, L), bool), np.zeros((B, Hkv, L), bool)
    for b in range(B):
        kind = kinds[b % len(kinds)]
        if kind == "all":
            low[b] = True
        elif kind == "first":            # all that the first query sees
            low[b, :, :L - T + 1] = True
        else:
            low[b] = np.random.default_rng(b).random((Hkv, L)) < 0.3
            low[b, :, 0] = False
            if kind == "high":
                high[b, :, L // 3] = True
                low[b, :, L // 3] = False
    A, bound = np.zeros((B, Hkv, L)), np.zeros((B, Hkv, L))
    scale = 1.0 / math.sqrt(128.0)
    for b in range(B):
        causal = np.tile(np.arange(L)[None] <= (L - T + np.arange(T))[:, None], (G, 1))
        for h in range(Hkv):
            s, size = K.scores_of(mode, rec, q[b, h * G:(h + 1) * G], b, h, L, scale)
            A[b, h], bound[b, h] = visible_weights(s, size, causal & ~low[b, h]) if not low[b, h].all() else (0.0, 0.0)
            if high[b, h].any():
                A[b, h] = np.nan         # (every row sees the token, and a row all tokens)
            for t in np.flatnonzero(low[b, h] | high[b, h]):
                sign = 1.0 if high[b, h, t] else -1.0
                if rec[1] is None:
                    rec[0][b, h, t, 0] = sign * np.inf
                else:
                    rec[1][b, h, t] = sign * np.sign(s[0, t]) * np.inf
    return rec, q, cap, A, bound


@pytest.mark.parametrize("mode,B,Hq,Hkv,T,L", [
    ("turbo4", 4, 8, 2, 1, 300),        # one kernel of clusters
    ("turbo4_asym", 4, 7, 1, 1, 90),
    ("turbo3", 4, 16, 2, 2, 1100),
    ("turbo4", 16, 16, 4, 1, 700),      # two kernels
    ("turbo4_asym", 16, 28, 4, 1, 300),
    ("turbo3", 16, 32, 4, 2, 200),
    ("turbo4", 4, 8, 2, 20, 500),       # a window of one query tile
    ("turbo4_asym", 4, 8, 2, 9, 300),
    ("turbo3", 4, 8, 2, 50, 400),       # two query tiles
    ("turbo4_asym", 4, 8, 2, 60, 700),
    ("turbo4", 4, 8, 2, 200, 700),      # pairs of query tiles
    ("turbo4_asym", 4, 8, 2, 130, 300),
])
def test_infinite_scores(dev, mode, B, Hq, Hkv, T, L):
    for kinds, status in ((("all", "first", "some", "high"), tqf.TQ_STATUS_SHORT_CONTEXT), (("some", "high"), 0)):
        rec, q, cap, A, bound = problem(mode, B, Hq, Hkv, T, L, kinds)
        cache = H.gpu_cache_from_records(mode, B, Hkv, cap, [L] * B, *rec, dev)
        old = np.random.default_rng(6).random((B, Hkv, cap)).astype(np.float32)
        for decay in (0.5, 0.0):
            w = torch.from_numpy(old).to(dev)
            ctx = tqf.Context()
            tqf.tq_attention_weights(ctx, cache, H.upload(q, dev), w, L, decay=decay)
            got = w.cpu().numpy()
            assert np.array_equal(got[:, :, L:], old[:, :, L:])
            base = np.where(np.arange(L) < L - T, old[:, :, :L] * np.float64(decay), 0.0)
            for b in range(B):
                nan = np.isnan(A[b])
                assert np.array_equal(np.isnan(got[b, :, :L]), nan), f"{kinds[b % len(kinds)]}, decay {decay}"
                off = np.abs(got[b, :, :L] - base[b] - A[b]) - bound[b] - 2.0 ** -22 * base[b]
                assert np.all(off[~nan] <= 0), f"{kinds[b % len(kinds)]}, decay {decay}: {off[~nan].max():.2e}"
            assert tqf.tq_get_status(ctx) == status
