"""Tree and packed attention where each row's softmax falls on one or two chosen tokens:
at tile and split boundaries, at the last context token, among the drafted ones, at the
diagonal, and beside tokens of the same score that the row must not see."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
from tests import helpers as H
from tests import serving_helpers as S
from tests import serving_needles as D
from tests.test_gpu_tree import random_trees, words_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_kv_cache_flash_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def boundaries(L):
    """Tokens beside the 32- and 128-token tiles' bounds and the ends."""
    at = {0, 1, 31, 32, L - 1} | {t + d for t in range(128, L + 1, 128) for d in (-1, 0)}
    return sorted(t for t in at if 0 <= t < L)


TREES = [
    # mode, Hq, Hkv, contexts, N
    ("turbo4", 32, 8, [900, 130], 40),           # tensor cores: 160 rows
    ("turbo3", 28, 4, [1537], 20),               # split over many CTAs
    ("turbo4k_3v", 16, 2, [255, 0, 640], 33),
    ("turbo4_asym", 28, 4, [700, 129], 33),      # fp16 K
    ("turbo3_asym", 8, 8, [383], 65),
    ("turbo4", 4, 4, [100], 256),                # the largest block
    ("turbo4", 8, 2, [640, 5], 4),               # the decode kernel: 16 rows
    ("turbo3", 8, 2, [300], 1),                  # 4 rows
    ("turbo3_asym", 14, 2, [511], 2),
    ("turbo3_table", 8, 2, [400, 31], 12),
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: f"{c[0]}-Hq{c[1]}-Hkv{c[2]}-B{len(c[3])}-N{c[4]}")
def test_tree_needles(dev, case):
    mode, Hq, Hkv, ctx_len, N = case
    B, G, L = len(ctx_len), Hq // Hkv, [c + N for c in ctx_len]
    cap = (max(L) + 15) // 16 * 16
    rng = np.random.default_rng(N + Hq)
    rec = H.random_cache(mode, B, Hkv, cap, 40 + N)
    nodes = random_trees(B, N, rng)
    q = np.zeros((B, Hq, N, 128), np.float16)
    units = {}
    for b in range(B):
        seen = np.ones((N, L[b]), bool)
        seen[:, ctx_len[b]:] = nodes[b]
        for h in range(Hkv):
            K, V = units[b, h] = S.kv_of(mode, rec, b, h, L[b])
            for j in range(N):
                vis, hid = np.flatnonzero(seen[j]), np.flatnonzero(~seen[j])
                places = boundaries(L[b]) + [ctx_len[b] - 1] + list(np.flatnonzero(nodes[b, j]) + ctx_len[b])
                for g in range(G):
                    if len(vis):
                        q[b, h * G + g, j] = D.needle_query(K, *D.pick(rng, set(vis.tolist()), hid.tolist(), places))
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, L, *rec, dev)
    qd, ctx = H.upload(q, dev), tqf.Context()
    out = torch.empty_like(qd)
    tqf.tq_tree_attention(ctx, cache, qd, out, torch.from_numpy(words_of(nodes)).to(dev), max(L))
    got = out.float().cpu().numpy()
    for (b, h), (K, V) in units.items():
        seen = np.ones((N, L[b]), bool)
        seen[:, ctx_len[b]:] = nodes[b]
        want, bound = D.needle_rows(q[b, h * G:(h + 1) * G].reshape(-1, 128), K, V, np.tile(seen, (G, 1)),
                                    H.MODE_BITS[mode][0] != 16)
        S.assert_rows(got[b, h * G:(h + 1) * G], want, bound, f"b{b} h{h}")


PREFILLS = [
    # mode, Hq, Hkv, contexts, new rows
    ("turbo4", 8, 2, [500, 0, 129], [130, 65, 1]),
    ("turbo3", 28, 4, [0, 383], [300, 20]),
    ("turbo4k_3v", 16, 2, [127, 0], [40, 129]),
    ("turbo4_asym", 28, 4, [640, 0], [20, 150]),
    ("turbo3_asym", 4, 4, [0, 257], [260, 5]),
]


@pytest.mark.parametrize("case", PREFILLS, ids=lambda c: f"{c[0]}-Hq{c[1]}-Hkv{c[2]}-n{sum(c[4])}")
def test_prefill_needles(dev, case):
    mode, Hq, Hkv, ctx_len, new = case
    B, G, L = len(new), Hq // Hkv, [a + b for a, b in zip(ctx_len, new)]
    cap = (max(L) + 15) // 16 * 16
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rng = np.random.default_rng(sum(new))
    rec = H.random_cache(mode, B, Hkv, cap, 60 + sum(new))
    q = np.zeros((cu[-1], Hq, 128), np.float16)
    units = {}
    for b in range(B):
        for h in range(Hkv):
            K, V = units[b, h] = S.kv_of(mode, rec, b, h, L[b])
            for j in range(new[b]):
                last = ctx_len[b] + j
                places = [t for t in boundaries(L[b]) if t <= last] + [last] * 3
                hid = [last + 1] if last + 1 < L[b] else []
                for g in range(G):
                    q[cu[b] + j, h * G + g] = D.needle_query(K, *D.pick(rng, set(range(last + 1)), hid, places))
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, L, *rec, dev)
    qd, ctx = H.upload(q, dev), tqf.Context()
    out = torch.empty_like(qd)
    tqf.tq_prefill_attention_packed(ctx, cache, qd, out, torch.from_numpy(cu).to(dev), max(L))
    assert tqf.tq_get_status(ctx) == 0
    got = out.float().cpu().numpy()
    for (b, h), (K, V) in units.items():
        last = np.repeat(ctx_len[b] + np.arange(new[b]), G)
        want, bound = D.needle_rows(q[cu[b]:cu[b + 1], h * G:(h + 1) * G].reshape(-1, 128), K, V,
                                    np.arange(L[b])[None, :] <= last[:, None], H.MODE_BITS[mode][0] != 16)
        S.assert_rows(got[cu[b]:cu[b + 1], h * G:(h + 1) * G], want, bound, f"b{b} h{h}")
