"""Packed and tree attention on the GPU where inputs are at the edge of what the
formats hold: NaN scores, norms of other sizes than a model's."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
from quantized_kv_cache_flash_gb300 import workloads as wl
from tests import helpers as H
from tests import serving_helpers as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_kv_cache_flash_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def chains(B, N, dev):
    """Masks [B, N, W] of a chain of N nodes."""
    return tqf.tq_tree_mask([i - 1 for i in range(N)]).to(dev).unsqueeze(0).repeat(B, 1, 1).contiguous()


NAN_CASES = [("turbo4", 32, 8, 40), ("turbo3", 28, 4, 64), ("turbo4_asym", 28, 4, 33),   # tensor cores
             ("turbo3", 8, 2, 4), ("turbo4_asym", 4, 2, 3), ("turbo3_table", 8, 2, 7)]   # the decode kernel


@pytest.mark.parametrize("mode,Hq,Hkv,N", NAN_CASES)
def test_tree_row_of_nan_scores_is_nan_at_every_split(dev, mode, Hq, Hkv, N):
    """A NaN query row: its output is NaN, the others are within the bound of their
    roundings (a row whose base moves takes its neighbours' along in the decode
    kernel, so they may round otherwise than beside a finite row), and no row counts
    as one that sees no token."""
    B, lengths, cap = 2, [3000 + N, 70 + N], 3104
    rec = H.random_cache(mode, B, Hkv, cap, 11)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, lengths, *rec, dev)
    q = H.upload(wl.random_fp16(12, (B, Hq, N, 128)), dev)
    mask, ctx = chains(B, N, dev), tqf.Context()
    got, G = torch.empty_like(q), Hq // Hkv
    lost = torch.zeros(B, Hq, N, dtype=torch.bool, device=dev)
    lost[0, 1, N - 1] = lost[1, Hq - 1, 0] = True
    q[lost] = float("nan")
    tqf.tq_tree_attention(ctx, cache, q, got, mask, max(lengths))
    assert bool(torch.isnan(got[lost]).all())
    assert bool(torch.isfinite(got[~lost]).all())
    for b, heads, h in ((0, slice(0, G), 0), (1, slice(Hq - G, Hq), Hkv - 1)):
        keep = ~lost[b, heads].cpu().numpy()
        K, V = S.kv_of(mode, rec, b, h, lengths[b])
        last = np.broadcast_to(lengths[b] - N + np.arange(N), keep.shape)[keep]
        rows, bound = S.attention_rows(q[b, heads].cpu().numpy()[keep], K, V,
                                       np.arange(lengths[b])[None, :] <= last[:, None], 1 / math.sqrt(128))
        S.assert_rows(got[b, heads].float().cpu().numpy()[keep], rows, bound, f"b{b}")
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("mode,Hq,Hkv,N", NAN_CASES)
def test_tree_with_nan_records_in_one_part_of_the_context(dev, mode, Hq, Hkv, N):
    """Records whose scores are NaN fill one 128-token part of a long context: every
    row sees them, so every row is NaN, however the context is split."""
    B, L, cap = 1, 3000 + N, 3104
    rec = H.random_cache(mode, B, Hkv, cap, 13)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, [L], *rec, dev)
    at = slice(1280, 1408)
    if mode == "turbo3_table":
        cache.k_data[:, 0, at, 48:] = 0x7F          # (table values of 0x7F7F: NaN)
    elif cache.k_norm is not None:
        cache.k_norm[:, 0, at] = float("nan")
    else:
        cache.k_data[:, 0, at] = float("nan")
    q = H.upload(wl.random_fp16(14, (B, Hq, N, 128)), dev)
    ctx, out = tqf.Context(), torch.zeros_like(q)
    tqf.tq_tree_attention(ctx, cache, q, out, chains(B, N, dev), L)
    G = Hq // Hkv
    assert bool(torch.isnan(out[:, :G]).all())
    assert bool(torch.isfinite(out[:, G:]).all())
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("mode,Hq,Hkv", [("turbo4", 8, 2), ("turbo3_asym", 28, 4)])
def test_prefill_row_of_nan_scores_is_nan(dev, mode, Hq, Hkv):
    new, cap = [300, 40], 304
    rec = H.random_cache(mode, 2, Hkv, cap, 15)
    cache = H.gpu_cache_from_records(mode, 2, Hkv, cap, new, *rec, dev)
    q, cu, ctx = H.upload(wl.random_fp16(16, (340, Hq, 128)), dev), i32([0, 300, 340], dev), tqf.Context()
    want, got = torch.empty_like(q), torch.empty_like(q)
    tqf.tq_prefill_attention_packed(ctx, cache, q, want, cu, 300)
    lost = torch.zeros(340, Hq, dtype=torch.bool, device=dev)
    lost[7, 1] = lost[299, Hq - 1] = lost[310, 0] = True
    q[lost] = float("nan")
    tqf.tq_prefill_attention_packed(ctx, cache, q, got, cu, 300)
    assert bool(torch.isnan(got[lost]).all())
    assert torch.equal(got[~lost], want[~lost])
    assert tqf.tq_get_status(ctx) == 0


# A term of P.V is rounded to fp16: at most 2^-11 of itself, or, below 2^-14, 2^-25.  The
# largest weight of a row over a tile whose largest V norm is nmax stands at 2^4 / nmax at
# least (a subnormal nmax counts as 2^-15 in the packed prefill), so what the second adds
# over n tokens is at most n 2^-25 nmax / 2^4, with V's vectors up to 1.2 times their norm.
# And an output element below 2^-14 is rounded by up to 2^-25, so a row of them by up to
# sqrt(128) 2^-25 in the 2-norm (row_bound's own absolute term, 2^-24, is for one).
def tiny_terms(n, nmax, v_rescale):
    return n * 2.0 ** -29 * max(nmax, 2.0 ** -15) * 1.2 * v_rescale + math.sqrt(128.0) * 2.0 ** -25


SIZES = {
    # the V norms of a cache: all small, down to the smallest; mixed from tile to tile; and
    # from token to token (the largest of each tile decide)
    "2^-11": lambda n, t: n * np.float16(2.0 ** -11),
    "2^-17": lambda n, t: n * np.float16(2.0 ** -17),
    "2^-21": lambda n, t: n * np.float16(2.0 ** -21),
    "tiles": lambda n, t: n * (2.0 ** -(7.0 * ((t // 128) % 4))).astype(np.float16),
    "rising": lambda n, t: n * (2.0 ** -(20.0 - 5 * (t // 128) % 25)).astype(np.float16),
    "large": lambda n, t: n * np.where((t // 128) % 2 == 1, 1500.0, 2.0 ** -12).astype(np.float16),
}


@pytest.mark.parametrize("size", sorted(SIZES))
@pytest.mark.parametrize("qs", [1.0, 8.0])
@pytest.mark.parametrize("mode,Hq,Hkv,N", [("turbo4", 8, 2, 30), ("turbo3_asym", 28, 4, 33), ("turbo3", 32, 8, 40)])
def test_tree_rows_over_norms_of_every_size(dev, mode, Hq, Hkv, N, qs, size):
    L, cap, G = 700 + N, 752, Hq // Hkv
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, 1, Hkv, cap, 17)]
    rec[3] = SIZES[size](rec[3], np.arange(cap)).astype(np.float16)
    nmax = float(rec[3][:, :, :L].max())
    vr = float(2.0 ** round(-math.log2(nmax)))
    cache = H.gpu_cache_from_records(mode, 1, Hkv, cap, [L], *rec, dev, v_rescale=vr)
    q = wl.random_fp16(18, (1, Hq, N, 128), scale=qs)
    qd, ctx = H.upload(q, dev), tqf.Context()
    out = torch.empty_like(qd)
    tqf.tq_tree_attention(ctx, cache, qd, out, chains(1, N, dev), L)
    assert tqf.tq_get_status(ctx) == 0
    got = out.float().cpu().numpy()
    seen = np.tile(np.arange(L)[None, :] <= (L - N + np.arange(N))[:, None], (G, 1))
    for h in range(Hkv):
        K, V = S.kv_of(mode, rec, 0, h, L, v_rescale=vr)
        want, bound = S.attention_rows(q[0, h * G:(h + 1) * G].reshape(-1, 128), K, V, seen, 1 / math.sqrt(128))
        S.assert_rows(got[0, h * G:(h + 1) * G], want, bound + tiny_terms(L, nmax, vr), f"h{h}")


@pytest.mark.parametrize("size", sorted(SIZES))
@pytest.mark.parametrize("qs", [1.0, 8.0])
@pytest.mark.parametrize("mode,Hq,Hkv", [("turbo4", 8, 2), ("turbo3_asym", 28, 4)])
def test_prefill_rows_over_norms_of_every_size(dev, mode, Hq, Hkv, qs, size):
    new, ctx_len, cap, G = [200, 61], [500, 0], 704, Hq // Hkv
    L = [a + b for a, b in zip(new, ctx_len)]
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, 2, Hkv, cap, 19)]
    rec[3] = SIZES[size](rec[3], np.arange(cap)).astype(np.float16)
    nmax = float(rec[3].max())
    vr = float(2.0 ** round(-math.log2(nmax)))
    cache = H.gpu_cache_from_records(mode, 2, Hkv, cap, L, *rec, dev, v_rescale=vr)
    q = wl.random_fp16(20, (261, Hq, 128), scale=qs)
    qd, ctx = H.upload(q, dev), tqf.Context()
    out = torch.empty_like(qd)
    tqf.tq_prefill_attention_packed(ctx, cache, qd, out, i32([0, 200, 261], dev), max(L))
    assert tqf.tq_get_status(ctx) == 0
    got, cu = out.float().cpu().numpy(), [0, 200, 261]
    for b in range(2):
        last = np.repeat(ctx_len[b] + np.arange(new[b]), G)
        for h in range(Hkv):
            K, V = S.kv_of(mode, rec, b, h, L[b], v_rescale=vr)
            want, bound = S.attention_rows(q[cu[b]:cu[b + 1], h * G:(h + 1) * G].reshape(-1, 128), K, V,
                                           np.arange(L[b])[None, :] <= last[:, None], 1 / math.sqrt(128))
            S.assert_rows(got[cu[b]:cu[b + 1], h * G:(h + 1) * G], want, bound + tiny_terms(L[b], nmax, vr), f"b{b} h{h}")


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan"), -65504.0])
@pytest.mark.parametrize("mode,Hq,Hkv,N", [("turbo4", 32, 8, 40), ("turbo4_asym", 28, 4, 33), ("turbo3", 8, 2, 6),
                                           ("turbo3_asym", 4, 2, 7)])
def test_tree_norms_of_unseen_tokens_may_be_anything(dev, mode, Hq, Hkv, N, value):
    """The last three nodes are padding that nobody sees, whatever their norms hold:
    every row is within its bound."""
    L, cap, G = 140 + N, 208, Hq // Hkv
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, 1, Hkv, cap, 27)]
    cache = H.gpu_cache_from_records(mode, 1, Hkv, cap, [L], *rec, dev)
    for t in (cache.k_norm, cache.v_norm):
        if t is not None:
            t[:, :, L - 3:L] = value
    seen = np.zeros((N, L), bool)
    seen[:, :L - N] = True
    for j in range(N):
        seen[j, L - N:min(L - N + j + 1, L - 3)] = True
    words = np.zeros((1, N, (N + 31) // 32), np.uint32)
    for j in range(N):
        for i in np.flatnonzero(seen[j, L - N:]):
            words[0, j, i >> 5] |= np.uint32(1 << (i & 31))
    q = wl.random_fp16(28, (1, Hq, N, 128))
    qd, ctx = H.upload(q, dev), tqf.Context()
    out = torch.empty_like(qd)
    tqf.tq_tree_attention(ctx, cache, qd, out, torch.from_numpy(words.view(np.int32)).to(dev), L)
    assert tqf.tq_get_status(ctx) == 0
    got = out.float().cpu().numpy()
    for h in range(Hkv):
        K, V = S.kv_of(mode, rec, 0, h, L)
        want, bound = S.attention_rows(q[0, h * G:(h + 1) * G].reshape(-1, 128), K, V, np.tile(seen, (G, 1)),
                                       1 / math.sqrt(128))
        S.assert_rows(got[0, h * G:(h + 1) * G], want, bound, f"h{h}")
