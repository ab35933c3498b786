"""Attention weights on the GPU (tq_attention_weights) against the 64-bit form: modes,
group sizes, from one query to whole prompts, masks, lengths, hints, decay and the
tokens that have a weight already; queries of 0, whose weights have a closed form, for
large calls; graphs, streams and contexts."""
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


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def close(got, want, bound, what=""):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    off = np.abs(got - want) - bound
    assert off.max() <= 0, f"{what}: {off.max():.3e} past the bound at {np.unravel_index(off.argmax(), off.shape)}"


CASES = [
    # mode, Hq, Hkv, contexts before the block, Tq, q scale
    ("turbo3", 4, 2, [0], 1, 1.0),                          # one token
    ("turbo4", 8, 2, [300, 17], 1, 1.0),                    # 4 rows
    ("turbo3", 28, 4, [517, 33, 0], 1, 1.0),                # 7 rows
    ("turbo4_asym", 28, 4, [700, 0, 129], 1, 1.0),
    ("turbo4k_3v", 8, 8, [250, 8], 3, 1.0),                 # G 1
    ("turbo3_asym", 16, 2, [1000, 31], 2, 4.0),             # 16 rows
    ("turbo4", 16, 1, [511, 63, 64, 65], 1, 1.0),           # 16 rows, lengths at stages' ends
    ("turbo4", 8, 2, [5, 1], 4, 8.0),                       # 16 rows over fewer tokens than a stage
    ("turbo3", 28, 4, [2000], 1, 24.0),                     # peaked
    ("turbo3", 8, 2, [40 + i for i in range(40)], 1, 1.0),  # over 32 sequences
    # (many units: two kernels; the ones above mostly take one)
    ("turbo4", 28, 4, [11 * i for i in range(12)], 1, 1.0),
    ("turbo3", 28, 4, [63 + i for i in range(12)], 1, 1.0),
    ("turbo3_asym", 28, 4, [200, 0, 31, 777], 1, 1.0),
    ("turbo4k_3v", 16, 2, [5 + 13 * i for i in range(20)], 2, 1.0),
    ("turbo3", 16, 2, [300 - 9 * i for i in range(20)], 2, 1.0),
    ("turbo4_asym", 16, 2, [90, 33, 0, 2, 500, 64], 2, 1.0),
    ("turbo4", 8, 2, [2 * i for i in range(40)], 1, 16.0),
    ("turbo4", 8, 2, [300, 2], 5, 1.0),                     # 20 rows
    ("turbo3", 28, 4, [517, 33], 16, 1.0),                  # 112 rows
    ("turbo4", 32, 4, [700, 0, 129, 1500], 16, 1.0),        # 128 rows
    ("turbo3_asym", 28, 4, [400, 90], 18, 4.0),             # 126 rows
    ("turbo3", 24, 8, [300, 1100], 43, 1.0),                # 129 rows
    ("turbo4_asym", 28, 4, [700, 0, 129], 33, 1.0),         # 231 rows
    ("turbo4", 32, 8, [900, 1, 260], 64, 1.0),              # 256 rows
    ("turbo3", 32, 8, [611], 65, 16.0),                     # just past them
    ("turbo3_asym", 8, 8, [127, 128, 129], 40, 1.0),        # rows of one head
    ("turbo4k_3v", 128, 1, [333], 3, 1.0),                  # G 128: 384 rows
    ("turbo4", 4, 4, [0, 100], 300, 1.0),                   # a prompt
    ("turbo4_asym", 16, 2, [0, 50], 270, 1.0),              # G 8: heads that end inside a tile
    ("turbo3", 4, 2, [1, 0, 640], 513, 4.0),
    ("turbo3", 8, 2, [30 + 7 * i for i in range(40)], 20, 1.0),   # over 32 groups of sequences
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}-b{len(c[3])}-t{c[4]}-q{c[5]}")
def test_against_the_64_bit_form(dev, case):
    mode, Hq, Hkv, ctxs, T, qs = case
    B, lengths = len(ctxs), [c + T for c in ctxs]
    cap = (max(lengths) + 15) // 16 * 16 + 16
    rec = H.random_cache(mode, B, Hkv, cap, 100 + T)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, lengths, *rec, dev)
    q = (wl.random_fp16(200 + T, (B, Hq, T, 128)).astype(np.float32) * qs).astype(np.float16)
    A, bound = K.weights(mode, rec, q, lengths, Hkv)
    old = np.random.default_rng(3).random((B, Hkv, cap)).astype(np.float32) * 4
    ctx = tqf.Context()
    qd = H.upload(q, dev)
    for decay in (1.0, 0.75, 0.0):
        # (what lies past the length, and with decay 0 everything, may be anything)
        w0 = old.copy()
        if decay == 0.0:
            w0[:] = np.nan
        w = torch.from_numpy(w0).to(dev)
        tqf.tq_attention_weights(ctx, cache, qd, w, max(lengths), decay=decay)
        for b, L in enumerate(lengths):
            base = np.where(np.arange(L) < L - T, (old[b, :, :L] * np.float64(decay)), 0.0)
            close(w[b, :, :L], base + A[b, :, :L], bound[b, :, :L] + 2.0 ** -22 * base, f"decay {decay} sequence {b}")
            assert np.array_equal(w[b, :, L:].cpu().numpy(), w0[b, :, L:], equal_nan=True)
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("mode,Hq,T", [("turbo4", 8, 1), ("turbo4_asym", 28, 1), ("turbo3", 8, 9), ("turbo3", 28, 80)])
def test_tokens_with_a_weight_already(dev, mode, Hq, T):
    B, Hkv, cap = 4, 4, 208
    lengths = [200, 199, 150, 81]
    rec = H.random_cache(mode, B, Hkv, cap, 11)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, lengths, *rec, dev)
    q = wl.random_fp16(12, (B, Hq, T, 128))
    A, bound = K.weights(mode, rec, q, lengths, Hkv)
    seen = [0, 200, 77, 500]      # none, all (and the token past the end), some, all
    old = np.random.default_rng(4).random((B, Hkv, cap)).astype(np.float32)
    w0 = old.copy()
    for b in range(B):
        w0[b, :, seen[b]:] = np.nan
    w = torch.from_numpy(w0).to(dev)
    ctx = tqf.Context()
    tqf.tq_attention_weights(ctx, cache, H.upload(q, dev), w, cap, decay=0.5, seen=i32(seen, dev))
    for b, L in enumerate(lengths):
        base = np.where(np.arange(L) < seen[b], 0.5 * old[b, :, :L], 0.0)
        close(w[b, :, :L], base + A[b, :, :L], bound[b, :, :L] + 2.0 ** -22 * base, f"sequence {b}")


@pytest.mark.parametrize("mode,Hq,T", [("turbo4", 8, 2), ("turbo3_asym", 8, 8), ("turbo3", 16, 70)])
def test_rows_that_see_no_token(dev, mode, Hq, T):
    """Sequences shorter than the block: the first queries add nothing; an empty one stays as it was."""
    B, Hkv, cap = 4, 2, 96
    lengths = [0, 1, T - 1, T + 3]
    rec = H.random_cache(mode, B, Hkv, cap, 21)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, lengths, *rec, dev)
    q = wl.random_fp16(22, (B, Hq, T, 128))
    A, bound = K.weights(mode, rec, q, lengths, Hkv)
    w = torch.full((B, Hkv, cap), 7.0, device=dev)
    ctx = tqf.Context()
    tqf.tq_attention_weights(ctx, cache, H.upload(q, dev), w, cap, decay=0.0)
    for b, L in enumerate(lengths):
        close(w[b, :, :L], A[b, :, :L], bound[b, :, :L]) if L else None
        assert torch.all(w[b, :, L:] == 7.0)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_SHORT_CONTEXT
    # the same block over sequences that hold it
    cache.lengths.fill_(T)
    tqf.tq_attention_weights(ctx, cache, H.upload(q, dev), w, cap, decay=0.0)
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("mode,Hq,T,hint", [("turbo4", 8, 1, 90), ("turbo3", 8, 2, 64), ("turbo4_asym", 8, 12, 100), ("turbo4", 4, 60, 77)])
def test_tokens_past_the_hint_are_not_looked_at(dev, mode, Hq, T, hint):
    B, Hkv, cap = 2, 2, 160
    lengths = [150, 80]
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, B, Hkv, cap, 31)]
    if rec[1] is not None:
        rec[1][:, :, hint:] = np.nan
    else:
        rec[0][:, :, hint:] = np.nan
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, lengths, *rec, dev)
    q = wl.random_fp16(32, (B, Hq, T, 128))
    A, bound = K.weights(mode, rec, q, lengths, Hkv, hint=hint)
    w = torch.full((B, Hkv, cap), 7.0, device=dev)
    tqf.tq_attention_weights(tqf.Context(), cache, H.upload(q, dev), w, hint, decay=0.0)
    for b, L in enumerate(lengths):
        n = min(L, hint)
        close(w[b, :, :n], A[b, :, :n], bound[b, :, :n])
        assert torch.all(w[b, :, n:] == 7.0)


@pytest.mark.parametrize("mode,T", [("turbo4", 2), ("turbo4_asym", 3), ("turbo3", 40), ("turbo4_asym", 40)])
def test_nan_stays_with_the_rows_and_tokens_that_meet_it(dev, mode, T):
    """A NaN query makes its row NaN: the tokens it sees, not the later ones; the same
    of a record that the first queries do not see, and of stale records past the length."""
    B, Hkv, Hq, cap, L = 2, 1, 1, 208, 180
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, B, Hkv, cap, 41)]
    k = rec[1] if rec[1] is not None else rec[0]
    k[:, :, L:] = np.nan                    # past the length
    k[1, :, L - 1] = np.nan                 # the last token: the last query alone sees it
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, [L, L], *rec, dev)
    q = np.array(wl.random_fp16(42, (B, Hq, T, 128)))
    q[0, 0, 0] = np.nan
    w = torch.zeros(B, Hkv, cap, device=dev)
    tqf.tq_attention_weights(tqf.Context(), cache, H.upload(q, dev), w, L, decay=0.0)
    got = w.cpu().numpy()
    assert np.all(np.isnan(got[0, 0, :L - T + 1])) and np.all(np.isfinite(got[0, 0, L - T + 1:L]))
    assert np.all(np.isnan(got[1, 0, :L]))   # (the last row is NaN and sees all)
    assert np.all(got[:, :, L:] == 0)
    # without the last query the second sequence is finite
    cache.lengths.fill_(L - 1)
    q[0, 0, 0] = 1
    w.zero_()               # (what lies past the length stays: the last token's NaN too)
    tqf.tq_attention_weights(tqf.Context(), cache, H.upload(q, dev), w, L, decay=0.0)
    assert torch.all(torch.isfinite(w))


@pytest.mark.parametrize("mode,Hq,Hkv,ctxs,T", [
    ("turbo3", 8, 1, [131000], 1),            # a long context of one sequence
    ("turbo4", 8, 2, [70000, 3], 2),
    ("turbo4_asym", 4, 1, [66000], 1),
    ("turbo3", 16, 2, [40000, 9], 20),        # windows
    ("turbo4_asym", 14, 2, [3000, 0], 1100),  # prompts: many pairs of query tiles
    ("turbo4", 128, 1, [7], 8192),            # more rows than a block of pairs holds
    ("turbo4", 64, 2, [0, 100], 4100),
])
def test_large_calls_by_their_closed_form(dev, mode, Hq, Hkv, ctxs, T):
    """Queries of 0 weigh all the tokens that they see alike: query j adds G / n_j to each
    of its n_j tokens."""
    B, lengths = len(ctxs), [c + T for c in ctxs]
    cap = (max(lengths) + 15) // 16 * 16
    cache = tqf.Cache(tqf.MODES[mode], B, Hkv, cap, dev)
    if cache.k_norm is not None:
        cache.k_data.random_(0, 256)
        cache.k_norm.uniform_(0.5, 20.0)
    else:
        cache.k_data.normal_()
    cache.lengths.copy_(i32(lengths, dev))
    w = torch.ones(B, Hkv, cap, device=dev)
    ctx = tqf.Context()
    q = torch.zeros(B, Hq, T, 128, dtype=torch.float16, device=dev)
    tqf.tq_attention_weights(ctx, cache, q, w, max(lengths), decay=1.0)
    G = Hq // Hkv
    for b, c in enumerate(ctxs):
        inv = 1.0 / (c + 1.0 + np.arange(T))
        tail = np.concatenate([np.cumsum(inv[::-1])[::-1], [0.0]])       # sum over queries j, j + 1, ..
        t = np.arange(lengths[b])
        want = G * tail[np.maximum(t - c, 0)]
        base = np.where(t < c, 1.0, 0.0)
        # exp2's error and that of the row's logarithm (numbers below 17), the sums in
        # chains of 32 rows, then of 256
        bound = want * (2 * K.EXP2 + 17 * 2.0 ** -23 + (64 + G * T / 256) * 2.0 ** -24) + 2.0 ** -23 * base
        close(w[b, :, :lengths[b]], np.tile(base + want, (Hkv, 1)), np.tile(bound, (Hkv, 1)), f"sequence {b}")
        assert torch.all(w[b, :, lengths[b]:] == 1)
    assert tqf.tq_get_status(ctx) == 0


def test_scale_and_a_codebook_of_its_own(dev):
    from oracle import tq_oracle as o
    B, Hkv, cap, L = 1, 2, 96, 90
    rec = H.random_cache("turbo4", B, Hkv, cap, 61)
    half = np.array([1, 2, 3, 5, 8, 13, 21, 34], np.float32) / 256
    cb = np.concatenate([-half[::-1], half]).tolist()
    cache = H.gpu_cache_from_records("turbo4", B, Hkv, cap, [L], *rec, dev)
    mine = tqf.Cache(tqf.MODES["turbo4"], B, Hkv, cap, dev, codebook_k=cb, codebook_v=cb)
    for a, c in ((mine.k_data, cache.k_data), (mine.k_norm, cache.k_norm), (mine.lengths, cache.lengths)):
        a.copy_(c)
    for T in (1, 30):
        q = wl.random_fp16(62, (B, 4, T, 128))
        w = torch.zeros(B, Hkv, cap, device=dev)
        tqf.tq_attention_weights(tqf.Context(), mine, H.upload(q, dev), w, L, decay=0.0, scale=0.02)
        for h in range(Hkv):
            s, size = K.scores_of("turbo4", rec, q[0, 2 * h:2 * h + 2], 0, h, L, 0.02, cbk=np.array(cb))
            seen = np.tile(np.arange(L)[None] <= (L - T + np.arange(T))[:, None], (2, 1))
            p = np.exp(np.where(seen, s, -np.inf) - np.where(seen, s, -np.inf).max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            close(w[0, h, :L], p.sum(0), p.sum(0) * (2 * K.SCORE * size.max() + 2.0 ** -18))


@pytest.mark.parametrize("T", [1, 24, 300])
def test_same_bits_again_on_other_streams_and_in_graphs(dev, T):
    """Eager, on another stream, replayed after the lengths have changed, and on a context
    that a larger call has used in between: the same bits."""
    mode, B, Hkv, Hq, cap = "turbo4", 3, 2, 8, 1008
    lengths = [1000, 700, 333]
    rec = H.random_cache(mode, B, Hkv, cap, 71)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, lengths, *rec, dev)
    q = H.upload(wl.random_fp16(72, (B, Hq, T, 128)), dev)
    ctx, w = tqf.Context(), torch.zeros(B, Hkv, cap, device=dev)
    run = lambda stream=None: tqf.tq_attention_weights(ctx, cache, q, w, cap, decay=0.0, stream=stream)  # noqa: E731
    run()
    first = w.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    w.zero_()
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    side.synchronize()
    assert torch.equal(w, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for ls in ([900, 1000, 301], lengths):
        cache.lengths.copy_(i32(ls, dev))
        w.zero_()
        g.replay()
        got = w.clone()
        w.zero_()
        tqf.tq_attention_weights(tqf.Context(), cache, q, w, cap, decay=0.0)
        assert torch.equal(got, w)
    big = torch.zeros(B, Hq, 400, 128, dtype=torch.float16, device=dev)
    tqf.tq_attention_weights(ctx, cache, big, torch.zeros_like(w), cap)      # (grows the workspace)
    w.zero_()
    g.replay()
    assert torch.equal(w, first) and tqf.tq_get_status(ctx) in (0, tqf.TQ_STATUS_SHORT_CONTEXT)


@pytest.mark.parametrize("mode,Hq,T", [("turbo4", 32, 5), ("turbo4", 32, 32), ("turbo3", 32, 9), ("turbo4_asym", 32, 20),
                                       ("turbo3", 32, 64)])
def test_cold_caches(dev, mode, Hq, T):
    """Copies that land late and out of order: the bits stay."""
    B, Hkv, cap = 8, 8, 4000
    cache = tqf.Cache(tqf.MODES[mode], B, Hkv, cap, dev)
    if cache.k_norm is not None:
        cache.k_data.random_(0, 256)
        cache.k_norm.uniform_(0.5, 20.0)
    else:
        cache.k_data.normal_()
    cache.lengths.fill_(cap)
    q = H.upload(wl.random_fp16(81, (B, Hq, T, 128)), dev)
    ctx, w = tqf.Context(), torch.zeros(B, Hkv, cap, device=dev)
    tqf.tq_attention_weights(ctx, cache, q, w, cap, decay=0.0)
    first = w.clone()
    assert abs(first.double().sum().item() - B * Hq * T) < 1e-4 * B * Hq * T
    other = torch.empty(300 << 20, dtype=torch.uint8, device=dev)
    for i in range(40):
        other.fill_(i)
        tqf.tq_attention_weights(ctx, cache, q, w, cap, decay=0.0)
        assert torch.equal(w, first)
    assert tqf.tq_get_status(ctx) == 0
