"""Attention weights of calls whose workspace would pass its bound, which are taken in blocks
of sequences, of KV heads or of queries: short sequences in caches (and with hints) that are
very long, many sequences, and more queries than a block holds, against the 64-bit form; and
long caches whose records lie past 32-bit offsets, with queries that tell them apart."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
from tests import helpers as H
from tests import keeping_helpers as K

pytestmark = pytest.mark.gpu

BOUND = 512 << 20      # of a call's workspace, where one KV head of one sequence keeps to it


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_kv_cache_flash_gb300 import build
    build.build()
    yield torch.device("cuda", 0)
    torch.cuda.empty_cache()


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def poisoned(mode, B, Hkv, cap, lengths, key, dev):
    """A cache with random records at its tokens and NaN keys everywhere else, and the
    records [B, Hkv, max(lengths), ..] on the host."""
    n = max(lengths)
    rec = H.random_cache(mode, B, Hkv, n, key)
    cache = tqf.Cache(tqf.MODES[mode], B, Hkv, cap, dev)
    (cache.k_data if cache.k_norm is None else cache.k_norm).fill_(float("nan"))
    cache.k_data[:, :, :n] = H.upload(rec[0], dev)
    if cache.k_norm is not None:
        cache.k_norm[:, :, :n] = H.upload(rec[1], dev)
    cache.lengths.copy_(i32(lengths, dev))
    return cache, rec


def queries(key, shape, dev):
    return torch.randn(shape, generator=torch.Generator(device=dev).manual_seed(key), device=dev).half()


def check(w, w0, mode, rec, q, lengths, seen, Hkv, decay, sequences):
    """Sequences of w [B, Hkv, cap] against the 64-bit form, w0 the weights before."""
    for b in sequences:
        L = lengths[b]
        one = [None if r is None else r[b:b + 1] for r in rec]
        A, bound = K.weights(mode, one, q[b:b + 1].cpu().numpy(), [L], Hkv)
        got = w[b].cpu().numpy().astype(np.float64)
        old = w0[b].cpu().numpy()
        base = np.where(np.arange(L) < seen[b], decay * old[:, :L].astype(np.float64), 0.0)
        off = np.abs(got[:, :L] - base - A[0, :, :L]) - bound[0, :, :L] - 2.0 ** -22 * base
        assert L == 0 or (np.all(np.isfinite(got[:, :L])) and off.max() <= 0), f"sequence {b}: {off.max():.2e}"
        assert np.array_equal(got[:, L:], old[:, L:]), f"sequence {b}"


def used(run):
    """Device memory that a call takes and keeps."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.mem_get_info()[0]
    run()
    torch.cuda.synchronize()
    return before - torch.cuda.mem_get_info()[0]


@pytest.mark.parametrize("mode,B,Hq,Hkv,T,cap", [
    ("turbo3", 5, 32, 8, 1, 850_000),         # 4 rows, 544 MB of scores: 3 sequences and 2
    ("turbo4_asym", 7, 28, 4, 1, 620_000),    # 7 rows, 556 MB
    ("turbo4", 2, 16, 2, 2, 2_200_000),       # 16 rows, 563 MB: a sequence and a sequence
    ("turbo4k_3v", 3, 32, 8, 1, 4_300_000),   # a sequence's 550 MB: KV heads of one
    ("turbo4_asym", 1, 32, 2, 1, 4_300_000),  # 16 rows: a KV head and a KV head
])
def test_steps_of_short_sequences_in_long_caches(dev, mode, B, Hq, Hkv, T, cap):
    lengths = [(0, T, 333, 64, 129, 17, 400)[(3 * b + 2) % 7] for b in range(B)]
    cache, rec = poisoned(mode, B, Hkv, cap, lengths, 500, dev)
    seen = [(1000, 0, 50)[b % 3] for b in range(B)]
    q = queries(501, (B, Hq, T, 128), dev)
    w = torch.rand(B, Hkv, cap, device=dev)
    w0, sums = w[:, :, :512].clone(), w[:, :, 512:].double().sum().item()
    ctx, sd = tqf.Context(), i32(seen, dev)
    got = used(lambda: tqf.tq_attention_weights(ctx, cache, q, w, cap, decay=0.5, seen=sd))
    assert got <= BOUND + (64 << 20)
    check(w[:, :, :512], w0, mode, rec, q, lengths, seen, Hkv, 0.5, range(B))
    assert w[:, :, 512:].double().sum().item() == sums
    assert tqf.tq_get_status(ctx) == (tqf.TQ_STATUS_SHORT_CONTEXT if min(lengths) < T else 0)


def test_a_captured_step_of_blocks(dev):
    """A step captured with the cache's capacity as its hint, replayed as the sequences grow."""
    mode, B, Hq, Hkv, cap = "turbo4", 3, 8, 8, 1_450_000
    cache, rec = poisoned(mode, B, Hkv, cap, [700] * B, 510, dev)
    w = torch.zeros(B, Hkv, cap, device=dev)
    q = queries(511, (B, Hq, 1, 128), dev)
    ctx = tqf.Context()
    run = lambda: tqf.tq_attention_weights(ctx, cache, q, w, cap, decay=0.0)  # noqa: E731
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for lengths in ([1, 700, 50], [333, 7, 699]):
        cache.lengths.copy_(i32(lengths, dev))
        w.fill_(3.0)
        g.replay()
        check(w[:, :, :720], torch.full((B, Hkv, 720), 3.0), mode, rec, q, lengths, [0] * B, Hkv, 0.0, range(B))
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("mode,B,Hkv,G,T", [
    ("turbo4", 601, 8, 2, 12),       # 4,808 units of a single query tile: 640 MB in one go
    ("turbo3", 2050, 2, 4, 35),      # 4,100 units of two
    ("turbo4k_3v", 600, 8, 16, 20),  # 4,800 of two pairs of them
])
def test_many_sequences(dev, mode, B, Hkv, G, T):
    lengths = [T + (7 * b) % 13 if b % 50 else b % 3 for b in range(B)]
    cache, rec = poisoned(mode, B, Hkv, 48, lengths, 520, dev)
    seen = [(9, 0, 30)[b % 3] for b in range(B)]
    q = queries(521, (B, G * Hkv, T, 128), dev)
    w = torch.rand(B, Hkv, 48, device=dev)
    w0, ctx, sd = w.clone(), tqf.Context(), i32(seen, dev)
    got = used(lambda: tqf.tq_attention_weights(ctx, cache, q, w, 48, decay=0.5, seen=sd))
    assert got <= BOUND + (64 << 20)
    half = B // 2
    check(w, w0, mode, rec, q, lengths, seen, Hkv, 0.5,
          sorted({0, 1, 2, 50, half - 1, half, half + 1, B - 2, B - 1, *range(3, B, B // 12)}))
    # every row's weights add to 1 (all sums together, off by their roundings)
    at = torch.arange(48, device=dev)
    L = i32(lengths, dev).view(-1, 1, 1)
    base = torch.where((at < sd.view(-1, 1, 1)) & (at < L), 0.5 * w0.double(), torch.where(at < L, 0.0, w0.double()))
    rows = G * Hkv * sum(min(n, T) for n in lengths)
    assert abs((w.double() - base).sum().item() - rows) < 1e-4 * rows
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_SHORT_CONTEXT


@pytest.mark.parametrize("mode", ["turbo4", "turbo3_asym"])
def test_queries_in_blocks(dev, mode):
    """Pairs of query tiles past the first block's: with a hint of 131,072, 64 pairs in blocks of
    51 (quantized K) or 63 (fp16 K), of other queries each."""
    B, Hq, Hkv, T, cap = 4, 512, 4, 128, 131072
    lengths = [328, 129, 250, 123]
    cache, rec = poisoned(mode, B, Hkv, cap, lengths, 530, dev)
    seen = [(100, 0, 1000)[b % 3] for b in range(B)]
    q = queries(531, (B, Hq, T, 128), dev)
    w = torch.rand(B, Hkv, cap, device=dev)
    w0, ctx, sd = w.clone(), tqf.Context(), i32(seen, dev)
    got = used(lambda: tqf.tq_attention_weights(ctx, cache, q, w, cap, decay=0.5, seen=sd))
    assert got <= BOUND + (64 << 20)
    check(w, w0, mode, rec, q, lengths, seen, Hkv, 0.5, range(B))
    for b in range(B):
        n = lengths[b]
        base = torch.where(torch.arange(n, device=dev) < seen[b], 0.5 * w0[b, :, :n].double(), 0.0)
        rows = Hq * min(n, T)
        assert abs((w[b, :, :n].double() - base).sum().item() - rows) < 1e-4 * rows
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_SHORT_CONTEXT


@pytest.mark.parametrize("mode,Hkv,cap,lengths,T", [
    ("turbo4_asym", 2, 6_000_000, [300, 64], 1),   # K rows of the last head 4.6 GB behind the first's
    ("turbo4_asym", 2, 6_000_000, [300, 64], 30),
    ("turbo4_asym", 2, 6_000_000, [300, 150], 70),
    ("turbo4", 8, 9_000_000, [200, 333], 1),       # codes of 9.2 GB, norms of 288 MB
    ("turbo4", 8, 9_000_000, [200, 333], 20),
    ("turbo3", 8, 9_000_000, [200, 333], 100),
])
def test_records_past_32_bit_offsets(dev, mode, Hkv, cap, lengths, T):
    """Every unit's records its own, NaN (or zero codes) wherever else an offset could lead."""
    B, G = len(lengths), 2
    cache, rec = poisoned(mode, B, Hkv, cap, lengths, 540, dev)
    q = queries(541, (B, G * Hkv, T, 128), dev)
    w = torch.full((B, Hkv, cap), 2.0, device=dev)
    ctx = tqf.Context()
    tqf.tq_attention_weights(ctx, cache, q, w, max(lengths), decay=0.0)
    n = max(lengths) + 16
    check(w[:, :, :n], torch.full((B, Hkv, n), 2.0), mode, rec, q, lengths, [0] * B, Hkv, 0.0, range(B))
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("mode,T", [("turbo4_asym", 1), ("turbo3", 2), ("turbo4_asym", 20), ("turbo4", 40),
                                    ("turbo3", 8)])   # (16 rows: 576 MB of scores for one KV head)
def test_tokens_past_2_gb_within_a_sequence(dev, mode, T):
    """8,999,000 tokens that score 0 but for some, most of them behind the first 8 million: a
    row's softmax has e^0 from each of the others that it sees."""
    cap, L, Hq = 9_000_000, 8_999_000, 2
    cache = tqf.Cache(tqf.MODES[mode], 1, 1, cap, dev)
    rng = np.random.default_rng(7)
    at = np.sort(np.concatenate([rng.choice(8_000_000, 30, replace=False), 8_000_000 + rng.choice(L - 8_000_000 - 64, 200, replace=False),
                                 L - 1 - np.arange(0, 60, 3)]))
    rec = H.random_cache(mode, 1, 1, len(at), 550)
    where = torch.from_numpy(at).to(dev)
    cache.k_data[:, :, where] = H.upload(rec[0], dev)
    if cache.k_norm is not None:     # (norms of 0 elsewhere)
        cache.k_norm[:, :, where] = H.upload(rec[1], dev)
    cache.lengths.fill_(L)
    q = queries(551, (1, Hq, T, 128), dev)
    scale = 1.0 / math.sqrt(128.0)
    s, size = K.scores_of(mode, rec, q[0].cpu().numpy(), 0, 0, len(at), scale)
    last = np.tile(L - T + np.arange(T), Hq)                       # the rows' last tokens
    seen = at[None] <= last[:, None]
    z = np.where(seen, np.exp(np.where(seen, s, 0.0)), 0.0).sum(1) + (last + 1 - seen.sum(1))
    w = torch.full((1, 1, cap), 2.0, device=dev)
    ctx = tqf.Context()
    tqf.tq_attention_weights(ctx, cache, q, w, cap, decay=0.0)
    got = w[0, 0].double()
    # scores' errors, the logarithm (24 at most: 1.5 steps of 2^-19), exp2's, the sums of a row's
    # 9 million terms (chains of 32, tiles, and shares of some hundred tiles)
    rel = 2 * K.SCORE * size.max() + 1.04 * 2.0 ** -19 + 2 * K.EXP2 + (400 + 2 * T) * 2.0 ** -24
    want = np.where(seen, np.exp(s) / z[:, None], 0.0).sum(0)
    assert np.all(np.abs(got[where].cpu().numpy() - want) <= rel * want)
    zero = torch.ones(L, dtype=torch.bool, device=dev)
    zero[where] = False
    # (of the others, those that every row sees have sum 1 / z)
    zero[L - T:] = False
    flat = float((1 / z).sum())
    assert torch.all(torch.abs(got[:L][zero] - flat) <= rel * flat)
    assert torch.all(got[L:] == 2) and tqf.tq_get_status(ctx) == 0
