"""Eviction by weight on the GPU (tq_cache_evict): places, records and weights equal to
the host's, in every mode, in place and into another cache, for every variant of the
selection; ties, NaN and infinite weights; bad counts; graphs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
from tests import helpers as H
from tests import keeping_helpers as K
from tests.test_gpu_cache_moves import make, parts

pytestmark = pytest.mark.gpu

MODES = sorted(tqf.MODES)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_kv_cache_flash_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def heavy(shape, seed, ties=True):
    """Weights over many magnitudes, some of them equal, some 0."""
    rng = np.random.default_rng(seed)
    w = np.exp(rng.standard_normal(shape) * 3).astype(np.float32)
    if ties:
        w[rng.random(shape) < 0.2] = 0
        w[rng.random(shape) < 0.2] = 1.25
    return w


def run_evict(dev, mode, cap, lengths, counts, sinks, recent, w, other, Hkv=2, seed=1, bad=(), hint=None, dst_cap=None,
              weights_in_place=False):
    B = len(lengths)
    src, rs = make(mode, B, Hkv, cap, lengths, seed, dev)
    dcap = cap if not other else dst_cap or (max(max(counts), 1) + 15) // 16 * 16
    dst, rd = (src, rs) if not other else make(mode, B, Hkv, dcap, [5 % dcap] * B, seed + 1, dev)
    before = [None if r is None else r.copy() for r in rs]
    mk = max(max(counts), 1)
    kept = torch.full((B, Hkv, mk), -7, dtype=torch.int32, device=dev)
    wd = torch.from_numpy(w).to(dev)
    nw = wd if weights_in_place else torch.full((B, Hkv, dcap), -7.0, device=dev)
    nw0 = nw.cpu().numpy()
    ctx = tqf.Context()
    tqf.tq_cache_evict(ctx, dst, src, wd, i32(counts, dev), kept, hint or cap, new_weights=nw, sinks=sinks, recent=recent)
    status = tqf.tq_get_status(ctx)
    want_kept, want_w = np.full((B, Hkv, mk), -7), nw0.copy()
    want_len = list(lengths) if not other else [5 % dcap] * B
    for b in range(B):
        if b in bad:
            continue
        for h in range(Hkv):
            at = K.evict(w[b, h], lengths[b], counts[b], sinks, recent)
            n = len(at)
            want_kept[b, h, :n] = at
            want_w[b, h, :n] = w[b, h, at]
            for r, s in zip(rd, before):
                if r is not None:
                    r[b, h, :n] = s[b, h, at]
        want_len[b] = min(lengths[b], counts[b])
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(nw.cpu().numpy(), want_w, equal_nan=True)
    assert dst.lengths.cpu().tolist() == want_len
    for got, r in zip(parts(dst), rd):
        if r is not None:
            assert np.array_equal(got.view(np.uint8), np.ascontiguousarray(r).view(np.uint8))
    if other:   # the source is left as it was
        assert src.lengths.cpu().tolist() == list(lengths)
        for got, r in zip(parts(src), before):
            if r is not None:
                assert np.array_equal(got.view(np.uint8), np.ascontiguousarray(r).view(np.uint8))
    if not weights_in_place:
        assert np.array_equal(wd.cpu().numpy(), w, equal_nan=True)
    return status


@pytest.mark.parametrize("other", [False, True], ids=["in_place", "other"])
@pytest.mark.parametrize("mode", MODES)
def test_every_mode(dev, mode, other):
    lengths, counts = [600, 257, 0, 31, 8, 500, 77], [300, 256, 5, 40, 8, 9, 12]
    w = heavy((7, 2, 608), 2)
    assert run_evict(dev, mode, 608, lengths, counts, 3, 5, w, other) == 0


@pytest.mark.parametrize("other", [False, True], ids=["in_place", "other"])
@pytest.mark.parametrize("mode", MODES)
def test_every_mode_with_many_units(dev, mode, other):
    """More units than CTAs that are resident at once: the first ones are done while the
    lengths of others are still read."""
    rng = np.random.default_rng(16)
    lengths = [int(x) for x in rng.integers(0, 1301, 100)]
    counts = [int(x) for x in rng.integers(12, 1200, 100)]
    bad = [int(b) for b in rng.choice(100, 9, replace=False)]
    for b in bad:
        counts[b], lengths[b] = -3, 900
    w = heavy((100, 8, 1312), 17)
    status = run_evict(dev, mode, 1312, lengths, counts, 3, 5, w, other, Hkv=8, bad=bad)
    assert status == tqf.TQ_STATUS_BAD_INDEX
    assert run_evict(dev, mode, 1312, [1300] * 100, [700] * 100, 0, 0, w, other, Hkv=8, weights_in_place=not other) == 0


@pytest.mark.parametrize("L,n", [
    (1, 1), (2, 1), (33, 32), (4096, 1), (4095, 2000),       # 8 keys a thread
    (4097, 4096), (8192, 3001), (8191, 17),                  # 16, or 8 of twice the threads
    (16384, 9000), (12001, 12000),                           # 32, or 16
    (32768, 20000), (20001, 5),                              # 32 of 1024 threads
    (32769, 1234), (70000, 40001),                           # weights read anew
])
@pytest.mark.parametrize("wide", [True, False], ids=["few_units", "many_units"])
def test_lengths(dev, L, n, wide):
    """Each variant of the selection (which goes by the longest sequence and the number of
    units), in place, over more than one round of the cluster that moves."""
    cap = (L + 15) // 16 * 16
    Hkv = 1 if wide else (160 if L <= 8192 else 154)
    if not wide and L > 20001:
        pytest.skip("one variant whatever the units")
    w = heavy((1, Hkv, cap), L)
    assert run_evict(dev, "turbo3", cap, [L], [n], min(2, n // 4), min(3, n // 4), w, False, Hkv=Hkv) == 0


@pytest.mark.parametrize("mode", ["turbo4_asym", "turbo4"])
@pytest.mark.parametrize("other", [False, True])
def test_many_rounds(dev, mode, other):
    w = heavy((2, 2, 9008), 5)
    assert run_evict(dev, mode, 9008, [9000, 5000], [7001, 3000], 4, 64, w, other) == 0


def test_weights_of_every_kind(dev):
    """Infinities, NaN (as -inf), zeros of both signs, subnormals and negative numbers; the
    first of equal ones stay."""
    rng = np.random.default_rng(9)
    kinds = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-45, -1e-45, 1e-40, -3.5, 2.0, 3.4e38, -3.4e38, -np.nan], np.float32)
    w = kinds[rng.integers(0, len(kinds), (3, 2, 1008))]
    for counts in ([1, 500, 999], [77, 300, 640], [1000, 90, 10]):
        for other in (False, True):
            assert run_evict(dev, "turbo3", 1008, [1000] * 3, counts, 0, 1, w, other) == 0
    same = np.zeros((3, 2, 1008), np.float32)      # all equal
    assert run_evict(dev, "turbo3", 1008, [1000, 999, 33], [500, 998, 1], 1, 0, same, False) == 0
    same[:] = np.nan
    assert run_evict(dev, "turbo3", 1008, [1000, 999, 33], [500, 998, 20], 2, 9, same, True) == 0


@pytest.mark.parametrize("other", [False, True])
def test_protected_tokens_alone(dev, other):
    w = heavy((4, 2, 208), 10)
    assert run_evict(dev, "turbo4", 208, [200, 21, 20, 19], [20] * 4, 8, 12, w, other) == 0
    assert run_evict(dev, "turbo4", 208, [200, 21, 1, 0], [0] * 4, 0, 0, w, other) == 0       # nothing stays
    assert run_evict(dev, "turbo4", 208, [200, 208, 10, 20], [20] * 4, 20, 0, w, other) == 0   # the first ones
    assert run_evict(dev, "turbo4", 208, [200, 208, 10, 20], [20] * 4, 0, 20, w, other) == 0   # the last ones


def test_weights_move_in_place(dev):
    w = heavy((3, 2, 3008), 11)
    assert run_evict(dev, "turbo4_asym", 3008, [3000, 2500, 100], [2400, 30, 200], 4, 10, w, False, weights_in_place=True) == 0


@pytest.mark.parametrize("other", [False, True])
def test_bad_counts_leave_their_sequences_untouched(dev, other):
    w = heavy((6, 2, 112), 12)
    lengths = [100, 100, 100, 100, 5, 100]
    # too few for the protected ones; below 0; fine; (max_keep is the largest: 60); few but
    # nothing to evict is fine too; fine
    counts = [7, -1, 8, 60, 5, 20]
    assert run_evict(dev, "turbo3", 112, lengths, counts, 4, 4, w, other, bad=(0, 1)) == tqf.TQ_STATUS_BAD_INDEX
    if other:     # more than the destination holds, and longer than the hint
        assert run_evict(dev, "turbo3", 112, lengths, [20, 60, 8, 10, 5, 33], 4, 4, w, True, bad=(1, 5),
                         dst_cap=32) == tqf.TQ_STATUS_CAPACITY
    assert run_evict(dev, "turbo3", 112, lengths, [20] * 6, 4, 4, w, other, bad=(0, 1, 2, 3, 5), hint=99) == tqf.TQ_STATUS_CAPACITY


def test_more_kept_than_the_list_holds(dev):
    cache, _ = make("turbo3", 2, 1, 64, [60, 60], 13, dev)
    kept = torch.full((2, 1, 10), -7, dtype=torch.int32, device=dev)
    ctx = tqf.Context()
    tqf.tq_cache_evict(ctx, cache, cache, torch.rand(2, 1, 64, device=dev), i32([11, 10], dev), kept, 64)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_BAD_INDEX
    assert cache.lengths.cpu().tolist() == [60, 10] and torch.all(kept[0] == -7)


@pytest.mark.parametrize("other", [False, True])
def test_replayed(dev, other):
    """A captured eviction goes by the lengths and weights of the replay."""
    mode, B, Hkv, cap = "turbo4", 2, 2, 512
    src, rec = make(mode, B, Hkv, cap, [500, 400], 14, dev)
    dst = make(mode, B, Hkv, 128, [0, 0], 15, dev)[0] if other else src
    w, kept = torch.rand(B, Hkv, cap, device=dev), torch.zeros(B, Hkv, 100, dtype=torch.int32, device=dev)
    count, ctx = i32([100, 90], dev), tqf.Context()
    go = lambda: tqf.tq_cache_evict(ctx, dst, src, w, count, kept, cap, sinks=1, recent=2)  # noqa: E731
    go()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for ls, seed in (([512, 50], 3), ([200, 101], 4)):
        src.lengths.copy_(i32(ls, dev))
        w.copy_(torch.from_numpy(heavy((B, Hkv, cap), seed)))
        for t, r in zip((src.k_data, src.k_norm, src.v_data, src.v_norm), rec):
            if t is not None:
                t.copy_(torch.from_numpy(r))
        g.replay()
        for b in range(B):
            for h in range(Hkv):
                at = K.evict(w[b, h].cpu().numpy(), ls[b], int(count[b]), 1, 2)
                assert np.array_equal(kept[b, h, :len(at)].cpu().numpy(), at)
                for t, r in zip((dst.k_data, dst.k_norm, dst.v_data, dst.v_norm), rec):
                    if t is not None:
                        assert np.array_equal(t[b, h, :len(at)].cpu().numpy().view(np.uint8), np.ascontiguousarray(r[b, h, at]).view(np.uint8))
        assert dst.lengths.cpu().tolist() == [min(a, int(c)) for a, c in zip(ls, count)]
    assert tqf.tq_get_status(ctx) == 0
