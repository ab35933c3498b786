"""Record moves on the GPU: keeping accepted tokens (tq_cache_compact) and
copying or forking sequences (tq_cache_copy), bit for bit against the same
moves of the arrays on the host, in every mode."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
from tests import helpers as H

pytestmark = pytest.mark.gpu

MODES = sorted(tqf.MODES)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_kv_cache_flash_gb300 import build
    build.build()
    return torch.device("cuda", 0)


def make(mode, B, Hkv, cap, lengths, key, dev):
    rec = H.random_cache(mode, B, Hkv, cap, key)
    return H.gpu_cache_from_records(mode, B, Hkv, cap, lengths, *rec, dev), [
        None if r is None else np.array(r) for r in rec]


def parts(c):
    return [None if t is None else t.cpu().numpy() for t in (c.k_data, c.k_norm, c.v_data, c.v_norm)]


def same(cache, want, lengths):
    for got, w in zip(parts(cache), want):
        assert (got is None) == (w is None)
        if got is not None:
            assert np.array_equal(got.view(np.uint8), np.ascontiguousarray(w).view(np.uint8))
    assert cache.lengths.cpu().tolist() == list(lengths)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def host_compact(rec, start, keep, count):
    for r in rec:
        if r is not None:
            for b, s in enumerate(start):
                src = [s + k for k in keep[b][:count[b]]]
                r[b, :, s:s + len(src)] = r[b][:, src]


@pytest.mark.parametrize("mode", MODES)
def test_compact_matches_the_host(dev, mode):
    B, Hkv, cap, N = 5, 3, 160, 77
    start = [0, 13, 83, 40, 7]
    keep = [[0, 5, 6, 30, 76], [1, 2, 3, 4, 5], [0, 1, 2, 0, 0], [76, 0, 0, 0, 0], [9, 9, 9, 9, 9]]
    count = [5, 5, 3, 1, 0]
    cache, rec = make(mode, B, Hkv, cap, [s + N for s in start], 41, dev)
    ctx = tqf.Context()
    tqf.tq_cache_compact(ctx, cache, i32(start, dev), i32(keep, dev), i32(count, dev), N)
    host_compact(rec, start, keep, count)
    same(cache, rec, [s + n for s, n in zip(start, count)])
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("mode", ["turbo3", "turbo4_asym", "turbo3_table"])
def test_compact_of_more_than_a_group_of_tokens(dev, mode):
    # overlapping moves over several groups of 32: every second, and all but the first
    B, Hkv, cap, N = 2, 2, 512, 300
    start, keep = [17, 200], [list(range(0, 300, 2)) + [0] * 149, list(range(1, 300))]
    count = [150, 299]
    cache, rec = make(mode, B, Hkv, cap, [s + N for s in start], 42, dev)
    ctx = tqf.Context()
    tqf.tq_cache_compact(ctx, cache, i32(start, dev), i32(keep, dev), i32(count, dev), N)
    host_compact(rec, start, keep, count)
    same(cache, rec, [167, 499])
    assert tqf.tq_get_status(ctx) == 0


def test_compact_leaves_bad_sequences_untouched(dev):
    B, cap, N = 8, 64, 8
    start = [0, -1, 60, 3, 3, 3, 3, 3]
    keep = [[1, 3, 5], [0, 1, 2], [0, 1, 2], [0, 8, 9], [2, 1, 3], [1, 1, 2], [0, 1, 2], [-1, 0, 1]]
    count = [3, 3, 3, 2, 3, 2, 4, 1]
    lengths = [20] * B
    cache, rec = make("turbo4", B, 2, cap, lengths, 43, dev)
    ctx = tqf.Context()
    tqf.tq_cache_compact(ctx, cache, i32(start, dev), i32(keep, dev), i32(count, dev), N)
    host_compact(rec, start[:1], keep, count)
    same(cache, rec, [3] + [20] * 7)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_BAD_INDEX
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("mode", MODES)
def test_copy_within_a_cache_matches_the_host(dev, mode):
    B, Hkv, cap = 7, 3, 608
    lengths = [600, 257, 0, 31, 8, 500, 77]
    cache, rec = make(mode, B, Hkv, cap, lengths, 51, dev)
    ctx = tqf.Context()
    # forks of 0, a whole copy of an empty sequence, a cut-off in place
    dst, src, n = [2, 4, 3, 5], [0, 0, 1, 5], [599, 0, 257, 499]
    tqf.tq_cache_copy(ctx, cache, cache, i32(dst, dev), i32(src, dev), 600, num_tokens=i32(n, dev))
    for d, s, m in zip(dst, src, n):
        for r in rec:
            if r is not None:
                r[d, :, :m] = r[s, :, :m]
        lengths[d] = m
    same(cache, rec, lengths)
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("mode", ["turbo3", "turbo4_asym", "turbo3_table"])
def test_copy_to_another_cache(dev, mode):
    src, rs = make(mode, 3, 2, 320, [300, 1, 0], 52, dev)
    dst, rd = make(mode, 4, 2, 1040, [9, 9, 9, 9], 53, dev)
    ctx = tqf.Context()
    tqf.tq_cache_copy(ctx, dst, src, i32([3, 0, 1], dev), i32([0, 1, 2], dev), 320)
    for d, s, m in ((3, 0, 300), (0, 1, 1)):
        for a, b in zip(rd, rs):
            if a is not None:
                a[d, :, :m] = b[s, :, :m]
    same(dst, rd, [1, 0, 9, 300])
    same(src, rs, [300, 1, 0])
    assert tqf.tq_get_status(ctx) == 0


def test_copy_skips_conflicts_and_bad_pairs(dev):
    lengths = [40, 30, 20, 10, 5, 6, 7, 8]
    cache, rec = make("turbo3", 8, 2, 64, lengths, 54, dev)
    small, rsm = make("turbo3", 2, 2, 16, [3, 3], 55, dev)
    ctx = tqf.Context()
    # 0 -> 4 and 1 -> 4 meet; 2 -> 0 would overwrite a source; 8 and -1 do not
    # exist; 2 -> 5 asks for more than there is; 3 -> 6 is fine
    pairs = [(0, 4, 40), (1, 4, 30), (2, 0, 20), (8, 7, 1), (0, -1, 1), (2, 5, 21), (3, 6, 10)]
    s, d, n = zip(*pairs)
    tqf.tq_cache_copy(ctx, cache, cache, i32(d, dev), i32(s, dev), 64, num_tokens=i32(n, dev))
    for r in rec:
        if r is not None:
            r[6, :, :10] = r[3, :, :10]
    lengths[6] = 10
    same(cache, rec, lengths)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_BAD_INDEX
    # past the destination's capacity, or past the hint
    tqf.tq_cache_copy(ctx, small, cache, i32([0], dev), i32([0], dev), 64)
    same(small, rsm, [3, 3])
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_CAPACITY
    tqf.tq_cache_copy(ctx, cache, cache, i32([7], dev), i32([0], dev), 39)
    same(cache, rec, lengths)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_CAPACITY


def test_many_pairs(dev):
    # more pairs than a CTA has threads
    B = 640
    cache, rec = make("turbo3", B, 1, 16, [7] * 300 + [0] * 340, 56, dev)
    ctx = tqf.Context()
    src, dst = [i % 300 for i in range(330)], [300 + i for i in range(330)]
    tqf.tq_cache_copy(ctx, cache, cache, i32(dst, dev), i32(src, dev), 16)
    for r in rec:
        if r is not None:
            r[300:630, :, :7] = r[src, :, :7]
    same(cache, rec, [7] * 630 + [0] * 10)
    assert tqf.tq_get_status(ctx) == 0


def test_moves_in_a_graph_and_on_another_stream(dev):
    cache, rec = make("turbo4", 3, 2, 128, [50, 0, 0], 57, dev)
    ctx = tqf.Context()
    args = (i32([1], dev), i32([0], dev))
    start, keep, count = i32([20, 10, 0], dev), i32([[0, 4], [3, 9], [0, 0]], dev), i32([2, 2, 0], dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tqf.tq_cache_copy(ctx, cache, cache, *args, 128, stream=side)   # an eager call creates the context
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tqf.tq_cache_copy(ctx, cache, cache, *args, 128)
        tqf.tq_cache_compact(ctx, cache, start, keep, count, 30)
    for r in rec:
        if r is not None:
            r[1, :, :50] = r[0, :, :50]
    before = [None if r is None else r.copy() for r in rec]
    for _ in range(2):
        # the replay starts from the same cache again
        H_reset(cache, before, [50, 50, 0])
        g.replay()
        torch.cuda.synchronize()
        want = [None if r is None else r.copy() for r in before]
        host_compact(want, [20, 10, 0], [[0, 4], [3, 9], [0, 0]], [2, 2, 0])
        same(cache, want, [22, 12, 0])
    assert tqf.tq_get_status(ctx) == 0


def H_reset(cache, rec, lengths):
    for t, r in zip((cache.k_data, cache.k_norm, cache.v_data, cache.v_norm), rec):
        if t is not None:
            t.copy_(torch.from_numpy(r))
    cache.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
