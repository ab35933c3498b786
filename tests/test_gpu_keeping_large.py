"""tq_attention_weights, tq_cache_evict and tq_verify_tree where offsets pass 32 bits, and
several calls at once."""
import numpy as np
import pytest
import torch

import quantized_kv_cache_flash_gb300 as tqf

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


@pytest.mark.parametrize("mode,Hkv,cap,ctxs,T", [
    ("turbo4_asym", 2, 6_000_000, [9, 1000], 1),       # the last head's K starts 4.6 GB behind the first's
    ("turbo4_asym", 2, 6_000_000, [9, 1000], 30),
    ("turbo4", 4, 9_000_000, [100, 700], 30),          # codes 4.0 GB
    ("turbo4", 4, 9_000_000, [100, 700], 2),
    ("turbo4_asym", 1, 9_000_000, [8_999_000], 1),     # tokens past 2 GB within one sequence
    ("turbo3", 1, 9_000_000, [8_999_000], 40),
])
def test_weights_of_a_long_cache(dev, mode, Hkv, cap, ctxs, T):
    """Queries of 0: query j adds G / n_j to each of its n_j tokens."""
    B, G = len(ctxs), 2
    lengths = [c + T for c in ctxs]
    cache = tqf.Cache(tqf.MODES[mode], B, Hkv, cap, dev)
    if cache.k_norm is not None:
        cache.k_norm.fill_(1.0)
    cache.lengths.copy_(i32(lengths, dev))
    w = torch.ones(B, Hkv, cap, device=dev)
    ctx = tqf.Context()
    q = torch.zeros(B, G * Hkv, T, 128, dtype=torch.float16, device=dev)
    tqf.tq_attention_weights(ctx, cache, q, w, max(lengths), decay=0.0)
    for b, c in enumerate(ctxs):
        n = c + 1.0 + torch.arange(T, device=dev, dtype=torch.float64)
        tail = torch.cat([torch.flip(torch.cumsum(torch.flip(1 / n, (0,)), 0), (0,)), torch.zeros(1, device=dev).double()])
        t = torch.arange(lengths[b], device=dev)
        want = G * tail[torch.clamp(t - c, min=0)]
        # log2 of at most 2^23.2 tokens: its error and one rounding, 1.5 steps of 2^-19, times
        # ln 2, beside exp2's 2^-22 and sums of at most 80 terms
        bound = want * (1.04 * 2.0 ** -19 + 2.0 ** -22 + 80 * 2.0 ** -24)
        for h in range(Hkv):
            assert torch.all(torch.abs(w[b, h, :lengths[b]].double() - want) <= bound)
            assert torch.all(w[b, h, lengths[b]:lengths[b] + 1000] == 1)
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("other", [False, True], ids=["in_place", "other"])
@pytest.mark.parametrize("mode,Hkv,cap,lengths", [
    ("turbo4_asym", 2, 6_000_000, [900, 5000]),
    ("turbo4_asym", 1, 9_000_000, [8_999_990]),
    ("turbo3", 1, 9_000_000, [8_999_990]),
])
def test_eviction_from_a_long_cache(dev, mode, Hkv, cap, lengths, other):
    B, n = len(lengths), 700
    cache = tqf.Cache(tqf.MODES[mode], B, Hkv, cap, dev)
    as_bytes = lambda t: t.view(torch.uint8).reshape(B, Hkv, t.shape[2], -1)  # noqa: E731
    for t in (cache.k_data, cache.v_data):
        as_bytes(t).random_(0, 256)
    cache.v_norm.copy_(torch.rand(cache.v_norm.shape, device=dev))
    cache.lengths.copy_(i32(lengths, dev))
    gen = torch.Generator(device=dev).manual_seed(3)
    w = torch.rand(B, Hkv, cap, device=dev, generator=gen)
    dst = tqf.Cache(tqf.MODES[mode], B, Hkv, 1008, dev) if other else cache
    want = []
    for b, L in enumerate(lengths):
        for h in range(Hkv):
            x = w[b, h, :L].clone()
            x[:4] = 2
            x[L - 32:] = 2
            at = torch.sort(torch.sort(x, descending=True, stable=True).indices[:n]).values
            want.append((b, h, at, as_bytes(cache.k_data)[b, h, at], as_bytes(cache.v_data)[b, h, at],
                         cache.v_norm[b, h, at]))
    kept = torch.zeros(B, Hkv, n, dtype=torch.int32, device=dev)
    ctx = tqf.Context()
    tqf.tq_cache_evict(ctx, dst, cache, w, i32([n] * B, dev), kept, max(lengths), sinks=4, recent=32)
    for b, h, at, k, v, vn in want:
        assert torch.equal(kept[b, h].long(), at)
        assert torch.equal(as_bytes(dst.k_data)[b, h, :n], k) and torch.equal(as_bytes(dst.v_data)[b, h, :n], v)
        assert torch.equal(dst.v_norm[b, h, :n], vn)
    assert dst.lengths.tolist() == [n] * B and tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("u", [0.0, 0.3, 0.71828, 1 - 2.0 ** -24])
def test_draw_from_a_long_row(dev, u):
    """Equal probabilities of 2^-28, one behind another in more than 2^30 bytes: floor(u V)."""
    B, N, V = 1, 2, (1 << 28) + 5
    target = torch.full((B, N, V), 2.0 ** -28, device=dev)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    keep, num, nxt = z(B, N), z(B), z(B)
    uni = torch.tensor([[u, 0.5]], device=dev)
    tqf.tq_verify_tree(tqf.Context(), z(B, N), i32([[-1, 0]], dev), target, None, uni, keep, num, nxt)
    # (the child's certain token has probability 2^-28: rejected, and token 0 is gone)
    x = float(np.float32(u))
    assert keep.tolist() == [[0, -1]] and num.tolist() == [1]
    assert nxt.tolist() == [int(x * (V - 1)) + 1]


def test_calls_at_once(dev):
    """Two contexts on two streams, the three calls on each: what each gives alone."""
    def side(seed):
        torch.manual_seed(seed)
        B, Hkv, cap, N, V = 4, 4, 3008, 8, 20000
        cache = tqf.Cache(tqf.MODES["turbo4"], B, Hkv, cap, dev)
        cache.k_data.random_(0, 256)
        cache.v_data.random_(0, 256)
        cache.k_norm.uniform_(0.5, 9.0)
        cache.v_norm.uniform_(0.5, 9.0)
        cache.lengths.copy_(i32([3000, 2500, 77, 1900], dev))
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
        s = dict(cache=cache, ctx=tqf.Context(), small=tqf.Cache(tqf.MODES["turbo4"], B, Hkv, 512, dev),
                 qs=[torch.randn(B, 4 * Hkv, T, 128, device=dev, dtype=torch.float16) for T in (1, 20, 50, 70)],
                 w=torch.zeros(B, Hkv, cap, device=dev), nw=torch.zeros(B, Hkv, 512, device=dev), n=i32([500, 400, 60, 36], dev),
                 kept=z(B, Hkv, 512), tok=torch.randint(0, V, (B, N), device=dev, dtype=torch.int32),
                 par=i32([[-1, 0, 0, 1, 1, 2, 3, 4]], dev), p=torch.softmax(torch.randn(B, N, V, device=dev), -1),
                 q=torch.softmax(torch.randn(B, N, V, device=dev), -1), u=torch.rand(B, N, device=dev), out=(z(B, N), z(B), z(B)))
        return s

    def run(s, stream):
        for q in s["qs"]:
            tqf.tq_attention_weights(s["ctx"], s["cache"], q, s["w"], 3000, decay=0.5, seen=s["cache"].lengths, stream=stream)
        tqf.tq_cache_evict(s["ctx"], s["small"], s["cache"], s["w"], s["n"], s["kept"], 3000, new_weights=s["nw"], sinks=4,
                           recent=32, stream=stream)
        tqf.tq_verify_tree(s["ctx"], s["tok"], s["par"], s["p"], s["q"], s["u"], *s["out"], stream=stream)

    def results(s):
        return [t.clone() for t in (s["w"], s["kept"], s["nw"], s["small"].k_data, s["small"].lengths, *s["out"])]

    sides, streams = [side(1), side(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    alone = []
    for s in sides:
        run(s, None)
        torch.cuda.synchronize()
        alone.append(results(s))
    for _ in range(10):
        for s in sides:
            s["w"].zero_()
            for t in (s["kept"], s["nw"], s["small"].lengths, *s["out"]):
                t.zero_()
        torch.cuda.synchronize()
        for s, st in zip(sides, streams):
            run(s, st)
        torch.cuda.synchronize()
        for s, a in zip(sides, alone):
            assert all(torch.equal(x, y) for x, y in zip(results(s), a))
            assert tqf.tq_get_status(s["ctx"]) in (0, tqf.TQ_STATUS_SHORT_CONTEXT)
