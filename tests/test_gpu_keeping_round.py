"""Eviction and verification as a server uses them together: prompts appended and
weighed, pressed into the decode's smaller cache, drafted trees verified and kept,
their tokens weighed, the cache evicted in place and decoded from; and the same round
captured into graphs that share a context."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
from quantized_kv_cache_flash_gb300 import workloads as wl
from tests import helpers as H
from tests import keeping_helpers as K
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


def records(cache):
    return [None if t is None else t.cpu().numpy() for t in (cache.k_data, cache.k_norm, cache.v_data, cache.v_norm)]


def same(a, b):
    """The same bits."""
    return np.array_equal(np.ascontiguousarray(a).view(np.uint8), np.ascontiguousarray(b).view(np.uint8))


def assert_decodes(mode, cache, ctx, q, hint):
    """The decode of q from the cache against 64 bits over its own records."""
    out = torch.zeros_like(q)
    tqf.tq_decode_attention(ctx, cache, q, out, hint)
    rec, lengths = records(cache), cache.lengths.cpu().tolist()
    B, Hq = q.shape[:2]
    Hkv = cache.num_kv_heads
    G = Hq // Hkv
    for b in range(B):
        for h in range(Hkv):
            k, v = S.kv_of(mode, rec, b, h, lengths[b])
            rows = q[b, h * G:(h + 1) * G, 0].cpu().numpy().astype(np.float64)
            want, bound = S.attention_rows(rows, k, v, np.ones((G, lengths[b]), bool), 1 / math.sqrt(128.0))
            S.assert_rows(out[b, h * G:(h + 1) * G, 0].cpu().numpy(), want, bound, f"decode {b}, {h}")


@pytest.mark.parametrize("mode", ["turbo4", "turbo3", "turbo4_asym"])
def test_a_round(dev, mode):
    B, Hq, Hkv, N, V, W = 3, 8, 2, 12, 700, 16
    lens = [300, 77, 190]
    cu = np.concatenate([[0], np.cumsum(lens)])
    rng = np.random.default_rng(21)
    prompt = tqf.Cache(tqf.MODES[mode], B, Hkv, 304, dev)
    ctx = tqf.Context()
    k, v = (H.upload(wl.random_fp16(80 + i, (cu[-1], Hkv, 128)), dev) for i in range(2))
    tqf.tq_encode_append_packed(ctx, prompt, k, v, i32(cu, dev))

    # the window at the prompts' ends weighs their tokens
    qw = wl.random_fp16(82, (B, Hq, W, 128))
    w0 = torch.zeros(B, Hkv, 304, device=dev)
    tqf.tq_attention_weights(ctx, prompt, H.upload(qw, dev), w0, 300, decay=0.0)
    A, bound = K.weights(mode, records(prompt), qw, lens, Hkv)
    assert np.all(np.abs(w0.cpu().numpy() - A) <= bound)

    # pressed into a smaller cache
    cache = tqf.Cache(tqf.MODES[mode], B, Hkv, 160, dev)
    w = torch.full((B, Hkv, 160), float("nan"), device=dev)
    kept = torch.zeros(B, Hkv, 100, dtype=torch.int32, device=dev)
    tqf.tq_cache_evict(ctx, cache, prompt, w0, i32([100, 100, 100], dev), kept, 300, new_weights=w, sinks=4, recent=W)
    assert cache.lengths.cpu().tolist() == [100, 77, 100]
    rp, rc = records(prompt), records(cache)
    for b in range(B):
        for h in range(Hkv):
            at = K.evict(w0[b, h].cpu().numpy(), lens[b], 100, 4, W)
            assert kept[b, h, :len(at)].cpu().tolist() == at.tolist()
            for a, c in zip(rp, rc):
                if a is not None:
                    assert same(c[b, h, :len(at)], a[b, h, at])
    assert_decodes(mode, cache, ctx, H.upload(wl.random_fp16(83, (B, Hq, 1, 128)), dev), 160)

    # two speculative steps
    for step in range(2):
        start = cache.lengths.clone()
        parents = [-1] + [int(rng.integers(0, i)) for i in range(1, N)]
        kd, vd = (H.upload(wl.random_fp16(90 + 2 * step + i, (B, Hkv, N, 128)), dev) for i in range(2))
        tqf.tq_encode_append(ctx, cache, kd, vd)
        q = H.upload(wl.random_fp16(94 + step, (B, Hq, N, 128)), dev)
        out = torch.zeros_like(q)
        tqf.tq_tree_attention(ctx, cache, q, out, tqf.tq_tree_mask(parents)[None].to(dev), 160)
        x = rng.standard_normal((B, N, V))
        target, draft = (np.exp(y) / np.exp(y).sum(-1, keepdims=True) for y in (x, x + 0.6 * rng.standard_normal(x.shape)))
        target, draft = target.astype(np.float32), draft.astype(np.float32)
        tok = rng.integers(0, V, (B, N)).astype(np.int32)
        for b in range(B):
            for i in range(1, N):
                tok[b, i] = min(np.searchsorted(np.cumsum(draft[b, parents[i]], dtype=np.float64), rng.random()), V - 1)
        u = rng.random((B, N), np.float32)
        keep, num, nxt = (torch.zeros(s, dtype=torch.int32, device=dev) for s in ((B, N), (B,), (B,)))
        tqf.tq_verify_tree(ctx, *(torch.from_numpy(np.asarray(y, t)).to(dev) for y, t in
                                  ((tok, np.int32), ([parents], np.int32), (target, np.float32), (draft, np.float32))),
                           torch.from_numpy(u).to(dev), keep, num, nxt)
        full = records(cache)
        tqf.tq_cache_compact(ctx, cache, start, keep, num, N)
        after = records(cache)
        for b in range(B):
            path, follow, _ = K.verify(tok[b], parents, target[b], draft[b], u[b])
            assert keep[b, :int(num[b])].cpu().tolist() == path and int(nxt[b]) == follow
            s = int(start[b])
            assert int(cache.lengths[b]) == s + len(path)
            for a, c in zip(full, after):
                if a is not None:
                    assert same(c[b, :, s:s + len(path)], a[b][:, [s + i for i in path]])
        # the accepted tokens have no weight yet: the last one's query weighs them with the others
        q1 = np.stack([q[b, :, int(num[b]) and int(keep[b, int(num[b]) - 1]):][:, :1].cpu().numpy() for b in range(B)])
        old = w.cpu().numpy().astype(np.float64)
        tqf.tq_attention_weights(ctx, cache, H.upload(q1, dev), w, 160, decay=0.5, seen=start)
        ls = cache.lengths.cpu().tolist()
        A, bound = K.weights(mode, after, q1, ls, Hkv)
        for b in range(B):
            base = np.where(np.arange(ls[b]) < int(start[b]), 0.5 * old[b, :, :ls[b]], 0.0)
            got = w[b, :, :ls[b]].cpu().numpy()
            assert np.all(np.abs(got - base - A[b, :, :ls[b]]) <= bound[b, :, :ls[b]] + 2.0 ** -22 * base)

    # back to 90 tokens, in place
    before, ws, ls = records(cache), w.cpu().numpy(), cache.lengths.cpu().tolist()
    tqf.tq_cache_evict(ctx, cache, cache, w, i32([90] * B, dev), kept, 160, new_weights=w, sinks=4, recent=8)
    after = records(cache)
    for b in range(B):
        for h in range(Hkv):
            at = K.evict(ws[b, h], ls[b], 90, 4, 8)
            for a, c in zip(before, after):
                if a is not None:
                    assert same(c[b, h, :len(at)], a[b, h, at])
            assert np.array_equal(w[b, h, :len(at)].cpu().numpy(), ws[b, h, at])
    assert cache.lengths.cpu().tolist() == [min(90, n) for n in ls]
    assert_decodes(mode, cache, ctx, H.upload(wl.random_fp16(99, (B, Hq, 1, 128)), dev), 160)
    assert tqf.tq_get_status(ctx) == 0


def test_a_captured_decode_loop_with_eviction(dev):
    """A step (append, decode, weights) and an eviction, each a graph of one context,
    replayed in turn as eager calls of another context are made: the same cache, bit for bit."""
    mode, B, Hq, Hkv, cap = "turbo4", 2, 8, 2, 128
    rec = H.random_cache(mode, B, Hkv, cap, 31)
    states = []
    for _ in range(2):
        c = H.gpu_cache_from_records(mode, B, Hkv, cap, [60, 41], *rec, dev)
        states.append(dict(cache=c, w=torch.zeros(B, Hkv, cap, device=dev), ctx=tqf.Context(),
                           k=torch.zeros(B, Hkv, 1, 128, dtype=torch.float16, device=dev),
                           v=torch.zeros(B, Hkv, 1, 128, dtype=torch.float16, device=dev),
                           q=torch.zeros(B, Hq, 1, 128, dtype=torch.float16, device=dev),
                           out=torch.zeros(B, Hq, 1, 128, dtype=torch.float16, device=dev),
                           kept=torch.zeros(B, Hkv, 48, dtype=torch.int32, device=dev), n=i32([48, 30], dev)))

    def step(s):
        tqf.tq_encode_append(s["ctx"], s["cache"], s["k"], s["v"])
        tqf.tq_decode_attention(s["ctx"], s["cache"], s["q"], s["out"], cap)
        tqf.tq_attention_weights(s["ctx"], s["cache"], s["q"], s["w"], cap, decay=0.9)

    def evict(s):
        tqf.tq_cache_evict(s["ctx"], s["cache"], s["cache"], s["w"], s["n"], s["kept"], cap, new_weights=s["w"], sinks=2, recent=9)

    eager, other = states
    # (one eager call each sizes the context; then back to the start)
    step(other), evict(other)
    for t, r in zip((other["cache"].k_data, other["cache"].k_norm, other["cache"].v_data, other["cache"].v_norm), rec):
        t.copy_(torch.from_numpy(r))
    other["cache"].lengths.copy_(i32([60, 41], dev))
    other["w"].zero_()
    graphs = []
    for f in (step, evict):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f(other)
        graphs.append(g)
    for i in range(40):
        for name, key in (("k", 100), ("v", 200), ("q", 300)):
            x = H.upload(wl.random_fp16(key + i, tuple(eager[name].shape)), dev)
            for s in states:
                s[name].copy_(x)
        step(eager)
        graphs[0].replay()
        if i % 7 == 6:
            evict(eager)
            graphs[1].replay()
        assert torch.equal(eager["out"], other["out"])
    a, b = ([t for t in (s["cache"].k_data, s["cache"].v_norm, s["cache"].lengths, s["w"], s["kept"])] for s in states)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert tqf.tq_get_status(eager["ctx"]) == 0 and tqf.tq_get_status(other["ctx"]) == 0
