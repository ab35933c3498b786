"""Evictions launched right behind the calls that write their weights, with nothing between:
the places go by the weights just written, eagerly and in graphs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
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


@pytest.mark.parametrize("mode,B,Hq,Hkv,T,cap", [
    ("turbo4", 2, 8, 2, 1, 3008),          # one kernel of clusters writes the weights,
    ("turbo3", 32, 32, 8, 1, 1504),        # the sums of a decode step,
    ("turbo4", 4, 8, 2, 30, 2000),         # a window's,
    ("turbo4_asym", 4, 8, 2, 200, 2000),   # those over pairs of query tiles;
    ("turbo3", 1, 4, 2, 1, 40000),         # weights read anew for each digit
])
def test_evictions_behind_the_weights(dev, mode, B, Hq, Hkv, T, cap):
    lengths = [cap - 13 * b for b in range(B)]
    n = [cap // 3 + b for b in range(B)]
    cache = tqf.Cache(tqf.MODES[mode], B, Hkv, cap, dev)
    small = tqf.Cache(tqf.MODES[mode], B, Hkv, (max(n) + 15) // 16 * 16, dev)
    if cache.k_norm is not None:
        cache.k_data.random_(0, 256)
        cache.k_norm.uniform_(0.5, 9.0)
    else:
        cache.k_data.normal_()
    cache.lengths.copy_(i32(lengths, dev))
    rounds, ctx, nd = 6, tqf.Context(), i32(n, dev)
    qs = torch.randn(rounds, B, Hq, T, 128, device=dev).half()
    w = torch.zeros(B, Hkv, cap, device=dev)
    kept = torch.zeros(rounds, B, Hkv, max(n), dtype=torch.int32, device=dev)
    ws = torch.zeros(rounds, B, Hkv, cap, device=dev)
    others = [torch.zeros(B, Hkv, small.capacity, device=dev) for _ in range(2)]

    def go():
        for i in range(rounds):
            # (the last eviction has read the places that these weights go to)
            tqf.tq_attention_weights(ctx, cache, qs[i], w, cap, decay=0.0)
            tqf.tq_cache_evict(ctx, small, cache, w, nd, kept[i], cap, new_weights=others[i & 1], sinks=4, recent=9)
            ws[i].copy_(w)

    def look(what):
        torch.cuda.synchronize()
        for i in range(rounds):
            for b in range(0, B, 1 + B // 4):
                for h in range(Hkv):
                    want = K.evict(ws[i, b, h].cpu().numpy(), lengths[b], n[b], 4, 9)
                    assert kept[i, b, h, :n[b]].tolist() == want.tolist(), f"{what}, round {i}, sequence {b}, head {h}"

    go()
    look("eager")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for _ in range(2):
        qs.normal_()
        kept.zero_()
        w.fill_(float("inf"))
        g.replay()
        look("replayed")
    assert tqf.tq_get_status(ctx) == 0
