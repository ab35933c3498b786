"""Attention of drafted trees on the GPU: each row within the bound of its
roundings, over modes, group sizes, block sizes, masks and lengths, and the
round of a speculative step (append, tree, keep, fork, decode)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
from quantized_kv_cache_flash_gb300 import workloads as wl
from oracle import tq_oracle as o
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


def words_of(seen):
    """int32 mask words of boolean masks [B, N, N]."""
    B, N, _ = seen.shape
    W = (N + 31) // 32
    pad = np.zeros((B, N, 32 * W), np.uint64)
    pad[..., :N] = seen
    return (pad.reshape(B, N, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def random_trees(B, N, rng, padding=True):
    """Ancestor masks of random trees; every second sequence has padding nodes."""
    seen = np.zeros((B, N, N), bool)
    for b in range(B):
        real = N if b % 2 == 0 or not padding else max(1, N - N // 3)
        for i in range(real):
            p = int(rng.integers(-1, i)) if i else -1
            if p >= 0:
                seen[b, i] = seen[b, p]
            seen[b, i, i] = True
    return seen


CASES = [
    # mode, Hq, Hkv, contexts before the block, N, shared mask, q scale
    ("turbo4", 8, 2, [300], 1, True, 1.0),                 # one node: a decode step
    ("turbo3", 28, 4, [517, 33], 16, False, 1.0),          # G 7
    ("turbo4_asym", 28, 4, [700, 0, 129], 33, False, 1.0),  # fp16 K, no context, odd
    ("turbo3_asym", 8, 8, [250, 8], 5, True, 1.0),         # G 1
    ("turbo4k_3v", 16, 2, [1000, 31], 17, False, 8.0),     # G 8
    ("turbo3_table", 8, 2, [200, 90], 12, False, 1.0),
    ("turbo4", 32, 8, [900, 1, 260], 64, False, 1.0),      # 256 rows
    ("turbo3", 32, 8, [611], 65, True, 1.0),               # just past two tiles of rows
    ("turbo4", 4, 4, [100, 700], 256, False, 1.0),         # the largest block
    ("turbo4", 128, 1, [333], 3, True, 1.0),               # G 128
    ("turbo3", 8, 2, [40 + i for i in range(40)], 9, False, 1.0),   # over 32 sequences
    ("turbo3", 28, 4, [517, 33], 16, False, 32.0),         # peaked rows
    ("turbo4_asym", 32, 8, [2000, 300], 40, True, 16.0),
    ("turbo4", 32, 8, [5000, 3], 48, False, 1.0),          # long: many splits of one unit
    ("turbo3_table", 32, 8, [700], 40, True, 1.0),
    ("turbo4", 16, 8, [30 + 7 * i for i in range(40)], 9, False, 1.0),   # more units than SMs
    ("turbo3_asym", 20, 4, [4200], 21, False, 1.0),        # CTAs of one unit each, many to merge
    ("turbo4k_3v", 12, 2, [100, 3000, 0, 17], 30, False, 4.0),   # CTAs that cross into other units
]


def run_case(dev, mode, Hq, Hkv, ctx_len, N, seen, qs=1.0, hint=None, cbk=None, key=0, edit=None, lengths=None):
    """The call on random records, checked row by row; returns (out, status)."""
    B, G = len(ctx_len), Hq // Hkv
    L = lengths or [c + N for c in ctx_len]
    hint = hint or max(L)
    cap = (max(L) + 15) // 16 * 16
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, B, Hkv, cap, 1300 + key + N)]
    if edit:
        edit(rec)
    q = wl.random_fp16(1301 + key + N, (B, Hq, N, 128), scale=qs)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, L, *rec, dev, v_rescale=0.5, codebook_k=cbk)
    ctx = tqf.Context()
    qd = H.upload(q, dev)
    out = torch.full_like(qd, float("nan"))
    mask = torch.from_numpy(words_of(seen)).to(dev)
    tqf.tq_tree_attention(ctx, cache, qd, out, mask, hint)
    torch.cuda.synchronize()
    status = tqf.tq_get_status(ctx)
    got = out.float().cpu().numpy()
    for b in range(B):
        vis = min(L[b], hint)
        m = np.zeros((N, vis), bool)
        for j in range(N):
            for t in range(vis):
                i = t - (L[b] - N)
                m[j, t] = i < 0 or seen[b if len(seen) > 1 else 0, j, i]
        for h in range(Hkv) if B * Hkv <= 16 else [b % Hkv]:
            K, V = S.kv_of(mode, rec, b, h, vis, cbk=cbk, v_rescale=0.5)
            rows = q[b, h * G:(h + 1) * G].reshape(-1, 128)
            want, bound = S.attention_rows(rows, K, V, np.tile(m, (G, 1)), 1 / math.sqrt(128))
            S.assert_rows(got[b, h * G:(h + 1) * G], want, bound, f"b{b} h{h}")
    return got, status


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-Hq{c[1]}-Hkv{c[2]}-B{len(c[3])}-N{c[4]}-q{c[6]:g}")
def test_tree_rows_within_their_bounds(dev, case):
    mode, Hq, Hkv, ctx_len, N, shared, qs = case
    rng = np.random.default_rng(N + len(ctx_len))
    seen = random_trees(1 if shared else len(ctx_len), N, rng)
    _, status = run_case(dev, mode, Hq, Hkv, ctx_len, N, seen, qs)
    # (a padding node over no context sees nothing)
    empty = any(c == 0 and not seen[b if not shared else 0].any(1).all() for b, c in enumerate(ctx_len))
    assert status == (tqf.TQ_STATUS_SHORT_CONTEXT if empty else 0)


@pytest.mark.parametrize("mode,Hq,Hkv,N", [("turbo4", 8, 2, 37), ("turbo3", 32, 8, 64), ("turbo4_asym", 28, 4, 50)])
def test_any_mask(dev, mode, Hq, Hkv, N):
    """Masks that no tree has: arbitrary bits, rows that see only others, none
    or all; set bits past the block are ignored."""
    rng = np.random.default_rng(N)
    seen = rng.random((2, N, N)) < 0.4
    seen[0, 3] = False
    seen[0, 4] = True
    _, status = run_case(dev, mode, Hq, Hkv, [0, 130], N, seen, key=7)
    assert status == tqf.TQ_STATUS_SHORT_CONTEXT


def test_bits_past_the_block_are_ignored(dev):
    mode, N, L, cap = "turbo4", 5, 133, 144
    rec = H.random_cache(mode, 1, 2, cap, 3)
    cache = H.gpu_cache_from_records(mode, 1, 2, cap, [L], *rec, dev)
    q = H.upload(wl.random_fp16(4, (1, 8, N, 128)), dev)
    seen = random_trees(1, N, np.random.default_rng(0))
    a, b = torch.empty_like(q), torch.empty_like(q)
    ctx = tqf.Context()
    w = torch.from_numpy(words_of(seen)).to(dev)
    tqf.tq_tree_attention(ctx, cache, q, a, w, L)
    tqf.tq_tree_attention(ctx, cache, q, b, w | ~0x1F, L)
    assert torch.equal(a, b)


@pytest.mark.parametrize("Hq,N", [(8, 6), (32, 48)])
def test_short_sequences_and_hints(dev, Hq, N):
    seen = random_trees(3, N, np.random.default_rng(5), padding=False)
    # shorter than the block (its first tokens do not exist), and empty
    _, status = run_case(dev, "turbo3", Hq, 2, [0, 0, 0], N, seen, key=9, lengths=[N - 2, 0, N + 300])
    assert status == tqf.TQ_STATUS_SHORT_CONTEXT
    # a hint that ends inside the block of the longest and before that of none
    run_case(dev, "turbo3", Hq, 2, [300, 10, 200], N, seen, key=10, hint=300 + N // 2)


@pytest.mark.parametrize("mode", ["turbo3", "turbo4"])
@pytest.mark.parametrize("Hq,N", [(8, 3), (32, 40)])
def test_codebook_of_other_levels(dev, mode, Hq, N):
    cbk = H.exact_lloyd_max(H.MODE_BITS[mode][0])
    run_case(dev, mode, Hq, 8, [400], N, random_trees(1, N, np.random.default_rng(2)), cbk=cbk, key=11)


@pytest.mark.parametrize("mode", ["turbo4", "turbo3_asym", "turbo3_table"])
@pytest.mark.parametrize("Hq,N", [(8, 6), (32, 40)])
def test_unseen_tokens_may_hold_anything(dev, mode, Hq, N):
    """Padding nodes whose K and V overflowed (or are NaN, as fp16 K) leave the
    rows that do not see them as they are."""
    B, Hkv, L = 2, 2, 140 + N
    cap = (L + 15) // 16 * 16
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, B, Hkv, cap, 77)]
    seen = random_trees(B, N, np.random.default_rng(8), padding=False)
    seen[:, :, N - 3:] = False     # three nodes that nobody sees, themselves included
    q = H.upload(wl.random_fp16(78, (B, Hq, N, 128)), dev)
    mask = torch.from_numpy(words_of(seen)).to(dev)
    outs = []
    for spoil in (False, True):
        cache = H.gpu_cache_from_records(mode, B, Hkv, cap, [L] * B, *rec, dev)
        if spoil:
            at = slice(L - 3, L)
            if cache.v_norm is not None:
                cache.v_norm[:, :, at] = float("inf")
            if cache.k_norm is not None:
                cache.k_norm[:, :, at] = float("inf")
            if cache.k_data.dtype == torch.float16:
                cache.k_data[:, :, at] = float("nan")
            if mode == "turbo3_table":
                for t in (cache.k_data, cache.v_data):
                    tab = t[:, :, at, 48:].contiguous().view(torch.float16)
                    t[:, :, at, 48:] = torch.where(tab < 0, -math.inf, math.inf).half().view(torch.uint8)
        ctx, out = tqf.Context(), torch.empty_like(q)
        tqf.tq_tree_attention(ctx, cache, q, out, mask, L)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    assert bool(torch.isfinite(outs[0]).all())


def test_a_chain_is_the_causal_block(dev):
    # the mask of a chain: decode attention of the same block
    mode, B, Hq, Hkv, N, L, cap = "turbo4", 2, 32, 8, 4, 900, 912
    rec = H.random_cache(mode, B, Hkv, cap, 21)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, [L, L - 301], *rec, dev)
    q = H.upload(wl.random_fp16(22, (B, Hq, N, 128)), dev)
    ctx = tqf.Context()
    a, b = torch.empty_like(q), torch.empty_like(q)
    mask = tqf.tq_tree_mask([-1, 0, 1, 2]).to(dev).unsqueeze(0)
    tqf.tq_tree_attention(ctx, cache, q, a, mask, L)
    tqf.tq_decode_attention(ctx, cache, q, b, L)
    assert torch.equal(a, b)


def test_contexts_graphs_and_streams(dev):
    """Calls of growing size on one context, a graph captured between them that
    is replayed after the workspace grew, and a side stream."""
    mode, Hkv, cap = "turbo3", 4, 2048
    rec = H.random_cache(mode, 3, Hkv, cap, 61)
    cache = H.gpu_cache_from_records(mode, 3, Hkv, cap, [700, 2000, 40], *rec, dev)
    ctx = tqf.Context()

    def args(N, seed):
        seen = random_trees(3, N, np.random.default_rng(seed))
        q = H.upload(wl.random_fp16(62 + seed, (3, 28, N, 128)), dev)
        return q, torch.empty_like(q), torch.from_numpy(words_of(seen)).to(dev)

    q, out, mask = args(8, 1)
    tqf.tq_tree_attention(ctx, cache, q, out, mask, cap)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tqf.tq_tree_attention(ctx, cache, q, out, mask, cap)
    q2, out2, mask2 = args(256, 2)
    tqf.tq_tree_attention(ctx, cache, q2, out2, mask2, cap)       # a larger workspace
    first = out2.clone()
    out.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2.fill_(float("nan"))
    torch.cuda.synchronize()
    tqf.tq_tree_attention(ctx, cache, q2, out2, mask2, cap, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out2, first)
    # (the third sequence's 40 tokens are fewer than 256 nodes)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_SHORT_CONTEXT


@pytest.mark.parametrize("mode", ["turbo3", "turbo4_asym"])
def test_speculative_round(dev, mode):
    """Prompts appended and prefilled packed, forked, a tree drafted and
    attended, its accepted path kept, and the next token decoded: the cache then
    holds what appending only the kept tokens would, and every output agrees."""
    Hq, Hkv, cap, new = 28, 4, 400, [211, 96]
    kb, vb = H.MODE_BITS[mode]
    cu = [0, 211, 307]
    rng = np.random.default_rng(17)
    k, v = wl.random_fp16(90, (307, Hkv, 128)), wl.random_fp16(91, (307, Hkv, 128))
    B, N = 4, 24
    cache, ctx = tqf.Cache(tqf.MODES[mode], B, Hkv, cap, dev), tqf.Context()
    # prompts into slots 0 and 2, forked to 1 and 3
    cu4 = [0, 211, 211, 307, 307]
    tqf.tq_encode_append_packed(ctx, cache, H.upload(k, dev), H.upload(v, dev), i32(cu4, dev))
    q = H.upload(wl.random_fp16(92, (307, Hq, 128)), dev)
    out = torch.empty_like(q)
    tqf.tq_prefill_attention_packed(ctx, cache, q, out, i32(cu4, dev), 211)
    tqf.tq_cache_copy(ctx, cache, cache, i32([1, 3], dev), i32([0, 2], dev), cap)
    start = cache.lengths.clone()
    kt, vt = wl.random_fp16(93, (B * N, Hkv, 128)), wl.random_fp16(94, (B * N, Hkv, 128))
    tqf.tq_encode_append_packed(ctx, cache, H.upload(kt, dev), H.upload(vt, dev),
                                i32([N * i for i in range(B + 1)], dev))
    parents = [[-1] + [int(rng.integers(-1, i)) for i in range(1, N)] for _ in range(B)]
    mask = torch.stack([tqf.tq_tree_mask(p) for p in parents]).to(dev)
    qt = H.upload(wl.random_fp16(95, (B, Hq, N, 128)), dev)
    ot = torch.empty_like(qt)
    tqf.tq_tree_attention(ctx, cache, qt, ot, mask, 211 + N)
    paths = []
    for p in parents:      # the path to the last node
        path, i = [], N - 1
        while i >= 0:
            path.append(i)
            i = p[i]
        paths.append(path[::-1])
    longest = max(len(p) for p in paths)
    keep = i32([p + [0] * (longest - len(p)) for p in paths], dev)
    tqf.tq_cache_compact(ctx, cache, start, keep, i32([len(p) for p in paths], dev), N)
    qd = H.upload(wl.random_fp16(96, (B, Hq, 1, 128)), dev)
    od = torch.empty_like(qd)
    tqf.tq_decode_attention(ctx, cache, qd, od, cap)
    torch.cuda.synchronize()
    assert tqf.tq_get_status(ctx) == 0

    # the same through one append of prompt and kept tokens per sequence
    for b in range(B):
        src = 0 if b < 2 else 2
        kk = np.concatenate([k[cu[src // 2]:cu[src // 2 + 1]], kt[b * N + np.array(paths[b])]])
        vv = np.concatenate([v[cu[src // 2]:cu[src // 2 + 1]], vt[b * N + np.array(paths[b])]])
        one, c1 = tqf.Cache(tqf.MODES[mode], 1, Hkv, cap, dev), tqf.Context()
        tqf.tq_encode_append_packed(c1, one, H.upload(kk, dev), H.upload(vv, dev), i32([0, len(kk)], dev))
        n = len(kk)
        assert int(cache.lengths[b]) == n == int(one.lengths[0])
        for a, w in ((cache.k_data, one.k_data), (cache.k_norm, one.k_norm), (cache.v_data, one.v_data),
                     (cache.v_norm, one.v_norm)):
            if a is not None:
                assert torch.equal(a[b, :, :n], w[0, :, :n])
        # the last node's row of the tree is the causal row of that path
        last = qt[b:b + 1, :, N - 1:].contiguous()
        o1 = torch.empty_like(last)
        tqf.tq_decode_attention(c1, one, last, o1, cap)
        H.assert_attention_close(ot[b, :, N - 1].float().cpu().numpy(), o1[0, :, 0].float().cpu().numpy(), "tree")
        o2 = torch.empty_like(last)
        tqf.tq_decode_attention(c1, one, qd[b:b + 1].contiguous(), o2, cap)
        H.assert_attention_close(od[b].float().cpu().numpy(), o2[0].float().cpu().numpy(), "decode")
