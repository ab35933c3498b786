"""Packed prompts on the GPU: the append (records equal to 64-bit decisions, bit
for bit) and the causal attention (each row within the bound of its roundings)
of sequences of different lengths back to back."""
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


def cum(n):
    return [0] + [int(x) for x in np.cumsum(n)]


def check_append(dev, mode, Hkv, cap, before, new, k, v, extra=0, stream=None):
    """Append packed rows and compare every byte of the cache with the host's."""
    B, (kb, vb) = len(new), H.MODE_BITS[mode]
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, B, Hkv, cap, 71)]
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, before, *rec, dev)
    ctx = tqf.Context()
    cu = cum(new)
    assert len(k) == cu[-1] + extra
    tqf.tq_encode_append_packed(ctx, cache, H.upload(k, dev), H.upload(v, dev), i32(cu, dev), stream=stream)
    torch.cuda.synchronize()
    table = mode in H.TABLE_MODES
    streams = [(2, 3, v, vb)] if kb == 16 else [(0, 1, k, kb), (2, 3, v, vb)]
    for data, norm, x, bits in streams:
        codes, norms = S.encode_exact(x, bits)
        if table:
            t = o.centroid_norm_table(norms, o.codebook(bits))
            codes = np.concatenate([codes, t.astype("<f2").view(np.uint8)], axis=-1)
        for b in range(B):
            if before[b] + new[b] <= cap:
                at = slice(before[b], before[b] + new[b])
                rec[data][b, :, at] = codes[cu[b]:cu[b + 1]].transpose(1, 0, 2)
                if not table:
                    rec[norm][b, :, at] = norms[cu[b]:cu[b + 1]].T
    if kb == 16:
        for b in range(B):
            if before[b] + new[b] <= cap:
                rec[0][b, :, before[b]:before[b] + new[b]] = k[cu[b]:cu[b + 1]].transpose(1, 0, 2)
    got = [None if t is None else t.cpu().numpy() for t in (cache.k_data, cache.k_norm, cache.v_data, cache.v_norm)]
    for name, g, w in zip(("k", "k_norm", "v", "v_norm"), got, rec):
        assert (g is None) == (w is None)
        if g is not None:
            assert np.array_equal(g.view(np.uint8), np.ascontiguousarray(w).view(np.uint8)), name
    after = [p + n if p + n <= cap else p for p, n in zip(before, new)]
    assert cache.lengths.cpu().tolist() == after
    return tqf.tq_get_status(ctx)


APPENDS = [
    # mode, Hkv, cap, lengths before, new tokens
    ("turbo3", 4, 64, [0], [1]),
    ("turbo4", 3, 128, [5, 0, 127, 64], [17, 0, 1, 64]),
    ("turbo4_asym", 2, 96, [0, 31, 7], [33, 1, 0]),
    ("turbo3_table", 1, 64, [3, 0], [9, 40]),
    ("turbo4k_3v", 8, 48, [0, 40, 16], [3, 8, 32]),
    # more than 4096 vectors: the tensor-core kernel, tiles that end inside a token
    ("turbo3", 8, 1024, [0, 999, 17], [700, 25, 3]),
    ("turbo4", 5, 1024, [1, 0, 0, 12], [0, 701, 300, 2]),
    ("turbo4_asym", 3, 1488, [0, 77], [1488, 3]),
    ("turbo3_asym", 1, 4608, [501], [4098]),
    ("turbo4k_3v", 7, 640, [0] * 40, [(37 * i) % 61 for i in range(40)]),
    ("turbo3_table", 4, 1200, [100, 200], [1100, 77]),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"{c[0]}-Hkv{c[1]}-n{sum(c[4])}")
def test_append_equals_64_bit_decisions(dev, case):
    mode, Hkv, cap, before, new = case
    n = sum(new) + 3
    k = wl.random_fp16(700 + n, (n, Hkv, 128))
    k[..., [5, 60, 90, 111]] = (k[..., [5, 60, 90, 111]].astype(np.float32) * 8).astype(np.float16)
    v = wl.random_fp16(701 + n, (n, Hkv, 128))
    # (three rows behind the last sequence are ignored)
    assert check_append(dev, mode, Hkv, cap, before, new, k, v, extra=3) == 0


@pytest.mark.parametrize("mode", ["turbo3", "turbo4"])
@pytest.mark.parametrize("n", [600, 60000])
def test_append_near_the_midpoints(dev, mode, n):
    """Enough vectors that many hold an element within fp32 error of a midpoint
    (600 take the small kernel, 60,000 the tensor cores), and constructed ones:
    zeros, single entries, constants, subnormals, the largest values."""
    k = wl.random_fp16(5, (n, 2, 128))
    v = wl.random_fp16(6, (n, 2, 128)) * np.float16(0.01)
    k[0] = 0
    k[1] = 0
    k[1, :, 7] = 3.5
    k[2] = 0.25
    k[3, :, ::2] = -0.25
    k[4] = np.float16(6e-8)
    k[5] = 5000.0
    k[6, 0] = np.where(np.arange(128) % 3 == 0, 4096.0, 2.0 ** -14)
    assert check_append(dev, mode, 2, (n + 15) // 16 * 16, [0, 3], [n - 5, 5], k, v) == 0


def test_append_over_capacity_and_bad_bounds(dev):
    k, v = wl.random_fp16(8, (60, 2, 128)), wl.random_fp16(9, (60, 2, 128))
    assert check_append(dev, "turbo3", 2, 32, [0, 20, 1], [10, 13, 31], k[:54], v[:54]) == tqf.TQ_STATUS_CAPACITY
    ctx = tqf.Context()
    for bad in ([0, 20, 10, 60], [0, 20, 40, 61], [-1, 20, 40, 60]):
        cache = tqf.Cache(tqf.MODES["turbo3"], 3, 2, 64, dev)
        tqf.tq_encode_append_packed(ctx, cache, H.upload(k, dev), H.upload(v, dev), i32(bad, dev))
        torch.cuda.synchronize()
        want = [b - a if b >= a >= 0 and b <= 60 else 0 for a, b in zip(bad, bad[1:])]
        assert cache.lengths.cpu().tolist() == want
        assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_BAD_INDEX
    # an overflowing norm is flagged and stored as inf
    k[3, 1] = 60000.0
    cache = tqf.Cache(tqf.MODES["turbo3"], 3, 2, 64, dev)
    tqf.tq_encode_append_packed(ctx, cache, H.upload(k, dev), H.upload(v, dev), i32([0, 20, 40, 60], dev))
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_NORM_OVERFLOW
    assert math.isinf(float(cache.k_norm[0, 1, 3]))


PREFILLS = [
    # mode, Hq, Hkv, lengths before, new rows, hint (None: the longest), q scale
    ("turbo4", 8, 2, [0], [1], None, 1.0),
    ("turbo3", 28, 4, [0, 0, 0], [300, 1, 77], None, 1.0),            # G 7
    ("turbo4", 8, 2, [500, 0, 3, 129], [0, 130, 65, 1], None, 1.0),   # an empty sequence, chunks
    ("turbo4_asym", 4, 2, [0, 257], [513, 100], None, 1.0),           # fp16 K
    ("turbo3_asym", 8, 8, [31, 0], [97, 260], None, 1.0),             # G 1
    ("turbo4k_3v", 16, 2, [1000, 3], [64, 33], None, 8.0),            # G 8, sharper rows
    ("turbo3", 128, 1, [5, 0], [3, 7], None, 1.0),                    # G 128: one position per tile
    ("turbo4", 8, 2, [0] * 70, [(13 * i) % 41 for i in range(70)], None, 1.0),   # over 32 sequences
    ("turbo3", 8, 2, [200, 30], [300, 100], 450, 1.0),                # hint below a length
    ("turbo4_asym", 28, 4, [700, 0], [20, 500], None, 32.0),
    ("turbo4", 8, 2, [1500, 0], [700, 40], None, 32.0),               # many tiles, bases that move late
    ("turbo3_asym", 12, 2, [2000, 5], [300, 1], None, 4.0),           # G 6, fp16 K
]


@pytest.mark.parametrize("case", PREFILLS, ids=lambda c: f"{c[0]}-Hq{c[1]}-Hkv{c[2]}-B{len(c[4])}-n{sum(c[4])}")
def test_prefill_rows_within_their_bounds(dev, case):
    mode, Hq, Hkv, ctx_len, new, hint, qs = case
    B, G = len(new), Hq // Hkv
    L = [a + b for a, b in zip(ctx_len, new)]
    hint = hint or max(L)
    cap = (max(L) + 15) // 16 * 16
    rec = H.random_cache(mode, B, Hkv, cap, 900 + sum(new))
    total = sum(new) + 2   # two rows of no sequence
    q = wl.random_fp16(901 + total, (total, Hq, 128), scale=qs)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, L, *rec, dev, v_rescale=0.5)
    ctx = tqf.Context()
    qd = H.upload(q, dev)
    out = torch.full_like(qd, 7.0)
    cu = cum(new)
    tqf.tq_prefill_attention_packed(ctx, cache, qd, out, i32(cu, dev), hint)
    torch.cuda.synchronize()
    assert tqf.tq_get_status(ctx) == 0
    got = out.float().cpu().numpy()
    assert np.all(got[cu[-1]:] == 7.0)
    heads = range(Hkv) if B < 32 else [0]
    for b in range(B):
        if new[b] == 0:
            continue
        vis = min(L[b], hint)
        for h in heads:
            K, V = S.kv_of(mode, rec, b, h, vis, v_rescale=0.5)
            last = L[b] - new[b] + np.arange(new[b])
            rows = q[cu[b]:cu[b + 1], h * G:(h + 1) * G].reshape(-1, 128)   # [n, G]
            seen = np.arange(vis)[None, :] <= np.repeat(last, G)[:, None]
            want, bound = S.attention_rows(rows, K, V, seen, 1 / math.sqrt(128))
            S.assert_rows(got[cu[b]:cu[b + 1], h * G:(h + 1) * G], want, bound, f"b{b} h{h}")


def test_prefill_agrees_with_the_padded_call(dev):
    """Equal blocks through both calls: each is within its row bounds of the exact
    row (the padded call rounds a term of P.V twice, the packed one once), so their
    distance is within the sum."""
    mode, B, Hq, Hkv, n, L, cap = "turbo3", 3, 28, 4, 150, 400, 400
    rec = H.random_cache(mode, B, Hkv, cap, 33)
    q = wl.random_fp16(34, (B, Hq, n, 128))
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, [L] * B, *rec, dev)
    ctx = tqf.Context()
    qd = H.upload(q, dev)
    a = torch.empty_like(qd)
    tqf.tq_prefill_attention(ctx, cache, qd, a, L)
    qp = qd.transpose(1, 2).reshape(B * n, Hq, 128).contiguous()
    b = torch.empty_like(qp)
    tqf.tq_prefill_attention_packed(ctx, cache, qp, b, i32(cum([n] * B), dev), L)
    got = b.view(B, n, Hq, 128).transpose(1, 2).float().cpu().numpy()
    for s in range(B):
        K, V = S.kv_of(mode, rec, s, 1, L)
        rows = q[s, 7:14].reshape(-1, 128)
        seen = np.arange(L)[None, :] <= np.tile(L - n + np.arange(n), 7)[:, None]
        _, bound = S.attention_rows(rows, K, V, seen, 1 / math.sqrt(128))
        S.assert_rows(got[s, 7:14], a[s, 7:14].float().cpu().numpy().astype(np.float64), 2 * bound, f"b{s}")


def test_prefill_bad_bounds_short_contexts_and_overflowed_norms(dev):
    mode, B, Hq, Hkv, cap = "turbo4", 3, 8, 2, 64
    rec = [np.array(r) for r in H.random_cache(mode, B, Hkv, cap, 35)]
    q = H.upload(wl.random_fp16(36, (60, Hq, 128)), dev)
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, [20, 20, 20], *rec, dev)
    ctx = tqf.Context()
    want = torch.empty_like(q)
    tqf.tq_prefill_attention_packed(ctx, cache, q, want, i32([0, 20, 40, 60], dev), cap)
    assert tqf.tq_get_status(ctx) == 0
    # (bounds that decrease make sequences overlap: only the status says so)
    for bad, b in (([0, 20, 10, 60], None), ([0, 20, 40, 61], 2), ([-1, 20, 40, 60], 0)):
        out = torch.full_like(q, 7.0)
        tqf.tq_prefill_attention_packed(ctx, cache, q, out, i32(bad, dev), cap)
        assert tqf.tq_get_status(ctx) & tqf.TQ_STATUS_BAD_INDEX
        if b is not None:
            keep = torch.arange(60, device=dev) // 20 == b
            assert bool((out[keep] == 7.0).all()) and torch.equal(out[~keep], want[~keep])
    # a sequence shorter than its block: the rows that see nothing are 0
    cache.lengths.copy_(i32([20, 5, 20], dev))
    out = torch.full_like(q, 7.0)
    tqf.tq_prefill_attention_packed(ctx, cache, q, out, i32([0, 20, 40, 60], dev), cap)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_SHORT_CONTEXT
    assert bool((out[20:35] == 0).all()) and torch.equal(out[:20], want[:20]) and torch.equal(out[40:], want[40:])
    assert bool(torch.isfinite(out).all()) and bool((out[35:40] != 0).any())
    # norms that overflowed at token 12 leave the rows before it alone
    cache.lengths.fill_(20)
    cache.v_norm[:, :, 12] = float("inf")
    cache.k_norm[:, :, 12] = float("inf")
    tqf.tq_prefill_attention_packed(ctx, cache, q, out, i32([0, 20, 40, 60], dev), cap)
    torch.cuda.synchronize()
    for b in range(3):
        assert torch.equal(out[20 * b:20 * b + 12], want[20 * b:20 * b + 12])


def test_packed_serving_round_in_a_graph(dev):
    """Append then prefill of packed prompts, eager and replayed from a graph,
    against the same tokens one sequence at a time (the same tiles, so the same
    bits)."""
    mode, Hq, Hkv, cap, new = "turbo3", 28, 4, 800, [257, 31, 700, 1]
    B, cu = len(new), cum(new)
    k, v = wl.random_fp16(80, (cu[-1], Hkv, 128)), wl.random_fp16(81, (cu[-1], Hkv, 128))
    q = wl.random_fp16(82, (cu[-1], Hq, 128))
    kd, vd, qd, cud = H.upload(k, dev), H.upload(v, dev), H.upload(q, dev), i32(cu, dev)
    cache, ctx = tqf.Cache(tqf.MODES[mode], B, Hkv, cap, dev), tqf.Context()
    out = torch.empty_like(qd)

    def step():
        cache.lengths.zero_()
        tqf.tq_encode_append_packed(ctx, cache, kd, vd, cud)
        tqf.tq_prefill_attention_packed(ctx, cache, qd, out, cud, 700)

    step()
    torch.cuda.synchronize()
    eager = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    assert tqf.tq_get_status(ctx) == 0
    for b in range(B):
        one, c1 = tqf.Cache(tqf.MODES[mode], 1, Hkv, cap, dev), tqf.Context()
        k1, v1, q1, e1 = (x[cu[b]:cu[b + 1]].contiguous() for x in (kd, vd, qd, eager))
        tqf.tq_encode_append_packed(c1, one, k1, v1, i32([0, new[b]], dev))
        o1 = torch.empty_like(q1)
        tqf.tq_prefill_attention_packed(c1, one, q1, o1, i32([0, new[b]], dev), new[b])
        assert torch.equal(e1, o1), b
        assert torch.equal(one.k_data[0, :, :new[b]], cache.k_data[b, :, :new[b]])
