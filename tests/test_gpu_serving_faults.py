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
