"""Packed appends whose list of bounds is wrong somewhere: each sequence goes by its
own two bounds, and every record inside the lengths is the one it should be."""
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


LISTS = [
    [0, 20, 10, 60],                     # the second decreases, the first and third share rows
    [0, 60, 0, 60, 30, 45],              # nested ranges
    [40, 60, 0, 25, 70, 5, 5, 60],       # one passes the end, one is empty
    [50, 10, 0],                         # none in order
    [0] + [7, 33] * 150 + [60],          # more sequences than threads, half of them decreasing
]


@pytest.mark.parametrize("cu", LISTS, ids=lambda c: "-".join(map(str, c[:6])))
@pytest.mark.parametrize("mode,Hkv,times", [("turbo3", 2, 1), ("turbo4_asym", 3, 1), ("turbo3_table", 2, 1),
                                            ("turbo4", 5, 20), ("turbo3_asym", 4, 20), ("turbo4k_3v", 5, 20)])
def test_records_of_every_sequence_in_order(dev, mode, Hkv, times, cu):
    # (times 20: more than 4096 vectors, the tensor-core kernel)
    cu = [times * x for x in cu]
    total, B, (kb, vb) = 60 * times, len(cu) - 1, H.MODE_BITS[mode]
    cap = 64 * times
    k, v = wl.random_fp16(21, (total, Hkv, 128)), wl.random_fp16(22, (total, Hkv, 128))
    before = [(3 * b) % 5 for b in range(B)]
    rec = [None if r is None else np.array(r) for r in H.random_cache(mode, B, Hkv, cap, 23)]
    cache = H.gpu_cache_from_records(mode, B, Hkv, cap, before, *rec, dev)
    ctx = tqf.Context()
    tqf.tq_encode_append_packed(ctx, cache, H.upload(k, dev), H.upload(v, dev),
                                torch.tensor(cu, dtype=torch.int32, device=dev))
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_BAD_INDEX
    streams = [(2, 3, v, vb)] if kb == 16 else [(0, 1, k, kb), (2, 3, v, vb)]
    enc = []
    for _, _, x, bits in streams:
        codes, norms = S.encode_exact(x, bits)
        if mode in H.TABLE_MODES:
            t = o.centroid_norm_table(norms, o.codebook(bits))
            codes = np.concatenate([codes, t.astype("<f2").view(np.uint8)], axis=-1)
        enc.append((codes, norms))
    after = list(before)
    for b in range(B):
        lo, hi = cu[b], cu[b + 1]
        if not (0 <= lo <= hi <= total):
            continue
        at = slice(before[b], before[b] + hi - lo)
        after[b] += hi - lo
        for (data, norm, _, _), (codes, norms) in zip(streams, enc):
            rec[data][b, :, at] = codes[lo:hi].transpose(1, 0, 2)
            if rec[norm] is not None:
                rec[norm][b, :, at] = norms[lo:hi].T
        if kb == 16:
            rec[0][b, :, at] = k[lo:hi].transpose(1, 0, 2)
    assert cache.lengths.cpu().tolist() == after
    # every byte of the cache, what no sequence in order names included
    for name, t, w in zip(("k", "k_norm", "v", "v_norm"), (cache.k_data, cache.k_norm, cache.v_data, cache.v_norm), rec):
        if w is not None:
            assert np.array_equal(t.cpu().numpy().view(np.uint8), np.ascontiguousarray(w).view(np.uint8)), name


@pytest.mark.parametrize("times", [1, 40])
def test_a_sequence_that_shares_its_rows_and_passes_the_capacity(dev, times):
    cu, total, cap = [0, 20 * times, 10 * times, 60 * times], 60 * times, 64 * times
    k, v = (H.upload(wl.random_fp16(24 + i, (total, 2, 128)), dev) for i in range(2))
    cache, ctx = tqf.Cache(tqf.MODES["turbo4"], 3, 2, cap, dev), tqf.Context()
    cache.lengths.copy_(torch.tensor([0, 0, 15 * times], dtype=torch.int32))
    tqf.tq_encode_append_packed(ctx, cache, k, v, torch.tensor(cu, dtype=torch.int32, device=dev))
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_BAD_INDEX | tqf.TQ_STATUS_CAPACITY
    assert cache.lengths.cpu().tolist() == [20 * times, 0, 15 * times]
    assert not bool(cache.v_data[2].any())
