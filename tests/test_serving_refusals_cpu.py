"""Calls on packed sequences, trees and record moves that are refused on the host
because the GPU would read a list at a bad address or while it is being written."""
import pytest

import quantized_kv_cache_flash_gb300 as tqf
from quantized_kv_cache_flash_gb300 import build as tqbuild
from tests.test_lib_cpu import FAKE, _cache
from tests.test_serving_cpu import LIST, LIST2, LIST3, OUT, Q, call


@pytest.fixture(scope="module")
def lib():
    tqbuild.build()
    return tqf.lib()


def far(**kw):
    """A cache that shares nothing with _cache()'s."""
    at = FAKE << 4
    return _cache(**{**dict(k_data=at, k_norm=at + (1 << 20), v_data=at + (2 << 20), v_norm=at + (3 << 20),
                            lengths=at + (4 << 20)), **kw})


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_lists(lib, off):
    bad = tqf.TQ_ERR_INVALID_ARG
    assert call(lib.tq_encode_append_packed, _cache(), Q, OUT, LIST + off, 5) == bad
    assert call(lib.tq_prefill_attention_packed, _cache(), Q, 4, LIST + off, 5, 32, 0.0, OUT) == bad
    assert call(lib.tq_tree_attention, _cache(), Q, 4, 8, 32, 0.0, LIST + off, 1, OUT) == bad
    for i in range(3):
        a = [LIST, LIST2, LIST3]
        a[i] += off
        assert call(lib.tq_cache_compact, _cache(), a[0], 8, a[1], a[2], 4) == bad
        assert call(lib.tq_cache_copy, far(), _cache(), a[0], a[1], a[2], 2, 64) == bad
    lengths = _cache().lengths + off
    for f, args in ((lib.tq_encode_append_packed, (Q, OUT, LIST, 5)),
                    (lib.tq_prefill_attention_packed, (Q, 4, LIST, 5, 32, 0.0, OUT)),
                    (lib.tq_tree_attention, (Q, 4, 8, 32, 0.0, LIST, 1, OUT)),
                    (lib.tq_decode_attention, (Q, 4, 1, 32, 0.0, OUT)),
                    (lib.tq_cache_compact, (LIST, 8, LIST2, LIST3, 4))):
        assert call(f, _cache(lengths=lengths), *args) == bad
    assert call(lib.tq_cache_copy, far(lengths=far().lengths + off), _cache(), LIST, LIST2, None, 2, 64) == bad


def test_lists_that_lie_in_the_lengths(lib):
    """The lengths are written while other CTAs of the call still read the lists."""
    bad = tqf.TQ_ERR_INVALID_ARG
    c = _cache(batch=3)
    at = c.lengths
    for i in range(3):
        for shared in (at, at + 8, at - 4):
            a = [LIST, LIST2, LIST3]
            a[i] = shared
            assert call(lib.tq_cache_compact, _cache(batch=3), a[0], 8, a[1], a[2], 4) == bad
            # within a cache, and from another one
            assert call(lib.tq_cache_copy, _cache(batch=3), _cache(batch=3), a[0], a[1], a[2], 2, 64) == bad
            assert call(lib.tq_cache_copy, _cache(batch=3), far(batch=3), a[0], a[1], a[2], 2, 64) == bad


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 32, -(1 << 31) - 1])
def test_numbers_past_32_bits(lib, n):
    """The binding refuses what the C call's integers would cut off to another number."""
    torch = pytest.importorskip("torch")
    cache, ctx = tqf.Cache(tqf.MODES["turbo3"], 2, 2, 32, "cpu"), tqf.Context()
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for name, f in (("max_len_hint", lambda: tqf.tq_prefill_attention_packed(ctx, cache, h(5, 4, 128), h(5, 4, 128), i(3), n)),
                    ("max_len_hint", lambda: tqf.tq_tree_attention(ctx, cache, h(2, 4, 3, 128), h(2, 4, 3, 128), i(1, 3, 1), n)),
                    ("max_len_hint", lambda: tqf.tq_cache_copy(ctx, cache, cache, i(2), i(2), n)),
                    ("num_drafted", lambda: tqf.tq_cache_compact(ctx, cache, i(2), i(2, 4), i(2), n))):
        with pytest.raises(ValueError, match=name):
            f()
