"""Argument errors of the packed, tree and record-move calls (all found on the
host before any CUDA call, so they run without a GPU), the host-only tree mask,
and the 64-bit forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import quantized_kv_cache_flash_gb300 as tqf
from quantized_kv_cache_flash_gb300 import build as tqbuild
from oracle import tq_oracle as o
from tests import serving_helpers as S
from tests.test_lib_cpu import FAKE, _cache


@pytest.fixture(scope="module")
def lib():
    tqbuild.build()
    return tqf.lib()


Q, OUT, LIST, LIST2, LIST3 = (FAKE + i * 65536 for i in range(1, 6))


def call(f, *args):
    ctx = ctypes.c_void_p(None)
    r = f(ctypes.byref(ctx), *[ctypes.byref(a) if isinstance(a, tqf.tq_cache) else a for a in args], None)
    assert ctx.value is None      # no context is created for a rejected call
    return r


def test_packed_append_errors(lib):
    f = lib.tq_encode_append_packed
    assert call(f, _cache(), Q, OUT, None, 5) == tqf.TQ_ERR_INVALID_ARG
    assert call(f, _cache(), Q, OUT, LIST, -1) == tqf.TQ_ERR_INVALID_ARG
    assert call(f, _cache(), None, OUT, LIST, 5) == tqf.TQ_ERR_INVALID_ARG
    assert call(f, _cache(), Q, OUT + 8, LIST, 5) == tqf.TQ_ERR_INVALID_ARG
    assert call(f, _cache(mode=9), Q, OUT, LIST, 5) == tqf.TQ_ERR_UNSUPPORTED
    assert call(f, _cache(hkv=8), Q, OUT, LIST, 1 << 28) == tqf.TQ_ERR_UNSUPPORTED   # 2^31 vectors
    assert call(f, _cache(), None, None, LIST, 0) == tqf.TQ_OK                       # no-op


def test_packed_prefill_errors(lib):
    f = lib.tq_prefill_attention_packed
    base = dict(c=_cache(), q=Q, hq=4, cu=LIST, total=5, hint=32, scale=0.0, out=OUT)

    def go(**kw):
        a = {**base, **kw}
        return call(f, a["c"], a["q"], a["hq"], a["cu"], a["total"], a["hint"], a["scale"], a["out"])

    for kw in (dict(cu=None), dict(total=-1), dict(q=None), dict(out=OUT + 2), dict(hq=3), dict(hq=0),
               dict(hint=0), dict(hint=65), dict(scale=-1.0), dict(scale=float("nan")),
               dict(c=_cache(v_rescale=float("inf")))):
        assert go(**kw) == tqf.TQ_ERR_INVALID_ARG, kw
    assert go(c=_cache(mode=5)) == tqf.TQ_ERR_UNSUPPORTED              # table records
    assert go(hq=2 * 129) == tqf.TQ_ERR_UNSUPPORTED                    # group over 128
    cb = [float(np.float32(x) * np.float32(1.0001)) for x in tqf.tq_lloyd_max_codebook(3)]
    assert go(c=_cache(cb=cb)) == tqf.TQ_ERR_UNSUPPORTED               # not fp16 levels
    assert go(total=0, q=None, out=None) == tqf.TQ_OK                  # no-op


def test_tree_errors(lib):
    f = lib.tq_tree_attention
    base = dict(c=_cache(cap=512), q=Q, hq=4, tq=8, hint=300, scale=0.0, mask=LIST, mb=1, out=OUT)

    def go(**kw):
        a = {**base, **kw}
        return call(f, a["c"], a["q"], a["hq"], a["tq"], a["hint"], a["scale"], a["mask"], a["mb"], a["out"])

    for kw in (dict(mask=None), dict(mask=LIST + 2), dict(mb=0), dict(mb=3), dict(q=None), dict(out=None),
               dict(tq=0), dict(tq=-1), dict(hq=3), dict(hint=0), dict(hint=513), dict(tq=200, hint=100),
               dict(scale=-0.5), dict(c=_cache(cap=512, lengths=None))):
        assert go(**kw) == tqf.TQ_ERR_INVALID_ARG, kw
    assert go(tq=257) == tqf.TQ_ERR_UNSUPPORTED
    assert go(hq=2 * 129) == tqf.TQ_ERR_UNSUPPORTED
    assert go(c=_cache(cap=512, head_dim=64)) == tqf.TQ_ERR_UNSUPPORTED


def test_compact_errors(lib):
    f = lib.tq_cache_compact
    base = dict(c=_cache(), start=LIST, n=8, keep=LIST2, count=LIST3, mk=4)

    def go(**kw):
        a = {**base, **kw}
        return call(f, a["c"], a["start"], a["n"], a["keep"], a["count"], a["mk"])

    for kw in (dict(start=None), dict(keep=None), dict(count=None), dict(n=0), dict(mk=0), dict(mk=9)):
        assert go(**kw) == tqf.TQ_ERR_INVALID_ARG, kw
    assert go(n=65) == tqf.TQ_ERR_CAPACITY


def test_copy_errors(lib):
    f = lib.tq_cache_copy
    far = dict(k_data=FAKE << 4, k_norm=(FAKE << 4) + (1 << 20), v_data=(FAKE << 4) + (2 << 20),
               v_norm=(FAKE << 4) + (3 << 20), lengths=(FAKE << 4) + (4 << 20))
    base = dict(d=_cache(**far), s=_cache(), ds=LIST, ss=LIST2, n=None, m=2, hint=64)

    def go(**kw):
        a = {**base, **kw}
        return call(f, a["d"], a["s"], a["ds"], a["ss"], a["n"], a["m"], a["hint"])

    for kw in (dict(ds=None), dict(ss=None), dict(m=-1), dict(hint=0), dict(hint=65),
               dict(d=_cache(mode=2, **far)), dict(d=_cache(hkv=4, **far)), dict(d=_cache(rot_seed=1, **far)),
               dict(d=_cache(v_rescale=2.0, **far)),
               dict(d=_cache(cb=[2 * x for x in tqf.tq_lloyd_max_codebook(3)], **far)),
               dict(d=_cache(cap=128)),                                  # one buffer, two shapes
               dict(d=_cache(**{**far, "k_data": _cache().k_data})),     # one buffer of several
               dict(d=_cache(**{**far, "v_data": _cache().v_data + 48})),   # buffers that overlap
               dict(d=_cache(**{**far, "lengths": _cache().lengths + 4}))):
        assert go(**kw) == tqf.TQ_ERR_INVALID_ARG, kw
    assert go(m=0) == tqf.TQ_OK
    assert go(m=1 << 30, hint=64, ds=LIST) == tqf.TQ_ERR_UNSUPPORTED     # 2^31 CTAs


def test_tree_mask(lib):
    rng = np.random.default_rng(0)
    for n in (1, 2, 31, 32, 33, 64, 200, 256):
        parents = [int(rng.integers(-1, i)) if i else -1 for i in range(n)]
        words = tqf.tq_tree_mask(parents).numpy().view(np.uint32)
        assert words.shape == (n, (n + 31) // 32)
        for j in range(n):
            want, i = set(), j
            while i >= 0:
                want.add(i)
                i = parents[i]
            assert {i for i in range(32 * words.shape[1]) if words[j, i >> 5] >> (i & 31) & 1} == want
    for bad in ([0], [-1, 1], [-1, -2], [-1, 2, 0]):
        with pytest.raises(tqf.TqError) as e:
            tqf.tq_tree_mask(bad)
        assert e.value.code == tqf.TQ_ERR_INVALID_ARG
    with pytest.raises(tqf.TqError) as e:
        tqf.tq_tree_mask([-1] * 257)
    assert e.value.code == tqf.TQ_ERR_UNSUPPORTED
    with pytest.raises(tqf.TqError):
        tqf.tq_tree_mask([])


def test_binding_refuses_wrong_tensors(lib):
    torch = pytest.importorskip("torch")
    cache = tqf.Cache(tqf.MODES["turbo3"], 2, 2, 32, "cpu")
    ctx = tqf.Context()
    h, i = torch.float16, torch.int32
    z = lambda *s, dt=h: torch.zeros(*s, dtype=dt)  # noqa: E731
    cu = z(3, dt=i)
    calls = [
        lambda: tqf.tq_encode_append_packed(ctx, cache, z(5, 3, 128), z(5, 3, 128), cu),           # heads
        lambda: tqf.tq_encode_append_packed(ctx, cache, z(5, 2, 128), z(4, 2, 128), cu),           # rows
        lambda: tqf.tq_encode_append_packed(ctx, cache, z(5, 2, 128).float(), z(5, 2, 128), cu),   # type
        lambda: tqf.tq_encode_append_packed(ctx, cache, z(5, 2, 128), z(5, 2, 128), z(4, dt=i)),   # bounds
        lambda: tqf.tq_encode_append_packed(ctx, cache, z(5, 2, 128), z(5, 2, 128), cu.long()),
        lambda: tqf.tq_encode_append_packed(ctx, cache, z(2, 5, 128).transpose(0, 1), z(5, 2, 128), cu),  # strides
        lambda: tqf.tq_prefill_attention_packed(ctx, cache, z(5, 4, 128), z(5, 4, 64), cu, 32),
        lambda: tqf.tq_prefill_attention_packed(ctx, cache, z(5, 4, 128), z(4, 4, 128), cu, 32),
        lambda: tqf.tq_tree_attention(ctx, cache, z(2, 4, 40, 128), z(2, 4, 40, 128), z(1, 40, 1, dt=i), 32),
        lambda: tqf.tq_tree_attention(ctx, cache, z(2, 4, 3, 128), z(2, 4, 3, 128), z(3, 3, 1, dt=i), 32),
        lambda: tqf.tq_tree_attention(ctx, cache, z(1, 4, 3, 128), z(1, 4, 3, 128), z(1, 3, 1, dt=i), 32),
        lambda: tqf.tq_cache_compact(ctx, cache, z(2, dt=i), z(3, 4, dt=i), z(2, dt=i), 8),
        lambda: tqf.tq_cache_copy(ctx, cache, cache, z(2, dt=i), z(3, dt=i), 32),
        # the right shapes, but not on a CUDA device
        lambda: tqf.tq_encode_append_packed(ctx, cache, z(5, 2, 128), z(5, 2, 128), cu),
    ]
    for c in calls:
        with pytest.raises(ValueError):
            c()


def test_plain_forms_agree_with_the_oracle():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((300, 128)).astype(np.float16)
    for bits in (3, 4):
        codes, norms = S.encode_exact(x, bits)
        idx, n16, u, _ = o.encode(x, o.codebook(bits), o.sign_vector(42))
        assert np.array_equal(o.unpack_codes(codes, bits), idx) and np.array_equal(norms, n16)
    q, K, V = rng.standard_normal((3, 128)), rng.standard_normal((50, 128)), rng.standard_normal((50, 128))
    seen = np.arange(50)[None, :] <= np.array([0, 30, 49])[:, None]
    got, bound = S.attention_rows(q, K, V, seen, 0.1)
    want = o.softmax_attention(q, K, V, 0.1, np.array([1, 31, 50]))
    assert np.allclose(got, want, atol=1e-13) and np.all(bound > 0)
    # the bound notices a term that is missing
    wrong, _ = S.attention_rows(q, K, V, seen & (np.arange(50) != 0), 0.1)
    with pytest.raises(AssertionError):
        S.assert_rows(wrong, want, bound)
