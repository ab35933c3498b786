"""Argument errors of the calls on attention weights, eviction and draft
verification (all found on the host before any CUDA call, so they run without a GPU),
and the 64-bit forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import quantized_kv_cache_flash_gb300 as tqf
from quantized_kv_cache_flash_gb300 import build as tqbuild
from tests import keeping_helpers as K
from tests.test_lib_cpu import FAKE, _cache
from tests.test_serving_cpu import LIST, LIST2, LIST3, OUT, Q, call
from tests.test_serving_refusals_cpu import far

BAD, NOT = tqf.TQ_ERR_INVALID_ARG, tqf.TQ_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    tqbuild.build()
    return tqf.lib()


def test_weights_errors(lib):
    base = dict(c=_cache(), q=Q, hq=4, tq=3, hint=32, scale=0.0, decay=1.0, seen=None, w=OUT)

    def go(**kw):
        a = {**base, **kw}
        return call(lib.tq_attention_weights, a["c"], a["q"], a["hq"], a["tq"], a["hint"], a["scale"], a["decay"],
                    a["seen"], a["w"])

    for kw in (dict(q=None), dict(q=Q + 8), dict(w=None), dict(w=OUT + 4), dict(hq=3), dict(hq=0), dict(tq=0),
               dict(tq=33), dict(hint=0), dict(hint=65), dict(scale=-1.0), dict(scale=float("inf")),
               dict(decay=-0.5), dict(decay=float("nan")), dict(decay=float("inf")), dict(seen=LIST + 2),
               dict(c=_cache(lengths=None)), dict(c=_cache(k_norm=None))):
        assert go(**kw) == BAD, kw
    assert go(c=_cache(mode=5)) == NOT                                  # table records
    assert go(hq=2 * 129) == NOT                                        # group over 128
    assert go(c=_cache(head_dim=64)) == NOT
    assert go(c=_cache(batch=40000, cap=16), hint=16) == NOT            # units
    cb = [float(np.float32(x) * np.float32(1.0001)) for x in tqf.tq_lloyd_max_codebook(3)]
    assert go(c=_cache(cb=cb)) == NOT                                   # not fp16 levels


def test_evict_errors(lib):
    W, NW, KEPT = (FAKE << 5), (FAKE << 5) + (1 << 20), (FAKE << 5) + (2 << 20)
    base = dict(d=far(), s=_cache(), w=W, nw=NW, n=LIST, kept=KEPT, mk=8, sinks=2, recent=3, hint=64)

    def go(**kw):
        a = {**base, **kw}
        return call(lib.tq_cache_evict, a["d"], a["s"], a["w"], a["nw"], a["n"], a["kept"], a["mk"], a["sinks"],
                    a["recent"], a["hint"])

    for kw in (dict(w=None), dict(w=W + 4), dict(nw=NW + 8), dict(n=None), dict(n=LIST + 1), dict(kept=None),
               dict(kept=KEPT + 2), dict(mk=0), dict(mk=-1), dict(sinks=-1), dict(recent=-1), dict(sinks=6),
               dict(sinks=9, recent=0), dict(hint=0), dict(hint=65),
               dict(d=far(batch=3)), dict(d=far(mode=2)), dict(d=far(hkv=4)), dict(d=far(rot_seed=1)),
               dict(d=far(v_rescale=2.0)), dict(d=_cache(cap=128)), dict(d=_cache(v_data=_cache().v_data + 4096)),
               # written while they are read
               dict(n=far().lengths), dict(n=far().lengths - 4), dict(kept=far().lengths), dict(kept=_cache().lengths),
               dict(nw=W), dict(nw=W + 16), dict(d=_cache(), nw=W + 16), dict(nw=KEPT), dict(kept=W), dict(kept=LIST),
               dict(nw=far().lengths & ~15), dict(nw=_cache().lengths & ~15), dict(nw=LIST & ~15)):
        assert go(**kw) == BAD, kw
    assert go(d=far(head_dim=64)) == NOT
    big = dict(batch=1 << 15, hkv=1 << 14, cap=16)      # cache rows past 2^31
    assert go(d=far(**big), s=_cache(**big), hint=16) == NOT


def test_verify_errors(lib):
    P, D, U, KEEP, NUM, NEXT = ((FAKE << 5) + i * (1 << 22) for i in range(6))
    base = dict(tok=LIST, par=LIST2, pb=1, p=P, ldp=100, d=D, ldd=100, u=U, b=3, n=5, v=100, keep=KEEP, num=NUM, nxt=NEXT)

    def go(**kw):
        a = {**base, **kw}
        return call(lib.tq_verify_tree, a["tok"], a["par"], a["pb"], a["p"], a["ldp"], a["d"], a["ldd"], a["u"],
                    a["b"], a["n"], a["v"], a["keep"], a["num"], a["nxt"])

    for kw in (dict(b=0), dict(n=0), dict(v=0), dict(b=-1), dict(pb=2), dict(pb=0), dict(ldp=99), dict(ldd=99),
               dict(tok=None), dict(par=None), dict(p=None), dict(u=None), dict(keep=None), dict(num=None),
               dict(nxt=None), dict(tok=LIST + 1), dict(p=P + 2), dict(d=D + 3), dict(u=U + 1), dict(keep=KEEP + 2),
               dict(keep=LIST), dict(num=LIST2 + 8), dict(nxt=U + 4), dict(nxt=P + 4 * 14 * 100), dict(keep=D),
               dict(num=KEEP), dict(nxt=KEEP + 56), dict(nxt=NUM)):
        assert go(**kw) == BAD, kw
    assert go(n=257) == NOT
    assert go(v=(1 << 30) + 1, ldp=1 << 31, ldd=1 << 31) == NOT
    assert go(ldp=1 << 58) == NOT
    assert go(b=(1 << 24) + 1) == NOT


def test_binding_refuses_wrong_tensors(lib):
    torch = pytest.importorskip("torch")
    ctx = tqf.Context()
    cache, other = (tqf.Cache(tqf.MODES["turbo3"], 2, 2, c, "cpu") for c in (32, 16))
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    h = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    V = tqf.tq_verify_tree
    ok = dict(tokens=i(3, 5), parents=i(1, 5), target=f(3, 5, 7), draft=f(3, 5, 7), uniforms=f(3, 5), keep=i(3, 5),
              num_keep=i(3), next_token=i(3))
    calls = [
        lambda: tqf.tq_attention_weights(ctx, cache, h(2, 4, 128), f(2, 2, 32), 32),
        lambda: tqf.tq_attention_weights(ctx, cache, h(2, 4, 1, 128), f(2, 2, 31), 32),
        lambda: tqf.tq_attention_weights(ctx, cache, h(2, 4, 1, 128), f(2, 2, 32).half(), 32),
        lambda: tqf.tq_attention_weights(ctx, cache, h(2, 4, 1, 128).float(), f(2, 2, 32), 32),
        lambda: tqf.tq_attention_weights(ctx, cache, h(2, 1, 4, 128).transpose(1, 2), f(2, 2, 32), 32, seen=i(2)),
        lambda: tqf.tq_attention_weights(ctx, cache, h(2, 4, 1, 128), f(2, 2, 32), 32, seen=i(3)),
        lambda: tqf.tq_attention_weights(ctx, cache, h(2, 4, 1, 128), f(2, 2, 32), 1 << 32),
        lambda: tqf.tq_attention_weights(ctx, cache, h(2, 4, 1, 128), f(2, 2, 32), 32),     # not on a CUDA device
        lambda: tqf.tq_cache_evict(ctx, other, cache, f(2, 2, 16), i(2), i(2, 2, 8), 32),
        lambda: tqf.tq_cache_evict(ctx, other, cache, f(2, 2, 32), i(3), i(2, 2, 8), 32),
        lambda: tqf.tq_cache_evict(ctx, other, cache, f(2, 2, 32), i(2), i(2, 8), 32),
        lambda: tqf.tq_cache_evict(ctx, other, cache, f(2, 2, 32), i(2), i(2, 1, 8), 32),
        lambda: tqf.tq_cache_evict(ctx, other, cache, f(2, 2, 32), i(2), i(2, 2, 8), 32, new_weights=f(2, 2, 32)),
        lambda: tqf.tq_cache_evict(ctx, other, cache, f(2, 2, 32), i(2), i(2, 2, 8), 32, sinks=1 << 33),
        lambda: tqf.tq_cache_evict(ctx, other, cache, f(2, 2, 32), i(2), i(2, 2, 8), 32),   # not on a CUDA device
        lambda: V(ctx, **{**ok, "target": f(3, 35)}),
        lambda: V(ctx, **{**ok, "target": f(3, 5, 7).double()}),
        lambda: V(ctx, **{**ok, "target": f(3, 7, 5).transpose(1, 2)}),
        lambda: V(ctx, **{**ok, "target": f(3, 10, 7)[:, ::2]}),          # (rows of one distance, sequences of another)
        lambda: V(ctx, **{**ok, "target": f(1, 5, 7).expand(3, 5, 7)}),
        lambda: V(ctx, **{**ok, "draft": f(3, 5, 8)}),
        lambda: V(ctx, **{**ok, "tokens": i(3, 4)}),
        lambda: V(ctx, **{**ok, "parents": i(2, 5)}),
        lambda: V(ctx, **{**ok, "uniforms": f(3, 5).double()}),
        lambda: V(ctx, **{**ok, "keep": i(5, 3).t()}),
        lambda: V(ctx, **{**ok, "next_token": i(3).long()}),
        lambda: V(ctx, **ok),                                             # not on a CUDA device
    ]
    for k, c in enumerate(calls):
        with pytest.raises(ValueError):
            c()
            pytest.fail(f"call {k} was taken")


def test_row_distances(lib):
    """The rows' distance that the verification's C call gets."""
    torch = pytest.importorskip("torch")
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    on = tqf._On(f(1))
    assert tqf._rows("x", f(3, 5, 7), (3, 5, 7), on) == 7
    assert tqf._rows("x", f(3, 5, 16)[:, :, :7], (3, 5, 7), on) == 16
    assert tqf._rows("x", f(3, 1, 16)[:, :, 2:9], (3, 1, 7), on) == 16
    assert tqf._rows("x", f(1, 1, 16)[:, :, :7], (1, 1, 7), on) == 7
    assert tqf._rows("x", f(4, 6, 1), (4, 6, 1), on) == 1


# ---------------------------------------------------------------------------
# the 64-bit forms
# ---------------------------------------------------------------------------
def test_weights_form_against_single_rows():
    from tests import helpers as H
    from quantized_kv_cache_flash_gb300 import workloads as wl
    from oracle import tq_oracle as o
    rec = H.random_cache("turbo4", 2, 2, 48, 5)
    q = wl.random_fp16(7, (2, 4, 3, 128))
    lengths = [40, 2]
    A, bound = K.weights("turbo4", rec, q, lengths, 2)
    assert np.allclose(A[0].sum(-1), 2 * 3) and np.all(A[0, :, 40:] == 0)       # every row's weights add to 1
    assert np.allclose(A[1].sum(-1), 2 * 2)                                     # the first query sees nothing
    # by hand: the last query's weights as the attention of one-hot values gives them
    unit = H.oracle_unit_from_records("turbo4", *rec, 0, 1, 40)
    Kf, _ = o.unit_kv_full("turbo4", unit, o.codebook(4), o.codebook(4), o.sign_vector(42))
    want = np.zeros(40)
    for g in range(2):
        for j in range(3):
            n = 40 - 3 + j + 1
            want[:n] += o.softmax_attention(q[0, 2 + g, j:j + 1].astype(np.float64), Kf[:n], np.eye(n), 128 ** -0.5,
                                            np.array([n]))[0]
    assert np.allclose(A[0, 1, :40], want, atol=1e-14)
    assert np.all(bound[0, 1, :40] < 2e-3 * A[0, 1, :40] + 1e-30)


def test_evict_form():
    w = np.array([5, 1, 3, np.nan, 3, -np.inf, 0.0, -0.0, 3, 9], np.float32)
    assert K.evict(w, 10, 3, 0, 0).tolist() == [0, 2, 9]
    assert K.evict(w, 10, 5, 1, 1).tolist() == [0, 2, 4, 8, 9]
    assert K.evict(w, 10, 7, 1, 1).tolist() == [0, 1, 2, 4, 6, 8, 9]      # -0 and 0 are equal: the first
    assert K.evict(w, 10, 9, 0, 0).tolist() == [0, 1, 2, 3, 4, 6, 7, 8, 9]     # NaN and -inf too
    assert K.evict(w, 4, 4, 0, 0).tolist() == [0, 1, 2, 3] and K.evict(w, 10, 0, 0, 0).tolist() == []


def test_verify_form():
    t = np.array([[.5, .3, .2], [.1, .8, .1], [1, 0, 0.]])
    d = np.array([[.2, .2, .6], [1, 0, 0.], [1, 0, 0.]])
    par = [-1, 0, 1]
    # .9 * .6 = .54 >= .2: rejected; what is left of row 0 is (.3, .1, 0)
    assert K.verify([0, 2, 0], par, t, d, [.74, .9, 0])[:2] == ([0], 0)
    assert K.verify([0, 2, 0], par, t, d, [.76, .9, 0])[:2] == ([0], 1)
    # .3 * .6 = .18 < .2: accepted; node 2 is token 0: .05 * 1 < .1, and no child is left
    assert K.verify([0, 2, 0], par, t, d, [.999, .3, .05])[:2] == ([0, 1, 2], 0)
    assert K.verify([0, 2, 0], par, t, d, [.5, .3, .2])[:2] == ([0, 1], 1)
    # without draft rows a token is accepted with its own probability
    assert K.verify([0, 2, 0], par, t, None, [.1, .19, .2])[:2] == ([0, 1], 1)
    assert K.verify([0, 2, 0], par, t, None, [.63, .21, 0])[:2] == ([0], 1)
