"""Draft verification on the GPU (tq_verify_tree): paths and tokens equal to the 64-bit
form's, over trees and chains, with draft rows and without, vocabularies that end
anywhere, rows with padding behind them, and rows of every kind; the accepted tokens'
distribution; graphs."""
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


def softmax(x):
    p = np.exp(x - x.max(-1, keepdims=True))
    return (p / p.sum(-1, keepdims=True)).astype(np.float32)


def trees(B, N, kind, rng):
    """Parents [B, N]: a chain, random trees, or one node with many children."""
    par = np.full((B, N), -1, np.int32)
    for b in range(B):
        for i in range(1, N):
            par[b, i] = {"chain": i - 1, "star": 0 if i < 3 * N // 4 else int(rng.integers(0, i)),
                         "tree": int(rng.integers(max(0, i - 6), i))}[kind]
            if kind == "tree" and rng.random() < 0.1:
                par[b, i] = -1          # padding
    return par


def problem(B, N, V, kind, draft, seed, sharp=2.0, near=0.5):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((B, N, V)) * sharp
    p = softmax(x)
    q = softmax(x + near * rng.standard_normal((B, N, V))) if draft else None
    par = trees(B, N, kind, rng)
    tok = np.zeros((B, N), np.int32)
    for b in range(B):
        for i in range(N):
            row = (q if draft else p)[b, max(par[b, i], 0)].astype(np.float64)
            tok[b, i] = min(int(np.searchsorted(np.cumsum(row), rng.random() * row.sum())), V - 1)
    return tok, par, p, q, rng.random((B, N), np.float32)


def on(x, dev, pad=0, off=0):
    """Rows on the device, `pad` numbers behind each, `off` numbers before the first."""
    if x is None:
        return None
    B, N, V = x.shape
    t = torch.full((B, N, V + pad), float("nan"), device=dev) if off == 0 else \
        torch.full((B * N * (V + pad) + off,), float("nan"), device=dev)[off:].view(B, N, V + pad)
    t[:, :, :V] = torch.from_numpy(x)
    return t[:, :, :V]


def verify(dev, tok, par, p, q, u, ctx=None):
    B, N = tok.shape
    keep, num, nxt = (torch.full(s, -9, dtype=torch.int32, device=dev) for s in ((B, N), (B,), (B,)))
    tqf.tq_verify_tree(ctx or tqf.Context(), torch.from_numpy(tok).to(dev), torch.from_numpy(par).to(dev), p, q,
                       torch.from_numpy(u).to(dev), keep, num, nxt)
    return keep.cpu().numpy(), num.cpu().numpy(), nxt.cpu().numpy()


def check(got, tok, par, p, q, u, near=1e-12):
    keep, num, nxt = got
    B, N = tok.shape
    for b in range(B):
        path, follow, dist = K.verify(tok[b], par[b if len(par) > 1 else 0], p[b], None if q is None else q[b], u[b])
        # (no decision of these inputs is nearer to a border than what either side rounds)
        assert dist > near, f"sequence {b}: an input at a border ({dist:.1e})"
        assert keep[b, :num[b]].tolist() == path and np.all(keep[b, num[b]:] == -1), f"sequence {b}"
        assert nxt[b] == follow, f"sequence {b}"


@pytest.mark.parametrize("draft", [True, False], ids=["drawn", "looked_up"])
@pytest.mark.parametrize("B,N,V,kind", [
    (1, 1, 1, "chain"), (1, 1, 100, "chain"), (2, 2, 2, "chain"), (3, 6, 1000, "chain"), (5, 33, 257, "tree"),
    (1, 64, 32000, "tree"), (9, 16, 4099, "tree"), (17, 40, 50, "star"), (33, 256, 97, "tree"), (2, 256, 641, "star"),
    (80, 5, 1003, "tree"), (200, 9, 129, "star"), (1, 7, 150001, "star"), (20, 4, 40001, "tree"), (9, 3, 70001, "star"),
])
def test_against_the_64_bit_form(dev, B, N, V, kind, draft):
    """Batches for 16, 8, 4, 2 and 1 CTAs a sequence; rows that the registers hold and longer ones."""
    tok, par, p, q, u = problem(B, N, V, kind, draft, 1000 + N + V)
    ctx = tqf.Context()
    check(verify(dev, tok, par, on(p, dev), on(q, dev), u, ctx), tok, par, p, q, u)
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("near", [0.0, 4.0])
def test_drafts_that_are_the_target_or_far_from_it(dev, near):
    """Equal rows accept the first child each time; far ones reject most, several at a node."""
    tok, par, p, q, u = problem(12, 40, 500, "star", True, 5, near=near)
    check(verify(dev, tok, par, on(p, dev), on(q, dev), u), tok, par, p, q, u)


@pytest.mark.parametrize("pad_p,pad_q,off", [(0, 0, 1), (3, 3, 0), (1, 2, 0), (5, 0, 2), (64, 61, 3), (0, 7, 0)])
def test_rows_at_any_distance_and_alignment(dev, pad_p, pad_q, off):
    """What lies behind and between the rows (NaN here) does not count."""
    tok, par, p, q, u = problem(4, 12, 1001, "star", True, 6)
    check(verify(dev, tok, par, on(p, dev, pad_p, off), on(q, dev, pad_q), u), tok, par, p, q, u)


def test_one_tree_for_all(dev):
    tok, par, p, q, u = problem(6, 20, 300, "tree", True, 7)
    check(verify(dev, tok, par[:1].copy(), on(p, dev), on(q, dev), u), tok, par[:1], p, q, u)


@pytest.mark.parametrize("draft", [True, False])
def test_rows_with_zeros(dev, draft):
    """Truncated distributions (top-k): tokens of probability 0 are neither accepted nor drawn."""
    tok, par, p, q, u = problem(30, 24, 400, "star", draft, 8)
    p = np.where(p < np.sort(p, -1)[..., -20:-19], 0, p).astype(np.float32)
    p /= p.sum(-1, keepdims=True)
    if draft:
        q = np.where(q < np.sort(q, -1)[..., -8:-7], 0, q).astype(np.float32)
        q /= q.sum(-1, keepdims=True)
        for b in range(30):
            for i in range(24):
                r = q[b, max(par[b, i], 0)]
                tok[b, i] = np.argmax(r) if r[tok[b, i]] == 0 else tok[b, i]
    keep, num, nxt = verify(dev, tok, par, on(p, dev), on(q, dev), u)
    check((keep, num, nxt), tok, par, p, q, u)
    for b in range(30):
        for i in keep[b, 1:num[b]]:
            assert p[b, par[b, i], tok[b, i]] > 0
        assert p[b, keep[b, num[b] - 1], nxt[b]] > 0


def test_numbers_of_every_kind(dev):
    """NaN, negative and infinite entries, uniform numbers at and past the ends, rows
    without positive entries, the same token twice among siblings."""
    tok, par, p, q, u = problem(16, 10, 200, "star", True, 9)
    p[:, :, 3::7], q[:, :, 5::11] = np.nan, np.nan
    p[:, :, 4::17], q[:, :, 6::13] = -0.25, -np.inf
    u[1, :], u[2, :], u[3, :] = 0.0, -1.0, np.nan
    u[4, 1:] = 1.0
    tok[5, 1:] = tok[5, 1]
    p[6], q[6] = 0.0, 0.0
    p[7, 0], q[7, 0] = np.nan, 0.5
    p[8, :] = np.eye(200, dtype=np.float32)[17]
    q[9] = p[9]
    par[10, 1:] = -1
    ctx = tqf.Context()
    check(verify(dev, tok, par, on(p, dev), on(q, dev), u, ctx), tok, par, p, q, u)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_BAD_VALUE
    # without draft rows: the same token twice is rejected twice
    check(verify(dev, tok, par, on(p, dev), None, u, ctx), tok, par, p, None, u)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_BAD_VALUE


def test_nothing_left_after_a_rejection(dev):
    """All of the target's mass on a token that was rejected by a rounding: its row itself."""
    p = np.zeros((1, 2, 50), np.float32)
    q = np.zeros((1, 2, 50), np.float32)
    p[0, :, 20], q[0, :, 20] = 0.75, 1.0          # (a row that does not add up to 1)
    tok, par = np.array([[0, 20]], np.int32), np.array([[-1, 0]], np.int32)
    keep, num, nxt = verify(dev, tok, par, on(p, dev), on(q, dev), np.array([[0.3, 0.9]], np.float32))
    assert keep.tolist() == [[0, -1]] and num[0] == 1 and nxt[0] == 20


def test_bad_nodes_count_as_padding(dev):
    tok, par, p, q, u = problem(7, 12, 100, "chain", True, 10, near=0.0)
    tok[0, 3], tok[1, 4], par[2, 5], par[3, 6], par[4, 2] = 100, -1, 5, 11, -2
    tok[5, 0], par[5, 0] = -5, 77                  # (the first node's say nothing)
    ctx = tqf.Context()
    got = verify(dev, tok, par, on(p, dev), on(q, dev), u, ctx)
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_BAD_INDEX
    assert got[1].tolist() == [3, 4, 5, 6, 2, 12, 12]
    for b, i in ((2, 5), (3, 6), (4, 2)):
        par[b, i] = -1
    check(got, tok, par, p, q, u)
    verify(dev, tok[5:], par[5:], on(p[5:], dev), on(q[5:], dev), u[5:], ctx)
    assert tqf.tq_get_status(ctx) == 0


@pytest.mark.parametrize("draft", [True, False])
def test_accepted_tokens_are_distributed_as_the_targets(dev, draft):
    """The first token after the settled one, over many sequences: the target's frequencies
    within five standard deviations, whatever the draft."""
    rng = np.random.default_rng(11)
    B, V = 60000, 6
    p1, q1 = softmax(rng.standard_normal(V) * 1.2), softmax(rng.standard_normal(V) * 1.2)
    par = np.array([[-1, 0, 0, 0, 1]], np.int32)
    p = np.broadcast_to(p1, (B, 5, V)).copy()
    q = np.broadcast_to(q1, (B, 5, V)).copy()
    tok = rng.choice(V, size=(B, 5), p=q1.astype(np.float64) / q1.sum(dtype=np.float64)).astype(np.int32)
    if not draft:
        tok[:, 1:4] = [2, 0, 5]       # looked up: whatever they are
    keep, num, nxt = verify(dev, tok, par, on(p, dev), on(q, dev) if draft else None, rng.random((B, 5), np.float32))
    first = np.where(num > 1, tok[np.arange(B), np.maximum(keep[:, 1], 0)], nxt)
    got = np.bincount(first, minlength=V) / B
    assert np.all(np.abs(got - p1) < 5 * np.sqrt(p1 * (1 - p1) / B)), (got, p1)
    second = num > 2                  # a token after an accepted one is the target's too
    if draft:
        got = np.bincount(np.where(second, tok[:, 4], nxt)[keep[:, 1] == 1], minlength=V)
        n = got.sum()
        assert np.all(np.abs(got / n - p1) < 5 * np.sqrt(p1 * (1 - p1) / n))


def test_replayed_with_other_numbers(dev):
    B, N, V = 3, 20, 3001
    a = [problem(B, N, V, "star", True, s) for s in (12, 13)]
    t = [torch.from_numpy(x).to(dev) for x in a[0]]
    out = [torch.zeros(s, dtype=torch.int32, device=dev) for s in ((B, N), (B,), (B,))]
    ctx = tqf.Context()
    go = lambda: tqf.tq_verify_tree(ctx, t[0], t[1], t[2], t[3], t[4], *out)  # noqa: E731
    go()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for x in (a[1], a[0]):
        for d, s in zip(t, x):
            d.copy_(torch.from_numpy(s))
        g.replay()
        check([o.cpu().numpy() for o in out], *x)
    assert tqf.tq_get_status(ctx) == 0
