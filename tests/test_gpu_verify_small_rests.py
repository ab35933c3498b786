"""Draft verification where next to nothing is left after a rejection (a draft a hair from the
target): decisions and draws still equal the 64-bit form's, down to the sums' error bound."""
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


@pytest.mark.parametrize("B,V,apart", [(3, 700, 1e-3), (6, 5003, 1e-4), (20, 1999, 1e-4), (200, 300, 1e-3), (4, 30011, 1e-2)])
def test_small_rests(dev, B, V, apart):
    rng = np.random.default_rng(40 + V)
    N = 6
    p = rng.random((B, 1, V)) ** 3 + 1e-3
    p = np.repeat(p / p.sum(-1, keepdims=True), N, 1).astype(np.float32)
    q = p * (1 + apart * rng.standard_normal(p.shape))
    q = (q / q.sum(-1, keepdims=True, dtype=np.float64)).astype(np.float32)
    par = np.array([[-1, 0, 0, 0, 0, 0]], np.int32)
    tok = rng.integers(0, V, (B, N)).astype(np.int32)
    u = rng.random((B, N), np.float32)
    # the first two children are tokens that the draft has more of: rejected by the largest uniform number
    tok[:, 1:3] = np.argsort(p[:, 0] / q[:, 0], axis=-1)[:, :2]
    u[:, 1:3] = 1 - 2.0 ** -24
    keep, num, nxt = (torch.full(s, -9, dtype=torch.int32, device=dev) for s in ((B, N), (B,), (B,)))
    ctx = tqf.Context()
    up = lambda x: torch.from_numpy(x).to(dev)  # noqa: E731
    tqf.tq_verify_tree(ctx, up(tok), up(par), up(p), up(q), up(u), keep, num, nxt)
    keep, num, nxt = (t.cpu().numpy() for t in (keep, num, nxt))
    told = 0
    for b in range(B):
        path, follow, near = K.verify(tok[b], par[0], p[b], q[b], u[b])
        left = np.maximum(p[b, 0].astype(np.float64) - q[b, 0], 0.0).sum()
        # A sum drops less than two units of 2^-52 in each of at most 2^14 lanes: 2^-37 of what is
        # left, in each of the rests (at most five) that a decision goes by
        if near <= 6 * 2.0 ** -37 / left:
            continue
        told += 1
        assert keep[b, :num[b]].tolist() == path and nxt[b] == follow, f"sequence {b}"
    assert told > 0.9 * B and tqf.tq_get_status(ctx) == 0
