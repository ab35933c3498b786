"""Codes of packed appends against 64-bit decisions where fp32 sums go wrong: vectors
made so that the tensor core's sums lose as much as they can on the way to a value
beside a midpoint, and codebooks of other levels."""
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


def half(v):
    return np.float16(v).astype(np.float64)


def long_way_round(d, mid, rng):
    """An fp16 vector whose transform's entry d is 0.8e-6 of the norm above the
    midpoint: sixteen large products lead the sum past a power of two, 96 small ones
    follow that lose nearly a unit of its 25 bits each, and sixteen large ones lead
    back.  In 16-product steps with truncated addends the sum ends some 9e-6 of the norm
    too low."""
    p = np.zeros(128)
    big = half(256 * (1 + 0.9 * rng.random(16)))
    big = half(big * 2.0 ** math.ceil(math.log2(big.sum())) / big.sum() * 1.004)
    unit = 2.0 ** (math.floor(math.log2(big.sum())) - 25)
    p[:16] = big
    p[16:112] = 2 * unit * (1 - 2.0 ** -10)
    p[16:112:16] = unit * (1 - 2.0 ** -11)
    p[112:] = -big[rng.permutation(16)]
    for it in range(60):     # the last products bring the entry to its place
        n = math.sqrt(np.sum(p * p))
        gap = (mid * math.sqrt(128.0) + 0.8e-6) * n - p.sum()
        if abs(gap) < 0.3e-6 * n:
            break
        k = 112 + it % 8 if it < 30 else 120 + it % 3
        p[k] = half(gap + (0.0 if it >= 30 and abs(gap) <= 1e-3 * n and abs(p[k]) >= 1e-2 * n else p[k]))
    return (p * o.hadamard()[d] * o.sign_vector(42)).astype(np.float16)


def check_codes(dev, mode, k, v, cbk=None, cbv=None):
    """All codes of one packed append [n, Hkv, 128] equal to 64-bit decisions."""
    n, hkv, _ = k.shape
    kb, vb = H.MODE_BITS[mode]
    cache = tqf.Cache(tqf.MODES[mode], 1, hkv, (n + 15) // 16 * 16, dev, codebook_k=cbk, codebook_v=cbv)
    ctx = tqf.Context()
    tqf.tq_encode_append_packed(ctx, cache, H.upload(k, dev), H.upload(v, dev),
                                torch.tensor([0, n], dtype=torch.int32, device=dev))
    assert tqf.tq_get_status(ctx) == 0
    for data, x, bits, cb in ((cache.k_data, k, kb, cbk), (cache.v_data, v, vb, cbv)):
        codes, _ = S.encode_exact(x, bits, cb)
        got = data[0, :, :n].cpu().numpy().transpose(1, 0, 2)
        bad = np.flatnonzero((got != codes).any(-1).reshape(-1))
        assert len(bad) == 0, f"{len(bad)} vectors of {n * hkv}, the first {bad[:5]}"


@pytest.mark.parametrize("mode", ["turbo3", "turbo4"])
@pytest.mark.parametrize("n", [400, 4800])     # a warp per vector; the tensor cores
def test_sums_that_lose_what_they_can(dev, mode, n):
    bits = H.MODE_BITS[mode][0]
    cb = np.asarray(o.codebook(bits), np.float64)
    mids = 0.5 * (cb[:-1] + cb[1:])
    rng = np.random.default_rng(bits)
    x = wl.random_fp16(31, (n, 1, 128))
    for i in range(400):
        x[i, 0] = long_way_round(int(rng.integers(0, 128)), float(rng.choice(mids[mids > 0])), rng)
    check_codes(dev, mode, x, -x[::-1].copy())


def wide(bits):
    """Levels far from a normalised vector's, whose midpoints reach to entries of 1."""
    half_cb = np.array([0.05, 0.3, 0.6999, 1.3] if bits == 3 else [0.01, 0.06, 0.2, 0.5, 0.8, 0.95, 1.0498, 1.4], np.float32)
    return [-float(x) for x in half_cb[::-1]] + [float(x) for x in half_cb]


@pytest.mark.parametrize("mode", ["turbo3", "turbo4"])
@pytest.mark.parametrize("n", [2000, 60000])
def test_codebooks_of_wide_levels(dev, mode, n):
    """Vectors that lie almost along one row of the transform, their large entry
    within a few millionths of the midpoint near 1."""
    bits = H.MODE_BITS[mode][0]
    cb = wide(bits)
    mid = max(0.5 * (a + b) for a, b in zip(cb, cb[1:]) if 0.5 * (a + b) < 1.0)
    rng = np.random.default_rng(40 + bits)
    had, sign = o.hadamard(), o.sign_vector(42)
    d = rng.integers(0, 128, n)
    # u_d = cos of the angle to the row, spread over mid +- 3e-6
    tan = np.sqrt(1.0 / (mid + 3e-6 * rng.uniform(-1, 1, n)) ** 2 - 1.0)
    z = rng.standard_normal((n, 128))
    z -= (z * had[d]).sum(1, keepdims=True) / 128 * had[d]
    z *= (tan * math.sqrt(128.0) / np.linalg.norm(z, axis=1))[:, None]
    x = ((had[d] + z) * rng.uniform(1, 2000, (n, 1)) * sign).astype(np.float16).reshape(n, 1, 128)
    check_codes(dev, mode, x, x[::-1].copy(), cb, cb)
