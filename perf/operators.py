"""The cache and attention operators of speculative and ragged serving, as they are measured.

Five operators over the packed cache (records of 128-dim K/V vectors: 3- or
4-bit codes of the rotated direction plus an fp16 norm, or fp16 K):

  append   packed prompts of different lengths encoded into the cache
  prefill  causal attention of such packed prompts over the cache
  tree     attention of a tree of drafted tokens over the cache
  compact  keeping the accepted ones of the drafted tokens
  copy     copying and forking sequences of the cache

``run`` computes them in elementary torch operations, or, where ``own`` is
true, makes the calls of the library.  The record layout is the one documented
in include/tq.h.
"""
import math

import numpy as np
import torch

own = False

BITS = {"turbo4_asym": (16, 4), "turbo3": (3, 3), "turbo4": (4, 4), "turbo3_asym": (16, 3),
        "turbo4k_3v": (4, 3)}
ROT_SEED = 42
SCALE = 1.0 / math.sqrt(128.0)
GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user's draft of 16 tokens over a medium context: latency
        dict(name="tree16_turbo3_b1", op="tree", mode="turbo3", batch=1, hq=28, hkv=4, nodes=16,
             ctx_lo=8176, ctx_hi=8176, shared=True),
        # a batch of users, drafts of 64 tokens, a tree of each one's own
        dict(name="tree64_turbo4_b8", op="tree", mode="turbo4", batch=8, hq=32, hkv=8, nodes=64,
             ctx_lo=4000, ctx_hi=16384, shared=False),
        # fp16 K, an odd number of drafted tokens and odd contexts
        dict(name="tree33_turbo4asym_b3", op="tree", mode="turbo4_asym", batch=3, hq=28, hkv=4,
             nodes=33, ctx_lo=777, ctx_hi=16351, shared=False),
        # three short prompts that arrive together: latency
        dict(name="prefill_short_turbo3", op="prefill", mode="turbo3", hq=28, hkv=4, batch=3,
             new_lo=17, new_hi=300, ctx_lo=0, ctx_hi=0),
        # a server's ordinary batch of prompts of very different lengths
        dict(name="prefill_mixed_turbo4", op="prefill", mode="turbo4", hq=32, hkv=8, batch=12,
             new_lo=64, new_hi=4096, ctx_lo=0, ctx_hi=0),
        # long chunks behind contexts that the cache holds already, fp16 K
        dict(name="prefill_chunks_turbo4asym", op="prefill", mode="turbo4_asym", hq=28, hkv=4,
             batch=3, new_lo=2047, new_hi=8192, ctx_lo=0, ctx_hi=8191),
        # the append of the short prompts
        dict(name="append_short_turbo3", op="append", mode="turbo3", hkv=4, batch=3, new_lo=17,
             new_hi=300, ctx_lo=0, ctx_hi=0),
        # the append of a server's batch, some 20,000 tokens, behind odd contexts
        dict(name="append_mixed_turbo4", op="append", mode="turbo4", hkv=8, batch=32, new_lo=64,
             new_hi=4096, ctx_lo=0, ctx_hi=999),
        # one user's accepted path of 5 drafted tokens
        dict(name="compact_turbo3_b1", op="compact", mode="turbo3", hkv=4, batch=1, nodes=16, keep=5,
             ctx_lo=8176, ctx_hi=8176),
        # a batch's, with fp16 K
        dict(name="compact_turbo4asym_b32", op="compact", mode="turbo4_asym", hkv=8, batch=32,
             nodes=64, keep=9, ctx_lo=4000, ctx_hi=16384),
        # a finished prompt moves from the prefill's cache to the decode's
        dict(name="copy_prompt_turbo3", op="copy", mode="turbo3", hkv=4, sources=1, forks=1,
             len_lo=8191, len_hi=8191, other=True),
        # parallel sampling: eight prompts, each forked to three more sequences
        dict(name="copy_fork_turbo4_b8x3", op="copy", mode="turbo4", hkv=8, sources=8, forks=3,
             len_lo=4000, len_hi=16384, other=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["tree", "tree", "prefill", "prefill", "append", "compact", "copy"])
    mode = rng.choice(sorted(BITS))
    if op == "tree":
        hq, hkv = rng.choice([(4, 2), (28, 4), (32, 8), (8, 8), (16, 2)])
        batch, nodes = _log(rng, 1, 16), _log(rng, 1, 128)
        hi = _log(rng, 1, 16384)
        # as much context work as the largest listed case at most
        hi = max(1, min(hi, 8 * 8 * 16384 // (batch * hkv * max(1, nodes * (hq // hkv) // 128))))
        return dict(op=op, mode=mode, batch=batch, hq=hq, hkv=hkv, nodes=nodes,
                    ctx_lo=rng.randint(0, hi), ctx_hi=hi, shared=rng.random() < 0.5)
    if op == "prefill":
        hq, hkv = rng.choice([(4, 2), (28, 4), (32, 8), (8, 8), (16, 2)])
        batch = _log(rng, 1, 16)
        hi = _log(rng, 1, 4096)
        ctx = rng.choice([0, 0, _log(rng, 1, 4096)])
        while batch > 1 and hq * batch * hi * (hi + ctx) > 6_000_000_000:
            batch //= 2
        return dict(op=op, mode=mode, hq=hq, hkv=hkv, batch=batch, new_lo=rng.randint(1, hi),
                    new_hi=hi, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx)
    hkv = rng.choice([2, 4, 8])
    if op == "append":
        batch, hi = _log(rng, 1, 32), _log(rng, 1, 4096)
        return dict(op=op, mode=mode, hkv=hkv, batch=batch, new_lo=rng.randint(1, hi), new_hi=hi,
                    ctx_lo=0, ctx_hi=rng.choice([0, _log(rng, 1, 999)]))
    if op == "compact":
        nodes = _log(rng, 1, 128)
        hi = _log(rng, 1, 16384)
        return dict(op=op, mode=mode, hkv=hkv, batch=_log(rng, 1, 32), nodes=nodes,
                    keep=rng.randint(1, max(1, min(nodes // 2, 16))), ctx_lo=rng.randint(0, hi),
                    ctx_hi=hi)
    hi = _log(rng, 1, 16384)
    return dict(op=op, mode=mode, hkv=hkv, sources=_log(rng, 1, 8), forks=rng.randint(1, 3),
                len_lo=rng.randint(1, hi), len_hi=hi, other=rng.random() < 0.5)


def _spread(lo, hi, n, off=0.0, log=False):
    """n numbers over [lo, hi], the first of them hi."""
    got = []
    for i in range(n):
        f = 1.0 - ((i * GOLDEN + (off if i or off else 0.0)) % 1.0)
        x = lo * (hi / lo) ** f if log and lo > 0 else lo + (hi - lo) * f
        got.append(int(round(x)))
    return got


def _cap(n):
    return (n + 16 + 15) // 16 * 16


def _record(mode):
    """Bytes of a token of one KV head."""
    kb, vb = BITS[mode]
    return (256 if kb == 16 else 16 * kb + 2) + 16 * vb + 2


def work(case):
    op, mode, rec = case["op"], case["mode"], _record(case["mode"])
    if op == "tree":
        ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["batch"])
        n, hq, hkv = case["nodes"], case["hq"], case["hkv"]
        # a drafted token sees the context, and of the tree its ancestors: a few
        pairs = sum(c * n for c in ctx)
        return {"bytes": sum(c + n for c in ctx) * hkv * rec + 2 * case["batch"] * hq * n * 256,
                "flops": 512 * hq * pairs}
    if op == "prefill":
        new = _spread(case["new_lo"], case["new_hi"], case["batch"], log=True)
        ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["batch"], 0.5)
        pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
        return {"bytes": sum(n + c for n, c in zip(new, ctx)) * case["hkv"] * rec
                + 2 * sum(new) * case["hq"] * 256, "flops": 512 * case["hq"] * pairs}
    if op == "append":
        new = sum(_spread(case["new_lo"], case["new_hi"], case["batch"], log=True))
        # the rotation as a fast transform: 7 stages of 128 sums
        return {"bytes": new * case["hkv"] * (512 + rec), "flops": new * case["hkv"] * 2 * 7 * 128}
    if op == "compact":
        kept = case["batch"] * case["keep"]
        return {"bytes": 2 * kept * case["hkv"] * rec + 8 * kept + 16 * case["batch"], "flops": 0}
    n = _spread(case["len_lo"], case["len_hi"], case["sources"])
    # a source is read once, however many copies are made of it
    return {"bytes": (1 + case["forks"]) * sum(n) * case["hkv"] * rec, "flops": 0}


# ---------------------------------------------------------------------------
# the format: rotation, codebooks, records (plain form)
# ---------------------------------------------------------------------------
def _signs():
    st, got = ROT_SEED, []
    for _ in range(128):
        st = (st + 0x9E3779B97F4A7C15) & (2**64 - 1)
        z = st
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & (2**64 - 1)
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & (2**64 - 1)
        z ^= z >> 31
        got.append(-1.0 if z >> 63 else 1.0)
    return got


_CODEBOOKS = {}


def _codebook(bits):
    """Lloyd-Max levels of N(0, 1/128), rounded to fp16 values."""
    if bits not in _CODEBOOKS:
        n, sigma = 1 << bits, 1.0 / math.sqrt(128.0)
        c = [sigma * (-2.0 + 4.0 * j / (n - 1)) for j in range(n)]
        phi = lambda x: 0.3989422804014327 * math.exp(-0.5 * x * x)  # noqa: E731
        cdf = lambda x: 0.5 * math.erfc(-x / math.sqrt(2.0))  # noqa: E731
        for _ in range(200000):
            e = [-math.inf] + [0.5 * (a + b) / sigma for a, b in zip(c, c[1:])] + [math.inf]
            p = [0.0 if math.isinf(x) else phi(x) for x in e]
            new = [sigma * (p[j] - p[j + 1]) / (cdf(e[j + 1]) - cdf(e[j])) for j in range(n)]
            done = max(abs(a - b) for a, b in zip(c, new)) < 1e-15
            c = new
            if done:
                break
        _CODEBOOKS[bits] = [float(x) for x in np.array(c, np.float64).astype(np.float16)]
    return _CODEBOOKS[bits]


class _Format:
    """Constants of the records on one device."""

    def __init__(self, dev):
        h = torch.ones(1, 1, dtype=torch.float64)
        for _ in range(7):
            h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
        self.sign = torch.tensor(_signs(), dtype=torch.float64, device=dev)
        self.had = h.to(dev)
        self.rot32 = (self.had * self.sign / math.sqrt(128.0)).float()  # Rot(x) = x @ rot32.T
        self.level, self.mid = {}, {}
        for b in (3, 4):
            c = torch.tensor(_codebook(b), dtype=torch.float64, device=dev)
            half = 1 << (b - 1)
            code = torch.arange(1 << b, device=dev)
            rank, neg = code % half, code >= half
            self.level[b] = torch.where(neg, c[half - 1 - rank], c[half + rank]).float()  # by code
            self.mid[b] = 0.5 * (c[:-1] + c[1:])
        self.j = torch.arange(8, device=dev, dtype=torch.int32)


_FORMATS = {}


def _format(dev):
    if dev not in _FORMATS:
        _FORMATS[dev] = _Format(dev)
    return _FORMATS[dev]


def _half(x):
    """fp64 to fp16, rounded once (a conversion through fp32 rounds twice)."""
    f = x.float()
    tie = (f.view(torch.int32) & 0x1FFF) == 0x1000
    up = torch.nextafter(f, torch.full_like(f, math.inf))
    down = torch.nextafter(f, torch.full_like(f, -math.inf))
    d = x - f.double()
    return torch.where(tie & (d > 0), up, torch.where(tie & (d < 0), down, f)).half()


def _encode(x, bits, fmt):
    """fp16 vectors [..., 128] -> (records uint8 [..., 16 bits], norms fp16)."""
    xd = x.double()
    norm = xd.square().sum(-1).sqrt()
    u = (xd * fmt.sign) @ fmt.had / (math.sqrt(128.0) * norm).unsqueeze(-1)
    u = torch.where(norm.unsqueeze(-1) > 0, u, torch.zeros_like(u))
    # the nearest level, ties to the lower one
    idx = torch.bucketize(u, fmt.mid[bits]).int()
    del xd, u
    half = 1 << (bits - 1)
    neg = idx < half
    code = torch.where(neg, half - 1 - idx, idx - half) | (neg.int() << (bits - 1))
    j = fmt.j
    if bits == 4:
        c = code.view(*x.shape[:-1], 16, 8)
        w = ((c & 7) << (4 * j)).sum(-1)
        s = c >> 3
        w = w + (s[..., :4] << (8 * j[:4] + 7)).sum(-1) + (s[..., 4:] << (8 * j[:4] + 3)).sum(-1)
    else:
        c = code.view(*x.shape[:-1], 4, 4, 8)
        w = (c[..., :3, :] << (4 * j)).sum(-1)
        k = fmt.j[:3].view(3, 1)
        w = w + (((c[..., 3:, :] >> k) & 1) << (4 * j + 3)).sum(-1)
    w = torch.where(w >= 2**31, w - 2**32, w).int() if w.dtype == torch.int64 else w
    return w.contiguous().view(torch.uint8).view(*x.shape[:-1], 16 * bits), _half(norm)


def _decode(rec, norm, bits, fmt):
    """Records -> norm * level in the rotated basis, fp32 [..., 128]."""
    w = rec.view(torch.int32)
    j = fmt.j
    if bits == 4:
        w = w.view(*rec.shape[:-1], 16, 1)
        s = torch.cat([(w >> (8 * j[:4] + 7)) & 1, (w >> (8 * j[:4] + 3)) & 1], -1)
        code = ((w >> (4 * j)) & 7) | (s << 3)
    else:
        w = w.view(*rec.shape[:-1], 4, 3, 1)
        last = ((w >> (4 * j + 3)) & 1) << fmt.j[:3].view(3, 1)
        code = torch.cat([(w >> (4 * j)) & 7, last.sum(-2, keepdim=True).int()], -2)
    x = fmt.level[bits][code.reshape(*rec.shape[:-1], 128)]
    return x.mul_(norm.float().unsqueeze(-1))


# ---------------------------------------------------------------------------
# states
# ---------------------------------------------------------------------------
class _State:
    pass


def _vectors(shape, gen, dev, channels=None):
    x = torch.randn(shape, generator=gen, device=dev)
    if channels is not None:  # K has a few channels of large values
        x[..., channels] *= 8.0
    return x.half()


def _buffers(mode, batch, hkv, cap, dev):
    kb, vb = BITS[mode]
    z = lambda *s, dt: torch.zeros(*s, dtype=dt, device=dev)  # noqa: E731
    return {
        "k": z(batch, hkv, cap, 128, dt=torch.float16) if kb == 16
        else z(batch, hkv, cap, 16 * kb, dt=torch.uint8),
        "k_norm": None if kb == 16 else z(batch, hkv, cap, dt=torch.float16),
        "v": z(batch, hkv, cap, 16 * vb, dt=torch.uint8),
        "v_norm": z(batch, hkv, cap, dt=torch.float16),
        "lengths": z(batch, dt=torch.int32),
    }


def _fill(buf, mode, lengths, gen, dev):
    """Records of seeded vectors at the tokens below `lengths`."""
    kb, vb = BITS[mode]
    fmt = _format(dev)
    channels = torch.randperm(128, generator=gen, device=dev)[:4]
    hkv = buf["v"].shape[1]
    for b, n in enumerate(lengths):
        for t in range(0, n, 8192):
            m = min(8192, n - t)
            k = _vectors((hkv, m, 128), gen, dev, channels)
            v = _vectors((hkv, m, 128), gen, dev)
            if kb == 16:
                buf["k"][b, :, t:t + m] = k
            else:
                buf["k"][b, :, t:t + m], buf["k_norm"][b, :, t:t + m] = _encode(k, kb, fmt)
            buf["v"][b, :, t:t + m], buf["v_norm"][b, :, t:t + m] = _encode(v, vb, fmt)
    buf["lengths"].copy_(torch.tensor(lengths, dtype=torch.int32))


def _handle(buf, mode):
    """The library's cache over these records."""
    import quantized_kv_cache_flash_gb300 as tq
    kb, vb = BITS[mode]
    cache = tq.Cache(tq.MODES[mode], buf["v"].shape[0], buf["v"].shape[1], buf["v"].shape[2],
                     buf["v"].device, codebook_k=None if kb == 16 else _codebook(kb),
                     codebook_v=_codebook(vb), rot_seed=ROT_SEED)
    for mine, its in (("k", cache.k_data), ("k_norm", cache.k_norm), ("v", cache.v_data),
                      ("v_norm", cache.v_norm), ("lengths", cache.lengths)):
        if its is not None:
            its.copy_(buf[mine])
    buf.update(k=cache.k_data, k_norm=cache.k_norm, v=cache.v_data, v_norm=cache.v_norm,
               lengths=cache.lengths)
    return cache


def _tree(nodes, real, rng):
    """Words of a random tree's mask: bit i of row j: node j sees node i (its
    ancestors and itself); the nodes past `real` are padding and see none."""
    words = (nodes + 31) // 32
    rows = [0] * nodes
    for i in range(real):
        parent = int(rng.integers(-1, i)) if i else -1
        rows[i] = (rows[parent] if parent >= 0 else 0) | (1 << i)
    return [[(r >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for r in rows]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(dev).manual_seed(int(seed) * 2 + 1)
    rng = np.random.Generator(np.random.PCG64([int(seed), 7]))
    s, op, mode, hkv = _State(), case["op"], case["mode"], case["hkv"]
    s.op, s.mode, s.fmt = op, mode, _format(dev)
    if op == "tree":
        batch, n = case["batch"], case["nodes"]
        lengths = [c + n for c in _spread(case["ctx_lo"], case["ctx_hi"], batch)]
        s.buf = _buffers(mode, batch, hkv, _cap(max(lengths)), dev)
        _fill(s.buf, mode, lengths, gen, dev)
        s.q = _vectors((batch, case["hq"], n, 128), gen, dev)
        # (trees that fill the rows, and in a batch some that leave padding)
        masks = [_tree(n, n if b % 2 == 0 else max(1, n - n // 4), rng)
                 for b in range(1 if case["shared"] else batch)]
        s.mask = torch.from_numpy(np.array(masks, np.uint32).view(np.int32)).to(dev)
        s.hint, s.out = max(lengths), torch.zeros_like(s.q)
    elif op in ("prefill", "append"):
        batch = case["batch"]
        new = _spread(case["new_lo"], case["new_hi"], batch, log=True)
        ctx = _spread(case["ctx_lo"], case["ctx_hi"], batch, 0.5)
        total = sum(new)
        s.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]).astype(np.int32), device=dev)
        s.hint = max(a + b for a, b in zip(new, ctx))
        s.buf = _buffers(mode, batch, hkv, _cap(s.hint), dev)
        s.longest = max(new)
        if op == "prefill":
            _fill(s.buf, mode, [a + b for a, b in zip(new, ctx)], gen, dev)
            s.q = _vectors((total, case["hq"], 128), gen, dev)
            s.out = torch.zeros_like(s.q)
        else:
            s.start = torch.tensor(ctx, dtype=torch.int32, device=dev)
            channels = torch.randperm(128, generator=gen, device=dev)[:4]
            s.k = _vectors((total, hkv, 128), gen, dev, channels)
            s.v = _vectors((total, hkv, 128), gen, dev)
    elif op == "compact":
        batch, n, keep = case["batch"], case["nodes"], case["keep"]
        ctx = _spread(case["ctx_lo"], case["ctx_hi"], batch)
        s.buf = _buffers(mode, batch, hkv, _cap(max(ctx) + n), dev)
        _fill(s.buf, mode, [c + n for c in ctx], gen, dev)
        s.start = torch.tensor(ctx, dtype=torch.int32, device=dev)
        s.n = n
        # accepted paths from the root down; behind the root they take nodes
        # past the kept block, so that a repeated pass reads the same records
        rows, counts = [], []
        for _ in range(batch):
            m = int(rng.integers(1, keep + 1))
            rest = np.sort(rng.permutation(np.arange(keep, n))[:m - 1]) if n > keep else []
            row = [0] + [int(x) for x in rest]
            counts.append(len(row))
            rows.append(row + [0] * (keep - len(row)))
        s.keep = torch.tensor(rows, dtype=torch.int32, device=dev)
        s.count = torch.tensor(counts, dtype=torch.int32, device=dev)
    else:
        src, forks = case["sources"], case["forks"]
        lengths = _spread(case["len_lo"], case["len_hi"], src)
        cap = _cap(max(lengths))
        batch = src if case["other"] else src * (1 + forks)
        s.buf = _buffers(mode, batch, hkv, cap, dev)
        _fill(s.buf, mode, lengths + [0] * (batch - src), gen, dev)
        s.to = _buffers(mode, src * forks, hkv, cap, dev) if case["other"] else None
        first = 0 if case["other"] else src
        order = rng.permutation(src * forks)
        s.src = torch.tensor([int(i) % src for i in order], dtype=torch.int32, device=dev)
        s.dst = torch.tensor([first + int(i) for i in order], dtype=torch.int32, device=dev)
        s.hint = max(lengths)
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        s.ctx, s.cache = tq.Context(), _handle(s.buf, mode)
        if op == "copy":
            s.to_cache = s.cache if s.to is None else _handle(s.to, mode)
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(s):
    return {"tree": _run_tree, "prefill": _run_prefill, "append": _run_append,
            "compact": _run_compact, "copy": _run_copy}[s.op](s)


def _softmax_v(score, seen, v):
    """Rows of softmax(score where seen) . v; rows that see nothing give 0."""
    score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = score.sum(-1, keepdim=True)
    return (score @ v) / torch.where(total > 0, total, torch.ones_like(total))


def _plain_attention(s, q, seen, tokens):
    """q [B, Hq, T, 128] over the first `tokens` tokens of the cache; seen
    [B, T, tokens].  In the rotated basis: products of rotated vectors are the
    products of the vectors."""
    kb, vb = BITS[s.mode]
    buf, fmt = s.buf, s.fmt
    b, hq, t, _ = q.shape
    hkv = buf["v"].shape[1]
    qr = q.float()
    if kb == 16:
        k = buf["k"][:, :, :tokens].float()
    else:
        k = _decode(buf["k"][:, :, :tokens].contiguous(), buf["k_norm"][:, :, :tokens], kb, fmt)
        qr = qr @ fmt.rot32.T
    score = (qr.reshape(b, hkv, hq // hkv * t, 128) @ k.transpose(-1, -2)).mul_(SCALE)
    del k
    v = _decode(buf["v"][:, :, :tokens].contiguous(), buf["v_norm"][:, :, :tokens], vb, fmt)
    o = _softmax_v(score.view(b, hkv, hq // hkv, t, tokens), seen.view(b, 1, 1, t, tokens),
                   v.unsqueeze(2))
    return o.reshape(b, hq, t, 128) @ fmt.rot32  # the inverse rotation


def _run_tree(s):
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        tq.tq_tree_attention(s.ctx, s.cache, s.q, s.out, s.mask, s.hint)
        return s.out
    n, dev = s.q.shape[2], s.q.device
    base = (s.buf["lengths"] - n).view(-1, 1, 1)
    at = torch.arange(s.hint, device=dev).view(1, 1, -1) - base           # place in the draft
    word = (at // 32).clamp(0, s.mask.shape[2] - 1)
    bits = torch.gather(s.mask.expand(s.q.shape[0], -1, -1), 2, word.expand(-1, n, -1))
    seen = (at < 0) | ((at < n) & (((bits >> (at % 32)) & 1) == 1))
    return _plain_attention(s, s.q, seen, s.hint).half()


def _run_prefill(s):
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        tq.tq_prefill_attention_packed(s.ctx, s.cache, s.q, s.out, s.cu, s.hint)
        return s.out
    dev, cu = s.q.device, s.cu.long()
    new = (cu[1:] - cu[:-1]).view(-1, 1)
    j = torch.arange(s.longest, device=dev).view(1, -1)
    row = cu[:-1].view(-1, 1) + torch.minimum(j, new - 1)                 # [B, longest]
    seen = torch.arange(s.hint, device=dev) <= (s.buf["lengths"].view(-1, 1) - new + j).unsqueeze(-1)
    o = _plain_attention(s, s.q[row].transpose(1, 2), seen, s.hint)      # [B, Hq, longest, 128]
    rows = torch.arange(s.q.shape[0], device=dev)
    b = torch.searchsorted(cu, rows, right=True) - 1
    return o[b, :, rows - cu[b]].half()


def _run_append(s):
    # new prompts enter their slots: the lengths before the append are set first
    s.buf["lengths"].copy_(s.start)
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        tq.tq_encode_append_packed(s.ctx, s.cache, s.k, s.v, s.cu)
        return {x: t for x, t in s.buf.items() if t is not None}
    kb, vb = BITS[s.mode]
    buf, cu = s.buf, s.cu.long()
    tok = torch.arange(s.k.shape[0], device=s.k.device)
    b = torch.searchsorted(cu, tok, right=True) - 1
    pos = buf["lengths"].long()[b] + tok - cu[b]
    if kb == 16:
        buf["k"][b, :, pos] = s.k
    else:
        buf["k"][b, :, pos], buf["k_norm"][b, :, pos] = _encode(s.k, kb, s.fmt)
    buf["v"][b, :, pos], buf["v_norm"][b, :, pos] = _encode(s.v, vb, s.fmt)
    buf["lengths"] += s.cu[1:] - s.cu[:-1]
    return {x: t for x, t in buf.items() if t is not None}


def _run_compact(s):
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        tq.tq_cache_compact(s.ctx, s.cache, s.start, s.keep, s.count, s.n)
        return {x: t for x, t in s.buf.items() if t is not None}
    buf = s.buf
    i = torch.arange(s.keep.shape[1], device=s.keep.device).view(1, -1)
    b = torch.arange(s.keep.shape[0], device=s.keep.device).view(-1, 1)
    at = s.start.long().view(-1, 1)
    src = at + torch.where(i < s.count.view(-1, 1), s.keep, i)
    for x in ("k", "k_norm", "v", "v_norm"):
        if buf[x] is not None:
            buf[x][b, :, at + i] = buf[x][b, :, src]
    buf["lengths"].copy_(s.start + s.count)
    return {x: t for x, t in buf.items() if t is not None}


def _run_copy(s):
    to = s.buf if s.to is None else s.to
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        tq.tq_cache_copy(s.ctx, s.to_cache, s.cache, s.dst, s.src, s.hint)
        return {x: t for x, t in to.items() if t is not None}
    src, dst = s.src.long(), s.dst.long()
    n = s.buf["lengths"][src]
    live = torch.arange(s.hint, device=n.device) < n.view(-1, 1)          # [M, hint]
    for x in ("k", "k_norm", "v", "v_norm"):
        if to[x] is not None:
            m = live.view(len(src), 1, -1, *([1] * (to[x].dim() - 3)))
            to[x][dst, :, :s.hint] = torch.where(m, s.buf[x][src, :, :s.hint], to[x][dst, :, :s.hint])
    to["lengths"][dst] = n
    return {x: t for x, t in to.items() if t is not None}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _bit_places(bits):
    """Places of the rank bits (low first) and the sign bit of each dimension in a record."""
    got = []
    for d in range(128):
        if bits == 4:
            word, j = d // 8, d % 8
            sign = 8 * j + 7 if j < 4 else 8 * (j - 4) + 3
            got.append([32 * word + 4 * j + i for i in range(3)] + [32 * word + sign])
        else:
            quarter, e = d // 32, d % 32
            if e < 24:
                got.append([96 * quarter + 32 * (e // 8) + 4 * (e % 8) + i for i in range(3)])
            else:
                got.append([96 * quarter + 32 * i + 4 * (e - 24) + 3 for i in range(3)])
    return got


def _full(rec, norm, bits):
    """The vectors that records stand for, in the original basis, fp64."""
    dev = rec.device
    place = torch.tensor(_bit_places(bits), device=dev)
    bit = (rec[..., place >> 3] >> (place & 7)) & 1                       # [..., 128, bits]
    rank = (bit[..., :-1].int() << torch.arange(bits - 1, device=dev)).sum(-1)
    level = torch.tensor(_codebook(bits)[1 << (bits - 1):], dtype=torch.float64, device=dev)[rank]
    y = torch.where(bit[..., -1] == 1, -level, level) * norm.double().unsqueeze(-1)
    i = np.arange(128)
    had = np.array([[(-1.0) ** bin(a & b).count("1") for b in i] for a in i]) / math.sqrt(128.0)
    return (y @ torch.from_numpy(had).to(dev)) * torch.tensor(_signs(), dtype=torch.float64, device=dev)


def exact(case, seed):
    if case["op"] in ("compact", "copy"):
        return None  # nothing is computed there
    s = prepare(case, seed)
    kb, vb = BITS[s.mode]
    if case["op"] == "append":
        # the norms; the codes are whole numbers
        new = (s.cu[1:] - s.cu[:-1]).tolist()
        first = s.cu.tolist()
        got = {"k": None, "k_norm": None, "lengths": None, "v": None}
        for name, x in ([("v_norm", s.v)] if kb == 16 else [("k_norm", s.k), ("v_norm", s.v)]):
            full = torch.zeros(s.buf["v_norm"].shape, dtype=torch.float64, device=x.device)
            size = torch.linalg.vector_norm(x.double(), dim=-1)
            for b, n in enumerate(new):
                at = int(s.start[b])
                full[b, :, at:at + n] = size[first[b]:first[b] + n].T
            got[name] = full
        return got
    lengths = s.buf["lengths"].tolist()
    out = torch.zeros(s.q.shape, dtype=torch.float64, device=s.q.device)
    hkv = case["hkv"]
    group = case["hq"] // hkv
    first = s.cu.tolist() if case["op"] == "prefill" else None
    for b, n in enumerate(lengths):
        rows = s.q[b] if first is None else s.q[first[b]:first[b + 1]].transpose(0, 1)  # [Hq, T, 128]
        t = rows.shape[1]
        if first is None:
            words = s.mask[b if s.mask.shape[0] > 1 else 0].cpu().numpy().view(np.uint32)
            seen = np.ones((t, n), bool)
            for j in range(t):
                for i in range(t):
                    seen[j, n - t + i] = bool((int(words[j, i >> 5]) >> (i & 31)) & 1)
            seen = torch.from_numpy(seen).to(s.q.device)
        else:
            seen = torch.ones(t, n, dtype=torch.bool, device=s.q.device).tril(n - t)
        for h in range(hkv):
            k = s.buf["k"][b, h, :n].double() if kb == 16 else \
                _full(s.buf["k"][b, h, :n], s.buf["k_norm"][b, h, :n], kb)
            v = _full(s.buf["v"][b, h, :n], s.buf["v_norm"][b, h, :n], vb)
            for g in range(h * group, (h + 1) * group):
                score = (rows[g].double() @ k.T * SCALE).masked_fill(~seen, -math.inf)
                o = torch.nan_to_num(torch.softmax(score, -1)) @ v
                if first is None:
                    out[b, g] = o
                else:
                    out[first[b]:first[b + 1], g] = o
    return out
