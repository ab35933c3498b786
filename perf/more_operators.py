"""The operators that decide which tokens a cache keeps, as they are measured.

Three operators next to the packed cache (records of 128-dim K/V vectors: 3- or
4-bit codes of the rotated direction plus an fp16 norm, or fp16 K):

  weights  the softmax weight that each cached token gets from a block of
           queries, added up (for a single token, a window or a whole prompt)
  evict    dropping the tokens of least weight, within a cache or into another
  verify   which drafted tokens of a tree are accepted under the target's
           probabilities, and the token that follows them

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
        # one user's decode step that keeps its tokens' weights: latency
        dict(name="weights_step_turbo3_b1", op="weights", mode="turbo3", batch=1, hq=28, hkv=4, tq=1,
             ctx_lo=8176, ctx_hi=8176, decay=1.0),
        # a server's decode step, contexts of very different lengths
        dict(name="weights_step_turbo4_b32", op="weights", mode="turbo4", batch=32, hq=32, hkv=8, tq=1,
             ctx_lo=4000, ctx_hi=16384, decay=1.0),
        # fp16 K, odd contexts, older weights fading
        dict(name="weights_step_turbo4asym_b5", op="weights", mode="turbo4_asym", batch=5, hq=28, hkv=4,
             tq=1, ctx_lo=777, ctx_hi=16351, decay=0.98),
        # the last 64 tokens of a batch's prompts look back over them
        dict(name="weights_window64_turbo4_b8", op="weights", mode="turbo4", batch=8, hq=32, hkv=8, tq=64,
             ctx_lo=4000, ctx_hi=16384, decay=0.0),
        # every token of two prompts does
        dict(name="weights_prompt_turbo4asym_b2", op="weights", mode="turbo4_asym", batch=2, hq=28, hkv=4,
             tq=2047, ctx_lo=0, ctx_hi=511, decay=0.0),
        # one long sequence brought back to half, in place: latency
        dict(name="evict_half_turbo3_b1", op="evict", mode="turbo3", hkv=4, batch=1, len_lo=8191,
             len_hi=8191, keep_lo=4096, keep_hi=4096, sinks=4, recent=64, other=False),
        # a batch in place, fp16 K, lengths of which some need no eviction
        dict(name="evict_ragged_turbo4asym_b16", op="evict", mode="turbo4_asym", hkv=4, batch=16, len_lo=777,
             len_hi=16351, keep_lo=1000, keep_hi=4000, sinks=4, recent=128, other=False),
        # a batch of finished prompts pressed into the decode's smaller cache
        dict(name="evict_prompts_turbo4_b32", op="evict", mode="turbo4", hkv=8, batch=32, len_lo=4000,
             len_hi=16384, keep_lo=2048, keep_hi=2048, sinks=4, recent=64, other=True),
        # one user's chain of five drafted tokens: latency
        dict(name="verify_chain5_b1", op="verify", batch=1, nodes=6, vocab=32000, tree=False, draft=True),
        # a batch's trees of 64 nodes over a large vocabulary
        dict(name="verify_tree64_b8", op="verify", batch=8, nodes=64, vocab=131072, tree=True, draft=True),
        # tokens looked up in the prompt (no draft probabilities), an odd vocabulary
        dict(name="verify_lookup_b64", op="verify", batch=64, nodes=11, vocab=50001, tree=False, draft=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["weights", "weights", "weights", "evict", "evict", "verify", "verify"])
    if op == "verify":
        batch, nodes = _log(rng, 1, 64), _log(rng, 1, 64)
        vocab = min(_log(rng, 100, 200000), 8 * 64 * 131072 // (batch * nodes))
        return dict(op=op, batch=batch, nodes=nodes, vocab=vocab, tree=rng.random() < 0.5,
                    draft=rng.random() < 0.7)
    mode = rng.choice(sorted(BITS))
    if op == "evict":
        hi = _log(rng, 16, 16384)
        sinks, recent = rng.choice([0, 4]), rng.choice([0, min(hi // 4, 64)])
        keep = max(sinks + recent, 1, _log(rng, 1, hi))
        return dict(op=op, mode=mode, hkv=rng.choice([2, 4, 8]), batch=_log(rng, 1, 32),
                    len_lo=rng.randint(1, hi), len_hi=hi, keep_lo=rng.randint(max(1, sinks + recent), keep),
                    keep_hi=keep, sinks=sinks, recent=recent, other=rng.random() < 0.5)
    hq, hkv = rng.choice([(4, 2), (28, 4), (32, 8), (8, 8), (16, 2)])
    kind = rng.choice(["step", "step", "window", "prompt"])
    tq = {"step": rng.choice([1, 1, 2]), "window": _log(rng, 3, 128), "prompt": _log(rng, 16, 2048)}[kind]
    batch = _log(rng, 1, 32 if kind == "step" else 8 if kind == "window" else 2)
    hi = _log(rng, 1, 1024 if kind == "prompt" else 16384)
    if kind == "window":   # as many scores as the listed window's at most
        hi = max(1, min(hi, 8 * 32 * 64 * 10000 // (batch * hq * tq)))
    return dict(op=op, mode=mode, batch=batch, hq=hq, hkv=hkv, tq=tq, ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                decay=rng.choice([0.0, 0.9, 1.0]))


def _spread(lo, hi, n, off=0.0):
    """n numbers over [lo, hi], the first of them hi."""
    f = [1.0 - ((i * GOLDEN + (off if i or off else 0.0)) % 1.0) for i in range(n)]
    return [int(round(lo + (hi - lo) * x)) for x in f]


def _cap(n):
    return (n + 15) // 16 * 16


def _record(mode):
    """Bytes of a token of one KV head: K with its norm, V with its norm."""
    kb, vb = BITS[mode]
    return (256 if kb == 16 else 16 * kb + 2), 16 * vb + 2


def work(case):
    op = case["op"]
    if op == "verify":
        # the rows at the end of the accepted path, and the lists (a test of a
        # drafted token reads a number of each row)
        rows = case["batch"] * (2 if case["draft"] else 1)
        return {"bytes": 4 * rows * case["vocab"] + 24 * case["batch"] * case["nodes"], "flops": 2 * rows * case["vocab"]}
    k, v = _record(case["mode"])
    if op == "weights":
        ctx, n = _spread(case["ctx_lo"], case["ctx_hi"], case["batch"]), case["tq"]
        pairs = sum(c * n + n * (n + 1) // 2 for c in ctx)
        old = 4 if case["decay"] else 0
        return {"bytes": case["hkv"] * sum(c * (k + 4 + old) + n * (k + 4) for c in ctx)
                + case["batch"] * case["hq"] * n * 256, "flops": 256 * case["hq"] * pairs}
    lengths = _spread(case["len_lo"], case["len_hi"], case["batch"])
    keeps = _spread(case["keep_lo"], case["keep_hi"], case["batch"], 0.25)
    moved = sum(m if case["other"] or m < n else 0 for n, m in ((n, min(n, m)) for n, m in zip(lengths, keeps)))
    kept = sum(min(n, m) for n, m in zip(lengths, keeps))
    return {"bytes": case["hkv"] * (4 * sum(lengths) + 2 * moved * (k + v) + 8 * kept), "flops": 0}


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
        sign = torch.tensor(_signs(), dtype=torch.float64)
        self.rot32 = (h * sign / math.sqrt(128.0)).float().to(dev)  # Rot(x) = x @ rot32.T
        self.level, self.mid = {}, {}
        for b in (3, 4):
            c = torch.tensor(_codebook(b), dtype=torch.float64)
            half, code = 1 << (b - 1), torch.arange(1 << b)
            rank, neg = code % half, code >= half
            self.level[b] = torch.where(neg, c[half - 1 - rank], c[half + rank]).float().to(dev)  # by code
            self.mid[b] = (0.5 * (c[:-1] + c[1:])).float().to(dev)
        self.j = torch.arange(8, device=dev, dtype=torch.int32)


_FORMATS = {}


def _format(dev):
    if dev not in _FORMATS:
        _FORMATS[dev] = _Format(dev)
    return _FORMATS[dev]


def _pack(idx, bits, fmt):
    """Level numbers [..., 128] -> records uint8 [..., 16 bits]."""
    half, j = 1 << (bits - 1), fmt.j
    neg = idx < half
    code = torch.where(neg, half - 1 - idx, idx - half) | (neg.int() << (bits - 1))
    if bits == 4:
        c = code.view(*idx.shape[:-1], 16, 8)
        s = c >> 3
        w = ((c & 7) << (4 * j)).sum(-1) + (s[..., :4] << (8 * j[:4] + 7)).sum(-1) + (s[..., 4:] << (8 * j[:4] + 3)).sum(-1)
    else:
        c = code.view(*idx.shape[:-1], 4, 4, 8)
        w = (c[..., :3, :] << (4 * j)).sum(-1) + (((c[..., 3:, :] >> j[:3].view(3, 1)) & 1) << (4 * j + 3)).sum(-1)
    w = (w & 0xFFFFFFFF)
    w = torch.where(w >= 2**31, w - 2**32, w).int()
    return w.contiguous().view(torch.uint8).view(*idx.shape[:-1], 16 * bits)


def _levels(rec, norm, bits, fmt):
    """Records -> norm * level in the rotated basis, fp32 [..., 128]."""
    w = rec.view(torch.int32)
    j = fmt.j
    if bits == 4:
        w = w.view(*rec.shape[:-1], 16, 1)
        s = torch.cat([(w >> (8 * j[:4] + 7)) & 1, (w >> (8 * j[:4] + 3)) & 1], -1)
        code = ((w >> (4 * j)) & 7) | (s << 3)
    else:
        w = w.view(*rec.shape[:-1], 4, 3, 1)
        last = ((w >> (4 * j + 3)) & 1) << j[:3].view(3, 1)
        code = torch.cat([(w >> (4 * j)) & 7, last.sum(-2, keepdim=True).int()], -2)
    x = fmt.level[bits][code.reshape(*rec.shape[:-1], 128)]
    return x.mul_(norm.float().unsqueeze(-1))


# ---------------------------------------------------------------------------
# states
# ---------------------------------------------------------------------------
class _State:
    pass


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
    """Records at the tokens below `lengths`: codes of directions without a
    preferred axis (what the rotation leaves) and norms of vectors with a few
    large channels, or such fp16 vectors."""
    kb, vb = BITS[mode]
    fmt = _format(dev)
    channels = torch.randperm(128, generator=gen, device=dev)[:4]
    hkv = buf["v"].shape[1]
    for b, n in enumerate(lengths):
        for t in range(0, n, 16384):
            m = min(16384, n - t)
            for x, bits, size in (("k", kb, 19.5), ("v", vb, 11.3)):
                y = torch.randn(hkv, m, 128, generator=gen, device=dev)
                if bits == 16:
                    y[..., channels] *= 8.0
                    buf[x][b, :, t:t + m] = y.half()
                    continue
                y /= y.square().sum(-1, keepdim=True).sqrt()
                buf[x][b, :, t:t + m] = _pack(torch.bucketize(y, fmt.mid[bits]).int(), bits, fmt)
                r = 1.0 + 0.15 * torch.randn(hkv, m, generator=gen, device=dev)
                buf[x + "_norm"][b, :, t:t + m] = (size * r).clamp_(min=1.0).half()
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


def _parents(nodes, tree, rng):
    """Parents of a drafted tree's nodes, or of a chain's: node 0 is the last
    token that is settled, the others follow it or one another."""
    if not tree:
        return [i - 1 for i in range(nodes)]
    got = [-1]
    for i in range(1, nodes):
        # (up to four children, so that the tree is some six levels deep)
        free = [j for j in range(i) if got.count(j) < 4]
        got.append(free[min(len(free) - 1, int(rng.exponential(2.0)))])
    return got


def _prepare_verify(s, case, gen, rng, dev):
    b, n, v = case["batch"], case["nodes"], case["vocab"]
    # a tree of one shape for all, as the drafting model's expansion gives it
    s.parents = torch.tensor([_parents(n, case["tree"], rng)], dtype=torch.int32, device=dev)
    x = torch.randn(b, n, v, generator=gen, device=dev).mul_(2.5)
    s.target = torch.softmax(x, -1)
    if case["draft"]:
        x.add_(torch.randn(b, n, v, generator=gen, device=dev), alpha=0.5)
        s.draft = torch.softmax(x, -1)
        del x
    else:
        s.draft = None
    # a child's token is drawn from its parent's draft row (or, looked up, is
    # mostly what the target would say)
    up = s.parents[0].long().clamp(min=0)
    c = (s.draft if case["draft"] else s.target)[:, up].cumsum(-1)
    u = torch.rand(b, n, 1, generator=gen, device=dev) * c[..., -1:]
    s.tokens = torch.searchsorted(c, u).squeeze(-1).clamp_(max=v - 1).int()
    del c
    s.uniforms = torch.rand(b, n, generator=gen, device=dev)
    if own:
        z = lambda *sh: torch.zeros(*sh, dtype=torch.int32, device=dev)  # noqa: E731
        s.keep, s.num_keep, s.next = z(b, n), z(b), z(b)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(dev).manual_seed(int(seed) * 2 + 1)
    rng = np.random.Generator(np.random.PCG64([int(seed), 11]))
    s, op = _State(), case["op"]
    s.op = op
    if op == "verify":
        _prepare_verify(s, case, gen, rng, dev)
    else:
        mode, batch, hkv = case["mode"], case["batch"], case["hkv"]
        s.mode, s.fmt = mode, _format(dev)
        if op == "weights":
            n = case["tq"]
            lengths = [c + n for c in _spread(case["ctx_lo"], case["ctx_hi"], batch)]
            s.hint, s.decay = max(lengths), case["decay"]
            s.buf = _buffers(mode, batch, hkv, _cap(s.hint), dev)
            _fill(s.buf, mode, lengths, gen, dev)
            s.q = torch.randn(batch, case["hq"], n, 128, generator=gen, device=dev).half()
            # weights that earlier steps left
            s.weights = torch.rand(batch, hkv, _cap(s.hint), generator=gen, device=dev)
        else:
            lengths = _spread(case["len_lo"], case["len_hi"], batch)
            keeps = _spread(case["keep_lo"], case["keep_hi"], batch, 0.25)
            s.sinks, s.recent, s.hint, s.most = case["sinks"], case["recent"], max(lengths), max(keeps)
            s.buf = _buffers(mode, batch, hkv, _cap(s.hint), dev)
            _fill(s.buf, mode, lengths, gen, dev)
            s.start = torch.tensor(lengths, dtype=torch.int32, device=dev)
            s.count = torch.tensor(keeps, dtype=torch.int32, device=dev)
            cap = _cap(s.most) if case["other"] else _cap(s.hint)
            s.to = _buffers(mode, batch, hkv, cap, dev) if case["other"] else None
            # few heavy tokens, many light ones, some that nobody looked at
            w = torch.randn(batch, hkv, _cap(s.hint), generator=gen, device=dev).mul_(2.0).exp_()
            s.weights = torch.where(w < 0.1, torch.zeros_like(w), w)
            s.kept = torch.full((batch, hkv, s.most), -1, dtype=torch.int32, device=dev)
            s.new_weights = torch.zeros(batch, hkv, cap, device=dev)
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        s.ctx = tq.Context()
        if op != "verify":
            s.cache = _handle(s.buf, mode)
        if op == "evict":
            s.to_cache = s.cache if s.to is None else _handle(s.to, mode)
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------
def run(s):
    return {"weights": _run_weights, "evict": _run_evict, "verify": _run_verify}[s.op](s)


def _run_weights(s):
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        tq.tq_attention_weights(s.ctx, s.cache, s.q, s.weights, s.hint, decay=s.decay)
        return s.weights
    kb, buf, n = BITS[s.mode][0], s.buf, s.hint
    b, hq, t, _ = s.q.shape
    hkv = buf["v"].shape[1]
    q = s.q.float()
    # in the rotated basis: products of rotated vectors are the products of the vectors
    if kb == 16:
        k = buf["k"][:, :, :n].float()
    else:
        k = _levels(buf["k"][:, :, :n].contiguous(), buf["k_norm"][:, :, :n], kb, s.fmt)
        q = q @ s.fmt.rot32.T
    p = (q.reshape(b, hkv, hq // hkv * t, 128) @ k.transpose(-1, -2)).mul_(SCALE).view(b, hkv, hq // hkv, t, n)
    del k
    at = torch.arange(n, device=q.device)
    length = buf["lengths"].view(-1, 1, 1)
    seen = at <= length - t + torch.arange(t, device=q.device).view(1, -1, 1)      # [B, t, n]
    p.masked_fill_(~seen.view(b, 1, 1, t, n), -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    add = p.sum((2, 3))
    old = s.weights[:, :, :n]
    # the block's own tokens have no weight from before
    base = torch.where(at < length - t, old * s.decay, torch.zeros_like(old))
    s.weights[:, :, :n] = torch.where(at < length, base + add, old)
    return s.weights


def _run_evict(s):
    # (in place, the lengths before the eviction are set first)
    s.buf["lengths"].copy_(s.start)
    to = s.buf if s.to is None else s.to
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        tq.tq_cache_evict(s.ctx, s.to_cache, s.cache, s.weights, s.count, s.kept, s.hint, new_weights=s.new_weights,
                          sinks=s.sinks, recent=s.recent)
    else:
        n = s.hint
        w = s.weights[:, :, :n]
        at = torch.arange(n, device=w.device)
        length, count = s.start.view(-1, 1, 1).long(), s.count.view(-1, 1, 1).long()
        held = (at < s.sinks) | ((at >= length - s.recent) & (at < length)) | (length <= count)
        free = ((at < length) & ~held).expand_as(w)
        # of the others the heaviest, the first of equal ones
        order = torch.where(w.isnan(), torch.full_like(w, -math.inf), w).sort(dim=-1, descending=True, stable=True).indices
        is_free = free.gather(-1, order)
        take = is_free & (is_free.long().cumsum(-1) <= count - s.sinks - s.recent)
        keep = torch.zeros_like(free).scatter(-1, order, take) | (held & (at < length))
        src = (~keep).byte().sort(dim=-1, stable=True).indices[..., :s.most]           # kept ones first, in order
        m = src.shape[-1]
        live = torch.arange(m, device=w.device) < torch.minimum(length, count)
        live = live.expand_as(src)
        for x in ("k", "k_norm", "v", "v_norm"):
            if to[x] is not None:
                more = [1] * (to[x].dim() - 3)
                got = s.buf[x].gather(2, src.view(*src.shape, *more).expand(*src.shape, *to[x].shape[3:]))
                to[x][:, :, :m] = torch.where(live.view(*src.shape, *more), got, to[x][:, :, :m])
        s.new_weights[:, :, :m] = torch.where(live, s.weights.gather(-1, src), s.new_weights[:, :, :m])
        s.kept[:, :, :m] = torch.where(live, src.int(), s.kept[:, :, :m])
        to["lengths"].copy_(torch.minimum(s.start, s.count))
    return {"kept": s.kept, "weights": s.new_weights, **{x: t for x, t in to.items() if t is not None}}


def _run_verify(s):
    if own:
        import quantized_kv_cache_flash_gb300 as tq
        tq.tq_verify_tree(s.ctx, s.tokens, s.parents, s.target, s.draft, s.uniforms, s.keep, s.num_keep, s.next)
        return {"keep": s.keep, "num_keep": s.num_keep, "next": s.next}
    b, n, v = s.target.shape
    dev = s.target.device
    row = torch.arange(b, device=dev)
    at = torch.arange(v, device=dev)
    parents, tokens = s.parents.expand(b, -1).long(), s.tokens.long()
    cur, count = torch.zeros_like(row), torch.ones_like(row)
    keep = torch.full((b, n), -1, dtype=torch.int64, device=dev)
    keep[:, 0] = 0
    # what is left of the target's row, and its sum (64 bits: tokens at a border)
    left, total = s.target[:, 0].double(), torch.ones(b, dtype=torch.float64, device=dev)
    for i in range(1, n):
        x, u = tokens[:, i], s.uniforms[:, i].double()
        turn = parents[:, i] == cur
        if s.draft is None:
            q, qx = (at == x.unsqueeze(-1)).double(), torch.ones_like(u)
        else:
            q = s.draft[row, cur].double()
            qx = q[row, x]
        yes = turn & (u * qx * total < left[row, x])
        no = turn & ~yes
        less = (left - total.unsqueeze(-1) * q).clamp_(min=0.0)
        left = torch.where(yes.unsqueeze(-1), s.target[:, i].double(), torch.where(no.unsqueeze(-1), less, left))
        total = torch.where(yes, torch.ones_like(total), torch.where(no, less.sum(-1), total))
        keep[row, torch.where(yes, count, torch.full_like(count, n - 1))] = torch.where(
            yes, torch.full_like(cur, i), keep[row, torch.where(yes, count, torch.full_like(count, n - 1))])
        count = count + yes.long()
        cur = torch.where(yes, torch.full_like(cur, i), cur)
    # the token that follows: where the sum up to it first passes u of all
    left = torch.where((left.sum(-1) > 0).unsqueeze(-1), left, s.target[row, cur].double())
    c = left.cumsum(-1)
    follow = (c <= s.uniforms[:, :1].double() * c[:, -1:]).sum(-1)
    return {"keep": keep.int(), "num_keep": count.int(), "next": follow.int()}


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


def _exact_weights(s, case):
    kb, hkv, t = BITS[s.mode][0], case["hkv"], case["tq"]
    group = case["hq"] // hkv
    out = s.weights.double()
    for b, n in enumerate(s.buf["lengths"].tolist()):
        hidden = ~torch.ones(t, n, dtype=torch.bool, device=out.device).tril(n - t)
        for h in range(hkv):
            k = s.buf["k"][b, h, :n].double() if kb == 16 else \
                _full(s.buf["k"][b, h, :n], s.buf["k_norm"][b, h, :n], kb)
            got = torch.zeros(n, dtype=torch.float64, device=out.device)
            got[:max(n - t, 0)] = out[b, h, :max(n - t, 0)] * case["decay"] if case["decay"] else 0.0
            for g in range(h * group, (h + 1) * group):
                score = (s.q[b, g].double() @ k.T * SCALE).masked_fill(hidden, -math.inf)
                got += torch.nan_to_num(torch.softmax(score, -1)).sum(0)
            out[b, h, :n] = got
    return out


def _exact_verify(s, case):
    parents = s.parents[0].tolist()
    keeps, counts, follow = [], [], []
    for b in range(case["batch"]):
        token, u = s.tokens[b].tolist(), s.uniforms[b].double().tolist()
        path, at, tested = [0], 0, 0
        rest = s.target[b, 0].double()
        while True:
            # the first child of the path's end that has not been tried yet
            child = next((i for i in range(tested + 1, case["nodes"]) if parents[i] == at), None)
            if child is None:
                break
            tested = child
            q = torch.zeros_like(rest) if s.draft is None else s.draft[b, at].double()
            if s.draft is None:
                q[token[child]] = 1.0
            if u[child] * float(q[token[child]]) < float(rest[token[child]]):
                at = child
                path.append(at)
                rest = s.target[b, at].double()
            else:
                rest = torch.relu(rest - q)
                rest = rest / rest.sum() if float(rest.sum()) > 0 else rest
        if not float(rest.sum()) > 0:
            rest = s.target[b, at].double()
        sums = np.cumsum(rest.cpu().numpy())
        follow.append(int(np.searchsorted(sums, u[0] * sums[-1], side="right")))
        counts.append(len(path))
        keeps.append(path + [-1] * (case["nodes"] - len(path)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=s.tokens.device)  # noqa: E731
    return {"keep": i32(keeps), "num_keep": i32(counts), "next": i32(follow)}


def exact(case, seed):
    if case["op"] == "evict":
        return None  # nothing is computed there
    s = prepare(case, seed)
    return _exact_weights(s, case) if case["op"] == "weights" else _exact_verify(s, case)
