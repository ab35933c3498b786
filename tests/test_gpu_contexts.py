"""Contexts on the GPU: what a new one owes to work on other streams."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import quantized_kv_cache_flash_gb300 as tqf
from quantized_kv_cache_flash_gb300 import workloads as wl
from tests import helpers as H

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


@pytest.mark.parametrize("n", [40, 5000])   # a warp per vector; the tensor-core kernel with its tile counter
def test_first_call_on_a_side_stream_while_the_default_stream_is_busy(dev, n):
    """The first call of a context creates it.  Its counters and status word are
    zero for that call and nothing clears them behind it, whatever the default
    stream still has to do."""
    cap = (2 * n + 15) // 16 * 16
    k, v = (H.upload(wl.random_fp16(50 + i, (n, 1, 128)), dev) for i in range(2))
    cu = i32([0, n - 3, n], dev)
    cache = tqf.Cache(tqf.MODES["turbo3"], 2, 1, cap, dev)
    side = torch.cuda.Stream()
    tqf.tq_encode_append_packed(tqf.Context(), cache, k, v, cu, stream=side)   # (loads the kernels)
    torch.cuda.synchronize()
    cache.lengths.copy_(i32([0, cap], dev))      # the second sequence is full
    torch.cuda.synchronize()
    torch.cuda.synchronize()
    ctx = tqf.Context()
    torch.cuda._sleep(200_000_000)               # some 0.1 s of the default stream
    for _ in range(2):
        tqf.tq_encode_append_packed(ctx, cache, k, v, cu, stream=side)
    side.synchronize()
    assert not torch.cuda.default_stream().query()   # (the appends did not wait for it)
    torch.cuda.synchronize()
    assert cache.lengths.cpu().tolist() == [2 * (n - 3), cap]
    assert torch.equal(cache.v_data[0, 0, :n - 3], cache.v_data[0, 0, n - 3:2 * (n - 3)])
    assert tqf.tq_get_status(ctx) == tqf.TQ_STATUS_CAPACITY
    assert tqf.tq_get_status(ctx) == 0


def tree_args(B, Hq, N, dev):
    q = H.upload(wl.random_fp16(60 + N, (B, Hq, N, 128)), dev)
    return q, torch.empty_like(q), tqf.tq_tree_mask([i - 1 for i in range(N)]).to(dev).unsqueeze(0)


def taken(calls, cache, ctx):
    """Device memory that a context's calls allocate."""
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    for q, out, mask in calls:
        tqf.tq_tree_attention(ctx, cache, q, out, mask, 512)
    torch.cuda.synchronize()
    return before - torch.cuda.mem_get_info()[0]


def test_a_growing_context_holds_its_largest_workspace_alone(dev):
    """Calls of growing size, none captured: what the context holds in the end is what
    its largest call takes on a context of its own."""
    B, Hq, Hkv, cap = 8, 32, 8, 512
    rec = H.random_cache("turbo4", B, Hkv, cap, 64)
    cache = H.gpu_cache_from_records("turbo4", B, Hkv, cap, [cap] * B, *rec, dev)
    calls = [tree_args(B, Hq, N, dev) for N in (40, 96, 160, 256)]
    torch.cuda.empty_cache()
    taken(calls[-1:], cache, tqf.Context())      # (loads the kernels)
    grown, alone = tqf.Context(), tqf.Context()
    held = taken(calls, cache, grown)
    assert held > 50 << 20
    want = [c[1].clone() for c in calls]
    need = taken(calls[-1:], cache, alone)
    assert held <= need + (4 << 20)              # (the allocator's 2 MB steps)
    # the same with every call captured before the next grows: the graphs stay good
    graphs, ctx = [], tqf.Context()
    for q, out, mask in calls:
        tqf.tq_tree_attention(ctx, cache, q, out, mask, cap)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tqf.tq_tree_attention(ctx, cache, q, out, mask, cap)
        graphs.append(g)
    for (_, out, _), g, w in zip(calls, graphs, want):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert tqf.tq_get_status(ctx) == 0


def test_two_contexts_in_flight_on_two_streams(dev):
    """Calls of two contexts, each on a stream and a cache of its own, issued in turn
    without a wait between them: what each gives is what it gives alone."""
    B, Hq, Hkv, cap, N = 3, 32, 8, 2560, 40
    steps = 6

    def state(seed):
        rec = H.random_cache("turbo4", B, Hkv, cap, seed)
        cache = H.gpu_cache_from_records("turbo4", B, Hkv, cap, [2000, 700, 64], *rec, dev)
        k, v = (H.upload(wl.random_fp16(seed + i, (3 * N, Hkv, 128)), dev) for i in (1, 2))
        q = H.upload(wl.random_fp16(seed + 3, (B, Hq, N, 128)), dev)
        qp = H.upload(wl.random_fp16(seed + 4, (3 * N, Hq, 128)), dev)
        return dict(cache=cache, ctx=tqf.Context(), k=k, v=v, q=q, qp=qp,
                    cu=i32([0, N, 2 * N, 3 * N], dev), start=i32([2000, 700, 64], dev),
                    keep=i32([[0, 5, 7, 20]] * 3, dev), count=i32([4, 2, 0], dev),
                    mask=tqf.tq_tree_mask([i - 1 for i in range(N)]).to(dev).unsqueeze(0))

    def step(s, stream, outs):
        """One round of a speculative step: append, tree, prefill, keep, cut back."""
        with torch.cuda.stream(stream):
            s["cache"].lengths.copy_(s["start"])
            tqf.tq_encode_append_packed(s["ctx"], s["cache"], s["k"], s["v"], s["cu"])
            a, b = torch.empty_like(s["q"]), torch.empty_like(s["qp"])
            tqf.tq_tree_attention(s["ctx"], s["cache"], s["q"], a, s["mask"], cap)
            tqf.tq_prefill_attention_packed(s["ctx"], s["cache"], s["qp"], b, s["cu"], cap)
            tqf.tq_cache_compact(s["ctx"], s["cache"], s["start"], s["keep"], s["count"], N)
            d = torch.empty_like(s["q"][:, :, :1].contiguous())
            tqf.tq_decode_attention(s["ctx"], s["cache"], s["q"][:, :, :1].contiguous(), d, cap)
            outs.append((a, b, d, s["cache"].lengths.clone()))

    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    want = []
    for seed in (70, 80):
        outs = []
        s = state(seed)
        torch.cuda.synchronize()
        step(s, one, outs)
        torch.cuda.synchronize()
        want.append(outs[0])
        assert tqf.tq_get_status(s["ctx"]) == 0
    x, y = state(70), state(80)
    torch.cuda.synchronize()
    got = [], []
    torch.cuda._sleep(20_000_000)   # (the first calls of both are queued when the GPU gets to them)
    one.wait_stream(torch.cuda.current_stream())
    two.wait_stream(torch.cuda.current_stream())
    for _ in range(steps):
        step(x, one, got[0])
        step(y, two, got[1])
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, w))
    assert tqf.tq_get_status(x["ctx"]) == 0 and tqf.tq_get_status(y["ctx"]) == 0
