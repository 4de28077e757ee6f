"""What a call allocates itself -- workspace and out -- is work of the stream it launches on."""
import contextlib
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import paged_kv_cache_19_gb300 as kp
from attention_util import Cache
from gpu_util import i32

B, HQ, HK, D, MB = 3, 4, 2, 64, 5


def calls():
    """Every call that allocates: name -> function of the keyword arguments, over host tensors."""
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)                      # noqa: E731
    q, q4, t, n = bf(B, HQ, D), bf(B, HQ, 2, D), torch.zeros(B, MB, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    k, pool = bf(B, HK, D), SimpleNamespace(handle=1, _h=SimpleNamespace(value=1), head_dim=D, kv_heads=HK, device=0)
    return {
        "paged_norm_rope_append": lambda **kw: kp.paged_norm_rope_append(pool, q, k, k, t, n, **kw),
        "paged_decode_attention": lambda **kw: kp.paged_decode_attention(pool, q, t, n, 1.0, **kw),
        "paged_decode_attention_split_merge": lambda **kw: kp.paged_decode_attention_split_merge(pool, q, t, n, 1.0, **kw),
        "paged_merge_attention_states": lambda **kw: kp.paged_merge_attention_states(bf(2, 3, D), torch.zeros(2, 3), **kw),
        "paged_attention_multi_query": lambda **kw: kp.paged_attention_multi_query(pool, q4, t, n, 1.0, **kw),
        "paged_attention_masked": lambda **kw: kp.paged_attention_masked(pool, q4, t, n, 1.0, **kw),
        "paged_shared_prefix_attention": lambda **kw: kp.paged_shared_prefix_attention(pool, q, t, n, n[:2], n[:1], 1.0, **kw),
        "paged_decode_step": lambda **kw: kp.paged_decode_step(pool, k, k, q, t, n, 1.0, **kw),
        "paged_mla_decode_attention": lambda **kw: kp.paged_mla_decode_attention(pool, q, t, n, 1.0, **kw),
        "paged_mla_decode_step": lambda **kw: kp.paged_mla_decode_step(pool, k[:, 0], q, t, n, 1.0, **kw),
    }


NO_WORKSPACE = ("paged_norm_rope_append", "paged_merge_attention_states")


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", list(calls()))
def test_allocations_are_made_on_the_launch_stream(monkeypatch, name, raw):
    """Host tensors and a library that launches nothing; torch's stream context is a fake."""
    active, made, kept, launched = [], [], [], []
    side, here = SimpleNamespace(cuda_stream=78), SimpleNamespace(cuda_stream=12)

    @contextlib.contextmanager
    def context(s):
        active.append(s.cuda_stream)
        yield
        active.pop()

    def noted(f):
        def g(*a, **kw):
            made.append(active[-1] if active else None)
            return f(*a, **kw)
        return g

    class Launches:
        def __getattr__(self, what):
            def f(*a):
                launched.append(a[-1])
                return 0
            return f

    f = calls()[name]
    monkeypatch.setattr(torch.cuda, "stream", context)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: SimpleNamespace(cuda_stream=h))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: here)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append(s.cuda_stream), raising=False)
    for make in ("zeros", "empty", "empty_like"):
        monkeypatch.setattr(torch, make, noted(getattr(torch, make)))
    for size in ("paged_decode_workspace_size", "paged_multi_query_workspace_size", "paged_attention_masked_workspace_size",
                 "paged_shared_prefix_workspace_size", "paged_mla_workspace_size"):
        monkeypatch.setattr(kp, size, lambda *a: 64)
    monkeypatch.setattr(kp, "_need", lambda t, *a: t)
    monkeypatch.setattr(kp, "load_library", Launches)
    monkeypatch.setattr(kp, "_binding", Launches())
    made.clear()
    f(stream=78 if raw else side)
    # (the merge's own inputs are made in the call above, before its allocation)
    own = [s for s in made if s is not None]
    assert launched == [78] and own == [78] * (1 if name in NO_WORKSPACE else 2)
    assert kept == [12]                              # out, for the caller's stream
    if name != "paged_merge_attention_states":
        assert len(made) == len(own)


def delayed(c, s, junk):
    """Leaves s with cached memory full of junk, and the current stream busy for some milliseconds."""
    with torch.cuda.stream(s):
        t = torch.full((junk,), 0x5A, dtype=torch.uint8, device="cuda")
        u = torch.full_like(c.q, float("nan"))
        del t, u
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_a_call_on_another_stream_than_the_current_one(handle):
    """The current stream is busy when the call is made, and the next allocations on it overwrite
    what a workspace given back to it would lose."""
    groups = [(40, 60), (9, 30)]
    ctx = np.concatenate([[b * 16] * m for m, b in groups]) + np.arange(49) * 9 + 1
    c = Cache(ctx=ctx, hq=16, hk=4, d=128, bs=16, shared=groups, seed=11)
    off, blk, want = i32(c.offsets), i32(c.blocks), c.reference()
    q = c.q[:, :, 0].contiguous()
    out_of = {
        "masked": lambda **kw: kp.paged_attention_masked(c.pool, c.q, c.tables, c.lens, c.scale, **kw),
        "shared": lambda **kw: kp.paged_shared_prefix_attention(c.pool, c.q, c.tables, c.lens, off, blk, c.scale, **kw),
        "multi": lambda **kw: kp.paged_attention_multi_query(c.pool, c.q, c.tables, c.lens, c.scale, kv_split_tokens=64, **kw),
        "decode": lambda **kw: kp.paged_decode_attention(c.pool, q, c.tables, c.lens, c.scale,
                                                         kv_split_tokens=64, **kw),
    }
    need = kp.paged_shared_prefix_workspace_size(c.pool, c.B, 16, 1, c.max_blocks, 2)
    s = torch.cuda.Stream()
    for name, f in out_of.items():
        for _ in range(5):
            delayed(c, s, need)
            out = f(stream=s.cuda_stream if handle else s)
            torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")
            torch.cuda.current_stream().wait_stream(s)
            c.check(out.view(c.q.shape), None, want)
    assert c.pool.device_errors() == 0
    c.pool.destroy()


class Handle:
    """Another library's stream: all it has to have is its handle."""

    def __init__(self, s):
        self.cuda_stream = s.cuda_stream


@pytest.mark.gpu
def test_other_ways_to_name_a_stream():
    c = Cache(ctx=[300, 70], hq=8, hk=2, d=64, bs=16)
    want, s = c.reference(), torch.cuda.Stream()
    for stream in (Handle(s), s.cuda_stream, torch.cuda.ExternalStream(s.cuda_stream), torch.cuda.current_stream(),
                   torch.cuda.default_stream(), 0, 1, None):
        torch.cuda.synchronize()
        for f in (kp.paged_attention_masked, kp.paged_attention_multi_query):
            out = f(c.pool, c.q, c.tables, c.lens, c.scale, stream=stream)
            torch.cuda.synchronize()
            c.check(out, None, want)
    c.pool.destroy()


@pytest.mark.gpu
def test_norm_rope_append_on_another_stream_than_the_current_one():
    pool = kp.kv_pool_create(8, 16, 2, 64)
    x = torch.randn(5, 8, 64, device="cuda").bfloat16()
    tab, seq, pos = i32(np.arange(8)[None]), i32(np.zeros(5)), i32(np.arange(5) * 20)
    args = (pool, x[:, :4], x[:, 4:6], x[:, 6:], tab)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(10_000_000)
        out = kp.paged_norm_rope_append(*args, token_seq=seq, token_pos=pos, stream=s)
        torch.full_like(x, float("nan"))
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(out, x[:, :4])
    pool.destroy()


@pytest.mark.gpu
def test_a_side_stream_inside_a_capture():
    """Workspace and out come from the graph's memory; the replays read the lengths of their time."""
    groups = [(30, 9), (4, 40)]
    ctx = np.concatenate([[b * 16] * m for m, b in groups]) + np.arange(34) * 5 + 40
    c = Cache(ctx=ctx, hq=8, hk=2, d=64, bs=16, shared=groups, seed=3)
    off, blk = i32(c.offsets), i32(c.blocks)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.wait_stream(torch.cuda.current_stream())
        masked = kp.paged_attention_masked(c.pool, c.q, c.tables, c.lens, c.scale, stream=s)
        shared = kp.paged_shared_prefix_attention(c.pool, c.q, c.tables, c.lens, off, blk, c.scale, stream=s.cuda_stream)
        multi = kp.paged_attention_multi_query(c.pool, c.q, c.tables, c.lens, c.scale, kv_split_tokens=64, stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for less in (0, 39, 17):
        c.ctx = ctx - less
        c.lens.copy_(i32(c.ctx))
        g.replay()
        torch.full((1 << 22,), 0x5A, dtype=torch.uint8, device="cuda")      # what the graph holds is not handed out
        for got in (masked, shared, multi):
            c.check(got, None, c.reference())
    assert c.pool.device_errors() == 0
    del masked, shared, multi
    g.reset()
    c.pool.destroy()
