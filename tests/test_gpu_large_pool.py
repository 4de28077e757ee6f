"""The norm-rotation-append, masked and shared-prefix calls on blocks whose byte offsets pass 32
bits, and two of them at once: the same bits as on a small pool, one call after the other."""
import numpy as np
import pytest
import torch

import paged_kv_cache_19_gb300 as kp
from attention_util import Cache, sharing
from gpu_util import i32

pytestmark = pytest.mark.gpu

# K half of the pool: past 2^32 bytes (and past 2^31 elements of an 8-bit cache)
SIZES = [(False, 16, 150_000), (True, 32, 40_000)]


@pytest.mark.parametrize("fp8,bs,blocks", SIZES)
def test_offsets_past_32_bits(fp8, bs, blocks):
    hk = 8 if not fp8 else 32
    groups = [(6, 5), (1, 0), (3, 9)]
    own = np.random.default_rng(1).integers(1, 90, 10)
    ctx = np.concatenate([[b * bs] * m for m, b in groups]) + own
    c = Cache(ctx=ctx, hq=2 * hk, hk=hk, d=128, bs=bs, fp8=fp8, shared=groups, seed=4)
    big = kp.kv_pool_create(blocks, bs, hk, 128, "fp8_e4m3" if fp8 else "bf16")
    block_bytes = bs * hk * 128 * (1 if fp8 else 2)
    assert (blocks - c.nb) * block_bytes > 2 ** 32
    if fp8:
        big.set_scales(c.ks, c.vs)
    # the small pool's blocks, alternately at the far end and at the near one
    to = np.where(np.arange(c.nb) % 2 == 0, blocks - 1 - np.arange(c.nb), np.arange(c.nb))
    at = torch.from_numpy(to).cuda()
    for src, dst in zip(c.pool.raw_bytes(), big.raw_bytes()):
        dst[at] = src
    tab = i32(np.where(c.tab >= 0, to[np.maximum(c.tab, 0)], -1))

    def both(f):
        x, y = f(c.pool, c.tables), f(big, tab)
        assert torch.equal(x, y)
        return x

    both(lambda p, t: kp.paged_attention_masked(p, c.q, t, c.lens, c.scale, softcap=20.0, window=70))
    shared = both(lambda p, t: kp.paged_shared_prefix_attention(p, c.q, t, c.lens, i32(c.offsets), i32(c.blocks), c.scale))
    c.check(shared, None, c.reference())
    g = torch.Generator("cuda").manual_seed(2)
    qkv = torch.randn((10, 4 * hk, 128), device="cuda", generator=g).bfloat16()
    q, k, v = qkv[:, :2 * hk], qkv[:, 2 * hk:3 * hk], qkv[:, 3 * hk:]
    rope = torch.randn((int(ctx.max()), 128), device="cuda", generator=g)
    w = torch.rand(128, device="cuda", generator=g)
    both(lambda p, t: kp.paged_norm_rope_append(p, q, k, v, t, c.lens, q_weight=w, k_weight=w, rope_table=rope))
    for src, dst in zip(c.pool.raw_bytes(), big.raw_bytes()):
        assert torch.equal(dst[at], src)
    assert c.pool.device_errors() == 0 and big.device_errors() == 0
    big.destroy()
    c.pool.destroy()


def test_two_calls_at_once_on_two_streams():
    groups = [(20, 30), (7, 12)]
    ctx = np.concatenate([[b * 16] * m for m, b in groups]) + np.arange(27) * 11 + 1
    c = Cache(ctx=ctx, hq=32, hk=8, d=128, bs=16, shared=groups, seed=8)
    off, blk = i32(c.offsets), i32(c.blocks)
    ws = [torch.zeros(kp.paged_attention_masked_workspace_size(c.pool, 27, 32, 1, c.max_blocks), dtype=torch.uint8, device="cuda"),
          torch.zeros(kp.paged_shared_prefix_workspace_size(c.pool, 27, 32, 1, c.max_blocks, 2), dtype=torch.uint8, device="cuda")]
    calls = [lambda out: kp.paged_attention_masked(c.pool, c.q, c.tables, c.lens, c.scale, workspace=ws[0], out=out),
             lambda out: kp.paged_shared_prefix_attention(c.pool, c.q, c.tables, c.lens, off, blk, c.scale, workspace=ws[1],
                                                          out=out)]
    want = [torch.empty_like(c.q) for _ in calls]
    for f, o in zip(calls, want):
        f(o)
    c.check(want[0], None, c.reference())
    outs = [[torch.full_like(c.q, float("nan")) for _ in range(20)] for _ in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for i in range(20):
        for f, o, s in zip(calls, outs, streams):
            with torch.cuda.stream(s):
                f(o[i])
    torch.cuda.synchronize()
    for os_, w in zip(outs, want):
        assert all(torch.equal(o, w) for o in os_)
    assert c.pool.device_errors() == 0
    c.pool.destroy()


@pytest.mark.parametrize("fp8,bs,blocks", SIZES)
def test_the_shared_pass_past_32_bits(fp8, bs, blocks):
    """Groups that are computed once, every second of their blocks at the far end of a large pool."""
    hk = 8 if not fp8 else 32
    groups = [(30, 9), (1, 0), (13, 12)]
    own = np.random.default_rng(3).integers(1, 90, 44)
    ctx = np.concatenate([[b * bs] * m for m, b in groups]) + own
    c = Cache(ctx=ctx, hq=2 * hk, hk=hk, d=128, bs=bs, fp8=fp8, shared=groups, seed=5)
    assert sharing(c.offsets, c.blocks, bs) == [0, 2]
    big = kp.kv_pool_create(blocks, bs, hk, 128, "fp8_e4m3" if fp8 else "bf16")
    if fp8:
        big.set_scales(c.ks, c.vs)
    to = np.where(np.arange(c.nb) % 2 == 0, blocks - 1 - np.arange(c.nb), np.arange(c.nb))
    far = to[c.tab[0, :9]] * (bs * hk * 128 * (1 if fp8 else 2))
    assert (far > 2 ** 32).any() and (far < 2 ** 32).any()
    at = torch.from_numpy(to).cuda()
    for src, dst in zip(c.pool.raw_bytes(), big.raw_bytes()):
        dst[at] = src
    tab = i32(np.where(c.tab >= 0, to[np.maximum(c.tab, 0)], -1))
    off, blk = i32(c.offsets), i32(c.blocks)
    small, large = (kp.paged_shared_prefix_attention(p, c.q, t, c.lens, off, blk, c.scale)
                    for p, t in ((c.pool, c.tables), (big, tab)))
    assert torch.equal(small, large)
    c.check(large, None, c.reference())
    assert c.pool.device_errors() == 0 and big.device_errors() == 0
    big.destroy()
    c.pool.destroy()
