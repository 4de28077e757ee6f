"""The bounded waits of the shared prefix pass, of the kernel behind it, and of the streaming form of
paged_norm_rope_append, run out on purpose (as test_gpu_timeout does for the decode kernels): the
loads stop at a stage -- in the shared pass as if their own wait had run out -- the waits for it give
up (after 20 ms, or with the pass's loads), KV_DEVERR_TIMEOUT is set, the kernels end, the pool is as
it was, and the next call is exact."""
import contextlib

import numpy as np
import pytest
import torch

import paged_kv_cache_19_gb300 as kp
from attention_util import Cache, sharing
from gpu_util import i32
from test_gpu_norm_rope_append import POISON, Call

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def stalled(stage):
    kp.kv_debug_decode_stall(stage, 20_000_000)
    try:
        yield
        torch.cuda.synchronize()
    finally:
        kp.kv_debug_decode_stall(-1, 0)


CASES = {
    # every CTA with two tiles stops, in the pass and behind it; rows in two tiles, and in one
    "both": dict(groups=[(40, 300)], own=60, hq=8, hk=2, stage=3),
    "both-alternating": dict(groups=[(24, 300)], own=60, hq=8, hk=2, stage=3),
    "first-load": dict(groups=[(24, 300)], own=60, hq=8, hk=2, stage=0),
    # ranges of at most two tiles (four stages) in the pass, of six sub-blocks behind it
    "suffix": dict(groups=[(2, 130)], own=900, hq=4, hk=2, stage=5),
    # ranges of ten tiles (20 stages) in the pass, short units behind it
    "pass": dict(groups=[(128, 320)], own=16, hq=64, hk=8, stage=19),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(CASES))
def test_shared_prefix_attention(name, fp8):
    case = CASES[name]
    groups = case["groups"]
    members, blocks = groups[0]
    ctx = blocks * 16 + np.random.default_rng(1).integers(max(1, case["own"] // 2), case["own"] + 1, members)
    c = Cache(ctx=ctx, hq=case["hq"], hk=case["hk"], d=128, bs=16, shared=groups, fp8=fp8, seed=2)
    assert sharing(c.offsets, c.blocks, 16) == [0]
    off, blk = i32(c.offsets), i32(c.blocks)
    ws = torch.zeros(kp.paged_shared_prefix_workspace_size(c.pool, c.B, c.hq, 1, c.max_blocks, 1), dtype=torch.uint8,
                     device="cuda")
    before = [t.clone() for t in c.pool.raw_bytes()]
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device="cuda")

    def call():
        kp.paged_shared_prefix_attention(c.pool, c.q, c.tables, c.lens, off, blk, c.scale, workspace=ws, out=out, lse=lse)

    with stalled(case["stage"]):
        call()
    assert c.pool.device_errors() & kp.DEVERR_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(before, c.pool.raw_bytes()))
    ws.zero_()
    call()
    c.check(out, lse, c.reference())
    assert c.pool.device_errors() == 0
    c.pool.destroy()


@pytest.mark.parametrize("kw", [dict(hq=4, hk=2, d=128, bs=16, rope_dim=128), dict(hq=4, hk=4, d=128, bs=32, fp8=True)], ids=str)
def test_norm_rope_append_of_a_prompt(kw):
    """Tokens before the stage are written, the others are not."""
    n, stage = 2500, 2
    c = Call(batch=1, seq=np.zeros(n, int), pos=np.arange(n), **kw)
    ctas = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    assert n >= 3 * ctas                              # the streaming form
    lo = np.arange(ctas) * n // ctas
    done = np.zeros(n, bool)
    for s in range(stage):
        done[np.minimum(lo + s, n - 1)] = True
    out = torch.full((n, c.hq, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    with stalled(stage):
        c.run(out=out)
    assert c.pool.device_errors() == kp.DEVERR_TIMEOUT
    assert (out[torch.from_numpy(~done).cuda()] == 7.0).all()
    raw = c.pool.raw_bytes()[0].cpu()
    blk, slot = c.tab[0, np.arange(n) // c.bs], np.arange(n) % c.bs
    assert (raw[blk[~done], slot[~done]] == POISON).all() and not (raw[blk[done], slot[done]] == POISON).all(-1).all(-1).any()
    c.run(out=out)
    assert c.pool.device_errors() == 0
    c.check(out)
