"""paged_shared_prefix_attention against attention in 64 bits, and beside the attention that
shares nothing; one decode step of a forked batch with everything it needs."""
import numpy as np
import pytest
import torch

import paged_kv_cache_19_gb300 as kp
from attention_util import POISON, Cache, sharing
from gpu_util import i32

pytestmark = pytest.mark.gpu


def run(c, split=0, offsets=None, blocks=None, **kw):
    out = torch.full_like(c.q, float("nan"))
    lse = torch.full(c.q.shape[:3], float("nan"), device="cuda")
    kp.paged_shared_prefix_attention(c.pool, c.q, c.tables, c.lens,
                                     i32(c.offsets if offsets is None else offsets),
                                     i32(c.blocks if blocks is None else blocks), c.scale,
                                     kv_split_tokens=split, out=out, lse=lse, **kw)
    return out, lse


def batch(groups, bs, own, q_len=1, seed=0):
    """Context lengths: the group's blocks plus 1 .. own tokens and the new ones' room."""
    r = np.random.default_rng(seed)
    n = np.concatenate([[b * bs] * m for m, b in groups])
    return n + r.integers(q_len, own + q_len, len(n))


CASES = [
    # (groups as (members, blocks), block size, own tokens, heads, kv heads, head_dim, q_len, fp8)
    ([(2, 1)], 16, 5, 4, 4, 64, 1, False),
    ([(4, 32)], 16, 50, 32, 8, 128, 1, False),
    ([(3, 7), (1, 9), (2, 0), (5, 33)], 16, 100, 8, 2, 128, 1, False),
    ([(2, 3), (70, 20)], 32, 40, 8, 2, 128, 1, False),
    ([(33, 9)], 32, 90, 8, 1, 64, 1, False),
    ([(40, 17)], 16, 70, 7, 1, 128, 1, False),
    ([(9, 24), (20, 13)], 16, 60, 12, 4, 64, 3, False),
    ([(3, 50)], 32, 33, 16, 2, 128, 17, False),
    ([(2, 300)], 16, 500, 8, 8, 128, 1, False),
    ([(5, 16)], 32, 70, 8, 8, 128, 1, True),
    ([(3, 7), (90, 20)], 16, 40, 8, 2, 128, 1, True),
    ([(130, 33), (2, 4)], 32, 20, 4, 2, 128, 2, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: str(c).replace(" ", ""))
def test_matches_the_formula(case):
    groups, bs, own, hq, hk, d, q_len, fp8 = case
    c = Cache(ctx=batch(groups, bs, own, q_len), hq=hq, hk=hk, d=d, bs=bs, fp8=fp8, q_len=q_len, shared=groups)
    want = c.reference()
    for split in (0, bs):
        c.check(*run(c, split), want)
    assert c.pool.device_errors() == 0
    # and the attention that shares nothing agrees
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device="cuda")
    kp.paged_attention_multi_query(c.pool, c.q, c.tables, c.lens, c.scale, out=out, lse=lse)
    c.check(out, lse, want)
    c.pool.destroy()


def test_long_prefix_over_every_sm():
    """One run per kv head, cut into as many pieces as there are SMs."""
    c = Cache(ctx=np.array([20000 + 3, 20000 + 800]), hq=4, hk=1, d=128, bs=16, shared=[(2, 1250)], seed=3)
    c.check(*run(c), c.reference())
    c.pool.destroy()


@pytest.mark.parametrize("fp8", [False, True])
def test_few_members_behind_long_prefixes(fp8):
    """Runs cut into fewer pieces than there are SMs, beside short ones."""
    groups = [(2, 390), (3, 30), (2, 1)]
    c = Cache(ctx=batch(groups, 32, 50), hq=4, hk=1, d=128, bs=32, fp8=fp8, shared=groups, seed=6)
    c.check(*run(c), c.reference())
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_contexts_that_end_inside_the_shared_blocks():
    """Rows that see part of the prefix, or nothing: empty places of a padded batch."""
    ctx = np.array([80, 16 * 20, 0, 1, 16 * 20 + 9, 17, 129, 128])
    c = Cache(ctx=ctx, hq=8, hk=2, d=128, bs=16, shared=[(8, 20)])
    out, lse = run(c)
    c.check(out, lse, c.reference())
    assert not out[2].any() and (lse[2] == -float("inf")).all()
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_several_new_tokens_reaching_back_into_the_shared_blocks():
    c = Cache(ctx=np.array([16 * 9 + 2, 16 * 9, 5, 16 * 9 + 40]), hq=4, hk=2, d=64, bs=16, q_len=5, shared=[(4, 9)])
    c.check(*run(c), c.reference())
    c.pool.destroy()


def test_growing_scores_rescale_the_output():
    """Scores far apart, with the largest in late tiles."""
    groups = [(40, 64)]
    c = Cache(ctx=batch(groups, 16, 9), hq=8, hk=2, d=128, bs=16, shared=groups, q_scale=6.0, seed=8)
    k, _, _, _ = c.pool.tensors()
    for t in range(0, 1024, 61):
        at = c.tab[0, t // 16], t % 16
        k[at] *= 1.0 + t / 300
    c.k = k.float().cpu().double().numpy()
    out, size, lse, top = c.reference()
    # the fp32 scores' error grows with the sums: 128 2^-24 sum|q k| scale, here up to 2^-6 of them
    c.check(*run(c), (out, size, lse, top * 4))
    c.pool.destroy()


@pytest.mark.parametrize("scale", [0.0, -0.05])
def test_scales_that_are_not_positive(scale):
    groups = [(10, 12)]
    c = Cache(ctx=batch(groups, 16, 30), hq=8, hk=2, d=64, bs=16, shared=groups)
    c.scale = scale
    c.check(*run(c), c.reference())
    c.pool.destroy()


def test_extreme_queries_on_an_8_bit_cache():
    """Rows of zeros, rows far above and far below the range of f16."""
    groups = [(6, 12)]
    c = Cache(ctx=batch(groups, 16, 30), hq=8, hk=2, d=128, bs=16, shared=groups, fp8=True)
    f = torch.tensor([0.0, 2.0 ** -40, 2.0 ** 20, 1.0, 2.0 ** -14, 2.0 ** -130], device="cuda")[:, None, None, None]
    c.scale *= 2.0 ** -20
    c.q = (c.q.float() * f).to(torch.bfloat16)
    c.q64 = c.q.double().cpu().numpy()
    c.check(*run(c), c.reference())
    c.pool.destroy()


def test_poison_behind_the_contexts_and_bad_blocks():
    """Blocks of nobody hold NaN; an invalid id in the shared part is skipped for all members."""
    groups = [(7, 10), (3, 6)]
    for fp8 in (False, True):
        c = Cache(ctx=batch(groups, 16, 50), hq=8, hk=2, d=128, bs=16, shared=groups, fp8=fp8)
        tab = c.tab.copy()
        tab[:7, 4] = -1
        tab[7:, 5] = 10 ** 6
        c.tables = i32(tab)
        got = run(c)
        assert c.pool.device_errors() == kp.DEVERR_BLOCK_ID
        want = c.reference(lambda b, pos, t: (t > pos) | (t // 16 == (4 if b < 7 else 5)))
        c.check(*got, want)
        c.pool.destroy()


@pytest.mark.parametrize("fp8", [False, True])
def test_poison_and_bad_blocks_in_groups_that_save_much(fp8):
    groups = [(21, 10), (30, 8)]
    c = Cache(ctx=batch(groups, 16, 50), hq=8, hk=2, d=128, bs=16, shared=groups, fp8=fp8)
    tab = c.tab.copy()
    tab[:21, 4] = -1
    tab[21:, 5] = 10 ** 6
    c.tables = i32(tab)
    got = run(c)
    assert c.pool.device_errors() == kp.DEVERR_BLOCK_ID
    c.check(*got, c.reference(lambda b, pos, t: (t > pos) | (t // 16 == (4 if b < 21 else 5))))
    c.pool.destroy()


def test_extreme_queries_in_a_group_that_saves_much():
    groups = [(24, 12)]
    c = Cache(ctx=batch(groups, 16, 30), hq=8, hk=2, d=128, bs=16, shared=groups, fp8=True)
    f = torch.tensor([0.0, 2.0 ** -40, 2.0 ** 20, 1.0, 2.0 ** -14, 2.0 ** -130] * 4, device="cuda")[:, None, None, None]
    c.scale *= 2.0 ** -20
    c.q = (c.q.float() * f).to(torch.bfloat16)
    c.q64 = c.q.double().cpu().numpy()
    c.check(*run(c), c.reference())
    c.pool.destroy()


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
@pytest.mark.parametrize("fp8", [False, True])
def test_scales_in_a_group_that_saves_much(scale, fp8):
    groups = [(16, 12)]
    c = Cache(ctx=batch(groups, 16, 30), hq=8, hk=2, d=128, bs=16, shared=groups, fp8=fp8)
    c.scale = scale
    c.check(*run(c), c.reference())
    c.pool.destroy()


def test_several_new_tokens_in_groups_that_save_much():
    """Contexts that end inside the shared blocks, at their end and behind it, some of length 0."""
    ctx = np.concatenate([np.full(20, 16 * 9) + np.arange(20) - 6, [5, 0, 16 * 9], np.full(18, 16 * 9 + 40)])
    c = Cache(ctx=ctx, hq=4, hk=2, d=64, bs=16, q_len=5, shared=[(41, 9)])
    c.check(*run(c), c.reference())
    c.pool.destroy()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("members", [2, 3, 5, 6, 9])
def test_groups_on_both_sides_of_the_sharing_rule(members, fp8):
    """The same bits' meaning whether a group is computed once or not: groups that save 1,536 to
    2,560 tokens next to each other."""
    groups = [(members, b) for b in (1536 // 32 // (members - 1), 2048 // 32 // (members - 1), 2048 // 32 // (members - 1) + 1,
                                     2560 // 32 // (members - 1))]
    c = Cache(ctx=batch(groups, 32, 40), hq=4, hk=2, d=128, bs=32, fp8=fp8, shared=groups, seed=members)
    c.check(*run(c), c.reference())
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_bad_groups_share_nothing_and_are_right():
    groups = [(7, 10), (3, 6)]
    c = Cache(ctx=batch(groups, 16, 50), hq=8, hk=2, d=128, bs=16, shared=groups)
    want = c.reference()
    for off, blk in (([0, 8, 7, 10], [10, 1, 6]), ([-1, 7, 10], [10, 6]), ([0, 7, 11], [10, 6]),
                     ([0, 7, 10], [10, -1]), ([0, 7, 10], [10, 1000])):
        c.check(*run(c, offsets=off, blocks=blk), want)
        assert c.pool.device_errors() == kp.DEVERR_GROUP
    # groups that cover part of the batch, empty ones among them, or none
    for off, blk in (([2, 2, 6, 6], [10, 9, 10]), ([7, 10], [6]), ([0], []), ([1, 4, 4, 7, 9], [9, 3, 10, 6]),
                     ([3, 3], [2]), ([10, 10], [1])):
        c.check(*run(c, offsets=off, blocks=np.array(blk, int)), want)
        assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_more_groups_than_threads():
    groups = [(1 + (i % 3), i % 4) for i in range(700)]
    c = Cache(ctx=batch(groups, 16, 20), hq=2, hk=1, d=64, bs=16, shared=groups)
    c.check(*run(c), c.reference())
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_more_sequences_than_threads_around_the_groups():
    """Sequences before, between and behind groups, over several rounds of the partition."""
    groups = [(1, 0)] * 200 + [(3, 5), (1, 2), (170, 2), (2, 9)] + [(1, 1)] * 150
    c = Cache(ctx=batch(groups, 16, 30), hq=4, hk=4, d=64, bs=16, shared=groups)
    want = c.reference()
    c.check(*run(c), want)
    o = np.array(c.offsets)
    # only the groups in the middle are named
    c.check(*run(c, offsets=o[200:205], blocks=c.blocks[200:204]), want)
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_repeated_calls_give_the_same_bits():
    """The pieces and their merge order are fixed (chunks of the own part too)."""
    groups = [(40, 40), (9, 3)]
    c = Cache(ctx=batch(groups, 16, 700), hq=16, hk=4, d=128, bs=16, shared=groups)
    ws = torch.zeros(kp.paged_shared_prefix_workspace_size(c.pool, c.B, 16, 1, c.max_blocks, 2, 64),
                     dtype=torch.uint8, device="cuda")
    first = run(c, 64, workspace=ws)
    for _ in range(20):
        again = run(c, 64, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    c.check(*first, c.reference())
    c.pool.destroy()


def test_another_stream_and_a_replayed_graph_with_other_groups():
    groups = [(6, 30), (5, 12)]
    c = Cache(ctx=batch(groups, 16, 100), hq=8, hk=2, d=128, bs=16, shared=groups)
    want = c.reference()
    ws = torch.zeros(kp.paged_shared_prefix_workspace_size(c.pool, c.B, 8, 1, c.max_blocks, 2), dtype=torch.uint8,
                     device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(c, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    c.check(*got, want)
    out = torch.empty_like(c.q)
    off, blk = i32(c.offsets), i32(c.blocks)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kp.paged_shared_prefix_attention(c.pool, c.q, c.tables, c.lens, off, blk, c.scale, workspace=ws, out=out)
    for o, b in (([0, 6, 11], [30, 12]), ([0, 6, 11], [20, 0]), ([6, 8, 11], [3, 12]), ([3, 3, 6], [1, 29])):
        off.copy_(i32(o))
        blk.copy_(i32(b))
        g.replay()
        c.check(out, None, want)
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_one_workspace_for_masked_and_shared_calls_of_any_size():
    groups = [[(2, 40)], [(30, 9), (3, 25)], [(64, 4)], [(2, 2)]]
    cs = [Cache(ctx=batch(g, 16, 300), hq=8 * hk, hk=hk, d=128, bs=16, shared=g, seed=hk) for g, hk in zip(groups, (1, 4, 8, 2))]
    need = 0
    for c in cs:
        for split in (0, 16):
            need = max(need, kp.paged_attention_masked_workspace_size(c.pool, c.B, c.hq, 1, c.max_blocks, 0, split),
                       kp.paged_shared_prefix_workspace_size(c.pool, c.B, c.hq, 1, c.max_blocks, len(c.blocks), split))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    wants = [c.reference() for c in cs]
    for split in (16, 0):
        for c, want in zip(cs, wants):
            c.check(*run(c, split, workspace=ws), want)
            out = torch.full_like(c.q, float("nan"))
            kp.paged_attention_masked(c.pool, c.q, c.tables, c.lens, c.scale, kv_split_tokens=split, workspace=ws, out=out)
            c.check(out, None, want)
    for c in cs:
        assert c.pool.device_errors() == 0
        c.pool.destroy()


def test_refusals():
    c = Cache(ctx=[40, 50], hq=4, hk=2, d=64, bs=16, shared=[(2, 1)])
    off, blk = i32(c.offsets), i32(c.blocks)
    lib = kp.load_library()
    out = torch.zeros_like(c.q)
    need = kp.paged_shared_prefix_workspace_size(c.pool, 2, 4, 1, c.max_blocks, 1)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def call(**kw):
        a = dict(q=c.q.data_ptr(), hq=4, q_len=1, tab=c.tables.data_ptr(), mb=c.max_blocks, ctx=c.lens.data_ptr(), B=2,
                 off=off.data_ptr(), blk=blk.data_ptr(), n=1, scale=0.1, split=0, ws=ws.data_ptr(), bytes=need,
                 out=out.data_ptr())
        a.update(kw)
        return lib.paged_shared_prefix_attention(c.pool.handle, *a.values(), None, None)

    for kw in (dict(q=None), dict(out=None), dict(tab=None), dict(ctx=None), dict(off=None), dict(blk=None), dict(n=-1),
               dict(hq=3), dict(q_len=0), dict(mb=0), dict(B=-1), dict(scale=float("inf")), dict(split=5), dict(ws=None),
               dict(bytes=need - 1), dict(off=off.data_ptr() + 2), dict(ws=ws.data_ptr() + 8)):
        assert call(**kw) == kp.KV_ERR_INVALID_ARG, kw
    assert call(q_len=5000) == kp.KV_ERR_UNSUPPORTED
    assert call(B=0) == kp.KV_OK
    torch.cuda.synchronize()
    assert not out.any() and c.pool.device_errors() == 0
    with pytest.raises(ValueError):
        run(c, offsets=[0, 1, 2])
    with pytest.raises(kp.KVError):
        kp.paged_shared_prefix_workspace_size(c.pool, 2, 4, 1, c.max_blocks, -1)
    latent = kp.kv_mla_pool_create(2, 16)
    with pytest.raises(kp.KVError):
        kp.paged_shared_prefix_workspace_size(latent, 2, 4, 1, 4, 1)
    latent.destroy()
    c.pool.destroy()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_step_of_a_forked_batch(fp8):
    """Prompt and forks through the block manager; every step norms, rotates and appends the new
    tokens and attends over the shared prompt; the same step without sharing, and with a window,
    agrees with 64-bit attention over the cache as stored."""
    hq, hk, d, bs, n = 8, 2, 128, 16, 5
    bm = kp.BlockManager(64, bs)
    pool = kp.kv_pool_create(64, bs, hk, d, "fp8_e4m3" if fp8 else "bf16")
    if fp8:
        pool.set_scales([0.01, 0.02], [0.015, 0.01])
    for t in pool.raw_bytes():
        t.fill_(POISON)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    w = [torch.rand(d, generator=gen, device="cuda") + 0.5 for _ in range(2)]
    a = np.arange(200)[:, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
    rope = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()
    prompt = 100
    bm.add_sequence(0)
    assert bm.append_slots(0, prompt) is None
    tab, _ = bm.build_tables([0], 12)
    x = rand(prompt, hq + 2 * hk, d)
    kp.paged_norm_rope_append(pool, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], tab.cuda(), q_weight=w[0], k_weight=w[1],
                              rope_table=rope, token_seq=i32(np.zeros(prompt)), token_pos=i32(np.arange(prompt)))
    for child in range(1, n):
        bm.fork(0, child)
    seqs = list(range(n))
    for step in range(3):
        copies = [cp for s in seqs if (cp := bm.append_slots(s, 1)) is not None]
        if copies:
            kp.kv_copy_blocks(pool, i32(copies))
        order, off, blk = bm.prefix_groups(seqs)
        assert order.tolist() == seqs and off.tolist() == [0, n] and blk.tolist() == [prompt // bs]
        tab, ctx = bm.build_tables(seqs, 12)
        tab, ctx = tab.cuda(), ctx.cuda()
        x = rand(n, hq + 2 * hk, d)
        q = kp.paged_norm_rope_append(pool, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], tab, ctx, q_weight=w[0],
                                      k_weight=w[1], rope_table=rope)
        out, lse = torch.empty_like(q), torch.empty(n, hq, device="cuda")
        kp.paged_shared_prefix_attention(pool, q, tab, ctx, off.cuda(), blk.cuda(), d ** -0.5, out=out, lse=lse)
        win = kp.paged_attention_masked(pool, q, tab, ctx, d ** -0.5, window=30, softcap=20.0)
        # the oracle over the cache's own bytes
        c = object.__new__(Cache)
        c.B, c.hq, c.hk, c.d, c.bs, c.q_len, c.scale, c.pool = n, hq, hk, d, bs, 1, d ** -0.5, pool
        c.ctx, c.tab, c.q64 = ctx.cpu().numpy(), tab.cpu().numpy(), q.double().cpu().numpy()[:, :, None]
        k, v, ks, vs = (t.float().cpu().double().numpy() for t in pool.tensors())
        c.k, c.v = k * ks[:, None], v * vs[:, None]
        c.check(out, lse, c.reference())
        c.check(win, None, c.reference(lambda b, pos, t: (t > pos) | (t <= pos - 30), softcap=20.0))
    assert pool.device_errors() == 0
    pool.destroy()
    bm.close()


@pytest.mark.parametrize("scale", [2.0 ** -129, 1.5 * 2.0 ** -132, 2.0 ** -100, 1.0, 2.0 ** 100, 1.25 * 2.0 ** 116])
def test_the_ends_of_the_values_scale(scale):
    """Every scale that kv_pool_set_scales takes, where the outputs are numbers of bf16: values of one
    sign, codes 64 .. 448, so that an output is at least 64 scales and sum p|v| is the output itself.

    Beside check's bound (twice 2^-8 of the output, probabilities and output rounded, and the scores'
    2^-12), an output below 2^-126 is rounded by up to 2^-134, half a step of bf16's last numbers."""
    groups = [(40, 12), (30, 20), (3, 0)]
    c = Cache(ctx=batch(groups, 16, 300), hq=8, hk=2, d=128, bs=16, shared=groups, fp8=True, seed=13)
    scale = float(np.float32(scale))
    v = c.pool.tensors()[1]
    codes = torch.from_numpy(np.random.default_rng(2).uniform(64, 448, v.shape).astype(np.float32)).to(v.dtype)
    seen = ~torch.isnan(v.float())
    v.copy_(torch.where(seen, codes.cuda().float(), float("nan")).to(v.dtype))
    c.v = v.float().cpu().double().numpy()
    c.pool.set_scales(c.ks, [scale] * 2)
    want, _, want_lse, top = c.reference()          # in units of the scale
    masked = torch.full_like(c.q, float("nan"))
    kp.paged_attention_masked(c.pool, c.q, c.tables, c.lens, c.scale, out=masked)
    shared, lse = run(c)
    assert c.pool.device_errors() == 0 and (np.abs(lse.double().cpu().numpy() - want_lse) <= 2.0 ** -12 + 2.0 ** -19 * top).all()
    want = want * scale                             # (64 bits: far from the ends of their range)
    assert np.isfinite(want).all() and (np.abs(want) >= 2.0 ** -127).all() and want.max() < 2.0 ** 127
    bound = (2.0 ** -7 + 2.0 ** -12 + 2.0 ** -19 * top[..., None]) * want + 2.0 ** -134
    for got in (masked, shared):
        assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
    c.pool.destroy()


@pytest.mark.parametrize("fp8", [False, True])
def test_groups_that_share_behind_many_that_do_not(fp8):
    """The shared pass looks 320 or 448 groups over at a time: ones that share in the first round, in
    later ones, and at the very end."""
    groups = ([(1, 1)] * 10 + [(17, 8)] + [(1, 1)] * 400 + [(20, 9)] + [(1, 0)] * 500 + [(30, 5), (2, 3)] + [(1, 2)] * 60
              + [(140, 1)])
    c = Cache(ctx=batch(groups, 16, 20), hq=2, hk=1, d=128 if fp8 else 64, bs=16, fp8=fp8, shared=groups, seed=7)
    assert sharing(c.offsets, c.blocks, 16) == [10, 411, 912, 974]
    want = c.reference()
    c.check(*run(c), want)
    # only the groups from the second round on are named
    c.check(*run(c, offsets=c.offsets[330:], blocks=c.blocks[330:]), want)
    assert c.pool.device_errors() == 0
    c.pool.destroy()


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_groups_beside_ones_that_share(fp8):
    """A block count that breaks the rule: its group shares nothing, the others do.  Offsets that do:
    nothing is shared.  Empty groups and sequences of no group between ones that share."""
    groups = [(30, 10), (20, 16), (25, 12)]
    c = Cache(ctx=batch(groups, 16, 50), hq=8, hk=2, d=128, bs=16, shared=groups, fp8=fp8)
    want = c.reference()
    o, far = [0, 30, 50, 75], c.max_blocks + 1
    for off, blk in ((o, [-1, 16, 12]), (o, [10, far, 12]), (o, [10, 16, -(2 ** 31)]), (o, [2 ** 31 - 1, -1, 12]),
                     ([0, 30, 29, 75], [10, 16, 12]), ([-1, 30, 50, 75], [10, 16, 12]), ([0, 30, 50, 76], [10, 16, 12]),
                     ([0, 2 ** 31 - 1, 50, 75], [10, 16, 12])):
        c.check(*run(c, offsets=off, blocks=np.array(blk)), want)
        assert c.pool.device_errors() == kp.DEVERR_GROUP
    for off, blk in (([0, 30, 30, 30, 50, 75, 75], [10, 16, 9, 16, 12, 4]), ([2, 29, 30, 30, 49], [10, 3, 16, 15]),
                     ([31, 50], [16]), ([50, 50, 75], [9, 12])):
        assert sharing(off, blk, 16)
        c.check(*run(c, offsets=off, blocks=np.array(blk)), want)
        assert c.pool.device_errors() == 0
    c.pool.destroy()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_step_of_a_batch_forked_behind_a_long_prompt(fp8):
    """As test_a_decode_step_of_a_forked_batch, with a prompt long enough to be computed once: prompt,
    forks and groups through the block manager, the new tokens appended, attention over the cache."""
    hq, hk, d, bs, n, prompt, mb = 8, 2, 128, 16, 6, 533, 40
    bm = kp.BlockManager(80, bs)
    pool = kp.kv_pool_create(80, bs, hk, d, "fp8_e4m3" if fp8 else "bf16")
    if fp8:
        pool.set_scales([0.01, 0.02], [0.015, 0.01])
    for t in pool.raw_bytes():
        t.fill_(POISON)
    gen = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    w = [torch.rand(d, generator=gen, device="cuda") + 0.5 for _ in range(2)]
    a = np.arange(600)[:, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
    rope = torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()
    bm.add_sequence(0)
    bm.append_slots(0, prompt)
    tab, _ = bm.build_tables([0], mb)
    x = rand(prompt, hq + 2 * hk, d)
    kp.paged_norm_rope_append(pool, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], tab.cuda(), q_weight=w[0], k_weight=w[1],
                              rope_table=rope, token_seq=i32(np.zeros(prompt)), token_pos=i32(np.arange(prompt)))
    for child in range(1, n):
        bm.fork(0, child)
    bm.add_sequence(n)                                # and one of its own
    bm.append_slots(n, 20)
    seqs = [n, *range(n)]
    tab, _ = bm.build_tables([n], mb)
    x = rand(20, hq + 2 * hk, d)
    kp.paged_norm_rope_append(pool, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], tab.cuda(), q_weight=w[0], k_weight=w[1],
                              rope_table=rope, token_seq=i32(np.zeros(20)), token_pos=i32(np.arange(20)))
    for step in range(3):
        copies = [cp for s in seqs if (cp := bm.append_slots(s, 1)) is not None]
        if copies:
            kp.kv_copy_blocks(pool, i32(copies))
        order, off, blk = bm.prefix_groups(seqs)
        assert sharing(off.numpy(), blk.tolist(), bs) == [1] and blk.tolist() == [0, prompt // bs]
        tab, ctx = bm.build_tables([seqs[i] for i in order.tolist()], mb)
        tab, ctx = tab.cuda(), ctx.cuda()
        x = rand(n + 1, hq + 2 * hk, d)
        q = kp.paged_norm_rope_append(pool, x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], tab, ctx, q_weight=w[0],
                                      k_weight=w[1], rope_table=rope)
        out, lse = torch.empty_like(q), torch.empty(n + 1, hq, device="cuda")
        kp.paged_shared_prefix_attention(pool, q, tab, ctx, off.cuda(), blk.cuda(), d ** -0.5, out=out, lse=lse)
        c = object.__new__(Cache)                     # the oracle over the cache's own bytes
        c.B, c.hq, c.hk, c.d, c.bs, c.q_len, c.scale, c.pool = n + 1, hq, hk, d, bs, 1, d ** -0.5, pool
        c.ctx, c.tab, c.q64 = ctx.cpu().numpy(), tab.cpu().numpy(), q.double().cpu().numpy()[:, :, None]
        k, v, ks, vs = (t.float().cpu().double().numpy() for t in pool.tensors())
        c.k, c.v = k * ks[:, None], v * vs[:, None]
        c.check(out, lse, c.reference())
    assert pool.device_errors() == 0
    pool.destroy()
    bm.close()
