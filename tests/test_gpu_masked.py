"""paged_attention_masked against attention in 64 bits: capped scores, distance bias, windows,
document starts and visible prefixes, over pools whose unseen blocks are poisoned or gone."""
import numpy as np
import pytest
import torch

import paged_kv_cache_19_gb300 as kp
from attention_util import Cache
from gpu_util import i32

pytestmark = pytest.mark.gpu


def hide(window=0, first=None, prefix=None):
    def f(b, pos, t):
        h = t > pos
        if prefix is not None:
            h &= t >= prefix[b]
        if window:
            h |= t <= pos - window
        if first is not None:
            h |= t < first[b]
        return h
    return f


def run(c, split=0, lse=True, **kw):
    out = torch.full_like(c.q, float("nan"))
    l = torch.full(c.q.shape[:3], float("nan"), device="cuda") if lse else None  # noqa: E741
    kp.paged_attention_masked(c.pool, c.q, c.tables, c.lens, c.scale, kv_split_tokens=split, out=out, lse=l, **kw)
    return out, l


def slopes_of(hq):
    return torch.tensor(2.0 ** (-8.0 * np.arange(1, hq + 1) / hq), dtype=torch.float32)


SHAPES = [
    dict(hq=4, hk=4, d=64, bs=16, ctx=[1, 17, 64, 129]),
    dict(hq=32, hk=8, d=128, bs=16, ctx=[300, 5, 1024, 16]),
    dict(hq=8, hk=1, d=128, bs=32, ctx=[33, 2000]),
    dict(hq=6, hk=2, d=64, bs=32, ctx=[1, 31, 32, 500], q_len=1),
    dict(hq=16, hk=2, d=128, bs=16, ctx=[7, 40, 700], q_len=7),
    dict(hq=4, hk=2, d=64, bs=16, ctx=[40, 333], q_len=33),
    dict(hq=8, hk=4, d=128, bs=32, ctx=[3, 65, 900], q_len=3, fp8=True),
    dict(hq=32, hk=32, d=128, bs=16, ctx=[100, 1], fp8=True),
    dict(hq=4, hk=1, d=128, bs=16, ctx=[9, 1000], q_len=5, fp8=True),
]
RULES = ["none", "cap", "alibi", "window1", "window", "first", "prefix", "all"]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(f"{k}{v}" for k, v in s.items()).replace(" ", ""))
def test_matches_the_formula(shape, rule):
    c = Cache(seed=len(shape) + len(rule), **shape)
    r = np.random.default_rng(5)
    kw, ref, first, prefix, window = {}, {}, None, None, 0
    if rule in ("cap", "all"):
        kw["softcap"] = ref["softcap"] = 2.0 if rule == "cap" else 30.0
    if rule in ("alibi", "all"):
        s = slopes_of(c.hq)
        kw["alibi_slopes"], ref["slopes"] = s.cuda(), s.numpy()
    if rule.startswith("window") or rule == "all":
        kw["window"] = window = 1 if rule == "window1" else 37
    if rule in ("first", "all"):
        first = r.integers(0, c.ctx + 1)            # may leave rows without a key
        kw["first_keys"] = i32(first)
    if rule in ("prefix", "all"):
        prefix = r.integers(0, c.ctx + 20)          # may reach past the context
        kw["prefix_lens"] = i32(prefix)
    want = c.reference(hide(window, first, prefix), **ref)
    for split in (0, c.bs, 5 * c.bs):
        c.check(*run(c, split, **kw), want)
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_no_rule_is_the_plain_attention():
    """No mask at all and a mask that hides nothing: paged_attention_multi_query up to rounding."""
    for q_len in (1, 4):
        c = Cache(ctx=[50, 900, 4], hq=8, hk=2, d=128, bs=16, q_len=q_len)
        want = c.reference()
        c.check(*run(c), want)
        c.check(*run(c, window=10 ** 9, softcap=0.0, first_keys=i32([0, -3, 0]), prefix_lens=i32([0, 0, -1])), want)
        out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device="cuda")
        kp.paged_attention_multi_query(c.pool, c.q, c.tables, c.lens, c.scale, out=out, lse=lse)
        c.check(out, lse, want)
        c.pool.destroy()


@pytest.mark.parametrize("kw", [dict(hk=2, d=128, bs=16), dict(hk=4, d=64, bs=16), dict(hk=8, d=128, bs=16, fp8=True),
                                dict(hk=1, d=128, bs=32, fp8=True), dict(hk=2, d=64, bs=32)], ids=str)
@pytest.mark.parametrize("ctx", [[500, 90, 4], [505, 88, 61], [511, 57, 73]])
def test_freed_blocks_before_a_window_are_not_looked_at(kw, ctx):
    c = Cache(ctx=ctx, hq=8, q_len=2, **kw)
    bs = kw["bs"]
    want = c.reference(hide(40))
    tab = c.tab.copy()
    raw = c.pool.raw_bytes()
    for b in range(3):
        lo = max(0, c.ctx[b] - 2 - 40 + 1) // bs
        for j in range(lo):
            for t in raw:
                t[tab[b, j]] = 0xFF
            tab[b, j] = [-1, 10 ** 6][j % 2]
    c.tables = i32(tab)
    c.check(*run(c, window=40), want)
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_nan_and_infinite_keys_and_values_behind_the_masks():
    """Slots of a visible block that no row sees may hold anything."""
    c = Cache(ctx=[61, 30], hq=4, hk=2, d=64, bs=32, q_len=1)
    first = np.array([37, 29])
    want = c.reference(hide(0, first))
    k, v, _, _ = c.pool.tensors()
    for b in range(2):
        for t in range(first[b]):
            at = c.tab[b, t // 32], t % 32
            k[at] = [float("nan"), float("inf"), -float("inf")][t % 3]
            v[at] = [float("inf"), float("nan"), -float("inf")][t % 3]
    c.check(*run(c, first_keys=i32(first)), want)
    c.pool.destroy()


def test_large_and_small_caps_keep_small_scores():
    """tanh near zero and saturated: a cap far above the scores changes nothing, one far below
    them flattens all keys."""
    c = Cache(ctx=[200], hq=4, hk=2, d=64, bs=16)
    plain = c.reference()
    c.check(*run(c, softcap=1e6), plain)
    for cap in (1e-3, 0.7, 1e30):
        c.check(*run(c, softcap=cap), c.reference(softcap=cap))
    c.pool.destroy()


def test_long_context_with_bias_and_every_split():
    c = Cache(ctx=[20011, 3], hq=8, hk=1, d=128, bs=16, seed=9)
    s = slopes_of(8)
    want = c.reference(slopes=s.numpy())
    for split in (0, 16, 4096):
        c.check(*run(c, split, alibi_slopes=s.cuda()), want)
    c.pool.destroy()


def test_padded_batch_bad_lengths_and_bad_blocks():
    """Context 0 gives 0 and -inf; lengths out of range are clamped, bad blocks skipped, both flagged."""
    c = Cache(ctx=[40, 0, 33], hq=4, hk=2, d=64, bs=16)
    out, lse = run(c, window=20)
    assert c.pool.device_errors() == 0
    c.check(out, lse, c.reference(hide(20)))
    assert not out[1].any() and (lse[1] == -float("inf")).all()
    c.lens = i32([40, -5, 1000])
    run(c)
    assert c.pool.device_errors() & kp.DEVERR_CONTEXT
    c.lens = i32([40, 0, 33])
    tab = c.tab.copy()
    tab[0, 1] = -7            # the second half of a 32-token piece of work
    c.tables = i32(tab)
    got = run(c)
    assert c.pool.device_errors() == kp.DEVERR_BLOCK_ID
    c.check(*got, c.reference(lambda b, pos, t: (t > pos) | ((b == 0) & (t // 16 == 1))))
    c.pool.destroy()


@pytest.mark.parametrize("kw", [dict(hk=2, d=64, bs=16), dict(hk=4, d=128, bs=16, fp8=True), dict(hk=4, d=128, bs=32, fp8=True),
                                dict(hk=1, d=128, bs=16)], ids=str)
def test_bad_blocks_anywhere_are_skipped(kw):
    c = Cache(ctx=[200, 77], hq=8, q_len=3, **kw)
    bs = kw["bs"]
    bad = {(0, 0), (0, 3), (0, 5), (1, 1), (1, 2)}
    tab = c.tab.copy()
    for i, (b, j) in enumerate(bad):
        tab[b, j] = [-1, 10 ** 6, c.nb][i % 3]
    c.tables = i32(tab)
    out = run(c, prefix_lens=i32([0, 0]))
    assert c.pool.device_errors() == kp.DEVERR_BLOCK_ID
    c.check(*out, c.reference(lambda b, pos, t: (t > pos) | np.isin(t // bs, [j for bb, j in bad if bb == b])))
    c.pool.destroy()


def test_workspace_is_reused_streams_and_graphs():
    """One zeroed workspace over many calls, another stream, and a graph replayed with new lengths."""
    c = Cache(ctx=[700, 90, 300], hq=8, hk=2, d=128, bs=16)
    need = kp.paged_attention_masked_workspace_size(c.pool, 3, 8, 1, c.max_blocks, 200, 32)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = c.reference(hide(200))
    for _ in range(3):
        c.check(*run(c, 32, window=200, workspace=ws), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(c, 32, window=200, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    c.check(*got, want)
    out = torch.empty_like(c.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kp.paged_attention_masked(c.pool, c.q, c.tables, c.lens, c.scale, window=200, kv_split_tokens=32,
                                  workspace=ws, out=out)
    c.ctx = np.array([650, 16, 1])
    c.lens.copy_(i32(c.ctx))
    for _ in range(2):
        g.replay()
        c.check(out, None, c.reference(hide(200)))
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_one_workspace_for_batches_of_any_size():
    """A workspace of the largest call, zeroed once, under calls of other shapes: every call has to
    find its counters at zero, whatever the ones before left in the rest."""
    cs = [Cache(ctx=[900] * b, hq=8 * hk, hk=hk, d=128, bs=16, q_len=q, seed=b) for b, hk, q in
          ((2, 1, 1), (40, 4, 1), (5, 2, 3), (64, 1, 1), (3, 4, 2))]
    ws = torch.zeros(max(kp.paged_attention_masked_workspace_size(c.pool, c.B, c.hq, c.q_len, c.max_blocks, 0, s)
                         for c in cs for s in (0, 16)), dtype=torch.uint8, device="cuda")
    wants = [c.reference() for c in cs]
    for s in (16, 0):
        for c, want in zip(cs, wants):
            c.check(*run(c, s, workspace=ws), want)
    for c in cs:
        assert c.pool.device_errors() == 0
        c.pool.destroy()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hk,q_len", [(4, 1), (2, 1), (1, 1), (4, 3), (2, 2), (1, 3)])
def test_units_cut_into_many_pieces(hk, q_len, fp8):
    """Two sequences over the whole grid: pieces merged in groups, then the groups; the same bits
    every time."""
    c = Cache(ctx=[15000, 4100], hq=8 * hk, hk=hk, d=128, bs=16, q_len=q_len, fp8=fp8, seed=3)
    ws = torch.zeros(kp.paged_attention_masked_workspace_size(c.pool, 2, c.hq, q_len, c.max_blocks, 0, 16),
                     dtype=torch.uint8, device="cuda")
    want = c.reference()
    for split in (0, 16):
        first = run(c, split, workspace=ws)
        c.check(*first, want)
        for _ in range(5):
            again = run(c, split, workspace=ws)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_window_shrinks_the_workspace():
    c = Cache(ctx=[700], hq=8, hk=2, d=128, bs=16)
    size = lambda w: kp.paged_attention_masked_workspace_size(c.pool, 1, 8, 1, c.max_blocks, w, 16)  # noqa: E731
    assert size(17) < size(100) < size(0) == size(1 << 30) == size(44 * 16)
    c.pool.destroy()


def test_many_sequences():
    """More sequences than a CTA has threads, most of them short or empty, and one long one."""
    r = np.random.default_rng(2)
    ctx = r.integers(0, 40, 700)
    ctx[333] = 3000
    c = Cache(ctx=ctx, hq=2, hk=1, d=64, bs=16)
    c.check(*run(c, window=50), c.reference(hide(50)))
    c.check(*run(c), c.reference())
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_repeated_calls_give_the_same_bits():
    c = Cache(ctx=[3000, 17, 900], hq=8, hk=2, d=128, bs=16, q_len=3)
    ws = torch.zeros(kp.paged_attention_masked_workspace_size(c.pool, 3, 8, 3, c.max_blocks, 0, 16), dtype=torch.uint8,
                     device="cuda")
    first = run(c, 16, workspace=ws)
    for _ in range(20):
        again = run(c, 16, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    c.pool.destroy()


def test_refusals():
    c = Cache(ctx=[40, 30], hq=4, hk=2, d=64, bs=16)
    before = c.q.clone()
    for kw in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")), dict(softcap=1e-45),
               dict(window=-1), dict(split=7), dict(split=-16), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"), split=16)):
        with pytest.raises(kp.KVError) as e:
            run(c, **kw)
        assert e.value.status == kp.KV_ERR_INVALID_ARG
    for kw in (dict(alibi_slopes=torch.ones(3, device="cuda")), dict(first_keys=i32([1])), dict(prefix_lens=i32([1, 2, 3])),
               dict(alibi_slopes=torch.ones(4, dtype=torch.float64, device="cuda"))):
        with pytest.raises(ValueError):
            run(c, **kw)
    with pytest.raises(ValueError):
        kp.paged_attention_masked(c.pool, c.q, c.tables[:1], c.lens, c.scale)
    with pytest.raises(kp.KVError):
        kp.paged_attention_masked(c.pool, c.q, c.tables, c.lens, float("nan"))
    with pytest.raises(kp.KVError):
        kp.paged_attention_masked(c.pool, c.q[:, :3].contiguous(), c.tables, c.lens, c.scale)
    assert torch.equal(c.q, before) and c.pool.device_errors() == 0
    empty = kp.paged_attention_masked(c.pool, c.q[:0], c.tables[:0], c.lens[:0], c.scale, window=3)
    assert empty.shape[0] == 0
    c.pool.destroy()


def test_sparse_tensors_raise():
    """Torch throws for their strides and memory; the calls turn that into a ValueError."""
    c = Cache(ctx=[40, 30], hq=4, hk=2, d=64, bs=16)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    out, off, blk = torch.empty_like(c.q), i32([0, 2]), i32([1])
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    base = dict(pool=c.pool, q=c.q, block_tables=c.tables, context_lens=c.lens, out=out)
    for call, kw in ((kp.paged_attention_masked, dict(base, scale=1.0, workspace=ws, first_keys=c.lens)),
                     (kp.paged_shared_prefix_attention, dict(base, scale=1.0, workspace=ws, group_offsets=off, group_blocks=blk)),
                     (kp.paged_norm_rope_append, dict(base, q=c.q[:, :, 0], k=kv, v=kv))):
        for name, t in kw.items():
            if isinstance(t, torch.Tensor):
                with pytest.raises((ValueError, RuntimeError)):
                    call(**dict(kw, **{name: t.to_sparse()}))
    assert c.pool.device_errors() == 0
    c.pool.destroy()


def test_a_stage_that_never_lands_times_out():
    c = Cache(ctx=[900], hq=4, hk=1, d=128, bs=16)
    kp.kv_debug_decode_stall(3, 20_000_000)
    try:
        run(c, 256, window=500)
        torch.cuda.synchronize()
    finally:
        kp.kv_debug_decode_stall(-1, 0)
    assert c.pool.device_errors() & kp.DEVERR_TIMEOUT
    c.check(*run(c, 256, window=500), c.reference(hide(500)))
    c.pool.destroy()


def test_the_largest_caps_and_scales():
    """Scores are kept in log2 units: a cap or a scale whose product with log2(e) is no fp32 number is
    refused (it made every score NaN); the largest cap that has one changes nothing."""
    c = Cache(ctx=[61, 300], hq=4, hk=2, d=64, bs=16)
    want = c.reference()
    top = float(np.finfo(np.float32).max) / 1.4427
    for cap in (top, 2.0 ** 127, 2.0 ** 100, 2.0 ** 60):
        c.check(*run(c, softcap=cap), want)
    with pytest.raises(kp.KVError):
        run(c, softcap=3e38)
    c.scale = 3e38
    with pytest.raises(kp.KVError):
        run(c)
    with pytest.raises(kp.KVError):
        kp.paged_shared_prefix_attention(c.pool, c.q, c.tables, c.lens, i32([0, 2]), i32([1]), c.scale)
    assert c.pool.device_errors() == 0
    c.pool.destroy()
