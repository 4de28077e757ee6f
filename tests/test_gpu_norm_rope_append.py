"""paged_norm_rope_append against the formula in 64 bits: per-head RMS norm, rotary rotation,
and the append to the paged pool."""
import numpy as np
import pytest
import torch

import paged_kv_cache_19_gb300 as kp
from gpu_util import i32

pytestmark = pytest.mark.gpu

POISON = 0xFF


def rope_table(positions, dim, seed=0):
    """Cosines and sines of position * 10000^(-2i/dim), float32 [positions, dim]."""
    a = np.arange(positions)[:, None] * 10000.0 ** (-2 * np.arange(dim // 2) / dim)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def reference(x, w, eps, table, pos, interleaved):
    """x [T, H, d] float64 -> (normed and rotated, largest |number| of each normed row)."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    top = np.abs(y).max(-1, keepdims=True)
    if table is not None:
        half = table.shape[1] // 2
        c = table[pos, :half].astype(np.float64)[:, None]
        s = table[pos, half:].astype(np.float64)[:, None]
        ia = np.arange(half) * 2 if interleaved else np.arange(half)
        ib = ia + 1 if interleaved else ia + half
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia] = a * c - b * s
        y[..., ib] = b * c + a * s
    return y, top


# fp32 arithmetic before the one rounding: the norm's factor is off by at most
# (d + 8) 2^-24 / 2 + 2^-22 < 2^-17 of itself (d <= 128 terms of one sign, one rsqrt of 2 ulp,
# three products), the rotation adds 4 roundings of two terms no larger than the row's top:
# together below 2^-15 of the top.
def bf16_bound(ref, top):
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * top


def e4m3_bound(ref, top):
    return 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 + 2.0 ** -14 * top


class Call:
    """One call's inputs: `n` tokens of a batch over a poisoned pool of shuffled blocks."""

    def __init__(self, *, hq, hk, d, bs, fp8=False, norm=True, rope_dim=0, interleaved=False, batch=3, q_len=1,
                 ctx=None, pos=None, seq=None, fused=True, seed=0, eps=1e-6):
        r = np.random.default_rng(seed)
        self.hq, self.hk, self.d, self.bs, self.fp8, self.q_len = hq, hk, d, bs, fp8, q_len
        self.interleaved, self.eps = interleaved, eps
        if seq is None:
            ctx = np.asarray(ctx)
            batch = len(ctx)
            self.seq = np.repeat(np.arange(batch), q_len)
            self.pos = np.repeat(ctx - q_len, q_len) + np.tile(np.arange(q_len), batch)
            self.explicit = False
        else:
            self.seq, self.pos = np.asarray(seq), np.asarray(pos)
            self.explicit = True
        top = int(self.pos.max()) + 1
        self.mb = -(-top // bs)
        self.nb = batch * self.mb + 2
        self.tab = r.permutation(self.nb)[:batch * self.mb].reshape(batch, self.mb)
        n = len(self.seq)
        x = torch.from_numpy(r.standard_normal((n, hq + 2 * hk, d))).to(torch.bfloat16)
        self.x = x.double().numpy()
        if fused:
            x = x.cuda()
            self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        else:
            self.q, self.k, self.v = (x[:, a:b].contiguous().cuda() for a, b in
                                      ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
        self.qw = r.uniform(0.5, 1.5, d).astype(np.float32) if norm else None
        self.kw = r.uniform(0.5, 1.5, d).astype(np.float32) if norm else None
        self.table = rope_table(top, rope_dim) if rope_dim else None
        self.pool = kp.kv_pool_create(self.nb, bs, hk, d, "fp8_e4m3" if fp8 else "bf16")
        self.ks = np.ones(hk)
        self.vs = np.ones(hk)
        if fp8:
            self.ks = r.uniform(0.004, 0.02, hk).astype(np.float32)
            self.vs = r.uniform(0.004, 0.02, hk).astype(np.float32)
            self.pool.set_scales(self.ks, self.vs)
        for t in self.pool.raw_bytes():
            t.fill_(POISON)
        self.ctx = i32(ctx) if ctx is not None else None
        dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        self.dqw, self.dkw, self.dtable, self.dtab = dev(self.qw), dev(self.kw), dev(self.table), i32(self.tab)

    def run(self, **kw):
        a = dict(q_weight=self.dqw, k_weight=self.dkw, eps=self.eps, rope_table=self.dtable,
                 interleaved=self.interleaved, q_len=self.q_len)
        if self.explicit:
            a.update(token_seq=i32(self.seq), token_pos=i32(self.pos))
        a.update(kw)
        return kp.paged_norm_rope_append(self.pool, self.q, self.k, self.v, self.dtab, self.ctx, **a)

    def check(self, out, written=None, q_written=None):
        """Queries, written slots, and everything else left as it was."""
        n = len(self.seq)
        written = np.ones(n, bool) if written is None else written
        q_written = np.ones(n, bool) if q_written is None else q_written
        pos = np.maximum(self.pos, 0)
        if self.table is not None:
            pos = np.minimum(pos, len(self.table) - 1)
        hq, hk = self.hq, self.hk
        q, qt = reference(self.x[:, :hq], self.qw, self.eps, self.table, pos, self.interleaved)
        k, kt = reference(self.x[:, hq:hq + hk], self.kw, self.eps, self.table, pos, self.interleaved)
        v = self.x[:, hq + hk:]
        got = out.double().cpu().numpy().reshape(n // self.q_len, hq, self.q_len, self.d).transpose(0, 2, 1, 3)
        got = got.reshape(n, hq, self.d)
        assert (np.abs(got - q) <= bf16_bound(q, qt))[q_written].all()
        rows = torch.ones(self.pool.num_blocks, self.bs, dtype=torch.bool)
        for half, ref, top, scale in ((0, k, kt, self.ks), (1, v, 0.0, self.vs)):
            raw = self.pool.raw_bytes()[half].cpu()
            vals = self.pool.tensors()[half].float().double().cpu().numpy()
            for i in np.nonzero(written)[0]:
                blk, slot = self.tab[self.seq[i], self.pos[i] // self.bs], self.pos[i] % self.bs
                rows[blk, slot] = False
                y = vals[blk, slot]
                if self.fp8:
                    want = np.clip(ref[i] / scale[:, None], -448, 448)
                    bound = e4m3_bound(want, (top[i] if half == 0 else 0.0) / scale[:, None])
                else:
                    want = ref[i]
                    bound = bf16_bound(want, top[i]) if half == 0 else 0.0
                assert (np.abs(y - want) <= bound).all(), (half, i)
            assert (raw[rows] == POISON).all()
        self.pool.destroy()


CASES = [
    dict(hq=4, hk=4, d=64, bs=16, rope_dim=64, ctx=[1]),
    dict(hq=32, hk=8, d=128, bs=16, rope_dim=128, ctx=[1, 16, 17, 300]),
    dict(hq=32, hk=8, d=128, bs=32, rope_dim=128, interleaved=True, ctx=[5, 64, 65], fused=False),
    dict(hq=7, hk=7, d=128, bs=16, rope_dim=32, ctx=[9, 33]),
    dict(hq=6, hk=2, d=64, bs=32, rope_dim=16, interleaved=True, ctx=[40]),
    dict(hq=8, hk=1, d=128, bs=16, rope_dim=0, ctx=[18, 2]),
    dict(hq=5, hk=1, d=64, bs=16, norm=False, rope_dim=48, ctx=[100, 1, 31]),
    dict(hq=16, hk=4, d=128, bs=16, rope_dim=128, q_len=5, ctx=[5, 21, 100]),
    dict(hq=32, hk=32, d=128, bs=32, fp8=True, norm=False, rope_dim=64, interleaved=True, q_len=3, ctx=[3, 33, 70]),
    dict(hq=32, hk=8, d=128, bs=16, fp8=True, rope_dim=128, ctx=[1, 17, 300, 16]),
    dict(hq=12, hk=12, d=128, bs=16, fp8=True, rope_dim=96, fused=False, ctx=[77]),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()).replace(" ", ""))
def test_matches_the_formula(kw):
    c = Call(**kw)
    out = torch.full((len(c.seq) // c.q_len, c.hq, c.q_len, c.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert c.run(out=out) is out
    assert c.pool.device_errors() == 0
    c.check(out)


def test_ragged_prompt_pieces():
    """Tokens of several sequences in any order, more than fill one launch's first wave."""
    r = np.random.default_rng(4)
    seq = np.repeat([2, 0, 3], [700, 1, 500])
    pos = np.concatenate([np.arange(13, 713), [8], np.arange(500)])
    order = r.permutation(len(seq))
    c = Call(hq=8, hk=4, d=128, bs=16, rope_dim=128, batch=4, seq=seq[order], pos=pos[order])
    out = c.run()
    assert c.pool.device_errors() == 0 and out.shape == (1201, 8, 128)
    c.check(out)


@pytest.mark.parametrize("kw", [dict(hq=4, hk=2, d=128, bs=16, rope_dim=128), dict(hq=5, hk=1, d=64, bs=32, rope_dim=32, norm=False),
                                dict(hq=4, hk=4, d=128, bs=32, rope_dim=64, interleaved=True, fp8=True),
                                dict(hq=64, hk=16, d=128, bs=16, rope_dim=0)],
                         ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_long_prompts(kw):
    """Enough tokens for every CTA's ring to go round; some of them bad, one batch of q_len tokens."""
    r = np.random.default_rng(5)
    n = 3001 if kw["hq"] < 64 else 1300
    seq = np.sort(r.integers(0, 4, n))
    pos = np.concatenate([np.arange((seq == b).sum()) + 7 * b for b in range(4)])
    c = Call(batch=4, seq=seq, pos=pos, **kw)
    bad = np.zeros(n, bool)
    bad[[0, 31, 32, 700, n - 1]] = True
    c.seq[bad] = [-1, 4, 10 ** 9, -5, 99]
    out = torch.full((n, c.hq, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out)
    assert c.pool.device_errors() == kp.DEVERR_SEQ
    assert (out[torch.from_numpy(bad).cuda()] == 7.0).all()
    c.seq[bad] = 0
    c.check(out, written=~bad, q_written=~bad)
    if kw["hq"] == 4 and not kw.get("fp8"):
        c = Call(ctx=r.integers(5, 40, 301), q_len=5, **kw)
        out = torch.empty((301, 4, 5, c.d), dtype=torch.bfloat16, device="cuda")
        c.run(out=out)
        assert c.pool.device_errors() == 0
        c.check(out)


def test_without_norm_and_rotation_it_is_the_append():
    """Same pool bytes as paged_kv_append, queries copied."""
    for fp8 in (False, True):
        c = Call(hq=8, hk=4, d=128, bs=16, fp8=fp8, norm=False, ctx=[1, 20, 47])
        out = c.run()
        assert torch.equal(out, c.q)
        mine = [t.clone() for t in c.pool.raw_bytes()]
        for t in c.pool.raw_bytes():
            t.fill_(POISON)
        kp.paged_kv_append(c.pool, c.k.contiguous(), c.v.contiguous(), c.dtab, c.ctx)
        for a, b in zip(mine, c.pool.raw_bytes()):
            assert torch.equal(a, b)
        c.pool.destroy()


@pytest.mark.parametrize("repeat", [1, 4])
def test_every_bf16_value_rounds_as_the_append_does(repeat):
    """All 65,536 bf16 patterns under many scales: quotients at, next to and far from the values
    where the code changes, powers of two, and scales at the ends of the range."""
    r = np.random.default_rng(5)
    scales = np.concatenate([r.uniform(0.001, 0.1, 9), [1.0, 2.0 ** -7, 1 / 3, 0.3, 1e-40, 2.0 ** -149, 3e38, 1e-30, 1e30, 2.0 ** 100,
                                                        1.5 * 2.0 ** -99, 448.0, 7.0, 0.9999999, 1.0000001, 17 / 16, 15 / 8]])
    scales = np.resize(scales.astype(np.float32), 32)
    n = 512 * repeat
    rows = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(512, 1, 128)
    rows = rows.expand(512, 32, 128).repeat(repeat, 1, 1).cuda()
    q = torch.zeros(n, 8, 128, dtype=torch.bfloat16, device="cuda")
    pool = kp.kv_pool_create(n // 32, 32, 32, 128, "fp8_e4m3")
    pool.set_scales(scales, scales[::-1].copy())
    tab = i32(r.permutation(n // 32)[None])
    seq, pos = i32(np.zeros(n)), i32(np.arange(n))
    kp.paged_norm_rope_append(pool, q, rows, rows, tab, token_seq=seq, token_pos=pos)
    mine = [t.clone() for t in pool.raw_bytes()]
    for t in pool.raw_bytes():
        t.fill_(POISON)
    kp.paged_kv_append(pool, rows, rows, tab, None, token_seq=seq, token_pos=pos)
    for a, b in zip(mine, pool.raw_bytes()):
        assert torch.equal(a, b)
    pool.destroy()


def test_far_positions_and_extreme_rows():
    """Rows of zeros (the norm's eps), of tiny and of large numbers, infinities kept to their row."""
    c = Call(hq=4, hk=2, d=128, bs=16, rope_dim=128, batch=1, seq=[0] * 4, pos=[70000, 0, 69999, 31], eps=1e-5)
    c.x[0] = 0.0
    c.x[1] = np.float64(torch.tensor(2.0 ** -60, dtype=torch.bfloat16))
    c.x[2] *= 2.0 ** 40
    x = torch.from_numpy(c.x).to(torch.bfloat16)
    c.x = x.double().numpy()
    x = x.cuda()
    c.q, c.k, c.v = x[:, :4], x[:, 4:6], x[:, 6:]
    out = c.run()
    assert c.pool.device_errors() == 0
    c.check(out)


def test_bad_tokens_write_nothing_of_others():
    """Invalid sequence, position or block id: flagged; what the call leaves alone stays."""
    seq, pos = np.array([0, -1, 5, 1, 1, 0, 1]), np.array([3, 0, 0, -1, 64, 17, 2])
    c = Call(hq=4, hk=2, d=64, bs=16, rope_dim=64, batch=2, seq=seq, pos=np.clip(pos, 0, 63))
    c.pos = pos
    c.tab[0, 1] = 10 ** 6                     # sequence 0's second block is not in the pool
    c.dtab = i32(c.tab)
    out = torch.full((7, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out)
    assert c.pool.device_errors() == kp.DEVERR_SEQ | kp.DEVERR_POSITION | kp.DEVERR_BLOCK_ID
    assert (out[[1, 2, 3, 4]] == 7.0).all()
    ok = np.array([1, 0, 0, 0, 0, 0, 1], bool)
    c.check(out, written=ok, q_written=ok | (np.arange(7) == 5))


def test_positions_past_the_rotation_table_are_flagged():
    c = Call(hq=4, hk=2, d=64, bs=16, rope_dim=64, ctx=[3, 40])
    out = torch.full((2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out, rope_table=c.dtable[:39].contiguous())
    assert c.pool.device_errors() == kp.DEVERR_POSITION
    assert (out[1] == 7.0).all()
    ok = np.array([True, False])
    c.check(out, written=ok, q_written=ok)


def test_padded_batch_and_fewer_tokens_than_the_batch():
    """context 0 has no new token (flagged, as the append does); rows behind the tokens stay."""
    c = Call(hq=4, hk=2, d=64, bs=16, rope_dim=32, ctx=[3, 9])
    ctx = i32([3, 0, 9])
    tab = torch.cat([c.dtab, c.dtab])[[0, 1, 1]].contiguous()
    x = torch.stack([c.q[0], c.q[0], c.q[1]]), torch.stack([c.k[0], c.k[0], c.k[1]]), torch.stack([c.v[0], c.v[0], c.v[1]])
    out = torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kp.paged_norm_rope_append(c.pool, *x, tab, ctx, q_weight=c.dqw, k_weight=c.dkw, rope_table=c.dtable, out=out)
    assert c.pool.device_errors() == kp.DEVERR_POSITION
    assert (out[1] == 7.0).all()
    c.check(out[[0, 2]])


def test_another_stream_and_a_replayed_graph():
    c = Call(hq=8, hk=2, d=128, bs=16, rope_dim=128, ctx=[5, 50, 33])
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        c.run(out=out)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        c.run(out=out)
    out.zero_()
    for t in c.pool.raw_bytes():
        t.fill_(POISON)
    # the replay reads the lengths of its time
    c.ctx.copy_(i32([6, 49, 40]))
    c.pos = np.array([5, 48, 39])
    g.replay()
    torch.cuda.synchronize()
    c.check(out)


def test_refusals():
    c = Call(hq=4, hk=2, d=64, bs=16, rope_dim=64, ctx=[3, 9])
    lib = kp.load_library()
    out = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")

    def call(**kw):
        a = dict(q=c.q.data_ptr(), qs=8 * 64, k=c.k.data_ptr(), ks=8 * 64, v=c.v.data_ptr(), vs=8 * 64, heads=4, n=2,
                 qw=c.dqw.data_ptr(), kw=c.dkw.data_ptr(), eps=1e-6, rope=c.dtable.data_ptr(), npos=9, dim=64, style=0,
                 seq=None, pos=None, tab=c.dtab.data_ptr(), mb=c.mb, ctx=c.ctx.data_ptr(), batch=2, q_len=1,
                 out=out.data_ptr())
        a.update(kw)
        return lib.paged_norm_rope_append(c.pool.handle, *a.values(), None)

    some = c.ctx.data_ptr()
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(tab=None), dict(heads=0), dict(n=-1),
               dict(n=3), dict(batch=0), dict(mb=0), dict(mb=1 << 28), dict(q_len=0), dict(qw=None), dict(kw=None),
               dict(eps=-1.0), dict(eps=float("nan")), dict(dim=24), dict(dim=80), dict(dim=0), dict(npos=0),
               dict(style=2), dict(ctx=None), dict(qs=4 * 64 - 8), dict(ks=2 * 64 + 4), dict(vs=64),
               dict(q=c.q.data_ptr() + 8), dict(out=out.data_ptr() + 2), dict(rope=c.dtable.data_ptr() + 4),
               dict(seq=some, q_len=2), dict(pos=some, q_len=2)):
        assert call(**kw) == kp.KV_ERR_INVALID_ARG, kw
    assert call(n=1 << 28, seq=some, pos=some) == kp.KV_ERR_UNSUPPORTED
    assert call(n=0) == kp.KV_OK
    torch.cuda.synchronize()
    assert c.pool.device_errors() == 0 and not out.any()
    with pytest.raises(ValueError):
        kp.paged_norm_rope_append(c.pool, c.q, c.k[:1], c.v, c.dtab, c.ctx)
    with pytest.raises(ValueError):
        kp.paged_norm_rope_append(c.pool, c.q.transpose(0, 1), c.k, c.v, c.dtab, c.ctx)
    with pytest.raises(ValueError):
        kp.paged_norm_rope_append(c.pool, c.q, c.k, c.v, c.dtab, c.ctx, token_pos=i32([1]))
    with pytest.raises(ValueError):
        kp.paged_norm_rope_append(c.pool, c.q, c.k, c.v, c.dtab, c.ctx, q_len=3)
    latent = kp.kv_mla_pool_create(2, 16)
    assert lib.paged_norm_rope_append(latent.handle, c.q.data_ptr(), 512, c.k.data_ptr(), 512, c.v.data_ptr(), 512, 4, 2,
                                      None, None, 0.0, None, 0, 0, 0, None, None, c.dtab.data_ptr(), c.mb,
                                      c.ctx.data_ptr(), 2, 1, out.data_ptr(), None) == kp.KV_ERR_INVALID_ARG
    latent.destroy()
    c.pool.destroy()


@pytest.mark.parametrize("q_len,tokens", [(2, 3), (5, 4), (5, 9), (2, 1)])
def test_a_part_of_a_sequences_tokens_is_refused(q_len, tokens):
    """q_out has room for tokens / q_len sequences: a token behind them would be written past its end
    (row (tokens // q_len) * q_heads * q_len and on)."""
    c = Call(hq=4, hk=2, d=64, bs=16, rope_dim=64, q_len=q_len, ctx=[9, 20, 33])
    out = torch.zeros((3, 4, q_len, 64), dtype=torch.bfloat16, device="cuda")
    args = (c.q.data_ptr(), 512, c.k.data_ptr(), 512, c.v.data_ptr(), 512, 4)
    rest = (c.dqw.data_ptr(), c.dkw.data_ptr(), 1e-6, c.dtable.data_ptr(), len(c.table), 64, 0, None, None,
            c.dtab.data_ptr(), c.mb, c.ctx.data_ptr(), 3, q_len, out.data_ptr(), None)
    lib = kp.load_library()
    assert lib.paged_norm_rope_append(c.pool.handle, *args, tokens, *rest) == kp.KV_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert not out.any() and all((t == POISON).all() for t in c.pool.raw_bytes())
    assert lib.paged_norm_rope_append(c.pool.handle, *args, 3 * q_len, *rest) == kp.KV_OK
    assert c.pool.device_errors() == 0
    c.check(out)


@pytest.mark.parametrize("n", [12, 1800])
@pytest.mark.parametrize("eps", [0.0, 2.0 ** -140, 1e-30, 1e-6, 3e38])
def test_rows_whose_squares_leave_the_range_of_fp32(eps, n, monkeypatch):
    """The norm over the whole range of bf16 and of eps: rows of the smallest numbers, of the largest
    ones, and in between (both forms of the kernel).

    bf16_bound counts half a step as 2^-8 of the number, which holds from 2^-126 on.  Below, the
    steps of bf16 stay 2^-133 apart, so half a step is 2^-134 whatever the number (the fp32 numbers
    before it are off by 2^-149 there, inside the 2^-15 of the row's top or far below 2^-134)."""
    usual = bf16_bound
    monkeypatch.setitem(globals(), "bf16_bound", lambda ref, top: usual(ref, top) + 2.0 ** -134 * (np.abs(ref) < 2.0 ** -126))
    c = Call(hq=4, hk=2, d=128, bs=16, rope_dim=64, batch=1, seq=np.zeros(n, int), pos=np.arange(n), eps=eps)
    # standard normal numbers, at most 6 of them: 2^124 times that is finite in bf16
    by = np.array([2.0 ** e for e in (-131, -120, -90, -75, -64, -50, 0, 40, 61, 66, 90, 124)])
    x = torch.from_numpy(np.clip(c.x, -6, 6) * np.resize(by, n)[:, None, None]).to(torch.bfloat16)
    assert torch.isfinite(x).all()
    x[..., 0] = torch.where((x == 0).all(-1), torch.finfo(torch.bfloat16).smallest_normal, x[..., 0])
    c.x = x.double().numpy()
    # (the values are copied as they are; keys and queries are normed)
    x = x.cuda()
    c.q, c.k, c.v = x[:, :4], x[:, 4:6], x[:, 6:]
    out = c.run()
    assert c.pool.device_errors() == 0
    c.check(out)


def test_a_row_of_zeros_without_eps_is_not_a_number_and_stays_alone():
    """0 / 0, as the formula has it, in its own row only."""
    c = Call(hq=4, hk=2, d=128, bs=16, norm=True, rope_dim=0, ctx=[3, 9], eps=0.0)
    c.x[0, 1] = 0.0
    x = torch.from_numpy(c.x).to(torch.bfloat16).cuda()
    c.q, c.k, c.v = x[:, :4], x[:, 4:6], x[:, 6:]
    out = c.run()
    assert torch.isnan(out[0, 1]).all()
    c.x[0, 1] = 1.0
    out[0, 1] = torch.from_numpy(c.qw).cuda()
    c.check(out)


def test_a_rotation_table_without_rows_writes_nothing():
    c = Call(hq=4, hk=2, d=64, bs=16, rope_dim=64, ctx=[3, 9])
    out = torch.zeros_like(c.q)
    for table in (c.dtable[:0], c.dtable[:, :0].contiguous()):
        with pytest.raises(ValueError, match="rope_table"):
            c.run(out=out, rope_table=table)
    assert not out.any() and all((t == POISON).all() for t in c.pool.raw_bytes())
    c.pool.destroy()
