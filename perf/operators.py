"""The operators around paged decode attention, as cases to measure: their inputs, their plain
form in torch, their definition in 64 bits, and the library calls that compute them.

  * norm_rope_append: per-head RMS norm of queries and keys, the rotary rotation by position,
    and the store of keys and values into the paged cache, in one pass;
  * masked: attention over the paged cache whose scores are capped by a tanh, biased by
    distance, and masked by a window, a document start or a visible prefix;
  * shared_prefix: decode attention of a batch whose sequences share leading cache blocks,
    the shared part computed once for all members of a group.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- the cases
def listed():
    return [
        # one sequence of an interactive session: the call's latency is the token's latency
        dict(name="append-one", op="norm_rope_append", q_heads=32, kv_heads=8, head_dim=128, block_size=16,
             fp8=False, norm=True, rope_dim=128, interleaved=False, batch=1, q_len=1, tokens=0, ctx_hi=4096, lens=11),
        # the decode step of a serving batch, rows taken from one fused q|k|v projection
        dict(name="append-decode64", op="norm_rope_append", q_heads=32, kv_heads=8, head_dim=128, block_size=16,
             fp8=False, norm=True, rope_dim=128, interleaved=False, batch=64, q_len=1, tokens=0, ctx_hi=4096, lens=12),
        # a verify pass of 5 tokens over an 8-bit cache, half of each head rotated, pairs interleaved
        dict(name="append-verify-fp8", op="norm_rope_append", q_heads=32, kv_heads=32, head_dim=128, block_size=32,
             fp8=True, norm=False, rope_dim=64, interleaved=True, batch=37, q_len=5, tokens=0, ctx_hi=2048, lens=13),
        # prompts of a chunked prefill: ragged pieces of many sequences in one call
        dict(name="append-prefill", op="norm_rope_append", q_heads=32, kv_heads=8, head_dim=128, block_size=16,
             fp8=False, norm=True, rope_dim=128, interleaved=False, batch=9, q_len=1, tokens=8191, ctx_hi=2048, lens=14),

        # one short sequence with capped scores
        dict(name="masked-one", op="masked", q_heads=32, kv_heads=8, head_dim=128, block_size=16, fp8=False,
             batch=1, q_len=1, ctx_lo=300, ctx_hi=300, softcap=50.0, window=0, alibi=False, first=False,
             prefix=False, lens=21),
        # a serving batch on a layer with capped scores and a sliding window
        dict(name="masked-cap-window", op="masked", q_heads=32, kv_heads=8, head_dim=128, block_size=16, fp8=False,
             batch=64, q_len=1, ctx_lo=512, ctx_hi=4096, softcap=30.0, window=1000, alibi=False, first=False,
             prefix=False, lens=22),
        # long contexts with a bias by distance
        dict(name="masked-alibi-long", op="masked", q_heads=64, kv_heads=8, head_dim=128, block_size=16, fp8=False,
             batch=8, q_len=1, ctx_lo=32768, ctx_hi=131072, softcap=0.0, window=0, alibi=True, first=False,
             prefix=False, lens=23),
        # packed documents with a bidirectional prefix, 7 new tokens a sequence, 8-bit cache
        dict(name="masked-docs-fp8", op="masked", q_heads=32, kv_heads=32, head_dim=128, block_size=32, fp8=True,
             batch=33, q_len=7, ctx_lo=100, ctx_hi=2048, softcap=0.0, window=0, alibi=False, first=True,
             prefix=True, lens=24),

        # four samples of one short prompt
        dict(name="prefix-four", op="shared_prefix", q_heads=32, kv_heads=8, head_dim=128, block_size=16, fp8=False,
             batch=4, q_len=1, group=4, prefix=512, suffix=50, pad=0, lens=31),
        # a ragged batch whose groups of 8 share 512 tokens
        dict(name="prefix-groups", op="shared_prefix", q_heads=32, kv_heads=8, head_dim=128, block_size=16, fp8=False,
             batch=256, q_len=1, group=8, prefix=512, suffix=1500, pad=3, lens=32),
        # one system prompt over a batch on an 8-bit cache without grouped heads
        dict(name="prefix-system-fp8", op="shared_prefix", q_heads=32, kv_heads=32, head_dim=128, block_size=32,
             fp8=True, batch=128, q_len=1, group=128, prefix=2048, suffix=301, pad=0, lens=33),
        # a long shared document asked 128 questions
        dict(name="prefix-document", op="shared_prefix", q_heads=64, kv_heads=8, head_dim=128, block_size=16,
             fp8=False, batch=128, q_len=1, group=128, prefix=16384, suffix=500, pad=0, lens=34),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _layout(rng):
    fp8 = rng.random() < 0.3
    kv = rng.choice([1, 2, 4, 8, 8, 12, 32])
    g = rng.choice([1, 2, 3, 4, 4, 8, 8]) if kv < 32 else 1
    return dict(q_heads=kv * g, kv_heads=kv, head_dim=128 if fp8 else rng.choice([64, 128, 128]),
                block_size=rng.choice([16, 32]), fp8=fp8)


def draw(rng):
    op = rng.choice(["norm_rope_append", "masked", "shared_prefix"])
    c = dict(op=op, **_layout(rng), lens=rng.randrange(1 << 30))
    d = c["head_dim"]
    if op == "norm_rope_append":
        ragged = rng.random() < 0.4
        c.update(norm=rng.random() < 0.7, rope_dim=rng.choice([0, d // 2, d, d, d]),
                 interleaved=rng.random() < 0.3, batch=_log(rng, 1, 128),
                 q_len=1 if ragged else rng.choice([1, 1, 1, 2, 5]), tokens=0, ctx_hi=_log(rng, 64, 8192))
        if ragged:
            c.update(batch=_log(rng, 1, 16), tokens=_log(rng, 16, 4096), ctx_hi=_log(rng, 512, 4096))
        return c
    if op == "masked":
        batch = _log(rng, 1, 96)
        q_len = rng.choice([1, 1, 1, 2, 7, 33])
        hi = _log(rng, 1, max(64, min(65536, 120000 // batch // (8 if q_len > 7 else 1))))
        c.update(batch=batch, q_len=q_len, ctx_lo=q_len + rng.randrange(0, hi), ctx_hi=q_len + hi,
                 softcap=rng.choice([0.0, 20.0, 50.0]), window=rng.choice([0, 0, 1, _log(rng, 2, 4096)]),
                 alibi=rng.random() < 0.4, first=rng.random() < 0.3, prefix=rng.random() < 0.3)
        return c
    batch = _log(rng, 2, 200)
    prefix = _log(rng, 16, max(64, min(16384, 300000 // batch)))
    c.update(batch=batch, q_len=rng.choice([1, 1, 1, 3]), group=_log(rng, 1, batch),
             prefix=prefix, suffix=_log(rng, 4, 1000), pad=rng.choice([0, 0, 2]))
    return c


# --------------------------------------------------------------------------- sizes
def _lengths(case):
    """Context lengths (and, per operator, what else fixes the work) of a case: from the case alone."""
    r = np.random.RandomState(case["lens"] & 0x7FFFFFFF)
    B, q, bs = case["batch"], case["q_len"], case["block_size"]
    if case["op"] == "norm_rope_append":
        if case["tokens"]:
            # the call's tokens spread over the sequences in pieces that end anywhere
            cut = np.sort(r.randint(0, case["tokens"] + 1, B - 1)) if B > 1 else np.zeros(0, int)
            n = np.diff(np.concatenate([[0], cut, [case["tokens"]]]))
            start = r.randint(0, case["ctx_hi"], B)
            return {"n": n, "start": start, "ctx": start + n}
        return {"n": np.full(B, q), "ctx": q + r.randint(0, case["ctx_hi"], B)}
    if case["op"] == "masked":
        ctx = r.randint(case["ctx_lo"], case["ctx_hi"] + 1, B)
        # a document may begin after the first of the new tokens: those then see nothing
        first = np.minimum(r.randint(0, case["ctx_hi"], B), ctx - 1) if case["first"] else np.zeros(B, int)
        prefix = r.randint(0, ctx + 1) if case["prefix"] else np.zeros(B, int)
        return {"ctx": ctx, "first": first, "prefix": prefix}
    ng = -(-B // case["group"])
    blocks = np.maximum(1, np.round(case["prefix"] / bs * r.uniform(0.5, 1.0, ng))).astype(int)
    blocks[0] = max(1, case["prefix"] // bs)
    off = np.minimum(np.arange(ng + 1) * case["group"], B)
    of = np.repeat(np.arange(ng), np.diff(off))
    ctx = blocks[of] * bs + q - 1 + r.randint(1, case["suffix"] + 1, B)
    if case["pad"]:
        ctx[r.choice(B, min(case["pad"], B - 1), replace=False)] = 0      # empty places of a padded batch
    return {"ctx": ctx, "blocks": blocks, "off": off, "of": of}


def _intervals(case, L):
    """Visible keys [lo, hi) of each (sequence, query token) of a masked case."""
    q = case["q_len"]
    pos = L["ctx"][:, None] - q + np.arange(q)[None, :]
    lo = np.repeat(L["first"][:, None], q, 1)
    if case["window"]:
        lo = np.maximum(lo, pos - case["window"] + 1)
    hi = np.maximum(pos + 1, np.minimum(L["prefix"], L["ctx"])[:, None])
    return np.maximum(lo, 0), hi


def work(case):
    L = _lengths(case)
    hq, hk, d, B, q = case["q_heads"], case["kv_heads"], case["head_dim"], case["batch"], case["q_len"]
    e = 1 if case["fp8"] else 2
    if case["op"] == "norm_rope_append":
        n = int(L["n"].sum())
        b = n * (hq * d * 4 + 2 * hk * d * (2 + e)) + n * case["rope_dim"] * 4
        return {"bytes": b, "flops": n * (hq + hk) * (4 * d + 3 * case["rope_dim"])}
    rows = B * hq * q
    io = rows * (d * 4 + 4)
    if case["op"] == "masked":
        lo, hi = _intervals(case, L)
        keys = int(np.maximum(hi.max(1) - lo.min(1), 0).sum())
        pairs = int(np.maximum(hi - lo, 0).sum()) * hq
        return {"bytes": io + keys * hk * d * 2 * e, "flops": 4 * d * pairs}
    live = L["ctx"] > 0
    pre = L["blocks"][L["of"]] * case["block_size"]
    keys = int((L["blocks"] * case["block_size"]).sum() + np.where(live, L["ctx"] - pre, 0).sum())
    pairs = int(np.maximum(L["ctx"], 0).sum()) * q * hq
    return {"bytes": io + keys * hk * d * 2 * e, "flops": 4 * d * pairs}


# --------------------------------------------------------------------------- inputs
def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tables(ctx, bs, r, shared=None, spare=0, only=None):
    """Block tables over a shuffled pool: one row a sequence, -1 behind its blocks. shared:
    (group of each sequence, leading blocks of each group), held once. only(b, j): whether the
    block is in the pool at all (others name block 0 of the pool, which holds nothing)."""
    nb = -(-np.maximum(ctx, 0) // bs)
    if shared is not None:
        nb = np.maximum(nb, shared[1][shared[0]])
    tab = np.full((len(ctx), max(1, int(nb.max()))), -1, np.int64)
    total = 1 if only is not None else 0
    seen = {}
    for b in range(len(ctx)):
        n = int(nb[b])
        if only is not None:
            lo = only[b]
            tab[b, :lo] = 0
            tab[b, lo:n] = total + np.arange(n - lo)
            total += n - lo
        elif shared is not None:
            p, g = int(shared[1][shared[0][b]]), int(shared[0][b])
            if g not in seen:
                seen[g] = total
                total += p
            tab[b, :p] = seen[g] + np.arange(p)
            tab[b, p:n] = total + np.arange(n - p)
            total += n - p
        else:
            tab[b, :n] = total + np.arange(n)
            total += n
    total = max(total, 1) + spare
    perm = r.permutation(total)
    return np.where(tab >= 0, perm[np.maximum(tab, 0)], -1), total


def _pool(state, case, blocks, gen):
    """The cache of one layer: the library's pool, or two plain tensors of the same layout."""
    hk, d, bs = case["kv_heads"], case["head_dim"], case["block_size"]
    shape = (blocks, bs, hk, d)
    if case["fp8"]:
        ks = torch.rand(hk, generator=gen, device=DEV) * 0.01 + 0.008
        vs = torch.rand(hk, generator=gen, device=DEV) * 0.01 + 0.008
    else:
        ks = vs = torch.ones(hk, device=DEV)

    def values(scale):
        x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32 if case["fp8"] else torch.bfloat16)
        return (x / scale[:, None]).clamp_(-448, 448).to(torch.float8_e4m3fn) if case["fp8"] else x

    if own:
        import paged_kv_cache_19_gb300 as kp
        pool = kp.kv_pool_create(blocks, bs, hk, d, "fp8_e4m3" if case["fp8"] else "bf16")
        if case["fp8"]:
            pool.set_scales(ks.tolist(), vs.tolist())
        k, v, _, _ = pool.tensors()
        k.copy_(values(ks))
        v.copy_(values(vs))
        state["pool"] = pool
    else:
        k, v = values(ks), values(vs)
    state.update(k=k, v=v, ks=ks, vs=vs)


def _rope_table(positions, dim):
    """cos and sin of position * 10000^(-2i/dim), in 64 bits, rounded once."""
    i = torch.arange(dim // 2, dtype=torch.float64, device=DEV)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (-2 * i / dim)
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    L = _lengths(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.RandomState(seed & 0x7FFFFFFF)
    hq, hk, d, B, q, bs = (case[x] for x in ("q_heads", "kv_heads", "head_dim", "batch", "q_len", "block_size"))
    s = {"case": case, "scale": 1.0 / math.sqrt(d)}

    if case["op"] == "norm_rope_append":
        # blocks that the call does not write are not in this layer's small pool
        lo = (L["ctx"] - L["n"]) // bs
        tab, blocks = _tables(L["ctx"], bs, r, only=lo)
        _pool(s, case, blocks, gen)
        n = int(L["n"].sum())
        qkv = torch.randn((n, hq + 2 * hk, d), generator=gen, device=DEV, dtype=torch.bfloat16)
        s.update(q=qkv[:, :hq], key=qkv[:, hq:hq + hk], val=qkv[:, hq + hk:], tables=_i32(tab), ctx=_i32(L["ctx"]))
        s["qw"] = s["kw"] = s["rope"] = s["seq"] = s["pos"] = None
        if case["norm"]:
            s["qw"] = torch.rand(d, generator=gen, device=DEV) + 0.5
            s["kw"] = torch.rand(d, generator=gen, device=DEV) + 0.5
        if case["rope_dim"]:
            s["rope"] = _rope_table(int(L["ctx"].max()), case["rope_dim"])
        seq = np.repeat(np.arange(B), L["n"])
        pos = np.concatenate([np.arange(c - m, c) for c, m in zip(L["ctx"], L["n"])])
        s["at"] = (_i32(seq).long(), _i32(pos).long())
        if case["tokens"]:
            s.update(seq=_i32(seq), pos=_i32(pos))
            s["out"] = torch.empty((n, hq, d), dtype=torch.bfloat16, device=DEV)
        else:
            s["out"] = torch.empty((B, hq, q, d), dtype=torch.bfloat16, device=DEV)
        return s

    shared = None if case["op"] == "masked" else (L["of"], L["blocks"])
    tab, blocks = _tables(L["ctx"], bs, r, shared=shared, spare=3)
    _pool(s, case, blocks, gen)
    s.update(tables=_i32(tab), ctx=_i32(L["ctx"]),
             q=torch.randn((B, hq, q, d), generator=gen, device=DEV, dtype=torch.bfloat16),
             out=torch.empty((B, hq, q, d), dtype=torch.bfloat16, device=DEV),
             lse=torch.empty((B, hq, q), dtype=torch.float32, device=DEV))
    if case["op"] == "masked":
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device=DEV) / hq) if case["alibi"] else None
        s["first"] = _i32(L["first"]) if case["first"] else None
        s["prefix"] = _i32(L["prefix"]) if case["prefix"] else None
    else:
        s.update(off=_i32(L["off"]), blocks=_i32(L["blocks"]))
    if own:
        import paged_kv_cache_19_gb300 as kp
        if case["op"] == "masked":
            need = kp.paged_attention_masked_workspace_size(s["pool"], B, hq, q, tab.shape[1], case["window"])
        else:
            need = kp.paged_shared_prefix_workspace_size(s["pool"], B, hq, q, tab.shape[1], len(L["blocks"]))
        s["ws"] = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm_rope_append": _plain_append, "masked": _plain_masked, "shared_prefix": _plain_prefix}[op](s)
    import paged_kv_cache_19_gb300 as kp
    c = s["case"]
    if op == "norm_rope_append":
        kp.paged_norm_rope_append(s["pool"], s["q"], s["key"], s["val"], s["tables"], s["ctx"], q_weight=s["qw"],
                                  k_weight=s["kw"], eps=1e-6, rope_table=s["rope"], interleaved=c["interleaved"],
                                  q_len=c["q_len"], token_seq=s["seq"], token_pos=s["pos"], out=s["out"])
        return s["out"], s["k"], s["v"]
    if op == "masked":
        kp.paged_attention_masked(s["pool"], s["q"], s["tables"], s["ctx"], s["scale"], softcap=c["softcap"],
                                  window=c["window"], alibi_slopes=s["slopes"], first_keys=s["first"],
                                  prefix_lens=s["prefix"], workspace=s["ws"], out=s["out"], lse=s["lse"])
    else:
        kp.paged_shared_prefix_attention(s["pool"], s["q"], s["tables"], s["ctx"], s["off"], s["blocks"], s["scale"],
                                         workspace=s["ws"], out=s["out"], lse=s["lse"])
    return s["out"], s["lse"]


def _norm_rope(x, w, table, pos, interleaved):
    """One row a head: x / rms(x) * w, then the first rope_dim numbers rotated in pairs."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    if table is None:
        return x
    half = table.shape[1] // 2
    cos, sin = table[pos][:, None, :half], table[pos][:, None, half:]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _store(pool, x, scale, blk, slot, fp8):
    x = (x / scale[:, None]).clamp(-448, 448) if fp8 else x
    bits = x.to(pool.dtype).view(torch.uint8 if fp8 else torch.int16)
    pool.view(bits.dtype)[blk, slot] = bits


def _plain_append(s):
    c = s["case"]
    seq, pos = s["at"]
    q = _norm_rope(s["q"], s["qw"], s["rope"], pos, c["interleaved"])
    k = _norm_rope(s["key"], s["kw"], s["rope"], pos, c["interleaved"])
    v = s["val"].float()
    blk = s["tables"][seq, pos // c["block_size"]].long()
    _store(s["k"], k, s["ks"], blk, pos % c["block_size"], c["fp8"])
    _store(s["v"], v, s["vs"], blk, pos % c["block_size"], c["fp8"])
    q = q.to(torch.bfloat16)
    if not c["tokens"]:
        q = q.view(c["batch"], c["q_len"], c["q_heads"], -1).transpose(1, 2).contiguous()
    return q, s["k"], s["v"]


def _gathered(s, pool, scale):
    """The cached rows of every sequence as fp32 [batch, tokens, kv_heads, head_dim]."""
    rows = pool.view(torch.uint8)[s["tables"].clamp(min=0).long()].view(pool.dtype).flatten(1, 2).float()
    return rows * scale[:, None] if s["case"]["fp8"] else rows


def _attend(s, score, seen):
    """softmax over the seen keys and the sum of values; rows that see none give 0 and -inf."""
    c = s["case"]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).nan_to_num(neginf=0.0)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    out = torch.einsum("bhgqt,bthd->bhgqd", p, _gathered(s, s["v"], s["vs"]))
    lse = (total.log() + top).squeeze(-1)
    shape = (c["batch"], c["q_heads"], c["q_len"])
    return out.reshape(*shape, -1).to(torch.bfloat16), lse.reshape(shape)


def _scores(s):
    c = s["case"]
    g = c["q_heads"] // c["kv_heads"]
    q = s["q"].float().view(c["batch"], c["kv_heads"], g, c["q_len"], -1)
    score = torch.einsum("bhgqd,bthd->bhgqt", q, _gathered(s, s["k"], s["ks"])) * s["scale"]
    t = torch.arange(score.shape[-1], device=DEV)
    pos = s["ctx"][:, None] - c["q_len"] + torch.arange(c["q_len"], device=DEV)
    return score, t, pos[:, None, None, :, None]


def _plain_masked(s):
    c = s["case"]
    score, t, pos = _scores(s)
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    if s["slopes"] is not None:
        slope = s["slopes"].view(1, c["kv_heads"], -1, 1, 1)
        score = score - slope * (pos - t).abs()
    seen = t <= pos
    each = lambda x: x[:, None, None, None, None]  # noqa: E731
    if s["prefix"] is not None:
        seen = seen | (t < each(torch.minimum(s["prefix"], s["ctx"])))
    if c["window"]:
        seen = seen & (t > pos - c["window"])
    if s["first"] is not None:
        seen = seen & (t >= each(s["first"]))
    return _attend(s, score, seen)


def _plain_prefix(s):
    score, t, pos = _scores(s)
    return _attend(s, score, t <= pos)


# --------------------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_append(s) if case["op"] == "norm_rope_append" else _exact_attention(s)


def _exact_append(s):
    c, d = s["case"], s["case"]["head_dim"]
    seq, pos = s["at"]

    def turned(x, w):
        y = x.double()
        if w is not None:
            y = y / ((y ** 2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
        z = y.clone()
        for i in range(c["rope_dim"] // 2):
            # the rotation by the table's own cosines and sines: they are an input
            co, si = s["rope"][pos, i].double()[:, None], s["rope"][pos, c["rope_dim"] // 2 + i].double()[:, None]
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + c["rope_dim"] // 2)
            z[..., a] = co * y[..., a] - si * y[..., b]
            z[..., b] = si * y[..., a] + co * y[..., b]
        return z

    q, k = turned(s["q"], s["qw"]), turned(s["key"], s["kw"])
    pools = []
    for pool, x, scale in ((s["k"], k, s["ks"]), (s["v"], s["val"].double(), s["vs"])):
        whole = pool.double()
        at = s["tables"][seq, torch.div(pos, c["block_size"], rounding_mode="floor")].long()
        whole[at, pos % c["block_size"]] = (x / scale.double()[:, None]).clamp(-448.0, 448.0) if c["fp8"] else x
        pools.append(whole)
    if not c["tokens"]:
        q = q.reshape(c["batch"], c["q_len"], c["q_heads"], d).permute(0, 2, 1, 3).contiguous()
    return q, pools[0], pools[1]


def _exact_attention(s):
    c = s["case"]
    hk, n, bs = c["kv_heads"], c["q_len"], c["block_size"]
    g = c["q_heads"] // hk
    out = torch.zeros(tuple(s["q"].shape), dtype=torch.float64, device=DEV)
    lse = torch.full(tuple(s["q"].shape[:3]), -math.inf, dtype=torch.float64, device=DEV)
    masked = c["op"] == "masked"
    for b, ctx in enumerate(s["ctx"].tolist()):
        if ctx <= 0:
            continue
        ids = s["tables"][b, :-(-ctx // bs)].long()
        k = s["k"][ids].double().reshape(-1, hk, c["head_dim"])[:ctx] * s["ks"].double()[:, None]
        v = s["v"][ids].double().reshape(-1, hk, c["head_dim"])[:ctx] * s["vs"].double()[:, None]
        at = torch.arange(ctx - n, ctx, device=DEV)[:, None]
        t = torch.arange(ctx, device=DEV)[None, :]
        hidden = t > at
        if masked:
            if s["prefix"] is not None:
                hidden = hidden & (t >= int(s["prefix"][b]))
            if c["window"]:
                hidden = hidden | (at - t >= c["window"])
            if s["first"] is not None:
                hidden = hidden | (t < int(s["first"][b]))
        for h in range(hk):
            x = s["q"][b, h * g:(h + 1) * g].double() @ k[:, h].T / math.sqrt(c["head_dim"])
            if masked and c["softcap"]:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            if masked and s["slopes"] is not None:
                x = x - s["slopes"][h * g:(h + 1) * g].double()[:, None, None] * (at - t).abs().double()
            x = torch.where(hidden, -math.inf, x)
            z = torch.logsumexp(x, -1)
            lse[b, h * g:(h + 1) * g] = z
            p = torch.where(hidden, 0.0, (x - torch.where(z > -math.inf, z, 0.0)[..., None]).exp())
            out[b, h * g:(h + 1) * g] = p @ v[:, h]
    return out, lse
