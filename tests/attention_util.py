"""A paged cache of shuffled blocks with known contents, and attention over it in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

import paged_kv_cache_19_gb300 as kp
from gpu_util import i32

POISON = 0xFF          # a NaN in bf16 and in e4m3: slots that nothing should use


class Cache:
    """Batch of sequences in one pool.  shared: per group (members, leading blocks they share);
    slots at or past a sequence's context, and blocks of nobody, are poisoned."""

    def __init__(self, *, ctx, hq, hk, d, bs, fp8=False, q_len=1, shared=None, seed=0, spare=3, q_scale=1.0):
        r = np.random.default_rng(seed)
        self.ctx = np.asarray(ctx)
        B = len(self.ctx)
        self.B, self.hq, self.hk, self.d, self.bs, self.fp8, self.q_len = B, hq, hk, d, bs, fp8, q_len
        self.scale = d ** -0.5
        self.offsets = self.blocks = None
        nb = -(-self.ctx // bs)
        own = np.zeros(B, int)                 # leading blocks that are the group's
        group = np.arange(B)
        if shared is not None:
            sizes = [m for m, _ in shared]
            assert sum(sizes) == B
            self.offsets = np.concatenate([[0], np.cumsum(sizes)])
            self.blocks = np.array([n for _, n in shared])
            group = np.repeat(np.arange(len(sizes)), sizes)
            own = self.blocks[group]
            nb = np.maximum(nb, own)
        self.max_blocks = max(1, int(nb.max()))
        self.tab = np.full((B, self.max_blocks), -1)
        total, seen = 0, {}
        for b in range(B):
            if group[b] not in seen:
                seen[group[b]] = total
                total += own[b]
            self.tab[b, :own[b]] = seen[group[b]] + np.arange(own[b])
            n = nb[b] - own[b]
            self.tab[b, own[b]:nb[b]] = total + np.arange(n)
            total += n
        self.nb = total + spare
        perm = r.permutation(self.nb)
        self.tab = np.where(self.tab >= 0, perm[np.maximum(self.tab, 0)], -1)
        self.pool = kp.kv_pool_create(self.nb, bs, hk, d, "fp8_e4m3" if fp8 else "bf16")
        self.ks = self.vs = np.ones(hk)
        if fp8:
            self.ks, self.vs = (r.uniform(0.008, 0.02, hk).astype(np.float32) for _ in range(2))
            self.pool.set_scales(self.ks, self.vs)
        k, v, _, _ = self.pool.tensors()
        used = torch.zeros(self.nb, bs, dtype=torch.bool)
        for b in range(B):
            for j in range(nb[b]):
                n = bs if j < own[b] else int(np.clip(self.ctx[b] - j * bs, 0, bs))
                used[self.tab[b, j], :n] = True
        for t, raw, s in zip((k, v), self.pool.raw_bytes(), (self.ks, self.vs)):
            x = torch.from_numpy(r.standard_normal((self.nb, bs, hk, d)).astype(np.float32))
            if fp8:
                x = (x / torch.from_numpy(s)[:, None]).clamp(-448, 448)
            t.copy_(x.to(t.dtype))
            raw[(~used).cuda()] = POISON
        self.k = k.float().cpu().double().numpy() * np.asarray(self.ks)[:, None]
        self.v = v.float().cpu().double().numpy() * np.asarray(self.vs)[:, None]
        q = torch.from_numpy(r.standard_normal((B, hq, q_len, d)) * q_scale).to(torch.bfloat16)
        self.q64 = q.double().numpy()
        self.q = q.cuda()
        self.tables, self.lens = i32(self.tab), i32(self.ctx)

    def reference(self, hide=None, softcap=0.0, slopes=None):
        """(out, sum p|v|, lse, largest |score|) in 64 bits; hide(b, pos [q,1], t [1,n]) -> keys a
        query does not see beside the future ones (returned mask replaces the causal one)."""
        shape = self.q64.shape
        out, size = np.zeros(shape), np.zeros(shape)
        lse, top = np.full(shape[:3], -np.inf), np.zeros(shape[:3])
        g = self.hq // self.hk
        for b in range(self.B):
            n = int(self.ctx[b])
            if n <= 0:
                continue
            t = np.arange(n)
            blk, slot = self.tab[b, t // self.bs], t % self.bs
            pos = (n - self.q_len + np.arange(self.q_len))[:, None]
            hidden = hide(b, pos, t[None]) if hide is not None else t[None] > pos
            dead = hidden.all(0)                       # keys nobody sees may hold anything
            kb, vb = self.k[blk, slot], self.v[blk, slot]
            kb, vb = np.where(dead[:, None, None], 0.0, kb), np.where(dead[:, None, None], 0.0, vb)
            for h in range(self.hq):
                x = self.q64[b, h] @ kb[:, h // g].T * self.scale
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                if slopes is not None:
                    x = x - float(slopes[h]) * np.abs(pos - t[None])
                x = np.where(hidden, -np.inf, x)
                m = x.max(1, keepdims=True)
                some = np.isfinite(m[:, 0])
                p = np.exp(x - np.where(np.isfinite(m), m, 0.0))
                p = np.where(hidden, 0.0, p)
                z = p.sum(1)
                w = p / np.where(z > 0, z, 1.0)[:, None]
                out[b, h] = w @ vb[:, h // g]
                size[b, h] = w @ np.abs(vb[:, h // g])
                lse[b, h, some] = np.log(z[some]) + m[some, 0]
                top[b, h] = np.abs(np.where(hidden, 0.0, x)).max(1)
        return out, size, lse, top

    def check(self, got, got_lse, ref):
        """Per number: the probabilities are rounded once to bf16 or fp16 (half a step, 2^-8 of
        each, so 2^-8 of sum p|v|) and the output once to bf16 (2^-8 of it); the scores' fp32 sums
        of d <= 128 products are off by at most 128 2^-24 sum|q k| scale, under 2^-13 for these
        numbers, which moves a probability by as much.  The capped and biased scores carry 2^-20
        of themselves."""
        out, size, lse, top = ref
        o = got.double().cpu().numpy().reshape(out.shape)
        slack = 2.0 ** -12 + 2.0 ** -19 * top
        bound = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + slack[..., None]) * size + 1e-7
        bad = ~(np.abs(o - out) <= bound)
        assert not bad.any(), (np.argwhere(bad)[:3], np.abs(o - out).max())
        if got_lse is not None:
            s = got_lse.double().cpu().numpy().reshape(lse.shape)
            live = np.isfinite(lse)
            assert (s[~live] == -np.inf).all()
            off = np.abs(s[live] - lse[live])
            assert (off <= slack[live]).all(), off.max()


SHARE_TOKENS = 2048    # what a group has to save, (members - 1) x shared tokens, to be computed once


def sharing(offsets, blocks, bs):
    """Indexes of the groups that the shared pass computes."""
    n = np.diff(np.asarray(offsets))
    return [g for g in range(len(n)) if n[g] >= 2 and blocks[g] > 0 and (n[g] - 1) * blocks[g] * bs >= SHARE_TOKENS]
