"""Inputs of the windowed-attention and 4-bit-cache tests, and the bound their outputs are held to."""
import numpy as np
import torch

import oracle

ALL = 2 ** 31 - 1


def int32(x):
    return torch.tensor(x, dtype=torch.int32)


class WindowCase:
    """Contexts `ctx`, the last `new` positions of each queried (None: one, without query_start_loc).  Pool rows that no
    query sees are NaN, table entries of blocks that none sees are -1, and `tail` rows of queries belong to nobody."""

    def __init__(self, seed, ctx, new, window, sinks, *, q_heads, kv_heads, head_dim, block_size, dtype, tail=0,
                 unified=False, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        m = [1] * len(ctx) if new is None else list(new)
        low = [max(n - x + 1 - window, 0) for n, x in zip(ctx, m)]
        seen = [[j for j in range(n) if j < min(sinks, lo) or j >= lo] if x else [] for n, x, lo in zip(ctx, m, low)]
        used = [sorted({j // block_size for j in s}) for s in seen]
        self.num_blocks = sum(map(len, used)) + 3
        cap = max(max((-(-n // block_size) for n in ctx), default=1), 1) + 1
        ids = torch.randperm(self.num_blocks, generator=g).tolist()
        self.table = torch.full((len(ctx), cap), -1, dtype=torch.int32)
        rows = (self.num_blocks, block_size, kv_heads, head_dim)
        if unified:
            self.pool = torch.full((self.num_blocks, 2) + rows[1:], float("nan")).to(dtype)
            self.k, self.v = self.pool[:, 0], self.pool[:, 1]
        else:
            self.k, self.v = (torch.full(rows, float("nan")).to(dtype) for _ in range(2))
        self.block_size, self.dtype, self.window, self.sinks = block_size, dtype, window, sinks
        self.ctx_list, self.new_list, self.seen = list(ctx), m, seen
        for b, blocks in enumerate(used):
            for j in blocks:
                self.table[b, j] = ids.pop()
            if not seen[b]:
                continue
            at = np.array(seen[b])
            blk, tok = self.table[b, at // block_size].long(), torch.from_numpy(at % block_size)
            self.k[blk, tok] = (gain * torch.randn((at.size,) + rows[2:], generator=g)).to(dtype)
            self.v[blk, tok] = torch.randn((at.size,) + rows[2:], generator=g).to(dtype)
        total = sum(m)
        self.q = torch.randn((total + tail, q_heads, head_dim), generator=g).to(dtype)
        self.qsl = None if new is None else int32(np.concatenate([[0], np.cumsum(m)]))
        self.ctx = int32(list(ctx))
        self.scale = head_dim ** -0.5

    def row_of(self, b, j):
        return int(self.table[b, j // self.block_size]), j % self.block_size

    def device(self):
        if hasattr(self, "pool"):
            p = self.pool.cuda()
            k, v = p[:, 0], p[:, 1]
        else:
            k, v = self.k.cuda(), self.v.cuda()
        return dict(q=self.q.cuda(), query_start_loc=None if self.qsl is None else self.qsl.cuda(), k_pool=k, v_pool=v,
                    block_table=self.table.cuda(), context_lens=self.ctx.cuda())

    def oracle(self):
        return oracle.window.window_attention(self.q, self.qsl, self.k, self.v, self.table, self.ctx, self.scale,
                                              self.window, self.sinks)

    def most_seen(self):
        return max(max(map(len, self.seen), default=0), 1)


def bound(dtype, ref, spread, size, keys, head_dim, weight, floor=0.0):
    """How far an output may be from the 64-bit one.

    Output: half a step of the result, and below the type's smallest normal number, where all numbers lie eps * tiny
    apart, half of that.  Score: a dot product of head_dim products in 32 bits is off by head_dim + 4
    half steps of its absolute products (`size`, natural-log units; the scale and the log2 domain are two of them), the
    exponential's argument by one more and the exponential itself by 2^-22; a weight is off by that relative amount, in
    the numerator and in the denominator.  Sums over the keys: keys + 16 half steps (partitions and warps add a few).
    `weight`: how far a weight is rounded for the product with V, relative; `floor`: absolutely, times the values."""
    u32 = 2.0 ** -24
    rel = 2 * ((head_dim + 4) * u32 * size[:, :, None] + 2.0 ** -22) + 2 * (keys + 16) * u32 + weight * (1 + weight)
    half = torch.finfo(dtype).eps / 2
    return (half * np.maximum(np.abs(ref), torch.finfo(dtype).tiny) + spread * rel + floor + 1e-30) * (1 + half)


def pool_bound(case, ref, spread, size, cuda_cores=False):
    """The bound of paged_attention_window: tensor cores round weights to the pool's type (in fp16 by at least 2^-25)."""
    weight = 0.0 if case.dtype == torch.float32 or cuda_cores else torch.finfo(case.dtype).eps / 2
    finite = case.v[torch.isfinite(case.v)].double().abs()
    floor = case.most_seen() * 2.0 ** -25 * float(finite.max()) if weight and case.dtype == torch.float16 and finite.numel() else 0.0
    return bound(case.dtype, ref, spread, size, case.most_seen(), case.q.shape[2], weight, floor)


def pack(rows):
    """(codes, params) of rows [.., D] on the CPU, packed as the format says, 64 values at a time in float64 (the oracle's
    exact form is for small inputs; this one agrees with it on these, which a test checks)."""
    x = rows.double().unflatten(-1, (-1, 64))
    lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    f = lambda t: t.float().double()  # noqa: E731
    r = float(np.float32(1) / np.float32(15))  # (a product of two fp32 numbers is exact in 64 bits)
    s = f(f(hi * r) - f(lo * r)).to(torch.bfloat16).double()
    bad = ~torch.isfinite(x).all(-1)
    none = s < 2.0 ** -126
    step = torch.where(none | bad, 1.0, s)
    z = torch.round(-lo / step).clamp(0, 15)
    c = (torch.round(x / step[..., None]) + z[..., None]).clamp(0, 15)
    z, c = torch.where(none | bad, 0.0, z), torch.where((none | bad)[..., None], 0.0, c)
    s = torch.where(bad, float("nan"), torch.where(none, 0.0, s))
    c = c.to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([s, z], -1).flatten(-2).to(torch.bfloat16)


class PackedCase(WindowCase):
    """The same for the 4-bit cache: rows that no query sees have scale NaN."""

    def __init__(self, seed, ctx, window, sinks, *, dtype, **kw):
        super().__init__(seed, ctx, None, window, sinks, dtype=torch.float32, **kw)
        (self.kc, self.kp), (self.vc, self.vp) = pack(self.k), pack(self.v)
        self.q, self.dtype = self.q.to(dtype), dtype

    def cache(self, pa):
        return pa.Q4Cache(self.kc.cuda(), self.vc.cuda(), self.kp.cuda(), self.vp.cuda())

    def device(self):
        return dict(q=self.q.cuda(), block_table=self.table.cuda(), context_lens=self.ctx.cuda())

    def oracle(self):
        k, v = (torch.from_numpy(oracle.window.q4_values(c, p)) for c, p in ((self.kc, self.kp), (self.vc, self.vp)))
        rows, ref, spread, _ = oracle.window.window_attention(self.q, None, k, v, self.table, self.ctx, self.scale,
                                                              self.window, self.sinks)
        # what the score's sums are made of: query values times codes, and times zeros (fp32: times code - zero)
        top = 15 if self.dtype == torch.float32 else 2 * 15
        q = self.q.double().abs().unflatten(-1, (-1, 64)).sum(-1).numpy()  # [B, Hq, groups]
        scales = np.zeros(q.shape)
        group = q.shape[1] // self.kp.shape[2]
        for b, at in enumerate(self.seen):
            for j in at:
                s = self.kp[self.row_of(b, j)][:, 0::2].double().numpy()
                scales[b] = np.fmax(scales[b], np.repeat(s, group, 0))
        return rows, ref, spread, self.scale * (q * scales * top).sum(-1)

    def bound(self, ref, spread, size):
        # weight * scale: three parts of bf16, each half a step of what the one before left; or fp16, half a step, at least
        # 2^-25 of numbers whose largest scale counts 2^5 or more: times codes of at most 15, for every key
        if self.dtype == torch.float32:
            return bound(self.dtype, ref, spread, size, self.most_seen(), self.q.shape[2], 2.0 ** -24)
        scales = torch.nan_to_num(self.vp[..., 0::2].double(), nan=0.0)
        floor = self.most_seen() * 2.0 ** -30 * 15 * float(scales.max())
        return bound(self.dtype, ref, spread, size, self.most_seen(), self.q.shape[2], 2.0 ** -11, floor)
