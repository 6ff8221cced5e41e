"""Inputs of the drafted-tree tests, and the bound their outputs are held to."""
import numpy as np
import torch


def random_parents(rng, new):
    """A tree for every sequence: each node hangs on the history or on a node before it."""
    return np.array([rng.integers(-1, j) if rng.random() < 0.6 else j - 1 for m in new for j in range(m)], np.int64)


def mask_of(parents, new, words, tail=0):
    """Ancestor-or-self words of the nodes, with `tail` rows of ones behind them (never to be read)."""
    total = int(sum(new))
    out = np.zeros((total + tail, words), np.uint64)
    t0 = 0
    for m in new:
        for j in range(m):
            p = parents[t0 + j]
            if p >= 0:
                out[t0 + j] = out[t0 + p]
            out[t0 + j, j // 64] |= np.uint64(1) << np.uint64(j % 64)
        t0 += m
    out[total:] = ~np.uint64(0)
    return torch.from_numpy(out.view(np.int64))


class TreeCase:
    """History lengths `hist` and tree sizes `new`; every pool row that holds no token is NaN."""

    def __init__(self, seed, hist, new, *, q_heads, kv_heads, head_dim, block_size, dtype, words=1, tail=0, gain=1.0,
                 unified=False):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        n = [h + m for h, m in zip(hist, new)]
        used = [-(-x // block_size) for x in n]
        self.num_blocks = sum(used) + 3
        cap = max(max(used), 1) + 1
        ids = torch.randperm(self.num_blocks, generator=g)
        self.table = torch.full((len(n), cap), -1, dtype=torch.int32)
        shape = (self.num_blocks, block_size, kv_heads, head_dim)
        if unified:
            pool = torch.full((self.num_blocks, 2) + shape[1:], float("nan")).to(dtype)
            self.k, self.v = pool[:, 0], pool[:, 1]
            self.pool = pool
        else:
            self.k, self.v = (torch.full(shape, float("nan")).to(dtype) for _ in range(2))
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = ids[at:at + u].to(torch.int32)
            for j in range(n[b]):
                blk = int(self.table[b, j // block_size])
                self.k[blk, j % block_size] = (gain * torch.randn(shape[2:], generator=g)).to(dtype)
                self.v[blk, j % block_size] = torch.randn(shape[2:], generator=g).to(dtype)
            at += u
        total = sum(new)
        self.q = torch.randn((total + tail, q_heads, head_dim), generator=g).to(dtype)
        self.qsl = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
        self.ctx = torch.tensor(n, dtype=torch.int32)
        self.hist, self.new, self.block_size = list(hist), list(new), block_size
        self.mask = mask_of(random_parents(rng, new), new, words, tail) if words else None
        self.scale = head_dim ** -0.5
        self.dtype = dtype

    def row_of(self, b, j):
        """(block, token) of position j of sequence b."""
        return int(self.table[b, j // self.block_size]), j % self.block_size

    def device(self):
        if hasattr(self, "pool"):
            p = self.pool.cuda()
            k, v = p[:, 0], p[:, 1]
        else:
            k, v = self.k.cuda(), self.v.cuda()
        return dict(q=self.q.cuda(), query_start_loc=self.qsl.cuda(),
                    tree_mask=None if self.mask is None else self.mask.cuda(), k_pool=k, v_pool=v,
                    block_table=self.table.cuda(), context_lens=self.ctx.cuda())


def bound(dtype, ref, spread, size, keys: int, head_dim: int, values: float, tensor_cores: bool):
    """How far an output may be from the 64-bit one.

    Output: half a step of the result.  Score: a dot product of head_dim products in 32 bits is off by
    head_dim + 2 half steps of its absolute products (`size`, natural-log units; the scale and the log2
    domain are two of them), the exponential's argument by one more and the exponential itself by 2^-22;
    a weight is off by that relative amount, in the numerator and in the denominator.  Sums over the
    keys: keys + 16 half steps (partitions and warps add a few).  Tensor cores also round each weight to
    the pool's type (half a step; in fp16 at least 2^-25, the half step of the smallest numbers, of
    weights whose largest is 1 or more)."""
    u32 = 2.0 ** -24
    rel = 2 * ((head_dim + 4) * u32 * size[:, :, None] + 2.0 ** -22) + 2 * (keys + 16) * u32
    half = torch.finfo(dtype).eps / 2
    tol = half * np.abs(ref) + spread * rel + 1e-30
    if tensor_cores:
        tol = tol + spread * half * (1 + half)
        if dtype == torch.float16:
            tol = tol + keys * 2.0 ** -25 * values
    return tol * (1 + half)
