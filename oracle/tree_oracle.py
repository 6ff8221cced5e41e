"""CPU oracle of the drafted-tree calls.  TEST INFRASTRUCTURE ONLY (see paged_oracle.py).

Plain definitions: a step's index arrays sequence by sequence and token by token; tree attention as a
two-pass softmax in float64 over exactly the keys a node sees; the accepted rows moved one by one."""
from __future__ import annotations

import numpy as np

from .paged_oracle import gather_history, repeat_kv, to_f64, to_int


def ancestors(parents, j: int) -> list:
    """Node ``j`` and its ancestors in a tree given by ``parents`` (-1: the history)."""
    seen = [j]
    while parents[seen[-1]] >= 0:
        seen.append(int(parents[seen[-1]]))
    return seen


def step_tables(history_lens, new_lens, block_table, block_counts, free_blocks, free_count: int, block_size: int,
                tokens: int, parents=None, mask_words: int = 0) -> dict:
    """A step's tables for a batch in which every sequence fits."""
    hist, new = to_int(history_lens), to_int(new_lens)
    table, counts, free = to_int(block_table).copy(), to_int(block_counts).copy(), to_int(free_blocks)
    par = None if parents is None else to_int(parents)
    qsl, ctx = [0], []
    slots, pos = np.full(tokens, -1, np.int64), np.zeros(tokens, np.int64)
    mask = np.zeros((tokens, mask_words), np.uint64)
    for b in range(hist.size):
        while counts[b] * block_size < hist[b] + new[b]:
            free_count -= 1
            table[b, counts[b]] = free[free_count]
            counts[b] += 1
        for j in range(int(new[b])):
            t, p = qsl[-1] + j, int(hist[b]) + j
            slots[t] = table[b, p // block_size] * block_size + p % block_size
            pos[t] = p
            if par is not None:
                line = ancestors(par[qsl[-1]:], j)
                pos[t] = hist[b] + len(line) - 1
                for s in line:
                    mask[t, s // 64] |= np.uint64(1) << np.uint64(s % 64)
        qsl.append(qsl[-1] + int(new[b]))
        ctx.append(int(hist[b] + new[b]))
    return dict(block_table=table, block_counts=counts, free_count=free_count, query_start_loc=np.array(qsl),
                context_lens=np.array(ctx), slot_mapping=slots, positions=pos, tree_mask=mask.view(np.int64))


def sees(mask, row: int, m: int, r: int) -> np.ndarray:
    """Which of a sequence's ``m`` nodes its node ``r`` (query row ``row``) sees; ``mask`` None: a chain."""
    if mask is None:
        return np.arange(m) <= r
    words = to_int(mask)[row].view(np.uint64)
    s = np.arange(m)
    return ((words[s // 64] >> (s % 64).astype(np.uint64)) & np.uint64(1)).astype(bool)


def paged_tree_attention(q, query_start_loc, mask, k_pool, v_pool, block_table, context_lens, scale: float):
    """``(rows, out, spread)``: the query rows that belong to a sequence, their outputs, and per output the
    sum of the absolute weighted values and per row and head the largest sum of absolute products of a
    score (what rounding errors scale with), all float64."""
    qf, qsl, lens = to_f64(q), to_int(query_start_loc), to_int(context_lens)
    S, Hkv = int(k_pool.shape[1]), int(k_pool.shape[2])
    Hq, D = qf.shape[1:]
    rows, out, spread, size = [], [], [], []
    for b in range(lens.size):
        m, n = int(qsl[b + 1] - qsl[b]), int(lens[b])
        if m == 0:
            continue
        k = repeat_kv(gather_history(k_pool, block_table[b], n, S), Hq // Hkv)
        v = repeat_kv(gather_history(v_pool, block_table[b], n, S), Hq // Hkv)
        for r in range(m):
            row = int(qsl[b]) + r
            see = np.concatenate([np.ones(n - m, bool), sees(mask, row, m, r)])
            rows.append(row)
            if not see.any():
                out.append(np.zeros((Hq, D)))
                spread.append(np.zeros((Hq, D)))
                size.append(np.zeros(Hq))
                continue
            ks, vs = k[see], v[see]
            with np.errstate(all="ignore"):
                z = scale * np.einsum("hd,nhd->hn", qf[row], ks)
                p = np.exp(z - z.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                out.append(np.einsum("hn,nhd->hd", p, vs))
                spread.append(np.einsum("hn,nhd->hd", p, np.abs(vs)))
                size.append((abs(scale) * np.einsum("hd,nhd->hn", np.abs(qf[row]), np.abs(ks))).max(1))
    return np.array(rows, int), np.array(out), np.array(spread), np.array(size)


def paged_kv_accept(k_pool, v_pool, accepted, accepted_lens, history_lens, block_table):
    """Copies of the pools (one layer) with the accepted rows moved, one after the other."""
    k, v = k_pool.clone(), v_pool.clone()
    S = int(k.shape[1])
    acc, n, hist, table = (to_int(x) for x in (accepted, accepted_lens, history_lens, block_table))
    for b in range(n.size):
        for i in range(int(n[b])):
            src, dst = int(hist[b] + acc[b, i]), int(hist[b]) + i
            for pool in (k, v):
                pool[table[b, dst // S], dst % S] = pool[table[b, src // S], src % S].clone()
    return k, v
