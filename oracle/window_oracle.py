"""CPU oracle of the windowed attention and of the 4-bit cache.  TEST INFRASTRUCTURE ONLY (see paged_oracle.py).

Plain definitions: a two-pass softmax in float64 over exactly the positions a query sees; groups packed by comparing
every value with every point of their grid, in exact arithmetic."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch

from .paged_oracle import repeat_kv, slot_of, to_f64, to_int

GROUP = 64


def seen_positions(position: int, window: int, sinks: int) -> np.ndarray:
    """What a query at ``position`` attends to."""
    j = np.arange(position + 1)
    return j[(j > position - window) | (j < sinks)]


def attend(q, k, v, scale: float):
    """``(out, spread, size)`` of one query ``[Hq, D]`` over ``k, v [n, Hq, D]``: the attention, the sum of the absolute
    weighted values, and per head the largest sum of absolute products of a score."""
    with np.errstate(all="ignore"):
        z = scale * np.einsum("hd,nhd->hn", q, k)
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        return (np.einsum("hn,nhd->hd", p, v), np.einsum("hn,nhd->hd", p, np.abs(v)),
                (scale * np.einsum("hd,nhd->hn", np.abs(q), np.abs(k))).max(1))


def window_attention(q, query_start_loc, k_pool, v_pool, block_table, context_lens, scale: float, window: int,
                     sinks: int):
    """``(rows, out, spread, size)`` (see :func:`attend`) of the query rows that belong to a sequence; None for
    ``query_start_loc``: one query per sequence."""
    qf, lens = to_f64(q), to_int(context_lens)
    qsl = np.arange(lens.size + 1) if query_start_loc is None else to_int(query_start_loc)
    k_flat, v_flat = (to_f64(p).reshape(-1, *p.shape[2:]) for p in (k_pool, v_pool))
    S, n_rep = int(k_pool.shape[1]), qf.shape[1] // int(k_pool.shape[2])
    rows, res = [], []
    for b in range(lens.size):
        m, n = int(qsl[b + 1] - qsl[b]), int(lens[b])
        table = to_int(block_table[b])
        for r in range(m):
            row = int(qsl[b]) + r
            rows.append(row)
            if n == 0:
                res.append((np.zeros(qf.shape[1:]), np.zeros(qf.shape[1:]), np.zeros(qf.shape[1])))
                continue
            slots = [slot_of(table, int(j), S) for j in seen_positions(n - m + r, window, sinks)]
            res.append(attend(qf[row], repeat_kv(k_flat[slots], n_rep), repeat_kv(v_flat[slots], n_rep), scale))
    out, spread, size = (np.array(x) for x in zip(*res))
    return np.array(rows, int), out, spread, size


def _nearest(x: Fraction, s: Fraction) -> int:
    """x / s rounded to the nearest whole number, halves to the even one."""
    q = x / s
    low = q.numerator // q.denominator
    rest = q - low
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and low % 2):
        low += 1
    return low


def pack_group(x) -> tuple:
    """(codes, scale, zero) of 64 values."""
    x = [float(v) for v in x]
    if not all(np.isfinite(x)):
        return [0] * len(x), float("nan"), 0
    lo, hi = min(0.0, *x), max(0.0, *x)
    f32 = np.float32
    r = f32(1) / f32(15)
    scale = float(torch.tensor(f32(hi) * r - f32(lo) * r).to(torch.bfloat16))
    if scale < 2.0 ** -126:
        return [0] * len(x), 0.0, 0
    s = Fraction(scale)
    zero = min(max(_nearest(Fraction(-lo), s), 0), 15)
    return [min(max(_nearest(Fraction(v), s) + zero, 0), 15) for v in x], scale, zero


def q4_pack(x):
    """(codes uint8 ``[.., D / 2]``, params float64 ``[.., D / 32]``) of rows ``x [.., D]``."""
    xf = to_f64(x)
    lead, D = xf.shape[:-1], xf.shape[-1]
    codes, params = np.zeros(lead + (D,), np.uint8), np.zeros(lead + (D // 32,))
    for at in np.ndindex(lead):
        for g in range(D // GROUP):
            c, s, z = pack_group(xf[at][g * GROUP:(g + 1) * GROUP])
            codes[at][g * GROUP:(g + 1) * GROUP] = c
            params[at][2 * g:2 * g + 2] = s, z
    return codes[..., 0::2] | (codes[..., 1::2] << 4), params


def q4_values(codes, params) -> np.ndarray:
    """The float64 values that codes ``[.., D / 2]`` and params ``[.., D / 32]`` stand for."""
    c, p = to_int(codes).astype(np.int64), to_f64(params)
    D = 2 * c.shape[-1]
    both = np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], D // GROUP, GROUP)
    s, z = p[..., 0::2, None], p[..., 1::2, None]
    with np.errstate(all="ignore"):
        return (s * (both - z)).reshape(*c.shape[:-1], D)
