"""The operators that keep long contexts affordable, on real sizes: attention over a sliding window with a few first
tokens that stay visible, and a cache held in 4 bits (rows packed into it, blocks unpacked from it, attention over it).

`run` computes an operator in its plain form (elementary torch operations in 32 bits, in 64 where a value next to a
border decides), or with `own` through the calls of the package.  `exact` computes the same from the definition in 64
bits."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEVICE = "cuda"
GROUP = 64        # values of a row that share a scale and a zero point
ALL = 2147483647  # a window that hides nothing


# ------------------------------------------------------------------------------------------------ cases
def _window(name, batch, ctx, chunk, window, sinks, heads, head_dim, block_size, dtype):
    """ctx: inclusive range of the context lengths, the chunk among them; chunk: of the queries per sequence (None: one
    each, without query_start_loc)."""
    return dict(name=name, op="window", batch=batch, ctx_lo=ctx[0], ctx_hi=ctx[1], chunks=chunk is not None,
                new_lo=chunk[0] if chunk else 1, new_hi=chunk[1] if chunk else 1, window=window, sinks=sinks,
                q_heads=heads[0], kv_heads=heads[1], head_dim=head_dim, block_size=block_size, dtype=dtype)


def _q4(name, batch, ctx, heads, head_dim, block_size, dtype, window=ALL, sinks=0):
    return dict(name=name, op="q4", batch=batch, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=1, new_hi=1, window=window,
                sinks=sinks, q_heads=heads[0], kv_heads=heads[1], head_dim=head_dim, block_size=block_size, dtype=dtype)


def _store(name, batch, hist, new, kv_heads, head_dim, block_size, dtype):
    """new: inclusive range of the rows that each sequence packs; the blocks that they lie in are unpacked again."""
    return dict(name=name, op="store", batch=batch, hist_lo=hist[0], hist_hi=hist[1], new_lo=new[0], new_hi=new[1],
                kv_heads=kv_heads, head_dim=head_dim, block_size=block_size, dtype=dtype)


def _unpack(name, blocks, kv_heads, head_dim, block_size, dtype):
    return dict(name=name, op="unpack", blocks=blocks, kv_heads=kv_heads, head_dim=head_dim, block_size=block_size,
                dtype=dtype)


def listed():
    return [
        # one request on a small model: latency
        _window("window_one", 1, (1000, 1000), None, 256, 4, (12, 12), 64, 16, "fp16"),
        # the serving batch of the decode benchmark behind a window
        _window("window_serving", 64, (512, 4096), None, 1024, 4, (32, 8), 128, 16, "bf16"),
        # long documents behind a long window; what lies before it has been given back to the pool
        _window("window_long", 16, (32768, 131000), None, 8192, 64, (32, 8), 128, 16, "bf16"),
        # prompts in chunks
        _window("window_prompts", 8, (2048, 8192), (2048, 2048), 1024, 4, (32, 8), 128, 16, "bf16"),
        # single tokens beside chunks of uneven length on a small model
        _window("window_mixed", 24, (300, 2047), (1, 300), 500, 3, (12, 12), 64, 32, "fp16"),
        # one decode step of the serving batch packed
        _store("store_step", 64, (511, 4095), (1, 1), 8, 128, 16, "bf16"),
        # the prefill benchmark's chunk packed, and back as the values that the next chunk attends to
        _store("store_prompts", 128, (0, 1024), (256, 256), 8, 128, 32, "bf16"),
        # a short shared prefix of a small model unpacked for the next chunk
        _unpack("unpack_prefix", 33, 12, 64, 16, "fp16"),
        # the histories of a batch of prompts unpacked
        _unpack("unpack_histories", 5000, 8, 128, 16, "bf16"),
        # one request on a small model: latency
        _q4("q4_one", 1, (900, 900), (12, 12), 64, 16, "fp16"),
        # the serving batch of the decode benchmark
        _q4("q4_serving", 64, (512, 4096), (32, 8), 128, 16, "bf16"),
        # few requests with long documents
        _q4("q4_long", 4, (32768, 131000), (32, 8), 128, 16, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "q4", "q4", "q4", "store", "unpack"])
    kv, group = rng.choice([1, 2, 3, 4, 8, 12]), rng.choice([1, 2, 4, 8, 16])
    head_dim, block_size = rng.choice([64, 128]), rng.choice([16, 16, 32, 64, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    row = kv * head_dim * (4 if dtype == "fp32" else 2)  # bytes of one token's keys
    if op == "store":
        new_hi = _log(rng, 1, 2000)
        batch = max(1, min(_log(rng, 1, 128), int(6e7 / (row * new_hi))))
        c = _store("", batch, (0, _log(rng, 1, 4000)), (rng.choice([0, 1, new_hi]), new_hi), kv, head_dim, block_size, dtype)
    elif op == "unpack":
        c = _unpack("", max(1, min(_log(rng, 1, 5000), int(1.6e8 / (row * block_size)))), kv, head_dim, block_size, dtype)
    elif op == "q4":
        ctx_hi = _log(rng, 1, 65536)
        window, sinks = rng.choice([(ALL, 0), (ALL, 0), (_log(rng, 1, 8192), rng.choice([0, 1, 4, 33]))])
        seen = min(ctx_hi, window + sinks)
        batch = max(1, min(_log(rng, 1, 128), int((3e8 if dtype != "fp32" else 1e8) / (kv * head_dim * 1.125 * seen))))
        c = _q4("", batch, (rng.choice([1, ctx_hi // 2 + 1]), ctx_hi), (kv * group, kv), head_dim, block_size, dtype,
                window, sinks)
    else:
        ctx_hi = _log(rng, 1, 65536)
        window, sinks = _log(rng, 1, 8192), rng.choice([0, 1, 4, 16, 100])
        chunk = None
        most = 4e8 if dtype != "fp32" else 1e8  # bytes
        batch = min(_log(rng, 1, 128), int(most / (2 * row * min(ctx_hi, window + sinks))))
        if rng.random() < 0.5:
            # at most about 60 GFLOP (small blocks and single precision, off the tensor cores' fast path: 0.5)
            flops = 6e10 if dtype != "fp32" and block_size >= 16 else 5e8
            most = flops / (4 * head_dim * kv * group * min(ctx_hi, window + sinks))
            new_hi = max(1, min(_log(rng, 1, 2000), ctx_hi, int(most)))
            # (the plain form's scores: at most 6e8)
            keys = min(ctx_hi, window + sinks + new_hi)
            new_hi = max(1, min(new_hi, int(6e8 / (kv * group * keys))))
            batch = min(batch, int(most / new_hi), int(6e8 / (kv * group * keys * new_hi)))
            chunk = (rng.choice([1, new_hi // 2 + 1]), new_hi)
        c = _window("", max(1, batch), (rng.choice([chunk[1] if chunk else 1, ctx_hi]), ctx_hi), chunk, window, sinks,
                    (kv * group, kv), head_dim, block_size, dtype)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ inputs
def _rng(case, seed):
    return np.random.default_rng([seed, 78])


def _spread(case, what):
    """The lengths of a batch, evenly over their range: the same for every seed, which only shuffles them."""
    return np.rint(np.linspace(case[what + "_hi"], case[what + "_lo"], case["batch"])).astype(np.int64)


def _pairs_of_lengths(case):
    """Context and chunk lengths, the longest chunk in the longest context."""
    return np.maximum(_spread(case, "ctx"), _spread(case, "new")), _spread(case, "new")


def _int(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(DEVICE)


def _positions(case, ctx, new):
    """[sequence, place] positions that some query of the sequence sees, packed to the left, and whether there is one."""
    low = np.maximum(ctx - new + 1 - case["window"], 0)  # of the first query
    first = np.minimum(np.minimum(case["sinks"], low), ctx)
    place = np.arange(int((first + ctx - low).max()))[None, :]
    pos = np.where(place < first[:, None], place, place - first[:, None] + low[:, None])
    return pos, pos < ctx[:, None]


def _paged(case, ctx, new, rng):
    """A table whose entries are real where some query looks, and -1 elsewhere; the number of blocks."""
    bs, cap = case["block_size"], int(-(-ctx.max() // case["block_size"]))
    pos, real = _positions(case, ctx, new)
    used = np.zeros((case["batch"], cap), bool)
    used[np.nonzero(real)[0], pos[real] // bs] = True
    num_blocks = int(used.sum()) + 5
    table = np.full(used.shape, -1, np.int64)
    table[used] = rng.permutation(num_blocks)[:int(used.sum())]
    return table, num_blocks


def _rows(shape, dtype, g, keys):
    """Normal values; of keys, one channel in sixteen is far larger than the others."""
    x = torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)
    if keys:
        gain = torch.ones(shape[-2:], device=DEVICE, dtype=x.dtype)
        gain.view(-1)[::16] = 6.0
        x *= gain
    return x


def _pack(x):
    """The codes (two in a byte, the even dimension in the low half) and the (scale, zero) pairs of rows x[..., dim]:
    of every 64 values, scale = (largest - smallest) / 15 in bf16, zero = round(-smallest / scale), code = round(x /
    scale) + zero, with the smallest at most 0 and the largest at least 0."""
    v = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
    scale = (hi / 15 - lo / 15).to(torch.bfloat16)
    scale = torch.where(scale < 2.0 ** -126, 0, scale)
    step = torch.where(scale == 0, 1, scale).double()
    zero = torch.round(-lo / step).clamp(0, 15)
    code = (torch.round(v / step[..., None]) + zero[..., None]).clamp(0, 15)
    code, zero = torch.where(scale[..., None] == 0, 0, code), torch.where(scale == 0, 0, zero)
    code = code.to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.stack([scale, zero.to(torch.bfloat16)], -1).flatten(-2)


def _unpacked(codes, params, dtype):
    """The values that packed rows stand for, in 32 bits, and rounded to `dtype` where one is given."""
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, GROUP)).float()
    p = params.float().unflatten(-1, (-1, 2))
    v = (p[..., 0:1] * (code - p[..., 1:2])).flatten(-2)
    return v.to(dtype) if dtype else v


def _packed_pool(case, num_blocks, g, keys):
    return _pack(_rows((num_blocks, case["block_size"], case["kv_heads"], case["head_dim"]), torch.float32, g, keys))


def _empty_cache(case, num_blocks):
    shape = (num_blocks, case["block_size"], case["kv_heads"])
    codes = [torch.zeros(shape + (case["head_dim"] // 2,), dtype=torch.uint8, device=DEVICE) for _ in range(2)]
    params = [torch.zeros(shape + (case["head_dim"] // 32,), dtype=torch.bfloat16, device=DEVICE) for _ in range(2)]
    return (*codes, *params)


def prepare(case, seed):
    rng, g = _rng(case, seed), torch.Generator(device=DEVICE).manual_seed(seed)
    return {"window": _prepare_attention, "q4": _prepare_attention, "store": _prepare_store,
            "unpack": _prepare_unpack}[case["op"]](case, rng, g)


def _prepare_attention(case, rng, g):
    ctx, new = _pairs_of_lengths(case)
    order = rng.permutation(case["batch"])
    ctx, new = ctx[order], new[order]
    dtype = DTYPES[case["dtype"]]
    table, num_blocks = _paged(case, ctx, new, rng)
    s = dict(case=case, table=_int(table), ctx=_int(ctx), new=_int(new), qsl=None)
    if case["op"] == "q4":
        (kc, kp), (vc, vp) = _packed_pool(case, num_blocks, g, True), _packed_pool(case, num_blocks, g, False)
        s["cache"] = (kc, vc, kp, vp)
    else:
        shape = (num_blocks, case["block_size"], case["kv_heads"], case["head_dim"])
        s["k"], s["v"] = _rows(shape, dtype, g, True), _rows(shape, dtype, g, False)
        if case["chunks"]:
            s["qsl"] = _int(np.concatenate([[0], np.cumsum(new)]))
    # (queries of a size that leaves the scores of the large key channels in the range of a trained model's)
    s["q"] = 0.4 * torch.randn((int(new.sum()), case["q_heads"], case["head_dim"]), generator=g, device=DEVICE, dtype=dtype)
    s["out"] = torch.empty_like(s["q"])
    return s


def _prepare_store(case, rng, g):
    bs, batch = case["block_size"], case["batch"]
    hist, new = rng.permutation(_spread(case, "hist")), rng.permutation(_spread(case, "new"))
    first, end = hist // bs, -(-(hist + new) // bs)
    end = np.where(new == 0, first, end)
    num_blocks = int((end - first).sum()) + 3
    ids = rng.permutation(num_blocks)
    at = np.cumsum(end - first) - (end - first)
    seq = np.repeat(np.arange(batch), new)
    pos = hist[seq] + np.arange(seq.size) - (np.cumsum(new) - new)[seq]
    slots = ids[at[seq] + pos // bs - first[seq]] * bs + pos % bs
    dtype = DTYPES[case["dtype"]]
    used = num_blocks - 3
    rows = (seq.size, case["kv_heads"], case["head_dim"])
    pool = (used,) + (bs,) + rows[1:]
    return dict(case=case, k_new=_rows(rows, dtype, g, True), v_new=_rows(rows, dtype, g, False),
                slots=_int(slots, torch.int64), cache=_empty_cache(case, num_blocks),
                pairs=_int(np.stack([ids[:used], np.arange(used)], 1), torch.int64),
                k=torch.empty(pool, dtype=dtype, device=DEVICE), v=torch.empty(pool, dtype=dtype, device=DEVICE))


def _prepare_unpack(case, rng, g):
    n, dtype = case["blocks"], DTYPES[case["dtype"]]
    (kc, kp), (vc, vp) = _packed_pool(case, n + 7, g, True), _packed_pool(case, n + 7, g, False)
    pool = (n, case["block_size"], case["kv_heads"], case["head_dim"])
    return dict(case=case, cache=(kc, vc, kp, vp),
                pairs=_int(np.stack([rng.permutation(n + 7)[:n], rng.permutation(n)], 1), torch.int64),
                k=torch.empty(pool, dtype=dtype, device=DEVICE), v=torch.empty(pool, dtype=dtype, device=DEVICE))


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    return {"window": _run_window, "q4": _run_q4, "store": _run_store, "unpack": _run_unpack}[state["case"]["op"]](state)


def _run_window(s):
    case = s["case"]
    if own:
        import pagedattention_kv_cache_paged_gb300 as pa
        return pa.paged_attention_window(s["q"], s["qsl"], s["k"], s["v"], s["table"], s["ctx"], case["window"],
                                         case["sinks"], out=s["out"])
    return _plain_attention(s, lambda block, row: (s["k"][block, row].float(), s["v"][block, row].float()))


def _run_q4(s):
    case = s["case"]
    if own:
        import pagedattention_kv_cache_paged_gb300 as pa
        return pa.paged_attention_decode_q4(s["q"], pa.Q4Cache(*s["cache"]), s["table"], s["ctx"], window=case["window"],
                                            sinks=case["sinks"], out=s["out"])
    kc, vc, kp, vp = s["cache"]
    return _plain_attention(s, lambda block, row: (_unpacked(kc[block, row], kp[block, row], None),
                                                   _unpacked(vc[block, row], vp[block, row], None)))


def _plain_attention(s, rows_of):
    case = s["case"]
    bs, dim, kv, nodes = case["block_size"], case["head_dim"], case["kv_heads"], case["new_hi"]
    group, batch = case["q_heads"] // kv, case["batch"]
    window, sinks = case["window"], case["sinks"]
    ctx, new = s["ctx"].long(), s["new"].long()
    # positions that some query of a sequence sees, packed to the left
    low = (ctx - new + 1 - window).clamp(min=0)
    first = torch.minimum(low.clamp(max=sinks), ctx)
    most = min(case["ctx_hi"], sinks + window + nodes - 1)
    place = torch.arange(most, device=DEVICE)
    pos = torch.where(place < first[:, None], place, place - first[:, None] + low[:, None])
    real = pos < ctx[:, None]
    pos = torch.where(real, pos, 0)
    block = torch.gather(s["table"].long(), 1, torch.div(pos, bs, rounding_mode="floor")).clamp(min=0)
    k, v = (torch.where(real[:, :, None, None], x, 0.0).transpose(1, 2) for x in rows_of(block, pos % bs))
    # queries, padded to [batch, kv head, query * group, dim]
    start = torch.cumsum(new, 0) - new
    row = (start[:, None] + torch.arange(nodes, device=DEVICE)).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(batch, nodes, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, kv, -1, dim)
    at = (ctx - new)[:, None] + torch.arange(nodes, device=DEVICE)  # a query's position
    sees = real[:, None] & (pos[:, None] <= at[:, :, None]) & ((pos[:, None] > at[:, :, None] - window) |
                                                              (pos[:, None] < sinks))
    sees = sees[:, None, :, None].expand(-1, -1, -1, group, -1).reshape(batch, 1, -1, most)
    score = (q @ k.transpose(2, 3)) * dim ** -0.5
    score = torch.where(sees, score, float("-inf"))
    weight = torch.exp(score - score.amax(3, keepdim=True))
    out = (weight @ v) / weight.sum(3, keepdim=True)
    out = out.view(batch, kv, nodes, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, nodes, kv * group, dim)
    t = torch.arange(s["q"].shape[0], device=DEVICE)
    seq = torch.searchsorted(start + new, t, right=True)
    return out[seq, t - start[seq]].to(s["q"].dtype)


def _run_store(s):
    if own:
        import pagedattention_kv_cache_paged_gb300 as pa
        cache = pa.Q4Cache(*s["cache"])
        pa.paged_kv_write_q4(s["k_new"], s["v_new"], s["slots"], cache)
        pa.paged_kv_unpack_q4(cache, s["k"], s["v"], s["pairs"])
        return s["k"], s["v"]
    (kc, kp), (vc, vp) = _pack(s["k_new"]), _pack(s["v_new"])
    new = (kc, vc, kp, vp)
    block, row = torch.div(s["slots"], s["case"]["block_size"], rounding_mode="floor"), s["slots"] % s["case"]["block_size"]
    s["cache"][0][block, row], s["cache"][1][block, row] = new[0], new[1]
    s["cache"][2][block, row], s["cache"][3][block, row] = new[2], new[3]
    return _plain_unpack(s)


def _run_unpack(s):
    if own:
        import pagedattention_kv_cache_paged_gb300 as pa
        pa.paged_kv_unpack_q4(pa.Q4Cache(*s["cache"]), s["k"], s["v"], s["pairs"])
        return s["k"], s["v"]
    return _plain_unpack(s)


def _plain_unpack(s):
    src, dst = s["pairs"][:, 0], s["pairs"][:, 1]
    kc, vc, kp, vp = s["cache"]
    s["k"][dst] = _unpacked(kc[src], kp[src], s["k"].dtype)
    s["v"][dst] = _unpacked(vc[src], vp[src], s["v"].dtype)
    return s["k"], s["v"]


# ------------------------------------------------------------------------------------------------ what it takes
def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    head = case["kv_heads"] * case["head_dim"]
    packed = head // 2 + head // 16  # bytes of a token's keys in the cache
    if case["op"] == "unpack":
        tokens = case["blocks"] * case["block_size"]
        return {"bytes": 2 * tokens * (packed + head * size) + 16 * case["blocks"], "flops": 0}
    if case["op"] == "store":
        hist, new, bs = _spread(case, "hist"), _spread(case, "new"), case["block_size"]
        rows, blocks = int(new.sum()), int(np.where(new == 0, 0, -(-(hist % bs + new) // bs)).sum())
        # rows read, packed and written; their blocks read and written as values
        return {"bytes": rows * (2 * head * size + 2 * packed + 8) + 2 * blocks * bs * (packed + head * size) + 16 * blocks,
                "flops": 0}
    ctx, new = _pairs_of_lengths(case)
    keys = int(_positions(case, ctx, new)[1].sum())
    seen = 0
    for n, m in zip(ctx.tolist(), new.tolist()):
        p = np.arange(n - m, n)
        low = np.maximum(p + 1 - case["window"], 0)
        seen += int((p + 1 - low + np.minimum(low, case["sinks"])).sum())
    row = packed if case["op"] == "q4" else head * size
    return {"bytes": 2 * keys * row + 2 * int(new.sum()) * case["q_heads"] * case["head_dim"] * size
            + 4 * keys // case["block_size"], "flops": 4 * case["head_dim"] * case["q_heads"] * seen}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"window": _exact_attention, "q4": _exact_attention, "store": _exact_store, "unpack": _exact_unpack}[case["op"]](case, s)


def _values(codes, params):
    """scale * (code - zero) of packed rows, dimension by dimension."""
    out = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=codes.device)
    for d in range(out.shape[-1]):
        code = (codes[..., d // 2].int() >> (4 * (d % 2))) & 15
        out[..., d] = params[..., 2 * (d // GROUP)].double() * (code.double() - params[..., 2 * (d // GROUP) + 1].double())
    return out


def _exact_attention(case, s):
    bs, dim, kv = case["block_size"], case["head_dim"], case["kv_heads"]
    group = case["q_heads"] // kv
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
    t0 = 0
    for b in range(case["batch"]):
        n, m = int(s["ctx"][b]), int(s["new"][b])
        p = torch.arange(n - m, n, device=DEVICE)[:, None]
        j = torch.arange(n, device=DEVICE)
        j = j[(j < case["sinks"]) | (j > n - m - case["window"])]
        sees = (j <= p) & ((p - j < case["window"]) | (j < case["sinks"]))
        block, row = s["table"][b].long()[j // bs], j % bs
        for h in range(kv):
            if case["op"] == "q4":
                kc, vc, kp, vp = (x[block, row, h] for x in s["cache"])
                k, v = _values(kc, kp), _values(vc, vp)
            else:
                k, v = s["k"][block, row, h].double(), s["v"][block, row, h].double()
            q = s["q"][t0:t0 + m, h * group:(h + 1) * group].double()
            score = torch.einsum("mgd,nd->gmn", q, k) / math.sqrt(dim)
            weight = torch.softmax(score.masked_fill(~sees, float("-inf")), 2)
            out[t0:t0 + m, h * group:(h + 1) * group] = torch.einsum("gmn,nd->mgd", weight, v)
        t0 += m
    return out


def _exact_pack(x):
    """What rows are packed to, as values: from the definition, the grid point of every value by its distance to all
    sixteen (the nearer one; of two equally near ones the even quotient)."""
    x = x.double()
    out = torch.empty_like(x)
    for g in range(x.shape[-1] // GROUP):
        v = x[..., g * GROUP:(g + 1) * GROUP]
        lo, hi = v.amin(-1, keepdim=True).clamp(max=0.0), v.amax(-1, keepdim=True).clamp(min=0.0)
        # the scale's roundings are part of the definition: both quotients and their difference to 32 bits, then bf16
        scale = ((hi / 15).float().double() - (lo / 15).float().double()).float().bfloat16().double()
        none = scale < 2.0 ** -126
        scale = torch.where(none, 1.0, scale)
        q = torch.arange(-15, 16, device=x.device, dtype=torch.float64)
        q = q[torch.argsort(q % 2, stable=True)]  # the even ones first: argmin takes the first of equals

        def nearest(y):
            best = torch.full_like(y, float("inf"))
            at = torch.zeros_like(y)
            for i in q.tolist():
                d = (y - i * scale).abs()
                at = torch.where(d < best, i, at)
                best = torch.minimum(best, d)
            return at

        zero = nearest(-lo).clamp(0, 15)
        code = (nearest(v) + zero).clamp(0, 15)
        out[..., g * GROUP:(g + 1) * GROUP] = torch.where(none, 0.0, scale * (code - zero))
    return out


def _exact_store(case, s):
    bs, n = case["block_size"], s["pairs"].shape[0]
    out = []
    place = torch.full((n + 3,), -1, dtype=torch.int64, device=DEVICE)
    place[s["pairs"][:, 0]] = s["pairs"][:, 1]
    for new in (s["k_new"], s["v_new"]):
        pool = torch.zeros((n * bs, case["kv_heads"], case["head_dim"]), dtype=torch.float64, device=DEVICE)
        if new.numel():
            pool[place[s["slots"] // bs] * bs + s["slots"] % bs] = _exact_pack(new)
        out.append(pool.view(n, bs, case["kv_heads"], case["head_dim"]))
    return tuple(out)


def _exact_unpack(case, s):
    kc, vc, kp, vp = s["cache"]
    k, v = (torch.empty(s["k"].shape, dtype=torch.float64, device=DEVICE) for _ in range(2))
    k[s["pairs"][:, 1]] = _values(kc[s["pairs"][:, 0]], kp[s["pairs"][:, 0]])
    v[s["pairs"][:, 1]] = _values(vc[s["pairs"][:, 0]], vp[s["pairs"][:, 0]])
    return k, v
