"""The speculative-serving operators on real sizes: step tables from request lengths, attention of a drafted tree over
the paged cache, and keeping the accepted rows.

`run` computes an operator in its plain form (elementary torch operations in 32 bits), or with `own` through the calls
of the package.  `exact` computes the same from the definition in 64 bits."""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEVICE = "cuda"


# ------------------------------------------------------------------------------------------------ cases
def _tables(name, batch, hist, new, block_size, max_blocks, tokens, words):
    """hist, new: inclusive ranges of the lengths; tokens: rows of the padded token arrays; words: 64-node words of the
    tree mask (0: no trees)."""
    return dict(name=name, op="tables", batch=batch, hist_lo=hist[0], hist_hi=hist[1], new_lo=new[0], new_hi=new[1],
                block_size=block_size, max_blocks=max_blocks, tokens=tokens, words=words)


def _tree(name, batch, ctx, nodes, heads, head_dim, block_size, dtype, words, peaked=False):
    """ctx: inclusive range of the history lengths; nodes: of the tree sizes; words 0: chains instead of trees."""
    return dict(name=name, op="tree", batch=batch, hist_lo=ctx[0], hist_hi=ctx[1], new_lo=nodes[0], new_hi=nodes[1],
                q_heads=heads[0], kv_heads=heads[1], head_dim=head_dim, block_size=block_size, dtype=dtype, words=words,
                peaked=peaked)


def _accept(name, batch, layers, nodes, accepted, kv_heads, head_dim, block_size, dtype, hist):
    return dict(name=name, op="accept", batch=batch, layers=layers, nodes=nodes, acc_lo=accepted[0], acc_hi=accepted[1],
                kv_heads=kv_heads, head_dim=head_dim, block_size=block_size, dtype=dtype, hist_lo=hist[0],
                hist_hi=hist[1])


def listed():
    return [
        # one plain decode step of a handful of requests: a call that is all latency
        _tables("tables_decode", 4, (100, 900), (1, 1), 16, 64, 4, 0),
        # one speculative step of a full serving batch, trees of up to 16 drafted tokens, padded token arrays
        _tables("tables_drafts", 64, (512, 4096), (1, 16), 16, 260, 1024, 1),
        # wide trees of two mask words
        _tables("tables_wide_trees", 256, (1, 2000), (60, 128), 32, 128, 32768, 2),
        # the prompts of a large offline batch at once
        _tables("tables_prompts", 2048, (0, 0), (1, 1000), 16, 64, 1100000, 0),
        # one request with a short draft on a small model: latency
        _tree("tree_one", 1, (120, 128), (5, 5), (12, 12), 64, 16, "fp16", 1),
        # a small model's batch with uneven contexts
        _tree("tree_small_batch", 8, (1, 2048), (1, 26), (12, 12), 64, 16, "fp16", 1),
        # the serving batch of the decode benchmark, each request with a draft of up to 16
        _tree("tree_serving", 64, (512, 4080), (8, 16), (32, 8), 128, 16, "bf16", 1),
        # the same with trees as wide as one mask word
        _tree("tree_serving_wide", 64, (512, 4030), (48, 64), (32, 8), 128, 16, "bf16", 1),
        # few requests with long documents, some keys far above the rest
        _tree("tree_long", 4, (32768, 131000), (24, 32), (32, 8), 128, 16, "bf16", 1, True),
        # single precision, odd sizes
        _tree("tree_single", 16, (17, 1001), (1, 23), (8, 2), 64, 16, "fp32", 1),
        # one accepted draft in one layer of a small model
        _accept("accept_one", 1, 1, 8, (3, 3), 12, 64, 16, "fp16", (100, 120)),
        # the accepted drafts of the serving batch in all layers
        _accept("accept_serving", 64, 32, 16, (1, 8), 8, 128, 16, "bf16", (16, 200)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tables", "accept"])
    if op == "tables":
        batch, block_size = _log(rng, 1, 1024), rng.choice([16, 32, 64])
        words = rng.choice([0, 1, 2])
        new_hi = rng.randint(1, 64 * words) if words else _log(rng, 1, 900)
        hist_hi = _log(rng, 1, 4000)
        c = _tables("", batch, (0, hist_hi), (rng.choice([0, 1]), new_hi), block_size,
                    -(-(hist_hi + new_hi) // block_size) + 2, batch * new_hi + rng.randint(0, 64), words)
    elif op == "accept":
        nodes = rng.randint(2, 64)
        c = _accept("", _log(rng, 1, 64), _log(rng, 1, 32), nodes, (0, rng.randint(1, min(nodes, 16))),
                    rng.choice([1, 2, 8, 12]), rng.choice([64, 128]), rng.choice([16, 32]),
                    rng.choice(["bf16", "fp16", "fp32"]), (0, rng.randint(1, 200)))
    else:
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        kv, group = rng.choice([1, 2, 4, 8, 12]), rng.choice([1, 2, 4, 8, 16])
        head_dim = rng.choice([64, 128])
        hist_hi = _log(rng, 16, 32768)
        nodes = _log(rng, 1, 128 if dtype != "fp32" else 32)
        # at most about 400 MB of keys and values and 30 GFLOP (single precision: 2)
        keys = min(4e8 / (4 * kv * head_dim), (3e10 if dtype != "fp32" else 2e9) / (4 * kv * group * head_dim * nodes))
        batch = max(1, min(64, int(keys / (hist_hi + nodes))))
        words = rng.choice([0, 1, 1]) * -(-nodes // 64)
        c = _tree("", batch, (rng.choice([0, 1, hist_hi]), hist_hi), (rng.choice([1, nodes]), nodes), (kv * group, kv),
                  head_dim, rng.choice([16, 32, 64]), dtype, words, rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ inputs
def _rng(case, seed):
    return np.random.default_rng([seed, 77])


def _spread(case, what):
    """The lengths of a batch, evenly over their range: the same for every seed, which only shuffles them."""
    return np.rint(np.linspace(case[what + "_hi"], case[what + "_lo"], case["batch"])).astype(np.int64)


def _lengths(case, rng):
    return rng.permutation(_spread(case, "hist")), rng.permutation(_spread(case, "new"))


def _blocks(lengths, block_size):
    return int((-(-lengths // block_size)).sum())


def _parents(rng, new, rows):
    """Parents of every drafted token, numbered inside its own tree; -1 hangs on the history.  Half of the nodes
    continue the node before them, so that trees have some depth."""
    within = np.arange(int(new.sum())) - np.repeat(np.cumsum(new) - new, new)
    parent = np.where(rng.random(within.size) < 0.5, within - 1,
                      np.floor(rng.random(within.size) * (within + 1)).astype(np.int64) - 1)
    out = np.full(rows, -1, np.int64)
    out[:within.size] = parent
    return out


def _mask_words(parent, new, words):
    """Ancestor-or-self bits of every drafted token as signed 64-bit words, built node by node."""
    out = np.zeros((int(new.sum()), words), np.uint64)
    first = np.cumsum(new) - new
    start = np.repeat(first, new)
    within = np.arange(out.shape[0]) - start
    for j in range(int(new.max()) if new.size else 0):  # all trees' j-th nodes at once
        rows = np.nonzero(within == j)[0]
        p = parent[rows]
        has = p >= 0
        out[rows[has]] = out[start[rows[has]] + p[has]]
        out[rows, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


def _int(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(DEVICE)


def prepare(case, seed):
    return {"tables": _prepare_tables, "tree": _prepare_tree, "accept": _prepare_accept}[case["op"]](case, seed)


def _prepare_tables(case, seed):
    rng = _rng(case, seed)
    hist, new = _lengths(case, rng)
    batch, bs, cap = case["batch"], case["block_size"], case["max_blocks"]
    held = np.minimum(-(-hist // bs) + (rng.random(batch) < 0.2), cap)  # some rows still hold a spare block
    num_blocks = _blocks(hist, bs) + _blocks(new, bs) + batch + 8
    ids = rng.permutation(num_blocks)
    table = np.full((batch, cap), -1, np.int64)
    table[np.arange(cap)[None, :] < held[:, None]] = ids[:int(held.sum())]
    free = np.zeros(num_blocks, np.int64)
    n_free = num_blocks - int(held.sum())
    free[:n_free] = ids[int(held.sum()):]
    s = dict(case=case, hist=_int(hist), new=_int(new), table=_int(table), counts=_int(held), free=_int(free),
             free_state=_int([n_free, 0]), num_blocks=num_blocks, parents=None)
    if case["words"]:
        s["parents"] = _int(_parents(rng, new, case["tokens"]))
    t = case["tokens"]
    s["qsl"] = torch.zeros(batch + 1, dtype=torch.int32, device=DEVICE)
    s["ctx"] = torch.zeros(batch, dtype=torch.int32, device=DEVICE)
    s["slots"] = torch.zeros(t, dtype=torch.int64, device=DEVICE)
    s["pos"] = torch.zeros(t, dtype=torch.int32, device=DEVICE)
    s["mask"] = torch.zeros((t, case["words"]), dtype=torch.int64, device=DEVICE) if case["words"] else None
    return s


def _prepare_tree(case, seed):
    rng = _rng(case, seed)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    hist, new = _lengths(case, rng)
    bs, dtype = case["block_size"], DTYPES[case["dtype"]]
    used = -(-(hist + new) // bs)
    cap = int(-(-(case["hist_hi"] + case["new_hi"]) // bs))
    num_blocks = _blocks(hist, bs) + _blocks(new, bs) + 5
    table = np.full((case["batch"], cap), -1, np.int64)
    table[np.arange(cap)[None, :] < used[:, None]] = rng.permutation(num_blocks)[:int(used.sum())]
    shape = (num_blocks, bs, case["kv_heads"], case["head_dim"])
    k = torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)
    v = torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)
    if case["peaked"]:  # one key in a hundred far above the rest
        big = torch.rand(num_blocks * bs, generator=g, device=DEVICE) < 0.01
        k.view(num_blocks * bs, -1).mul_(torch.where(big, 8.0, 1.0).to(dtype)[:, None])
    total = int(new.sum())
    q = torch.randn((total, case["q_heads"], case["head_dim"]), generator=g, device=DEVICE, dtype=dtype)
    s = dict(case=case, q=q, k=k, v=v, table=_int(table), ctx=_int(hist + new),
             qsl=_int(np.concatenate([[0], np.cumsum(new)])), mask=None, out=torch.empty_like(q))
    if case["words"]:
        s["mask"] = _int(_mask_words(_parents(rng, new, total), new, case["words"]), torch.int64)
    return s


def _prepare_accept(case, seed):
    rng = _rng(case, seed)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    batch, bs, dtype = case["batch"], case["block_size"], DTYPES[case["dtype"]]
    hist, n_acc = rng.permutation(_spread(case, "hist")), rng.permutation(_spread(case, "acc"))
    order = np.argsort(rng.random((batch, case["nodes"])), axis=1)[:, :case["acc_hi"]]
    acc = np.full((batch, case["acc_hi"]), -1, np.int64)
    keep = np.arange(case["acc_hi"])[None, :] < n_acc[:, None]
    acc[keep] = np.sort(np.where(keep, order, case["nodes"]), axis=1)[keep]
    used = -(-(hist + case["nodes"]) // bs)
    cap = int(-(-(case["hist_hi"] + case["nodes"]) // bs))
    num_blocks = _blocks(hist, bs) + batch * -(-case["nodes"] // bs) + 3
    table = np.full((batch, cap), -1, np.int64)
    table[np.arange(cap)[None, :] < used[:, None]] = rng.permutation(num_blocks)[:int(used.sum())]
    shape = (case["layers"], num_blocks, bs, case["kv_heads"], case["head_dim"])
    k = torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)
    v = torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)
    return dict(case=case, k=k, v=v, acc=_int(acc), n_acc=_int(n_acc), hist=_int(hist), table=_int(table))


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    return {"tables": _run_tables, "tree": _run_tree, "accept": _run_accept}[state["case"]["op"]](state)


def _run_tables(s):
    if own:
        import pagedattention_kv_cache_paged_gb300 as pa
        pa.build_block_tables(s["hist"], s["new"], s["table"], s["counts"], s["free"], s["free_state"],
                              s["case"]["block_size"], s["num_blocks"], parents=s["parents"],
                              out=pa.StepTables(s["qsl"], s["ctx"], s["slots"], s["pos"], s["mask"]))
    else:
        _plain_tables(s)
    return {n: s[n] for n in ("table", "counts", "free_state", "qsl", "ctx", "slots", "pos", "mask")}


def _plain_tables(s):
    bs, words, tokens = s["case"]["block_size"], s["case"]["words"], s["case"]["tokens"]
    hist, new, counts, table = s["hist"].long(), s["new"].long(), s["counts"].long(), s["table"]
    ctx = hist + new
    ends = torch.cumsum(new, 0)
    held = torch.maximum(torch.div(ctx + bs - 1, bs, rounding_mode="floor"), counts)
    taken = torch.cumsum(held - counts, 0)
    col = torch.arange(table.shape[1], device=DEVICE)[None, :]
    fresh = (col >= counts[:, None]) & (col < held[:, None])
    at = s["free_state"][0].long() - 1 - ((taken - (held - counts))[:, None] + col - counts[:, None])
    table.copy_(torch.where(fresh, s["free"][at.clamp(0, s["free"].numel() - 1)], table))
    t = torch.arange(tokens, device=DEVICE)
    seq = torch.searchsorted(ends, t, right=True)
    real = seq < hist.numel()
    seq = seq.clamp(max=hist.numel() - 1)
    j = t - (ends - new)[seq]
    p = torch.where(real, hist[seq] + j, 0)
    block = table[seq, torch.div(p, bs, rounding_mode="floor")].long()
    s["slots"].copy_(torch.where(real, block * bs + p % bs, -1))
    if words:
        n = 64 * words
        reach = torch.zeros((hist.numel(), n, n), device=DEVICE)  # one step up, and staying
        jj = torch.where(real, j, 0)
        parent = s["parents"].long()
        reach.index_put_((seq, jj, parent.clamp(min=0)), (real & (parent >= 0)).float(), accumulate=True)
        reach = ((reach + torch.eye(n, device=DEVICE)) > 0).float()
        for _ in range(6 + words.bit_length()):  # 1, 2, 4, ... steps up
            reach = ((reach @ reach) > 0).float()
        rows = reach[seq, jj] * real[:, None]
        p = torch.where(real, hist[seq] + rows.sum(1).long() - 1, 0)
        bits = rows.long().view(tokens, words, 64) << torch.arange(64, device=DEVICE)
        s["mask"].copy_(bits.sum(2))
    s["pos"].copy_(p)
    s["qsl"][1:] = ends
    s["qsl"][0] = 0
    s["ctx"].copy_(ctx)
    s["counts"].copy_(held)
    s["free_state"][0] -= taken[-1]


def _run_tree(s):
    if own:
        import pagedattention_kv_cache_paged_gb300 as pa
        return pa.paged_attention_tree(s["q"], s["qsl"], s["mask"], s["k"], s["v"], s["table"], s["ctx"],
                                       max_nodes=s["case"]["new_hi"], out=s["out"])
    return _plain_tree(s)


def _plain_tree(s):
    case = s["case"]
    bs, nodes, dim, kv = case["block_size"], case["new_hi"], case["head_dim"], case["kv_heads"]
    group = case["q_heads"] // kv
    total, batch, cap = s["q"].shape[0], case["batch"], s["table"].shape[1] * bs
    ctx, qsl = s["ctx"].long(), s["qsl"].long()
    new = qsl[1:] - qsl[:-1]
    hist = ctx - new
    # queries, padded to [batch, kv head, node * group, dim]
    row = (qsl[:-1, None] + torch.arange(nodes, device=DEVICE)).clamp(max=total - 1)
    q = s["q"][row].float().view(batch, nodes, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, kv, -1, dim)
    # keys and values of the whole rows of the table, nothing where the context ends
    key = torch.arange(cap, device=DEVICE)
    inside = key < ctx[:, None]
    block = s["table"].long().clamp(min=0)
    k = torch.where(inside[:, :, None, None], s["k"][block].view(batch, cap, kv, dim).float(), 0.0).transpose(1, 2)
    v = torch.where(inside[:, :, None, None], s["v"][block].view(batch, cap, kv, dim).float(), 0.0).transpose(1, 2)
    # which keys a node sees: its history, and its ancestors and itself
    node = key[None, :] - hist[:, None]
    if s["mask"] is None:
        sees = node[:, None, :] <= torch.arange(nodes, device=DEVICE)[None, :, None]
    else:
        words = s["mask"][row]
        at = node.clamp(0, 64 * words.shape[2] - 1)
        word = torch.gather(words, 2, torch.div(at, 64, rounding_mode="floor")[:, None, :].expand(-1, nodes, -1))
        sees = (node < 0)[:, None, :] | (((word >> (at % 64)[:, None, :]) & 1) == 1)
    sees = (sees & inside[:, None, :])[:, None, :, None, :].expand(-1, -1, -1, group, -1).reshape(batch, 1, -1, cap)
    score = (q @ k.transpose(2, 3)) * dim ** -0.5
    score = torch.where(sees, score, float("-inf"))
    weight = torch.exp(score - score.amax(3, keepdim=True))
    out = (weight @ v) / weight.sum(3, keepdim=True)
    out = out.view(batch, kv, nodes, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, nodes, kv * group, dim)
    t = torch.arange(total, device=DEVICE)
    seq = torch.searchsorted(qsl[1:], t, right=True)
    return out[seq, t - qsl[seq]].to(s["q"].dtype)


def _run_accept(s):
    if own:
        import pagedattention_kv_cache_paged_gb300 as pa
        pa.paged_kv_accept(s["k"], s["v"], s["acc"], s["n_acc"], s["hist"], s["table"])
    else:
        bs, (batch, most) = s["case"]["block_size"], s["acc"].shape
        i = torch.arange(most, device=DEVICE)[None, :]
        keep = i < s["n_acc"][:, None]
        seq = torch.arange(batch, device=DEVICE)[:, None].expand(-1, most)[keep]
        src = (s["hist"][:, None] + s["acc"])[keep].long()
        dst = (s["hist"][:, None] + i)[keep].long()
        src_block, dst_block = s["table"][seq, src // bs].long(), s["table"][seq, dst // bs].long()
        k, v = s["k"][:, src_block, src % bs], s["v"][:, src_block, src % bs]
        s["k"][:, dst_block, dst % bs] = k
        s["v"][:, dst_block, dst % bs] = v
    return s["k"], s["v"]


# ------------------------------------------------------------------------------------------------ what it takes
def work(case):
    if case["op"] == "accept":
        rows = int(_spread(case, "acc").sum()) * case["layers"]
        return {"bytes": 4 * rows * case["kv_heads"] * case["head_dim"] * (4 if case["dtype"] == "fp32" else 2),
                "flops": 0}
    hist, new = _spread(case, "hist"), _spread(case, "new")
    total = int(new.sum())
    if case["op"] == "tables":
        fresh = total / case["block_size"]  # block ids read from the free list and written to the table
        per_token = 12 + (8 * case["words"])
        return {"bytes": case["tokens"] * per_token + (4 * total if case["words"] else 0) + 24 * case["batch"] + 8 * fresh,
                "flops": 0}
    size = 4 if case["dtype"] == "fp32" else 2
    keys = int(hist.sum()) + total
    sees = int(hist.sum()) * new.mean() + (new ** 1.5).sum()  # ancestors: about the root of the tree's size
    return {"bytes": (2 * keys * case["kv_heads"] + 2 * total * case["q_heads"]) * case["head_dim"] * size
            + 4 * keys / case["block_size"] + 8 * case["words"] * total,
            "flops": 4 * case["head_dim"] * case["q_heads"] * sees}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "tree": _exact_tree, "accept": _exact_accept}[case["op"]](case, s)


def _exact_tables(case, s):
    n = {k: s[k].cpu().numpy().copy() for k in ("hist", "new", "table", "counts", "free", "free_state")}
    bs, tokens, words = case["block_size"], case["tokens"], case["words"]
    parents = s["parents"].cpu().numpy() if words else None
    qsl, ctx = [0], []
    slots, pos = np.full(tokens, -1, np.int64), np.zeros(tokens, np.int64)
    mask = np.zeros((tokens, words), np.uint64)
    for b in range(case["batch"]):
        h, m = int(n["hist"][b]), int(n["new"][b])
        while n["counts"][b] * bs < h + m:
            n["free_state"][0] -= 1
            n["table"][b, n["counts"][b]] = n["free"][n["free_state"][0]]
            n["counts"][b] += 1
        t0, p = qsl[-1], np.arange(h, h + m)
        slots[t0:t0 + m] = n["table"][b, p // bs].astype(np.int64) * bs + p % bs
        pos[t0:t0 + m] = p
        for j in range(m if words else 0):
            up, depth = j, -1
            while up >= 0:
                mask[t0 + j, up // 64] |= np.uint64(1) << np.uint64(up % 64)
                up, depth = int(parents[t0 + up]), depth + 1
            pos[t0 + j] = h + depth
        qsl.append(t0 + m)
        ctx.append(h + m)
    i32 = np.int32
    return dict(table=n["table"], counts=n["counts"], free_state=n["free_state"], qsl=np.array(qsl, i32),
                ctx=np.array(ctx, i32), slots=slots, pos=pos.astype(i32), mask=mask.view(np.int64) if words else None)


def _exact_tree(case, s):
    bs, dim, kv = case["block_size"], case["head_dim"], case["kv_heads"]
    group = case["q_heads"] // kv
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEVICE)
    qsl, ctx = s["qsl"].tolist(), s["ctx"].tolist()
    for b in range(case["batch"]):
        t0, t1, n = qsl[b], qsl[b + 1], ctx[b]
        m = t1 - t0
        if m == 0:
            continue
        ids = s["table"][b, :-(-n // bs)].long()
        sees = torch.ones((m, n), dtype=torch.bool, device=DEVICE)
        if s["mask"] is None:
            sees[:, n - m:] = torch.ones((m, m), device=DEVICE).tril() > 0
        else:
            word = s["mask"][t0:t1].cpu().numpy().view(np.uint64)
            bit = np.arange(m, dtype=np.uint64)
            sees[:, n - m:] = torch.from_numpy((word[:, np.arange(m) // 64] >> (bit % np.uint64(64))) & np.uint64(1) > 0)
        for h in range(kv):
            k = s["k"][ids, :, h].reshape(-1, dim)[:n].double()
            v = s["v"][ids, :, h].reshape(-1, dim)[:n].double()
            q = s["q"][t0:t1, h * group:(h + 1) * group].double()
            score = torch.einsum("mgd,nd->gmn", q, k) / math.sqrt(dim)
            weight = torch.softmax(score.masked_fill(~sees, float("-inf")), 2)
            out[t0:t1, h * group:(h + 1) * group] = torch.einsum("gmn,nd->mgd", weight, v)
    return out


def _exact_accept(case, s):
    bs = case["block_size"]
    k, v = s["k"].double(), s["v"].double()
    table, acc, hist, n_acc = (s[x].tolist() for x in ("table", "acc", "hist", "n_acc"))
    for b in range(case["batch"]):
        for i in range(n_acc[b]):  # upward: a row is read before a later one is put in its place
            src, dst = hist[b] + acc[b][i], hist[b] + i
            for pool in (k, v):
                pool[:, table[b][dst // bs], dst % bs] = pool[:, table[b][src // bs], src % bs]
    return k, v
