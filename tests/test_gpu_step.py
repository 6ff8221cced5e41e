"""GPU parity of build_block_tables and paged_kv_accept (whole numbers and bit copies: equal to the
oracle's), and a run of the speculative step's calls together."""
import numpy as np
import pytest
import torch

import oracle
from tree_cases import random_parents

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean(cuda_lib):
    cuda_lib.device_error_flags(clear=True)
    yield
    cuda_lib.set_checked_mode(False)
    cuda_lib.device_error_flags(clear=True)


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32)


class State:
    """Tables of a batch with histories `hist`; `spare` more blocks than needed in some rows."""

    def __init__(self, seed, hist, new, block_size, cap=None, words=0, tail=0, spare=False, extra=3):
        rng = np.random.default_rng(seed)
        self.hist, self.new, self.S = list(hist), list(new), block_size
        B = len(hist)
        held = [-(-h // block_size) for h in hist]
        if spare:
            held = [c + int(rng.integers(0, 3)) for c in held]
        need = [max(0, -(-(h + m) // block_size) - c) for h, m, c in zip(hist, new, held)]
        self.num_blocks = sum(held) + sum(need) + extra
        self.cap = cap or max([c + n for c, n in zip(held, need)] + [1]) + 1
        ids = rng.permutation(self.num_blocks)
        self.table = torch.full((B, self.cap), -1, dtype=torch.int32)
        at = 0
        for b, c in enumerate(held):
            self.table[b, :c] = i32(ids[at:at + c])
            at += c
        self.counts = i32(held)
        self.free = torch.zeros(self.num_blocks, dtype=torch.int32)
        self.free[:self.num_blocks - at] = i32(ids[at:])
        self.state = i32([self.num_blocks - at, 0])
        self.tokens = sum(new) + tail
        self.words = words
        self.parents = None
        if words:
            self.parents = i32(np.concatenate([random_parents(rng, new), np.full(tail, 12345)]))

    def device(self):
        d = {k: getattr(self, k).cuda() for k in ("table", "counts", "free", "state")}
        d["parents"] = None if self.parents is None else self.parents.cuda()
        d["hist"], d["new"] = i32(self.hist).cuda(), i32(self.new).cuda()
        return d

    def build(self, pa, d, **kw):
        return pa.build_block_tables(d["hist"], d["new"], d["table"], d["counts"], d["free"], d["state"], self.S,
                                     self.num_blocks, num_tokens=self.tokens, parents=d["parents"],
                                     mask_words=self.words if self.words else None, **kw)

    def check(self, pa, d, out):
        ref = oracle.tree.step_tables(self.hist, self.new, self.table, self.counts, self.free, int(self.state[0]),
                                      self.S, self.tokens, self.parents, self.words)
        torch.cuda.synchronize()
        assert pa.device_error_flags() == 0
        for name in ("query_start_loc", "context_lens", "slot_mapping", "positions"):
            assert np.array_equal(getattr(out, name).cpu().numpy(), ref[name]), name
        if self.words:
            assert np.array_equal(out.tree_mask.cpu().numpy(), ref["tree_mask"])
        assert np.array_equal(d["table"].cpu().numpy(), ref["block_table"])
        assert np.array_equal(d["counts"].cpu().numpy(), ref["block_counts"])
        assert d["state"].cpu().tolist() == [ref["free_count"], 0]


@pytest.mark.parametrize("S", [1, 2, 16, 64, 256])
@pytest.mark.parametrize("words", [0, 1, 3])
@pytest.mark.parametrize("spare", [False, True])
def test_tables(cuda_lib, S, words, spare):
    hist = [0, 1, 15, 16, 17, 31, 32, 33, 255, 256, 257, 0, 700]
    new = [5, 1, 1, 1, 0, 1, 17, 64, 1, 30, 2, 0, 63]
    if words == 3:
        new[3], new[6] = 192, 129
    st = State(S + words, hist, new, S, words=words, tail=9, spare=spare)
    d = st.device()
    st.check(cuda_lib, d, st.build(cuda_lib, d))


@pytest.mark.parametrize("batch", [1, 2, 31, 1023, 1024, 1025, 2048, 3000])
@pytest.mark.parametrize("words", [0, 1])
def test_batches_across_the_chunks(cuda_lib, batch, words):
    rng = np.random.default_rng(batch)
    st = State(batch, rng.integers(0, 90, batch), rng.integers(0, 12, batch), 16, words=words, tail=5, spare=True)
    d = st.device()
    st.check(cuda_lib, d, st.build(cuda_lib, d))


@pytest.mark.parametrize("words", [0, 2])
@pytest.mark.parametrize("tail", [0, 20000])
def test_many_tokens_over_several_blocks(cuda_lib, words, tail):
    """Token ranges of several thread blocks that begin and end inside sequences; a sequence longer than
    a range; empty sequences at the borders."""
    rng = np.random.default_rng(4)
    new = [0, 0, 100] + list(rng.integers(0, 128, 700)) + [0, 0]
    if not words:
        new += [30000, 0, 9000]
    hist = rng.integers(0, 3000, len(new))
    st = State(5, hist, new, 16, words=words, tail=tail, spare=True)
    d = st.device()
    out = st.build(cuda_lib, d)
    st.check(cuda_lib, d, out)
    # the next step over the same arrays: the rows hold all they need by now
    st.table, st.counts, st.state = (d[k].cpu() for k in ("table", "counts", "state"))
    before = st.table.clone()
    st.check(cuda_lib, d, st.build(cuda_lib, d, out=out))
    assert torch.equal(d["table"].cpu(), before)


def test_every_sequence_empty(cuda_lib):
    st = State(1, [0, 5, 64], [0, 0, 0], 16, tail=4)
    d = st.device()
    st.check(cuda_lib, d, st.build(cuda_lib, d))
    st = State(1, [0, 5, 64], [0, 0, 0], 16, tail=0)
    d = st.device()
    st.check(cuda_lib, d, st.build(cuda_lib, d))


@pytest.mark.parametrize("many", [False, True])
def test_sequences_that_do_not_fit_get_nothing(cuda_lib, many):
    pa = cuda_lib
    pad = [3] * 1500 if many else []  # several thread blocks

    def run(hist, new, flag, which, words=0, **change):
        st = State(7, hist + [2] * len(pad), new + pad, 16, tail=5, words=words)
        d = st.device()
        for k, v in change.items():
            if k == "free":
                d["state"][0] = v
            else:
                d[{"m": "new", "h": "hist", "count": "counts"}[k]][1] = v
        before = {k: d[k].clone() for k in ("table", "counts", "state")}
        out = st.build(pa, d)
        torch.cuda.synchronize()
        assert pa.device_error_flags() == flag
        qsl = out.query_start_loc.cpu().tolist()
        for b in range(len(hist)):
            rows = slice(max(0, qsl[b]), qsl[b + 1])
            if b in which:
                assert (out.slot_mapping[rows] == -1).all() and (out.positions[rows] == 0).all()
                assert int(out.context_lens[b]) == 0
                assert torch.equal(d["table"][b], before["table"][b])
                assert int(d["counts"][b]) == int(before["counts"][b])
            else:
                assert (out.slot_mapping[rows] >= 0).all()
                assert int(out.context_lens[b]) == hist[b] + new[b]
        assert int(d["state"][1]) == 0
        took = int((d["counts"] - before["counts"]).sum())
        assert int(d["state"][0]) == max(int(before["state"][0]), 0) - took
        pa.set_checked_mode(True)
        d2 = st.device()
        for k in ("hist", "new", "parents"):
            d2[k] = d[k]
        for k, v in before.items():
            d2[k] = v
        with pytest.raises(pa.PagedAttnError) as e:
            st.build(pa, d2)
        assert e.value.status == pa.PA_ERANGE
        pa.set_checked_mode(False)

    hist, new = [20, 40, 16], [3, 30, 20]
    run(hist, new, pa.PA_DEVERR_CONTEXT_LEN, [1], m=-4)
    run(hist, new, pa.PA_DEVERR_CONTEXT_LEN, [1], h=-1)
    run(hist, new, pa.PA_DEVERR_CONTEXT_LEN | pa.PA_DEVERR_BLOCK_ID, [1], h=2 ** 31 - 1)
    run(hist, new, pa.PA_DEVERR_BLOCK_ID, [1], count=2)
    run(hist, new, pa.PA_DEVERR_BLOCK_ID, [1], count=77)
    if not many:
        run(hist, new, pa.PA_DEVERR_NO_BLOCKS, [1, 2], free=1)  # needs 0, 2 and 2 blocks
        run(hist, new, pa.PA_DEVERR_NO_BLOCKS, [2], free=3)
        run(hist, new, pa.PA_DEVERR_NO_BLOCKS, [1, 2], free=-5)
    run(hist, [3, 65, 20], pa.PA_DEVERR_TREE, [1], words=1)


def test_bad_parents_and_free_blocks_are_recorded(cuda_lib):
    pa = cuda_lib
    st = State(9, [20, 40], [3, 5], 16, words=1)
    for node, parent in ((1, 1), (1, 2), (2, -2), (0, 0), (2, 2 ** 31 - 1)):
        d = st.device()
        d["parents"][3 + node] = parent
        out = st.build(pa, d)
        assert pa.device_error_flags() == pa.PA_DEVERR_TREE
        assert int(out.positions[3 + node]) == 40 and int(out.tree_mask[3 + node, 0]) == 1 << node
    st = State(9, [16, 40], [3, 30], 16)
    d = st.device()
    d["free"][int(st.state[0]) - 1] = st.num_blocks
    out = st.build(pa, d)
    assert pa.device_error_flags() == pa.PA_DEVERR_BLOCK_ID
    assert (out.slot_mapping[:3] == -1).all() and int(d["table"][0, 1]) == -1
    assert (out.slot_mapping[3:] >= 0).all()


def test_tokens_past_the_arrays(cuda_lib):
    pa = cuda_lib
    st = State(9, [16, 40, 3], [3, 30, 5], 16)
    st.tokens = 20
    d = st.device()
    before = d["counts"].clone()
    out = st.build(pa, d)
    assert pa.device_error_flags() == pa.PA_DEVERR_QUERY_LOC
    assert out.context_lens.cpu().tolist() == [19, 0, 0] and out.query_start_loc.cpu().tolist() == [0, 3, 33, 38]
    assert (out.slot_mapping[:3] >= 0).all() and (out.slot_mapping[3:] == -1).all()
    assert torch.equal(d["counts"][1:], before[1:])


@pytest.mark.parametrize("tokens", [64, 30000])
def test_a_captured_step_advances(cuda_lib, tokens):
    """The same graph replayed: each replay grows the histories and takes blocks as it goes."""
    pa = cuda_lib
    B, S = 8, 16
    st = State(3, [0] * B, [0] * B, S, cap=40, extra=400)
    st.tokens = tokens
    d = st.device()
    out = st.build(pa, d)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        st.build(pa, d, out=out)
        d["hist"].copy_(out.context_lens)
    rng = np.random.default_rng(1)
    hist = [0] * B
    for _ in range(12):
        new = rng.integers(0, 9, B)
        d["new"].copy_(i32(new))
        st.hist, st.new = hist, list(new)
        st.table, st.counts, st.state, st.free = (d[k].cpu() for k in ("table", "counts", "state", "free"))
        g.replay()
        st.check(pa, d, out)
        hist = [h + int(m) for h, m in zip(hist, new)]


# ------------------------------------------------------------------------------------------------ accept
def accept_case(seed, hist, nodes, lens, S, H, D, dtype, layers=1, unified=False):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    B = len(hist)
    used = [-(-(h + nodes) // S) for h in hist]
    nb = sum(used) + 2
    ids = rng.permutation(nb)
    table = torch.full((B, max(used) + 1), -1, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = i32(ids[at:at + u])
        at += u
    if unified:
        pool = torch.randn((layers, nb, 2, S, H, D), generator=g).to(dtype)
        k, v = pool[:, :, 0], pool[:, :, 1]
    else:
        k, v = (torch.randn((layers, nb, S, H, D), generator=g).to(dtype) for _ in range(2))
    acc = torch.full((B, max(max(lens), 1)), -9, dtype=torch.int32)
    for b, n in enumerate(lens):
        acc[b, :n] = i32(np.sort(rng.permutation(nodes)[:n]))
    return k, v, acc, i32(lens), i32(hist), table


def check_accept(pa, case, unified=False):
    k, v, acc, lens, hist, table = case
    if unified:
        pool = torch.stack([k, v], 2).cuda()
        dk, dv = pool[:, :, 0], pool[:, :, 1]
    else:
        dk, dv = k.cuda(), v.cuda()
    if k.shape[0] == 1:
        pa.paged_kv_accept(dk[0], dv[0], acc.cuda(), lens.cuda(), hist.cuda(), table.cuda())
    else:
        pa.paged_kv_accept(dk, dv, acc.cuda(), lens.cuda(), hist.cuda(), table.cuda())
    torch.cuda.synchronize()
    for layer in range(k.shape[0]):
        rk, rv = oracle.tree.paged_kv_accept(k[layer], v[layer], acc, lens, hist, table)
        assert torch.equal(dk[layer].cpu(), rk) and torch.equal(dv[layer].cpu(), rv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("H,D", [(1, 64), (2, 128), (8, 128), (3, 8)])
@pytest.mark.parametrize("S", [1, 16, 64])
@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("unified", [False, True])
def test_accept(cuda_lib, dtype, H, D, S, layers, unified):
    case = accept_case(S + H, [0, 15, 16, 100, 7], 24, [0, 1, 24, 9, 5], S, H, D, dtype, layers, unified)
    check_accept(cuda_lib, case, unified)
    assert cuda_lib.device_error_flags() == 0


@pytest.mark.parametrize("lens", [[64, 65, 1], [200, 130, 0]])
def test_accept_long_lists(cuda_lib, lens):
    check_accept(cuda_lib, accept_case(3, [5, 0, 31], 220, lens, 16, 2, 64, torch.bfloat16, 2))
    assert cuda_lib.device_error_flags() == 0


@pytest.mark.parametrize("batch,layers", [(40, 40), (30, 41), (1, 700), (1300, 3)])
@pytest.mark.parametrize("H,D", [(1, 64), (2, 128)])
def test_accept_with_several_layers_to_a_block_of_threads(cuda_lib, batch, layers, H, D):
    rng = np.random.default_rng(batch)
    case = accept_case(batch, rng.integers(0, 20, batch).tolist(), 12, rng.integers(0, 12, batch).tolist(), 16, H, D,
                       torch.float16, layers)
    k, v, acc, lens, hist, table = case
    dk, dv = k.cuda(), v.cuda()
    cuda_lib.paged_kv_accept(dk, dv, acc.cuda(), lens.cuda(), hist.cuda(), table.cuda())
    # every layer as the oracle moves one: all of them side by side as the heads of one
    side = lambda x: x.permute(1, 2, 0, 3, 4).flatten(2, 3)
    rk, rv = oracle.tree.paged_kv_accept(side(k), side(v), acc, lens, hist, table)
    assert torch.equal(side(dk.cpu()), rk) and torch.equal(side(dv.cpu()), rv)
    assert cuda_lib.device_error_flags() == 0


def test_accept_lists_that_chain_through_each_other(cuda_lib):
    """Each row moves one place: every source is the destination of the entry after it."""
    case = list(accept_case(3, [5], 90, [80], 16, 2, 64, torch.float32))
    case[2] = i32(np.arange(1, 81))[None]
    check_accept(cuda_lib, case)
    case[2] = i32([[7, 7, 3, 3] + [4] * 1 + [80] * 75])  # the same node twice, not ascending, never below its place
    check_accept(cuda_lib, case)
    assert cuda_lib.device_error_flags() == 0


def test_accept_records_what_it_refuses(cuda_lib):
    pa = cuda_lib
    base = accept_case(3, [5, 20], 16, [4, 3], 16, 2, 64, torch.float32)

    def run(flag, same_rows, **change):
        k, v, acc, lens, hist, table = (x.clone() for x in base)
        if "acc" in change:
            acc[0, 1] = change["acc"]
        if "lens" in change:
            lens[0] = change["lens"]
        if "hist" in change:
            hist[0] = change["hist"]
        if "table" in change:
            table[0, 0] = change["table"]
        dk, dv = k[0].cuda(), v[0].cuda()
        args = (acc.cuda(), lens.cuda(), hist.cuda(), table.cuda())
        pa.paged_kv_accept(dk, dv, *args)
        torch.cuda.synchronize()
        assert pa.device_error_flags() == flag
        ref = oracle.tree.paged_kv_accept(k[0], v[0], acc[1:], lens[1:], hist[1:], table[1:])
        if same_rows:  # nothing of sequence 0 moved
            assert torch.equal(dk.cpu(), ref[0]) and torch.equal(dv.cpu(), ref[1])
        pa.set_checked_mode(True)
        with pytest.raises(pa.PagedAttnError) as e:
            pa.paged_kv_accept(dk, dv, *args)
        assert e.value.status == pa.PA_ERANGE
        pa.set_checked_mode(False)

    run(pa.PA_DEVERR_TREE, False, acc=0)
    run(pa.PA_DEVERR_TREE, False, acc=-1)
    run(pa.PA_DEVERR_CONTEXT_LEN, False, acc=10 ** 9)
    run(pa.PA_DEVERR_QUERY_LOC, True, lens=-1)
    run(pa.PA_DEVERR_QUERY_LOC, False, lens=10)
    run(pa.PA_DEVERR_CONTEXT_LEN, True, hist=-50)
    run(pa.PA_DEVERR_BLOCK_ID, False, table=-1)


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("graph", [False, True])
def test_speculative_steps(cuda_lib, dtype, graph):
    """Steps of a serving loop: tables from the lengths, the drafted rows written, the trees attended,
    some path of each accepted, its rows kept.  Every token has one key and one value for good, so what
    the cache holds, and every output, follows from the accepted tokens alone."""
    pa = cuda_lib
    B, S, H, G, D, L, nodes, T = 5, 16, 2, 4, 64, 2, 12, 64
    rng = np.random.default_rng(11)
    gen = torch.Generator().manual_seed(11)
    st = State(2, [0] * B, [0] * B, S, cap=24, words=1, extra=150)
    d = st.device()
    k = torch.full((L, st.num_blocks, S, H, D), float("nan"), dtype=dtype, device="cuda")
    v = k.clone()
    kn, vn = (torch.zeros((L, T, H, D), dtype=dtype, device="cuda") for _ in range(2))
    q = torch.zeros((L, T, H * G, D), dtype=dtype, device="cuda")
    outs = [torch.zeros((T, H * G, D), dtype=dtype, device="cuda") for _ in range(L)]
    acc, n_acc = torch.zeros((B, nodes), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    parents = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    tables = pa.build_block_tables(d["hist"], d["new"], d["table"], d["counts"], d["free"], d["state"], S,
                                   st.num_blocks, parents=parents)

    def step():
        pa.build_block_tables(d["hist"], d["new"], d["table"], d["counts"], d["free"], d["state"], S, st.num_blocks,
                              parents=parents, out=tables)
        for layer in range(L):
            pa.paged_kv_write(kn[layer], vn[layer], tables.slot_mapping, k[layer], v[layer])
            pa.paged_attention_tree(q[layer], tables.query_start_loc, tables.tree_mask, k[layer], v[layer], d["table"],
                                    tables.context_lens, out=outs[layer], max_nodes=nodes)
        pa.paged_kv_accept(k, v, acc, n_acc, d["hist"], d["table"])
        d["hist"].add_(n_acc)

    run = step
    if graph:
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        run = g.replay
    kept = [[] for _ in range(B)]  # per sequence the (key, value) of its accepted tokens, [L, H, D] each
    # half a step of the output, and (tensor cores) half a step of each weight, which the values' largest
    # bounds; 32-bit arithmetic: at most 256 keys and 64 products a score, each of order 10
    half = torch.finfo(dtype).eps / 2
    in_32 = 2.0 ** -24 * (2 * 256 + 2 * 64 * 10)
    for turn in range(14):
        new = rng.integers(0, nodes + 1, B) if turn else np.full(B, nodes)
        par = random_parents(rng, new)
        total = int(new.sum())
        hk, hv = (torch.randn((L, total, H, D), generator=gen).to(dtype) for _ in range(2))
        hq = torch.randn((L, total, H * G, D), generator=gen).to(dtype)
        d["new"].copy_(i32(new))
        parents[:total] = i32(par).cuda()
        kn[:, :total], vn[:, :total], q[:, :total] = hk.cuda(), hv.cuda(), hq.cuda()
        first = np.cumsum(new) - new
        lists = []
        for b in range(B):
            path = []
            if new[b]:
                path = oracle.tree.ancestors(par[first[b]:], int(rng.integers(0, new[b])))[::-1]
            lists.append(path)
            acc[b, :len(path)] = i32(path).cuda()
        n_acc.copy_(i32([len(p) for p in lists]))
        run()
        torch.cuda.synchronize()
        assert pa.device_error_flags() == 0
        for b in range(B):
            for j in range(int(new[b])):
                t = first[b] + j
                line = [first[b] + s for s in oracle.tree.ancestors(par[first[b]:], j)]
                assert int(tables.positions[t]) == len(kept[b]) + len(line) - 1
                for layer in range(L):
                    ks = torch.stack([x[0][layer] for x in kept[b]] + [hk[layer, s] for s in line]).double()
                    vs = torch.stack([x[1][layer] for x in kept[b]] + [hv[layer, s] for s in line]).double()
                    ks, vs = ks.repeat_interleave(G, 1), vs.repeat_interleave(G, 1)
                    z = torch.einsum("hd,nhd->hn", hq[layer, t].double(), ks) * D ** -0.5
                    ref = torch.einsum("hn,nhd->hd", torch.softmax(z, 1), vs)
                    most = float(vs.abs().max())
                    tol = (half * ref.abs() + (half + in_32) * most) * (1 + half)
                    assert ((outs[layer][t].double().cpu() - ref).abs() <= tol).all()
            kept[b] += [(hk[:, first[b] + s], hv[:, first[b] + s]) for s in lists[b]]
        assert d["hist"].cpu().tolist() == [len(x) for x in kept]
    held = int(d["counts"].sum())
    assert held + int(d["state"][0]) == st.num_blocks
    ids = torch.cat([d["table"][b, :int(d["counts"][b])] for b in range(B)] + [d["free"][:int(d["state"][0])]])
    assert sorted(ids.cpu().tolist()) == list(range(st.num_blocks))
