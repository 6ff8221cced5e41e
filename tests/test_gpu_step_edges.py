"""GPU tests of the step calls at the edges of what they allow: empty batches, chains of launches without another kernel
between them, views whose rows end with their memory."""
import numpy as np
import pytest
import torch

import oracle
from pagedattention_kv_cache_paged_gb300 import _abi

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clean(cuda_lib):
    cuda_lib.device_error_flags(clear=True)
    yield
    cuda_lib.set_checked_mode(False)
    cuda_lib.device_error_flags(clear=True)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("trees", [False, True])
@pytest.mark.parametrize("where", ["current", "stream", "raw", "default"])
def test_an_empty_batch_leaves_no_step_behind(cuda_lib, trees, where):
    """Arrays of an earlier step, written again for no sequences: no slot of that step is left, and what the call writes
    it writes in the order of its stream."""
    pa = cuda_lib
    table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    free, state = i32(list(range(16))), i32([16, 0])
    parents = i32([-1, 0, 1, -1, 0, 0, 0, 0, 0]) if trees else None
    t = pa.build_block_tables(i32([0, 0]), i32([3, 4]), table, i32([0, 0]), free, state, 16, 16, num_tokens=9, parents=parents)
    assert (t.slot_mapping[:7] >= 0).all()
    none = i32([])
    out = t._replace(query_start_loc=t.query_start_loc[:1], context_lens=t.context_lens[:0])
    torch.cuda.synchronize()
    side = torch.cuda.default_stream() if where == "default" else torch.cuda.Stream()
    if where != "current":
        with torch.cuda.stream(side):  # some 10 ms of waiting, then another writer of the same arrays
            torch.cuda._sleep(20_000_000)
            t.slot_mapping.fill_(77)
            t.query_start_loc.fill_(9)
    stream = {"current": None, "stream": side, "raw": side.cuda_stream, "default": 0}[where]
    with torch.cuda.stream(torch.cuda.Stream() if where == "default" else torch.cuda.current_stream()):
        got = pa.build_block_tables(none, none, table[:0], none, free, state, 16, 16, parents=parents, out=out, stream=stream)
        fresh = pa.build_block_tables(none, none, table[:0], none, free, state, 16, 16, num_tokens=9, parents=parents,
                                      stream=stream)
    torch.cuda.synchronize()
    assert got is out
    for o in (got, fresh):
        assert o.query_start_loc.cpu().tolist() == [0] and o.context_lens.numel() == 0
        assert (o.slot_mapping == -1).all() and (o.positions == 0).all() and o.slot_mapping.numel() == 9
        assert (o.tree_mask is not None) == trees and (not trees or (o.tree_mask == 0).all())
    assert state.cpu().tolist() == [15 - 1, 0] and pa.device_error_flags() == 0
    pool = torch.zeros((2, 16, 16, 1, 64), device="cuda")
    new = torch.ones((9, 1, 64), device="cuda")
    pa.paged_kv_write(new, new, got.slot_mapping, pool[0], pool[1])
    assert (pool == 0).all()


def test_checked_mode_reads_no_further_than_the_rows_of_a_view(cuda_lib):
    """Tables whose last row ends with its memory, though the stride of a row does not."""
    pa = cuda_lib
    torch.cuda.empty_cache()
    wide = torch.full((2, 10 * 2 ** 18), -9, dtype=torch.int32, device="cuda")  # 20 MiB, a segment of its own
    table = wide[:, 8:]
    table[:, :3] = i32([[0, 1, 2], [3, 4, 5]])
    lists = torch.full((2, 10 * 2 ** 18), -9, dtype=torch.int32, device="cuda")[:, -4:]
    lists[:, :2] = i32([[0, 3], [1, 2]])
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((6, 16, 2, 64), generator=g) for _ in range(2))
    q = torch.randn((8, 4, 64), generator=g)
    hist, ctx, qsl = i32([30, 40]), i32([34, 44]), i32([0, 4, 8])
    dk, dv = k.cuda(), v.cuda()
    pa.set_checked_mode(True)
    out = pa.paged_attention_tree(q.cuda(), qsl, None, dk, dv, table, ctx)
    pa.paged_kv_accept(dk, dv, lists, i32([2, 2]), hist, table)
    torch.cuda.synchronize()
    pa.set_checked_mode(False)
    small = table[:, :3].cpu()
    ref = oracle.tree.paged_tree_attention(q, qsl.cpu(), None, k, v, small, ctx.cpu(), 0.125)[1]
    # (a score of 64 products of order 1, weights and sums of 44 keys, in 32 bits: below 2^-24 * 4 * (64 + 44) times
    # values of 4)
    assert np.abs(out.cpu().double().numpy() - ref).max() < 2.0 ** -24 * 4 * 108 * 4
    want = oracle.tree.paged_kv_accept(k, v, lists.cpu(), i32([2, 2]).cpu(), hist.cpu(), small)
    assert torch.equal(dk.cpu(), want[0]) and torch.equal(dv.cpu(), want[1])
    # and what is wrong is found: an entry inside a context, an entry of a moved row
    table[1, 2] = 6
    pa.set_checked_mode(True)
    for call in (lambda: pa.paged_attention_tree(q.cuda(), qsl, None, dk, dv, table, ctx),
                 lambda: pa.paged_kv_accept(dk, dv, lists, i32([2, 2]), hist, table)):
        with pytest.raises(pa.PagedAttnError) as e:
            call()
        assert e.value.status == pa.PA_ERANGE


def test_checked_mode_without_memory_for_its_copy_returns(cuda_lib):
    """A list stride that no memory holds: an error code, and no exception out of the library."""
    pa = cuda_lib
    p = torch.zeros(2 ** 16, dtype=torch.int32, device="cuda").data_ptr()
    pa.set_checked_mode(True)
    before = pa.launch_count()
    assert pa.load_library().paged_kv_accept(p, p, 1, 0, p, 2 ** 61, 4, p, p, p, 8, 2, 4, 16, 1, 64, pa.PA_FP32, None,
                                             None) == _abi.PA_ECUDA
    assert pa.launch_count() == before


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("call", ["decode", "decode_cuda_cores", "decode_fp32", "decode_fused", "prefill", "tree", "tree_mma_sync",
                                  "tree_fp32", "chain"])
def test_tables_right_before_attention(cuda_lib, call, graph):
    """No launch between the tables of a step and the call that reads them: lengths, blocks and masks are those of this
    step every time, though the steps take turns between two batches that share all arrays."""
    pa = cuda_lib
    B, S, H, G, D = 48, 16, 4, 4, 128
    m = 1 if call.startswith("decode") else 6
    dtype = FP32 if call.endswith("fp32") else BF16
    g = torch.Generator(device="cuda").manual_seed(5)
    rng = np.random.default_rng(5)
    blocks = 2 * B * 72  # (a half for each batch: the fused call writes rows)
    k, v = (torch.randn((blocks, S, H, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((B * m, H * G, D), generator=g, device="cuda").to(dtype)
    new_k, new_v = (torch.randn((B, H, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    trees = call.startswith("tree")
    batches = []
    for i in range(2):
        held = rng.integers(0, 70, B) if i else np.sort(rng.integers(0, 30, B))
        ids = rng.permutation(B * 72) + i * B * 72
        table = np.full((B, 72), -1)
        table[np.arange(72)[None] < held[:, None]] = ids[:held.sum()]
        free = np.zeros(B * 72, np.int64)
        free[:B * 72 - held.sum()] = ids[held.sum():]
        parents = np.concatenate([[-1] + [rng.integers(-1, j) for j in range(1, m)] for _ in range(B)])
        batches.append(dict(hist=i32(held * S), table=i32(table), counts=i32(held), free=i32(free),
                            state=i32([B * 72 - held.sum(), 0]), parents=i32(parents) if trees else None))
    d = {n: x.clone() for n, x in batches[0].items() if n != "hist" and x is not None}
    new = i32([m] * B)
    t = pa.build_block_tables(batches[0]["hist"], new, d["table"], d["counts"], d["free"], d["state"], S, blocks,
                              num_tokens=B * m, parents=d.get("parents"))
    out = torch.empty_like(q)

    def step(i):
        for n in d:
            d[n].copy_(batches[i][n])
        pa.build_block_tables(batches[i]["hist"], new, d["table"], d["counts"], d["free"], d["state"], S, blocks,
                              parents=d.get("parents"), out=t)
        if call == "decode_fused":
            pa.paged_attention_decode_fused(q, new_k, new_v, t.slot_mapping, k, v, d["table"], t.context_lens, out=out)
        elif call.startswith("decode"):
            pa.paged_attention_decode(q, k, v, d["table"], t.context_lens, out=out, decode_kernel=int(call.endswith("cores")))
        elif call == "prefill":
            pa.paged_attention_prefill(q, t.query_start_loc, k, v, d["table"], t.context_lens, out=out)
        else:
            pa.paged_attention_tree(q, t.query_start_loc, t.tree_mask, k, v, d["table"], t.context_lens, out=out, max_nodes=m,
                                    kernel=int(call == "tree_mma_sync"))

    want = []
    for i in range(2):
        for n in d:
            d[n].copy_(batches[i][n])
        pa.build_block_tables(batches[i]["hist"], new, d["table"], d["counts"], d["free"], d["state"], S, blocks,
                              parents=d.get("parents"), out=t)
        torch.cuda.synchronize()
        assert int(t.slot_mapping.min()) >= 0
        step(i)  # (the fused call writes the same rows again)
        torch.cuda.synchronize()
        want.append(out.clone())
    # the reference batch on its own tables, without this call's history
    i = 1
    for n in d:
        d[n].copy_(batches[i][n])
    pa.build_block_tables(batches[i]["hist"], new, d["table"], d["counts"], d["free"], d["state"], S, blocks,
                          parents=d.get("parents"), out=t)
    torch.cuda.synchronize()
    rows, ref, _, _ = oracle.tree.paged_tree_attention(q.cpu(), t.query_start_loc.cpu(), None if t.tree_mask is None else
                                                       t.tree_mask.cpu(), k.cpu(), v.cpu(), d["table"].cpu(),
                                                       t.context_lens.cpu(), D ** -0.5)
    assert np.abs(want[1].double().cpu().numpy()[rows] - ref).max() < (1e-5 if dtype == FP32 else 2e-2)
    assert not torch.equal(want[0], want[1])
    kept = [torch.empty_like(out) for _ in range(40)]
    if graph:
        s = torch.cuda.Stream()
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr, stream=s):
            for j, o in enumerate(kept):
                step(j % 2)
                o.copy_(out)
        for _ in range(5):
            gr.replay()
    else:
        for j, o in enumerate(kept * 5):
            step(j % 2)
            o.copy_(out)
    torch.cuda.synchronize()
    for j, o in enumerate(kept):
        assert torch.equal(o, want[j % 2]), j
    assert pa.device_error_flags() == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("unified", [False, True])
def test_accept_with_the_layers_of_a_block_side_by_side(cuda_lib, dtype, unified):
    """Pools [num_blocks, layers, ..]: a layer is nearer than the next block."""
    L, NB, S, H, D = 3, 9, 16, 2, 64
    g = torch.Generator().manual_seed(2)
    pool = torch.randn((NB, L, 2, S, H, D), generator=g).to(dtype)
    dp = pool.cuda()
    if not unified:
        dp = [dp[:, :, i].contiguous() for i in range(2)]
    k, v = ((dp[:, :, i] if unified else dp[i]).transpose(0, 1) for i in range(2))
    acc, n_acc, hist = i32([[1, 2, 9], [0, 5, -3]]), i32([3, 2]), i32([13, 30])
    table = i32([[7, 2, -1, -1], [0, 5, 3, 1]])
    cuda_lib.paged_kv_accept(k, v, acc, n_acc, hist, table)
    assert cuda_lib.device_error_flags() == 0
    for layer in range(L):
        want = oracle.tree.paged_kv_accept(pool[:, layer, 0], pool[:, layer, 1], acc.cpu(), n_acc.cpu(), hist.cpu(),
                                           table.cpu())
        assert torch.equal(k[layer].cpu(), want[0]) and torch.equal(v[layer].cpu(), want[1])


@pytest.mark.parametrize("raw", [False, True])
def test_a_step_on_a_stream_given_to_the_calls(cuda_lib, raw):
    """Every call in the order of the stream it is given, behind what that stream has to do first."""
    pa = cuda_lib
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((40, 16, 2, 64), generator=g, device="cuda") for _ in range(2))
    q = torch.randn((9, 4, 64), generator=g, device="cuda")
    kn, vn = (torch.randn((9, 2, 64), generator=g, device="cuda") for _ in range(2))
    parents, acc, n_acc = i32([-1, 0, 0, 1, 1, -1, -1, 1, 2]), i32([[0, 2], [1, 3]]), i32([2, 2])

    def step(hist, stream, slow):
        pools = [k.clone(), v.clone()]
        table, counts, state = torch.full((2, 12), -1, dtype=torch.int32, device="cuda"), i32([7, 2]), i32([31, 0])
        table[0, :7], table[1, :2] = torch.arange(7, device="cuda"), torch.arange(7, 9, device="cuda")
        free = torch.arange(9, 40, dtype=torch.int32, device="cuda")
        h, m = i32([1, 1]), i32([5, 4])
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            if slow:
                torch.cuda._sleep(10_000_000)
            h.copy_(hist)
        s = stream.cuda_stream if raw else stream
        t = pa.build_block_tables(h, m, table, counts, free, state, 16, 40, parents=parents, stream=s)
        pa.paged_kv_write(kn, vn, t.slot_mapping, *pools, stream=s)
        out = pa.paged_attention_tree(q, t.query_start_loc, t.tree_mask, *pools, table, t.context_lens, max_nodes=5, stream=s)
        pa.paged_kv_accept(*pools, acc, n_acc, h, table, stream=s)
        return [out, *pools, table, counts, state, *t]

    hist = i32([100, 30])
    want = step(hist, torch.cuda.current_stream(), False)
    torch.cuda.synchronize()
    got = step(hist, torch.cuda.Stream(), True)
    torch.cuda.synchronize()
    assert pa.device_error_flags() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kernel", [0, 1])
def test_trees_of_many_mask_words(cuda_lib, kernel):
    """Trees of up to 700 nodes, some almost chains: masks as built, attention over them as the oracle has it."""
    pa = cuda_lib
    rng = np.random.default_rng(8)
    new, hist, words = [700, 3, 450, 0, 129], [20, 5, 0, 40, 100], 11
    parents = np.concatenate([[-1] + [j - 1 if rng.random() < 0.97 else rng.integers(-1, j) for j in range(1, m)]
                              for m in new if m])
    total = int(sum(new))
    held = [-(-h // 16) for h in hist]
    blocks = sum(-(-(h + m) // 16) for h, m in zip(hist, new)) + 2
    ids = rng.permutation(blocks)
    table = np.full((5, 50), -1)
    at = 0
    for b, c in enumerate(held):
        table[b, :c] = ids[at:at + c]
        at += c
    free = np.zeros(blocks, np.int64)
    free[:blocks - at] = ids[at:]
    args = [i32(table), i32(held), i32(free), i32([blocks - at, 0])]
    t = pa.build_block_tables(i32(hist), i32(new), *args, 16, blocks, parents=i32(parents), mask_words=words)
    ref = oracle.tree.step_tables(hist, new, i32(table).cpu(), i32(held).cpu(), i32(free).cpu(), blocks - at, 16, total,
                                  parents, words)
    for name in ("query_start_loc", "context_lens", "slot_mapping", "positions", "tree_mask"):
        assert np.array_equal(getattr(t, name).cpu().numpy(), ref[name]), name
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn((blocks, 16, 2, 64), generator=g) for _ in range(2))
    q = torch.randn((total, 4, 64), generator=g)
    for dtype, tol in ((BF16, 2e-2), (FP32, 1e-5)):
        out = pa.paged_attention_tree(q.to(dtype).cuda(), t.query_start_loc, t.tree_mask, k.to(dtype).cuda(),
                                      v.to(dtype).cuda(), args[0], t.context_lens, kernel=kernel)
        rows, want, _, _ = oracle.tree.paged_tree_attention(q.to(dtype), t.query_start_loc.cpu(), t.tree_mask.cpu(),
                                                            k.to(dtype), v.to(dtype), args[0].cpu(), t.context_lens.cpu(),
                                                            0.125)
        assert np.abs(out.cpu().double().numpy()[rows] - want).max() <= tol
    assert pa.device_error_flags() == 0


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_batch_of_30000_chains_of_one_node_is_a_decode_batch(cuda_lib, kernel, dtype):
    pa = cuda_lib
    B = 30000
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn((64, 16, 2, 64), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((B + 5, 8, 64), generator=g, device="cuda").to(dtype)
    q[B:] = float("nan")  # rows behind the last sequence
    table = torch.randint(0, 64, (B, 3), generator=g, device="cuda", dtype=torch.int32)
    ctx = torch.randint(1, 49, (B,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.full_like(q, 7.0)
    pa.paged_attention_tree(q, torch.arange(B + 1, dtype=torch.int32, device="cuda"), None, k, v, table, ctx, out=out,
                            max_nodes=1, kernel=kernel)
    want = pa.paged_attention_decode(q[:B].contiguous(), k, v, table, ctx, decode_kernel=1)
    assert pa.device_error_flags() == 0
    # (both within the framework's 2e-2 and 1e-5 of the definition)
    assert (out[:B].double() - want.double()).abs().max() <= (2e-5 if dtype == FP32 else 4e-2)
    assert (out[B:] == 7.0).all()


def test_checked_mode_looks_at_the_librarys_word_of_the_free_list(cuda_lib):
    pa = cuda_lib
    args = lambda word: (i32([0]), i32([5]), i32([[-1, -1]]), i32([0]), i32([3, 1]), i32([2, word]), 16, 8)
    pa.set_checked_mode(True)
    t = pa.build_block_tables(*args(0), num_tokens=5)
    assert t.slot_mapping.cpu().tolist() == list(range(16, 21))
    for word in (1, -1):
        with pytest.raises(pa.PagedAttnError) as e:
            pa.build_block_tables(*args(word), num_tokens=5)
        assert e.value.status == pa.PA_ERANGE
