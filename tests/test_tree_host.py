"""Refusals of the drafted-tree calls before anything is launched, and the oracle's own pins (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import pagedattention_kv_cache_paged_gb300 as pa
from tree_cases import TreeCase, mask_of, random_parents

P = 1 << 24  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    import os
    from pagedattention_kv_cache_paged_gb300 import _abi, build
    if not os.path.exists(_abi.LIB_PATH):
        build.build()
    return pa.load_library()


def call(lib, name, order, base, **change):
    v = dict(base, **change)
    return getattr(lib, name)(*[v[k] for k in order])


TREE = dict(out=P, q=P, qsl=P, total_q=8, mask=P, words=1, max_nodes=4, k=P, v=P, table=P, stride=4, ctx=P, batch=2,
            blocks=8, bs=16, scale=0.125, hq=8, hkv=2, d=64, dt=pa.PA_BF16, ws=None, ws_bytes=0, opts=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dt=7), "EDTYPE"), (dict(hq=6, hkv=4), "EINVAL"), (dict(hq=64, hkv=2), "EUNSUPPORTED"),
    (dict(d=96), "EUNSUPPORTED"), (dict(bs=12), "EUNSUPPORTED"), (dict(bs=512), "EUNSUPPORTED"), (dict(bs=0), "EINVAL"),
    (dict(batch=-1), "EINVAL"), (dict(total_q=-1), "EINVAL"), (dict(max_nodes=0), "EINVAL"), (dict(words=0), "EINVAL"),
    (dict(scale=0.0), "EINVAL"), (dict(scale=-1.0), "EINVAL"), (dict(scale=float("nan")), "EINVAL"),
    (dict(scale=float("inf")), "EINVAL"), (dict(out=None), "EINVAL"), (dict(q=P + 2), "EINVAL"), (dict(k=P + 8), "EINVAL"),
    (dict(qsl=None), "EINVAL"), (dict(ctx=None), "EINVAL"), (dict(table=None), "EINVAL"), (dict(stride=0), "EINVAL"),
    (dict(total_q=2 ** 31), "EINVAL"), (dict(blocks=0), "EINVAL"),
    (dict(opts="stride"), "EINVAL"), (dict(opts="kernel"), "EINVAL"),
    (dict(batch=0), "OK"), (dict(total_q=0), "OK"),
])
def test_tree_refusals(lib, change, status):
    change = dict(change)
    if change.get("opts") == "stride":
        change["opts"] = ctypes.byref(pa.make_opts(kv_block_stride_bytes=24))
    elif change.get("opts") == "kernel":
        change["opts"] = ctypes.byref(pa.make_opts(prefill_kernel=3))
    assert call(lib, "paged_attention_tree", list(TREE), TREE, **change) == getattr(pa, "PA_" + status)


def test_tree_workspace_of_bad_sizes_is_zero(lib):
    good = [2, 8, 4, 512, 16, 8, 2, 64, pa.PA_BF16]
    for i in range(8):
        bad = list(good)
        bad[i] = 0
        assert lib.paged_attention_tree_workspace_size(*bad, None) == 0
    assert lib.paged_attention_tree_workspace_size(*good[:8], 9, None) == 0


TABLES = dict(hist=P + 64, new=P + 128, batch=2, table=P, stride=8, cap=8, counts=P, free=P, free_n=16, state=P, blocks=16, bs=16,
              parents=None, qsl=P, ctx=P, slots=P, pos=P, tokens=8, mask=None, words=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), "EINVAL"), (dict(blocks=0), "EINVAL"), (dict(cap=0), "EINVAL"), (dict(cap=9), "EINVAL"),
    (dict(free_n=-1), "EINVAL"), (dict(tokens=-1), "EINVAL"), (dict(tokens=2 ** 31), "EINVAL"), (dict(bs=0), "EINVAL"),
    (dict(bs=24), "EUNSUPPORTED"), (dict(bs=512), "EUNSUPPORTED"), (dict(hist=None), "EINVAL"), (dict(new=None), "EINVAL"),
    (dict(table=None), "EINVAL"), (dict(counts=None), "EINVAL"), (dict(free=None), "EINVAL"), (dict(state=None), "EINVAL"),
    (dict(qsl=None), "EINVAL"), (dict(ctx=None), "EINVAL"), (dict(slots=None), "EINVAL"), (dict(pos=None), "EINVAL"),
    (dict(parents=P), "EINVAL"), (dict(parents=P, words=1), "EINVAL"), (dict(parents=P, mask=P), "EINVAL"),
    (dict(ctx=P + 64), "EINVAL"), (dict(ctx=P + 128), "EINVAL"), (dict(batch=0), "OK"),
    (dict(ctx=P + 68), "EINVAL"), (dict(ctx=P + 60), "EINVAL"), (dict(qsl=P + 56), "EINVAL"), (dict(counts=P + 132), "EINVAL"),
])
def test_tables_refusals(lib, change, status):
    assert call(lib, "build_block_tables", list(TABLES), TABLES, **change) == getattr(pa, "PA_" + status)


ACCEPT = dict(k=P, v=P, layers=1, layer_stride=0, acc=P, acc_stride=4, most=4, lens=P, hist=P, table=P, stride=8, batch=2,
              blocks=16, bs=16, hkv=2, d=64, dt=pa.PA_BF16, opts=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dt=5), "EDTYPE"), (dict(batch=-1), "EINVAL"), (dict(layers=-1), "EINVAL"), (dict(most=-1), "EINVAL"),
    (dict(most=5), "EINVAL"), (dict(layers=2), "EINVAL"), (dict(layers=2, layer_stride=24), "EINVAL"),
    (dict(k=None), "EINVAL"), (dict(v=P + 4), "EINVAL"), (dict(acc=None), "EINVAL"), (dict(lens=None), "EINVAL"),
    (dict(hist=None), "EINVAL"), (dict(table=None), "EINVAL"), (dict(stride=0), "EINVAL"), (dict(bs=0), "EINVAL"),
    (dict(d=4, hkv=1), "EUNSUPPORTED"), (dict(batch=0), "OK"), (dict(layers=0), "OK"), (dict(most=0), "OK"),
])
def test_accept_refusals(lib, change, status):
    assert call(lib, "paged_kv_accept", list(ACCEPT), ACCEPT, **change) == getattr(pa, "PA_" + status)


def test_the_binding_refuses_wrong_tensors(lib):
    case = TreeCase(1, [4, 5], [2, 3], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=torch.float32)
    good = dict(q=case.q, query_start_loc=case.qsl, tree_mask=case.mask, k_pool=case.k, v_pool=case.v,
                block_table=case.table, context_lens=case.ctx)
    for change in (dict(), dict(q=case.q[0]), dict(tree_mask=case.mask[:3]), dict(tree_mask=case.mask[:, :0]),
                   dict(block_table=case.table[:1]), dict(v_pool=case.v[:2]), dict(out=case.q[:2])):
        with pytest.raises(ValueError):
            pa.paged_attention_tree(**{**good, **change})
    n = torch.zeros(2, dtype=torch.int32)
    table, free = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    for kw in (dict(num_tokens=4), dict(), dict(parents=n, out=pa.StepTables(n, n, n, n, None))):
        with pytest.raises(ValueError):
            pa.build_block_tables(n, n, table, n, free, n, 16, 9, **kw)
    with pytest.raises(ValueError):
        pa.build_block_tables(n, n, table.t(), n, free, n, 16, 9, num_tokens=4)
    with pytest.raises(ValueError):
        pa.paged_kv_accept(case.k, case.v, torch.zeros((2, 3), dtype=torch.int32), n, n, table)
    with pytest.raises(ValueError):
        pa.paged_kv_accept(case.k, case.v, n, n, n, table)
    with pytest.raises(ValueError):
        pa.paged_kv_accept(case.k, case.v[None], torch.zeros((2, 3), dtype=torch.int32), n, n, table)


def test_the_oracle_of_a_chain_is_the_causal_chunk():
    case = TreeCase(2, [0, 9], [4, 5], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=torch.float32, words=0)
    rows, out, _, _ = oracle.tree.paged_tree_attention(case.q, case.qsl, None, case.k, case.v, case.table, case.ctx, 0.125)
    ref = oracle.paged_prefill(case.q, case.qsl, case.k, case.v, case.table, case.ctx, 0.125)
    for i, r in enumerate(rows):
        assert np.abs(out[i] - ref[r]).max() < 1e-13
    new = [4, 5]
    chain = np.concatenate([np.arange(m) - 1 for m in new])
    again = oracle.tree.paged_tree_attention(case.q, case.qsl, mask_of(chain, new, 1), case.k, case.v, case.table, case.ctx,
                                             0.125)[1]
    assert np.array_equal(again, out)


def test_the_oracle_of_a_tree_is_each_path_on_its_own():
    """A node's output is that of plain attention over its history and its own line of ancestors."""
    rng = np.random.default_rng(3)
    case = TreeCase(3, [6, 0], [7, 9], q_heads=2, kv_heads=1, head_dim=64, block_size=4, dtype=torch.float32)
    par = random_parents(rng, case.new)
    case.mask = mask_of(par, case.new, 1)
    out = oracle.tree.paged_tree_attention(case.q, case.qsl, case.mask, case.k, case.v, case.table, case.ctx, 0.3)[1]
    t = 0
    for b in range(2):
        k = oracle.repeat_kv(oracle.gather_history(case.k, case.table[b], int(case.ctx[b]), 4), 2)
        v = oracle.repeat_kv(oracle.gather_history(case.v, case.table[b], int(case.ctx[b]), 4), 2)
        for j in range(case.new[b]):
            line = list(range(case.hist[b])) + sorted(case.hist[b] + s for s in oracle.tree.ancestors(par[t - j:], j))
            ref = oracle.softmax_attention(case.q[t].double().numpy(), k[line], v[line], 0.3)
            assert np.abs(out[t] - ref).max() < 1e-12
            t += 1
