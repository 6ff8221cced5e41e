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
