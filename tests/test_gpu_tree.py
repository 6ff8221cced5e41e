"""GPU parity of paged_attention_tree against the float64 oracle, where it can go wrong."""
import numpy as np
import pytest
import torch

import oracle
from tree_cases import TreeCase, bound

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _clean(cuda_lib):
    cuda_lib.device_error_flags(clear=True)
    yield
    cuda_lib.set_checked_mode(False)
    cuda_lib.device_error_flags(clear=True)


def check(pa, case, got, kernel=0, flags=0):
    torch.cuda.synchronize()
    rows, ref, spread, size = oracle.tree.paged_tree_attention(case.q, case.qsl, case.mask, case.k, case.v, case.table,
                                                               case.ctx, case.scale)
    g = got.cpu().double().numpy()[rows]
    finite = torch.isfinite(case.v)
    values = float(case.v[finite].abs().max()) if finite.any() else 0.0
    tol = bound(case.dtype, ref, spread, size, int(case.ctx.max()), case.q.shape[2], values,
                case.dtype != FP32 and kernel != 1)
    assert np.isfinite(g).all()
    off = np.abs(g - ref) - tol
    assert (off <= 0).all(), f"worst excess {off.max()} at {np.unravel_index(off.argmax(), off.shape)}"
    assert pa.device_error_flags() == flags


def run(pa, case, **kw):
    d = case.device()
    return pa.paged_attention_tree(**d, scale=case.scale, **kw)


HIST, NEW = [0, 1, 63, 130, 17, 300], [5, 1, 16, 33, 0, 7]


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_ragged_trees(cuda_lib, kernel, dtype, D, G):
    case = TreeCase(10 * G + D, HIST, NEW, q_heads=2 * G, kv_heads=2, head_dim=D, block_size=16, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case, kernel=kernel, max_nodes=33), kernel)


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("S", [1, 2, 4, 8, 16, 32, 64, 128, 256])
def test_block_sizes(cuda_lib, kernel, dtype, S):
    case = TreeCase(S, [0, 100, 255], [70, 9, 3], q_heads=6, kv_heads=3, head_dim=64, block_size=S, dtype=dtype, words=2)
    check(cuda_lib, case, run(cuda_lib, case, kernel=kernel), 1 if S < 16 else kernel)


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("part", [16, 48, 128, 200, 256])
def test_split_contexts(cuda_lib, kernel, dtype, part):
    """Partitions that end inside a tile, before the tree, inside it and behind it."""
    case = TreeCase(part, [700, 0, 250, 129], [30, 64, 6, 1], q_heads=8, kv_heads=2, head_dim=128, block_size=16,
                    dtype=dtype)
    got = run(cuda_lib, case, kernel=kernel, partition_tokens=part)
    check(cuda_lib, case, got, kernel)


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("m", [1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_tree_sizes(cuda_lib, kernel, m):
    case = TreeCase(m, [77, 5], [m, 1], q_heads=4, kv_heads=1, head_dim=64, block_size=32, dtype=FP16, words=4)
    check(cuda_lib, case, run(cuda_lib, case, kernel=kernel), kernel)


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_chains(cuda_lib, kernel, dtype):
    """No mask: node r sees the ones before it, like a causal chunk."""
    case = TreeCase(3, [0, 40, 500], [90, 1, 20], q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=dtype, words=0)
    got = run(cuda_lib, case, kernel=kernel)
    check(cuda_lib, case, got, kernel)
    d = case.device()
    pre = cuda_lib.paged_attention_prefill(d["q"], d["query_start_loc"], d["k_pool"], d["v_pool"], d["block_table"],
                                           d["context_lens"], case.scale)
    check(cuda_lib, case, pre)


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("part", [0, 32])
def test_any_mask_and_rows_that_see_nothing(cuda_lib, kernel, dtype, part):
    case = TreeCase(5, [0, 0, 50, 64], [40, 3, 40, 64], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    g = torch.Generator().manual_seed(9)
    case.mask = torch.randint(-2 ** 63, 2 ** 63 - 1, case.mask.shape, generator=g)
    case.mask[::3] = 0  # with an empty history: zeros
    got = run(cuda_lib, case, kernel=kernel, partition_tokens=part)
    check(cuda_lib, case, got, kernel)
    assert (got[:40:3] == 0).all()


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("part", [0, 64])
def test_what_a_row_does_not_see_does_not_enter_it(cuda_lib, kernel, dtype, bad, part):
    """Non-finite keys and values in nodes that only some rows see: the others keep their results."""
    case = TreeCase(6, [90, 0, 128], [20, 50, 64], q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    for b in range(3):
        blk, tok = case.row_of(b, case.hist[b] + 7)
        case.v[blk, tok, :, 5:20] = bad
        blk, tok = case.row_of(b, case.hist[b] + 9)
        case.k[blk, tok] = bad
        blk, tok = case.row_of(b, case.hist[b] + 15)
        case.v[blk, tok] = bad
    got = run(cuda_lib, case, kernel=kernel, partition_tokens=part).cpu().double().numpy()
    rows, ref, spread, size = oracle.tree.paged_tree_attention(case.q, case.qsl, case.mask, case.k, case.v, case.table,
                                                               case.ctx, case.scale)
    fine = np.isfinite(ref) & np.isfinite(size)[:, :, None]
    assert fine.any() and not fine.all()
    values = float(case.v[torch.isfinite(case.v)].abs().max())
    size = np.where(np.isfinite(size), size, 0.0)
    tol = bound(dtype, np.where(fine, ref, 0), np.where(fine, spread, 0), size, int(case.ctx.max()), 64, values,
                dtype != FP32 and kernel != 1)
    assert (np.abs(got - ref)[fine] <= tol[fine]).all()
    # a value that a row sees and that is not finite leaves nothing finite in its column
    seen = ~np.isfinite(spread) & np.isfinite(size)[:, :, None]
    assert not np.isfinite(got[seen]).any()


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("part", [0, 64])
def test_rows_whose_every_score_is_minus_infinity(cuda_lib, kernel, part):
    """0 / 0, as the definition has it, and not the zeros of a row that sees nothing."""
    case = TreeCase(7, [100, 20], [3, 2], q_heads=2, kv_heads=1, head_dim=64, block_size=16, dtype=BF16)
    case.q = case.q.abs() + 0.5
    for j in range(103):
        blk, tok = case.row_of(0, j)
        case.k[blk, tok] = -float("inf")
    got = run(cuda_lib, case, kernel=kernel, partition_tokens=part)
    assert torch.isnan(got[:3]).all() and torch.isfinite(got[3:]).all()


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("gain", [0.0, 8.0, 200.0])
def test_flat_and_peaked_scores(cuda_lib, kernel, gain):
    case = TreeCase(8, [400, 33], [12, 40], q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=FP16, gain=gain)
    check(cuda_lib, case, run(cuda_lib, case, kernel=kernel, partition_tokens=128), kernel)


@pytest.mark.parametrize("kernel", [0, 1])
def test_rising_scores_move_the_maximum(cuda_lib, kernel):
    """Every tile holds a larger maximum than the one before it."""
    case = TreeCase(18, [640], [9], q_heads=4, kv_heads=1, head_dim=64, block_size=16, dtype=BF16)
    case.q = case.q.abs() + 0.25
    for j in range(649):
        blk, tok = case.row_of(0, j)
        case.k[blk, tok] = 0.02 * j
    check(cuda_lib, case, run(cuda_lib, case, kernel=kernel), kernel)


@pytest.mark.parametrize("kernel", [0, 1])
def test_rows_behind_the_last_sequence_stay(cuda_lib, kernel):
    case = TreeCase(11, [30, 200], [6, 10], q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=BF16, tail=21)
    out = torch.full_like(case.q, 7.0).cuda()
    got = run(cuda_lib, case, kernel=kernel, out=out, partition_tokens=64)
    assert got is out
    check(cuda_lib, case, got, kernel)
    assert (got[16:] == 7.0).all()


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_unified_pools_and_a_wider_table(cuda_lib, kernel, dtype):
    case = TreeCase(12, [30, 200, 1], [6, 10, 40], q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=dtype,
                    unified=True)
    d = case.device()
    wide = torch.full((3, 64), -5, dtype=torch.int32, device="cuda")
    wide[:, :case.table.shape[1]] = d["block_table"]
    d["block_table"] = wide[:, :case.table.shape[1]]
    check(cuda_lib, case, cuda_lib.paged_attention_tree(**d, scale=case.scale, kernel=kernel), kernel)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_offsets_past_32_bits(cuda_lib, dtype):
    """A pool of more than 2^32 bytes and 2^31 elements, the context in its last blocks."""
    S, H, D = 16, 8, 128
    blocks = 2 ** 31 // (S * H * D) + 20
    case = TreeCase(13, [60, 37], [9, 4], q_heads=16, kv_heads=H, head_dim=D, block_size=S, dtype=dtype)
    d = case.device()
    big = []
    for pool in (d["k_pool"], d["v_pool"]):
        p = torch.empty((blocks, S, H, D), dtype=dtype, device="cuda")
        p[-case.num_blocks:] = pool
        big.append(p)
    table = torch.where(d["block_table"] >= 0, d["block_table"] + (blocks - case.num_blocks), -1)
    d.update(k_pool=big[0], v_pool=big[1], block_table=table.to(torch.int32))
    check(cuda_lib, case, cuda_lib.paged_attention_tree(**d, scale=case.scale))


@pytest.mark.parametrize("kernel", [0, 1])
def test_bad_blocks_are_masked_and_recorded(cuda_lib, kernel):
    pa = cuda_lib
    case = TreeCase(14, [64, 100], [5, 6], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    good = run(pa, case, kernel=kernel).cpu()
    case.table[0, 1] = case.num_blocks + 9
    got = run(pa, case, kernel=kernel)
    torch.cuda.synchronize()
    assert torch.isfinite(got.float()).all()
    assert torch.equal(got[5:].cpu(), good[5:])
    assert pa.device_error_flags() == pa.PA_DEVERR_BLOCK_ID
    pa.set_checked_mode(True)
    with pytest.raises(pa.PagedAttnError) as e:
        run(pa, case, kernel=kernel)
    assert e.value.status == pa.PA_ERANGE


@pytest.mark.parametrize("kernel", [0, 1])
def test_sequences_that_do_not_fit_together_give_zeros(cuda_lib, kernel):
    pa = cuda_lib
    case = TreeCase(15, [64, 100, 3], [5, 6, 4], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    good = run(pa, case, kernel=kernel).cpu()
    for change, flag in ((dict(ctx=[69, 5, 7]), pa.PA_DEVERR_QUERY_LOC),
                         (dict(ctx=[69, 10 ** 6, 7]), pa.PA_DEVERR_CONTEXT_LEN),
                         (dict(ctx=[69, -3, 7]), pa.PA_DEVERR_QUERY_LOC | pa.PA_DEVERR_CONTEXT_LEN)):
        d = case.device()
        d["context_lens"] = torch.tensor(change["ctx"], dtype=torch.int32, device="cuda")
        got = pa.paged_attention_tree(**d, scale=case.scale, kernel=kernel).cpu()
        assert pa.device_error_flags() == flag
        assert torch.equal(got[:5], good[:5]) and torch.equal(got[11:], good[11:]) and (got[5:11] == 0).all()
    # more nodes than max_nodes: only the first max_nodes rows of the sequence are the call's
    out = torch.full_like(case.q, 7.0).cuda()
    run(pa, case, kernel=kernel, max_nodes=5, out=out)
    assert pa.device_error_flags() == pa.PA_DEVERR_QUERY_LOC
    assert torch.equal(out[:5].cpu(), good[:5]) and (out[5:10] == 0).all() and torch.equal(out[11:].cpu(), good[11:])
    # rows past total_q, and rows out of order
    d = case.device()
    for qsl in ([0, 5, 11, 16], [0, 5, 4, 8]):
        d["query_start_loc"] = torch.tensor(qsl, dtype=torch.int32, device="cuda")
        got = pa.paged_attention_tree(**d, scale=case.scale, kernel=kernel).cpu()
        assert pa.device_error_flags() == pa.PA_DEVERR_QUERY_LOC
        assert torch.equal(got[:4], good[:4])


@pytest.mark.parametrize("kernel", [0, 1])
def test_other_streams_and_a_captured_step_share_nothing(cuda_lib, kernel):
    """Two graphs and an eager call, each with its own scratch, replayed in turn and at once."""
    pa = cuda_lib
    cases = [TreeCase(20 + i, [900, 40 + i], [16, 9], q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=BF16)
             for i in range(2)]
    want = [run(pa, c, kernel=kernel, partition_tokens=64).cpu() for c in cases]
    ds = [c.device() for c in cases]
    torch.cuda.synchronize()  # the inputs, before other streams read them
    graphs, outs = [], []
    for c, d in zip(cases, ds):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            pa.paged_attention_tree(**d, scale=c.scale, kernel=kernel, partition_tokens=64)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(pa.paged_attention_tree(**d, scale=c.scale, kernel=kernel, partition_tokens=64))
        graphs.append((g, s))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        eager = pa.paged_attention_tree(**ds[0], scale=cases[0].scale, kernel=kernel, partition_tokens=64)
    torch.cuda.synchronize()
    assert torch.equal(outs[0].cpu(), want[0]) and torch.equal(outs[1].cpu(), want[1])
    assert torch.equal(eager.cpu(), want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = pa.paged_attention_tree(**ds[1], scale=cases[1].scale, kernel=kernel, partition_tokens=64, stream=stream)
        side.synchronize()
        assert torch.equal(got.cpu(), want[1])


@pytest.mark.parametrize("kernel", [0, 1])
def test_workspaces(cuda_lib, kernel):
    pa = cuda_lib
    case = TreeCase(30, [900, 300], [16, 9], q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    n = pa.tree_workspace_size(2, 25, 16, case.table.shape[1], 16, 8, 2, 64, BF16, partition_tokens=64,
                               kernel=kernel)
    assert n > 0
    auto = run(pa, case, kernel=kernel, partition_tokens=64, max_nodes=16)
    own = run(pa, case, kernel=kernel, partition_tokens=64, max_nodes=16,
              workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(auto, own)
    check(pa, case, run(pa, case, kernel=kernel, partition_tokens=64, workspace=None), kernel)
    with pytest.raises(pa.PagedAttnError) as e:
        run(pa, case, kernel=kernel, partition_tokens=64, max_nodes=16,
            workspace=torch.empty(n - 16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == pa.PA_EWORKSPACE


def test_the_same_call_gives_the_same_bits(cuda_lib):
    case = TreeCase(31, [1500, 60], [24, 50], q_heads=16, kv_heads=4, head_dim=128, block_size=16, dtype=BF16)
    first = run(cuda_lib, case)
    for _ in range(5):
        assert torch.equal(run(cuda_lib, case), first)


def test_an_empty_batch(cuda_lib):
    case = TreeCase(32, [5], [0], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    assert run(cuda_lib, case).shape == (0, 4, 64)
    d = case.device()
    d.update(q=torch.ones((3, 4, 64), dtype=BF16, device="cuda"), tree_mask=None,
             query_start_loc=torch.zeros(1, dtype=torch.int32, device="cuda"),
             block_table=d["block_table"][:0], context_lens=d["context_lens"][:0])
    cuda_lib.paged_attention_tree(**d)
    assert cuda_lib.device_error_flags() == 0


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [FP16, FP32])
@pytest.mark.parametrize("batch", [129, 384, 385, 900])
def test_more_sequences_than_threads(cuda_lib, kernel, dtype, batch):
    """Lengths are looked at in chunks of a CTA's threads; one sequence of a late chunk is refused."""
    rng = np.random.default_rng(batch)
    hist, new = rng.integers(0, 70, batch), rng.integers(0, 5, batch)
    hist[::17] = rng.integers(500, 900, len(hist[::17]))
    hist[:3] = new[:3] = 0
    new[batch - 2] = 3
    case = TreeCase(batch, hist.tolist(), new.tolist(), q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case, kernel=kernel, max_nodes=4), kernel)
    d = case.device()
    d["context_lens"][batch - 2] = 2
    got = cuda_lib.paged_attention_tree(**d, scale=case.scale, kernel=kernel, max_nodes=4)
    q0 = int(case.qsl[batch - 2])
    assert (got[q0:q0 + 3] == 0).all() and cuda_lib.device_error_flags() == cuda_lib.PA_DEVERR_QUERY_LOC
    got[q0:q0 + 3] = run(cuda_lib, case, kernel=kernel, max_nodes=4)[q0:q0 + 3]
    check(cuda_lib, case, got, kernel)


@pytest.mark.parametrize("dtype,G,m", [(BF16, 4, 16), (FP16, 8, 40), (FP32, 1, 12), (BF16, 1, 300)])
def test_many_long_calls_behind_one_another(cuda_lib, dtype, G, m):
    """Calls that overlap at their ends: the same bits every time, and no wait runs out."""
    rng = np.random.default_rng(m)
    case = TreeCase(m, rng.integers(0, 1500, 12).tolist(), rng.integers(1, m + 1, 12).tolist(), q_heads=8 * G, kv_heads=8,
                    head_dim=128, block_size=16, dtype=dtype, words=5)
    d = case.device()
    first = cuda_lib.paged_attention_tree(**d, scale=case.scale, max_nodes=m)
    outs = [torch.empty_like(first) for _ in range(4)]
    for i in range(200):
        cuda_lib.paged_attention_tree(**d, scale=case.scale, max_nodes=m, out=outs[i % 4])
    check(cuda_lib, case, first)
    assert all(torch.equal(o, first) for o in outs)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("kernel", [0, 1])
def test_the_largest_values(cuda_lib, dtype, kernel):
    """The largest finite numbers: where a row does not see them they do nothing, where it does they keep their
    size."""
    case = TreeCase(40, [70, 5], [24, 9], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    top = torch.finfo(dtype).max
    for b in range(2):
        for j, x in ((2, top), (3, -top)):
            blk, tok = case.row_of(b, case.hist[b] + j)
            case.v[blk, tok] = x
            case.k[blk, tok, :, :9] = x
    for row in range(33):
        case.mask[row] &= ~12
    check(cuda_lib, case, run(cuda_lib, case, kernel=kernel), kernel)
    blk, tok = case.row_of(0, 33)
    case.v[blk, tok, :, 7] = top
    check(cuda_lib, case, run(cuda_lib, case, kernel=kernel), kernel)


def test_more_work_than_positions_of_the_plan(cuda_lib):
    """Refused on the host, before the arrays matter."""
    pa = cuda_lib
    p = torch.zeros(64, dtype=torch.int64, device="cuda").data_ptr()
    assert pa.load_library().paged_attention_tree(p, p, p, 8, None, 0, 4, p, p, p, 2 ** 24, p, 2 ** 10, 8, 16, 0.125, 8, 2,
                                                  64, pa.PA_BF16, None, 0, None, None) == pa.PA_EUNSUPPORTED


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("entry", [0, 1, 2, 3, 5])
def test_what_an_earlier_sequence_left_does_not_stand_in_for_a_bad_block(cuda_lib, kernel, dtype, entry):
    """One CTA takes both sequences; every drafted key of the first is NaN."""
    pa = cuda_lib
    case = TreeCase(41, [100, 80], [60, 9], q_heads=4, kv_heads=1, head_dim=64, block_size=16, dtype=dtype)
    for j in range(60):
        blk, tok = case.row_of(0, 100 + j)
        case.k[blk, tok] = float("nan")
    case.table[1, entry] = -1
    got = run(pa, case, kernel=kernel, partition_tokens=8192)
    assert torch.isfinite(got[60:].float()).all()
    assert pa.device_error_flags() == pa.PA_DEVERR_BLOCK_ID
    case.k = torch.nan_to_num(case.k)
    case.v = torch.nan_to_num(case.v)
    assert torch.equal(got[60:], run(pa, case, kernel=kernel, partition_tokens=8192)[60:])


def test_long_fp32_contexts_keep_their_last_bits(cuda_lib):
    """One CTA sums up 12,000 keys.  Relative to the result, as root mean squares: 2^-24 for its rounding; partial
    sums of 16 keys that are cut off, at most 2^-22; 188 rounded additions to the running sums of each of four
    warps, at most 2^-24 each and of either sign, so about sqrt(188) / 2 of one, 2^-21.2; scores of size 1, off by
    four such steps, at most 2^-21, independent from key to key.  Below 2^-20 together; a sum whose every step is
    cut off comes to 188 * 6 * 2^-24 or 2^-14 at most, and to several times 2^-20 in fact."""
    case = TreeCase(42, [12000, 11000], [6, 3], q_heads=1, kv_heads=1, head_dim=64, block_size=32, dtype=FP32)
    got = run(cuda_lib, case, partition_tokens=16384)
    rows, ref, _, _ = oracle.tree.paged_tree_attention(case.q, case.qsl, case.mask, case.k, case.v, case.table, case.ctx,
                                                       case.scale)
    off = got.cpu().double().numpy()[rows] - ref
    assert np.sqrt((off ** 2).mean() / (ref ** 2).mean()) < 2.0 ** -20
