"""GPU parity of paged_attention_window against the float64 oracle, where it can go wrong."""
import numpy as np
import pytest
import torch

from window_cases import ALL, WindowCase, int32, pool_bound

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _clean(cuda_lib):
    cuda_lib.device_error_flags(clear=True)
    yield
    cuda_lib.set_checked_mode(False)
    cuda_lib.device_error_flags(clear=True)


def run(pa, case, **kw):
    return pa.paged_attention_window(**case.device(), window=case.window, sinks=case.sinks, scale=case.scale, **kw)


def check(pa, case, got, kernel=0, flags=0):
    torch.cuda.synchronize()
    rows, ref, spread, size = case.oracle()
    g = got.cpu().double().numpy()[rows]
    tol = pool_bound(case, ref, spread, size, cuda_cores=case.qsl is not None and kernel == 1)
    assert np.isfinite(g).all()
    off = np.abs(g - ref) - tol
    assert (off <= 0).all(), f"worst excess {off.max()} at {np.unravel_index(off.argmax(), off.shape)}"
    assert pa.device_error_flags() == flags


CTX = [1, 0, 17, 300, 129, 64, 1000]
NEW = [1, 0, 17, 40, 1, 64, 130]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("window,sinks", [(100, 4), (ALL, 0)])
def test_single_tokens(cuda_lib, dtype, D, G, window, sinks):
    case = WindowCase(10 * G + D, CTX, None, window, sinks, q_heads=2 * G, kv_heads=2, head_dim=D, block_size=16, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case))


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_chunks(cuda_lib, kernel, dtype, D, G):
    case = WindowCase(10 * G + D, CTX, NEW, 100, 4, q_heads=2 * G, kv_heads=2, head_dim=D, block_size=16, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case, kernel=kernel), kernel)


@pytest.mark.parametrize("chunks", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 127, 128, 129, 500, 5000])
@pytest.mark.parametrize("sinks", [0, 1, 16, 33, 200, 5000])
def test_windows_and_sinks(cuda_lib, chunks, dtype, window, sinks):
    """Sinks that end inside a block or tile, touch the window, lie in it or cover everything."""
    case = WindowCase(window + sinks, [640, 33, 260], [150, 33, 3] if chunks else None, window, sinks, q_heads=4, kv_heads=2,
                      head_dim=64, block_size=16, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case))


@pytest.mark.parametrize("chunks", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("S", [1, 2, 4, 8, 16, 32, 64, 128, 256])
def test_block_sizes(cuda_lib, chunks, dtype, S):
    case = WindowCase(S, [100, 7, 555], [70, 7, 9] if chunks else None, 60, 5, q_heads=6, kv_heads=3, head_dim=64,
                      block_size=S, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case), 1 if S < 16 else 0)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("part", [0, 1, 64, 200, 256, 4096])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_split_contexts(cuda_lib, dtype, part, workspace):
    case = WindowCase(part, [3000, 5, 700, 1201], None, 1100, 7, q_heads=8, kv_heads=2, head_dim=128, block_size=16,
                      dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case, partition_tokens=part, workspace=workspace))


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_windowless_single_tokens_agree_with_the_decode_call(cuda_lib, dtype):
    case = WindowCase(3, [40, 900, 1], None, ALL, 0, q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=dtype)
    d = case.device()
    check(cuda_lib, case, run(cuda_lib, case))
    check(cuda_lib, case, cuda_lib.paged_attention_decode(d["q"], d["k_pool"], d["v_pool"], d["block_table"],
                                                          d["context_lens"], case.scale))


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_rows_that_belong_to_nobody_stay(cuda_lib, kernel, dtype):
    case = WindowCase(4, [40, 300, 5], [11, 130, 5], 64, 2, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype,
                      tail=70)
    out = torch.full_like(case.q, 7.0).cuda()
    got = run(cuda_lib, case, kernel=kernel, out=out)
    check(cuda_lib, case, got, kernel)
    assert (got[146:] == 7.0).all()
    # and rows before the first sequence
    case.qsl = case.qsl + 3
    case.new_list[0] = 11
    out = torch.full_like(case.q, 7.0).cuda()
    got = run(cuda_lib, case, kernel=kernel, out=out)
    check(cuda_lib, case, got, kernel)
    assert (got[:3] == 7.0).all() and (got[149:] == 7.0).all()


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see_does_not_enter_it(cuda_lib, kernel, dtype, bad):
    """Non-finite keys and values that some rows of a chunk see (or none of a tile's): the others keep their results."""
    case = WindowCase(6, [400, 90, 64], [150, 90, 64], 70, 4, q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    for b, j in ((0, 2), (0, 200), (0, 260), (0, 330), (1, 0), (1, 60), (2, 31)):
        blk, tok = case.row_of(b, j)
        case.v[blk, tok, :, 5:20] = bad
    for b, j in ((0, 300), (1, 30)):
        case.k[case.row_of(b, j)] = bad
    got = run(cuda_lib, case, kernel=kernel).cpu().double().numpy()
    rows, ref, spread, size = case.oracle()
    fine = np.isfinite(ref) & np.isfinite(size)[:, :, None]
    assert fine.any() and not fine.all()
    size0 = np.where(np.isfinite(size), size, 0.0)
    tol = pool_bound(case, np.where(fine, ref, 0), np.where(fine, spread, 0), size0, kernel == 1)
    assert (np.abs(got - ref)[fine] <= tol[fine]).all()
    seen = ~np.isfinite(spread) & np.isfinite(size)[:, :, None]
    assert not np.isfinite(got[seen]).any()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("part", [0, 64])
def test_single_tokens_with_infinite_scores(cuda_lib, dtype, part):
    """Keys of -inf weigh nothing wherever they lie; nothing but them gives 0 / 0."""
    case = WindowCase(7, [400, 20, 300], None, 200, 4, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    case.q = case.q.abs() + 0.5
    for j in case.seen[0][:70] + case.seen[0][100:101]:
        case.k[case.row_of(0, j)] = -float("inf")
    for j in case.seen[1]:
        case.k[case.row_of(1, j)] = -float("inf")
    got = run(cuda_lib, case, partition_tokens=part).cpu().double().numpy()
    assert np.isnan(got[1]).all()
    keep = [0, 2]
    rows, ref, spread, size = case.oracle()
    size = np.where(np.isfinite(size), size, 100.0)  # (the scores that are left are far below that)
    tol = pool_bound(case, ref, spread, size)
    assert (np.abs(got - ref)[keep] <= tol[keep]).all()


@pytest.mark.parametrize("chunks", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_large_scores(cuda_lib, chunks, dtype):
    """Scores far apart: one key has all the weight, and the stabiliser moves often."""
    case = WindowCase(8, [500, 260], [40, 100] if chunks else None, 300, 4, q_heads=4, kv_heads=2, head_dim=64,
                      block_size=16, dtype=dtype, gain=60.0)
    got = run(cuda_lib, case).cpu().double().numpy()
    rows, ref, spread, size = case.oracle()
    assert (np.abs(got - ref) <= pool_bound(case, ref, spread, size)).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_refused_sequences_give_zeros(cuda_lib, dtype):
    case = WindowCase(9, [50, 60, 70], None, 30, 2, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    d = case.device()
    for wrong in (-1, 97):  # (the table holds 6 blocks)
        d["context_lens"] = int32([50, wrong, 70]).cuda()
        got = cuda_lib.paged_attention_window(**d, window=30, sinks=2, scale=case.scale)
        rows, ref, spread, size = case.oracle()
        tol = pool_bound(case, ref, spread, size)
        g = got.cpu().double().numpy()
        assert (np.abs(g - ref)[[0, 2]] <= tol[[0, 2]]).all() and (g[1] == 0).all()
        assert cuda_lib.device_error_flags() == cuda_lib.PA_DEVERR_CONTEXT_LEN
        cuda_lib.set_checked_mode(True)
        with pytest.raises(cuda_lib.PagedAttnError) as e:
            cuda_lib.paged_attention_window(**d, window=30, sinks=2)
        assert e.value.status == cuda_lib.PA_ERANGE
        cuda_lib.set_checked_mode(False)


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_refused_chunks_give_zeros(cuda_lib, kernel, dtype):
    case = WindowCase(9, [50, 60, 70], [20, 30, 70], 30, 2, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    d = case.device()
    for wrong in (-1, 97, 29):
        d["context_lens"] = int32([50, wrong, 70]).cuda()
        got = cuda_lib.paged_attention_window(**d, window=30, sinks=2, scale=case.scale, kernel=kernel)
        rows, ref, spread, size = case.oracle()
        tol = pool_bound(case, ref, spread, size, kernel == 1)
        g = got.cpu().double().numpy()
        keep = np.r_[:20, 50:120]
        assert (np.abs(g - ref)[keep] <= tol[keep]).all() and (g[20:50] == 0).all()
        assert cuda_lib.device_error_flags() & cuda_lib.PA_DEVERR_QUERY_LOC
        cuda_lib.set_checked_mode(True)
        with pytest.raises(cuda_lib.PagedAttnError) as e:
            cuda_lib.paged_attention_window(**d, window=30, sinks=2)
        assert e.value.status == cuda_lib.PA_ERANGE
        cuda_lib.set_checked_mode(False)


@pytest.mark.parametrize("chunks", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_bad_blocks_are_masked_and_recorded(cuda_lib, chunks, dtype):
    case = WindowCase(11, [200, 90], [30, 9] if chunks else None, 100, 20, q_heads=4, kv_heads=2, head_dim=64, block_size=16,
                      dtype=dtype)
    d = case.device()
    for j in (0, 8):  # a block of sinks and one of the window, which every query sees whole
        for wrong in (-1, case.num_blocks):
            d["block_table"][0, j] = wrong
            got = cuda_lib.paged_attention_window(**d, window=100, sinks=20, scale=case.scale).cpu().double().numpy()
            assert cuda_lib.device_error_flags() == cuda_lib.PA_DEVERR_BLOCK_ID
            assert np.isfinite(got).all()
            cuda_lib.set_checked_mode(True)
            with pytest.raises(cuda_lib.PagedAttnError):
                cuda_lib.paged_attention_window(**d, window=100, sinks=20)
            cuda_lib.set_checked_mode(False)
            d["block_table"][0, j] = case.table[0, j]
    # a sequence of nothing but bad blocks sees nothing
    d["block_table"][1] = -1
    got = cuda_lib.paged_attention_window(**d, window=100, sinks=20, scale=case.scale).cpu()
    assert (got[30:] == 0).all() if chunks else (got[1] == 0).all()


@pytest.mark.parametrize("chunks", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_checked_mode_lets_freed_blocks_be(cuda_lib, chunks, dtype):
    case = WindowCase(12, [640, 333], [50, 3] if chunks else None, 80, 3, q_heads=4, kv_heads=2, head_dim=64, block_size=16,
                      dtype=dtype)
    assert (case.table == -1).sum() > 20
    cuda_lib.set_checked_mode(True)
    check(cuda_lib, case, run(cuda_lib, case))


@pytest.mark.parametrize("chunks", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_unified_pools(cuda_lib, chunks, dtype):
    case = WindowCase(13, [640, 33], [50, 3] if chunks else None, 80, 3, q_heads=4, kv_heads=2, head_dim=128, block_size=16,
                      dtype=dtype, unified=True)
    check(cuda_lib, case, run(cuda_lib, case))


def test_views_and_a_wide_table(cuda_lib):
    """A table that is a view of a wider one, lengths that are a slice, queries at an offset."""
    case = WindowCase(14, [640, 33, 90], None, 80, 3, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    d = case.device()
    wide = torch.full((3, 100), -7, dtype=torch.int32, device="cuda")
    wide[:, 9:9 + case.table.shape[1]] = d["block_table"]
    d["block_table"] = wide[:, 9:9 + case.table.shape[1]]
    d["context_lens"] = torch.cat([int32([9, 9, 9]).cuda(), d["context_lens"]])[3:]
    d["q"] = torch.cat([d["q"][:1], d["q"]])[1:]
    check(cuda_lib, case, cuda_lib.paged_attention_window(**d, window=80, sinks=3, scale=case.scale))


@pytest.mark.parametrize("batch", [300, 2000])
def test_large_batches(cuda_lib, batch):
    rng = np.random.default_rng(batch)
    ctx = rng.integers(0, 40, batch).tolist()
    case = WindowCase(batch, ctx, None, 9, 2, q_heads=2, kv_heads=1, head_dim=64, block_size=16, dtype=BF16)
    check(cuda_lib, case, run(cuda_lib, case))
    new = [int(rng.integers(0, n + 1)) for n in ctx]
    case = WindowCase(batch, ctx, new, 9, 2, q_heads=2, kv_heads=1, head_dim=64, block_size=16, dtype=BF16)
    check(cuda_lib, case, run(cuda_lib, case))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_captured_call_follows_its_lengths(cuda_lib, dtype):
    """Two captured calls side by side in one graph, replayed with other lengths and tables in the same memory."""
    first = WindowCase(15, [640, 33, 90], None, 80, 3, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    other = WindowCase(16, [600, 640, 17], None, 80, 3, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    nb = max(first.num_blocks, other.num_blocks)
    d, e = first.device(), other.device()

    def grown(p):
        x = torch.zeros((nb,) + p.shape[1:], dtype=p.dtype, device="cuda")
        x[:p.shape[0]] = p
        return x

    d["k_pool"], d["v_pool"] = grown(d["k_pool"]), grown(d["v_pool"])
    outs = [torch.empty_like(d["q"]) for _ in range(2)]
    call = lambda: [cuda_lib.paged_attention_window(**d, window=80, sinks=3, scale=first.scale, out=o) for o in outs]  # noqa: E731
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    graph.replay()
    for o in outs:
        check(cuda_lib, first, o)
    d["k_pool"].copy_(grown(e["k_pool"]))
    d["v_pool"].copy_(grown(e["v_pool"]))
    for n in ("q", "block_table", "context_lens"):
        d[n].copy_(e[n])
    graph.replay()
    for o in outs:
        check(cuda_lib, other, o)


def test_calls_on_two_streams(cuda_lib):
    cases = [WindowCase(s, [3000, 700], None, 1100, 7, q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=BF16)
             for s in (17, 18)]
    devs = [c.device() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(20):
        for i in range(2):
            got[i] = cuda_lib.paged_attention_window(**devs[i], window=1100, sinks=7, scale=cases[i].scale, stream=streams[i])
    torch.cuda.synchronize()
    for c, g in zip(cases, got):
        check(cuda_lib, c, g)


def test_results_do_not_change_from_call_to_call(cuda_lib):
    case = WindowCase(19, [3000, 5, 700, 1201], None, 1100, 7, q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=BF16)
    first = run(cuda_lib, case)
    for _ in range(5):
        assert torch.equal(run(cuda_lib, case), first)
