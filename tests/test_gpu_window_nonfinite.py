"""Chunks behind a window over pools that hold values which are not finite: who sees them, and what that costs."""
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
    cuda_lib.device_error_flags(clear=True)


def check(pa, case, **kw):
    """Outputs are not finite exactly where a row sees such a value in the column, and the attention elsewhere."""
    got = pa.paged_attention_window(**case.device(), window=case.window, sinks=case.sinks, scale=case.scale, **kw)
    got = got.cpu().double().numpy()
    assert pa.device_error_flags() == 0
    bad = torch.where(torch.isfinite(case.v), 0.0, 1.0)
    kept = case.v.clone()
    with np.errstate(invalid="ignore"):
        rows, _, hit, size = case.oracle()
    seen = ~np.isfinite(hit)
    case.v.masked_fill_(bad.bool(), 0.0)
    _, ref, spread, size = case.oracle()
    tol = pool_bound(case, ref, spread, size, kw.get("kernel") == 1)
    case.v.copy_(kept)
    # (values made 0 for the oracle weigh nothing in the columns where nobody sees them)
    assert np.array_equal(~np.isfinite(got[rows]), seen)
    off = (np.abs(got[rows] - ref) - tol)[~seen]
    assert (off <= 0).all(), f"worst excess {off.max()}"
    return seen


SHAPES = [  # contexts, chunks, window, sinks, q heads, kv heads, head_dim, block size
    ([700, 300], [400, 300], 100, 4, 8, 2, 64, 16),
    ([700, 300], [400, 300], 100, 0, 2, 2, 128, 32),
    ([900, 5, 260], [700, 5, 130], 300, 33, 16, 1, 64, 16),
    ([900, 40], [260, 40], ALL, 0, 4, 1, 128, 16),
    ([520, 520], [300, 1], 17, 200, 12, 12, 64, 64),
    ([600], [600], 1, 1, 8, 1, 128, 16),
]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("kernel", [0, 1])
def test_a_few_values(cuda_lib, dtype, shape, seed, kernel):
    ctx, new, window, sinks, hq, hkv, D, S = SHAPES[shape]
    case = WindowCase(seed, ctx, new, window, sinks, q_heads=hq, kv_heads=hkv, head_dim=D, block_size=S, dtype=dtype)
    rng = np.random.default_rng([seed, shape])
    for b, n in enumerate(ctx):
        at = case.seen[b]
        # in the chunk, at the windows' beginnings, among the sinks and anywhere
        for j in {at[0], at[-1], at[rng.integers(len(at))], at[rng.integers(len(at))], max(n - new[b], 0), n - 1 - rng.integers(min(n, 20))}:
            if j in at and rng.random() < 0.6:
                blk, tok = case.row_of(b, j)
                case.v[blk, tok, rng.integers(hkv), rng.integers(D)] = [float("nan"), float("inf"), -float("inf")][rng.integers(3)]
    check(cuda_lib, case, kernel=kernel)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("every", [1, 2, 7])
def test_many_values(cuda_lib, dtype, every):
    """A token in so many of whose values one is NaN, each in another column."""
    case = WindowCase(3, [700, 90], [500, 90], 200, 4, q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    for b in range(2):
        for j in case.seen[b][::every]:
            case.v[case.row_of(b, j)][j % 2, 5 * j % 64] = float("nan")
    seen = check(cuda_lib, case)
    assert seen.any()


def test_large_values(cuda_lib):
    """Weights are 1 at most and their sums stay finite where their average does."""
    case = WindowCase(4, [150], [100], 50, 2, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    case.v = torch.where(torch.isfinite(case.v), case.v.sign() * 1e38 + case.v * 1e37, case.v.float()).to(BF16)
    check(cuda_lib, case)


def us(call, times=5):
    for _ in range(2):
        call()
    best = float("inf")
    for _ in range(times):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
    return best


@pytest.mark.parametrize("batch,rows,ctx,window,sinks", [(8, 2048, 4096, 1024, 4), (1, 2048, 8192, ALL, 0)])
def test_one_value_costs_no_more_than_the_call(cuda_lib, batch, rows, ctx, window, sinks):
    pa, S = cuda_lib, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    pools = torch.randn((2, batch * ctx // S, S, 8, 128), generator=g, device="cuda", dtype=BF16)
    table = torch.arange(batch * ctx // S, dtype=torch.int32, device="cuda").view(batch, -1)
    q = torch.randn((batch * rows, 32, 128), generator=g, device="cuda", dtype=BF16)
    qsl, lens = int32([rows * b for b in range(batch + 1)]).cuda(), int32([ctx] * batch).cuda()
    call = lambda: pa.paged_attention_window(q, qsl, pools[0], pools[1], table, lens, window, sinks)  # noqa: E731
    clean, fine = us(call), call()
    at = ctx - rows // 2 + 5  # a token of the chunk of the first sequence, in one column
    pools[1, at // S, at % S, :, 7] = float("nan")
    one, got = us(call), call()
    r = torch.arange(batch * rows, device="cuda")
    p = r % rows + ctx - rows
    sees = (r < rows) & (p >= at) & (p < at + window)
    want = sees[:, None, None] & (torch.arange(128, device="cuda") == 7)
    assert torch.equal(torch.isnan(got), want.expand_as(got))
    assert torch.equal(got[~sees], fine[~sees])
    pools[1, 0, 0, :, 7] = float("nan")  # and the first token, a sink or far from most rows
    both = us(call)
    assert max(one, both) <= 3 * clean + 300, (clean, one, both)
