"""Every key that a query sees counts once and no other does, at any length; and what is left when blocks or chunks are bad."""
import numpy as np
import pytest
import torch

import oracle
from window_cases import ALL, PackedCase, WindowCase, int32, pack, pool_bound

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _clean(cuda_lib):
    cuda_lib.device_error_flags(clear=True)
    yield
    cuda_lib.device_error_flags(clear=True)


FORMS = [("pool", BF16, 16), ("pool", FP16, 8), ("pool", FP32, 16), ("packed", BF16, 16), ("packed", FP32, 32),
         ("chunk", BF16, 16), ("chunk", FP16, 64), ("chunk", BF16, 8), ("chunk", FP32, 16)]
LENGTHS = [(1, 2, 15, 16, 17, 63, 64, 65), (100, 1000, 1023, 1025, 4095, 4097, 10_000, 33_333), (131_072, 131_073, 3, 77_777)]


@pytest.mark.parametrize("form,dtype,S", FORMS)
@pytest.mark.parametrize("lens", range(len(LENGTHS)))
@pytest.mark.parametrize("window,sinks", [(ALL, 0), (500, 37), (70_000, 5)])
@pytest.mark.parametrize("split", [dict(), dict(workspace=None)])
def test_every_key_counts_once(cuda_lib, form, dtype, S, lens, window, sinks, split):
    """Keys are 0, so that all weights are alike; of the values one in each dimension is not 0, of a token of its own.  Sums of
    weights are whole numbers below 2^24 (times a power of two): exact, so what is left is the quotient and its rounding."""
    pa, D, lens = cuda_lib, 64, LENGTHS[lens]
    if form == "chunk" and split:
        pytest.skip("chunks take no workspace")
    if form == "chunk" and (S < 16 or dtype == FP32) and max(lens) > 20_000:
        pytest.skip("a CTA a row: slow")
    rng = np.random.default_rng([len(lens), S, sinks])
    new = [min(n, 5) if form == "chunk" else 1 for n in lens]
    table = np.zeros((len(lens), -(-max(lens) // S)), np.int64)  # (block 0: values of 0)
    marks, blocks = [], [np.zeros((S, 1, D))]
    for b, n in enumerate(lens):
        low = n - window
        at = np.concatenate([[0, n - 1, low - 1, low, low + 1, sinks - 1, sinks, n - 2, n - 5, n // 2 // 16 * 16], rng.integers(n, size=D)])
        at = np.array([j % n for j in at[:D]])
        marks.append(at)
        for d, j in enumerate(at):
            if table[b, j // S] == 0:
                table[b, j // S] = len(blocks)
                blocks.append(np.zeros((S, 1, D)))
            blocks[table[b, j // S]][j % S, 0, d] = 15 * 2.0 ** 10
    v = torch.from_numpy(np.stack(blocks)).float()
    k, table_d, lens_d = torch.zeros_like(v), torch.from_numpy(table).to(torch.int32).cuda(), int32(list(lens)).cuda()
    q = torch.randn((sum(new), 2, D), generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    if form == "packed":
        (kc, kp), (vc, vp) = pack(k), pack(v)
        got = pa.paged_attention_decode_q4(q, pa.Q4Cache(*(x.cuda() for x in (kc, vc, kp, vp))), table_d, lens_d, window, sinks, **split)
    else:
        qsl = int32([0] + list(np.cumsum(new))).cuda() if form == "chunk" else None
        got = pa.paged_attention_window(q, qsl, k.to(dtype).cuda(), v.to(dtype).cuda(), table_d, lens_d, window, sinks, **split)
    assert pa.device_error_flags() == 0
    got, row = got.double().cpu().numpy(), 0
    half = torch.finfo(dtype).eps / 2
    for b, n in enumerate(lens):
        for r in range(new[b]):
            p = n - new[b] + r
            j = marks[b]
            sees = (j <= p) & ((j > p - window) | (j < sinks))
            count = min(p + 1, window + min(sinks, max(p + 1 - window, 0)))
            want = np.where(sees, 15 * 2.0 ** 10 / count, 0.0)
            assert (np.abs(got[row] - want) <= want * (half + 2.0 ** -21) * (1 + half)).all(), (n, r)
            row += 1


@pytest.mark.parametrize("what", ["one", "chunk", "cuda cores", "packed"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("wrong", [-1, 10 ** 6])
@pytest.mark.parametrize("blocks", [(0,), (8,), (1, 8, 11), (12,)])
def test_the_blocks_that_are_left(cuda_lib, what, dtype, wrong, blocks):
    """Blocks outside the pool are masked: the attention over the others."""
    pa, window, sinks, S = cuda_lib, 100, 20, 16
    kw = dict(q_heads=4, kv_heads=2, head_dim=64, block_size=S, dtype=dtype)
    chunks = what in ("chunk", "cuda cores")
    case = PackedCase(11, [200, 90], window, sinks, **kw) if what == "packed" else \
        WindowCase(11, [200, 90], [30, 9] if chunks else None, window, sinks, **kw)
    if what == "packed":
        k, v = (oracle.window.q4_values(c, p).reshape(-1, 2, 64) for c, p in ((case.kc, case.kp), (case.vc, case.vp)))
    else:
        k, v = (x.double().numpy().reshape(-1, 2, 64) for x in (case.k, case.v))
    d = case.device()
    for j in blocks:
        d["block_table"][0, j] = wrong
    if what == "packed":
        got = pa.paged_attention_decode_q4(cache=case.cache(pa), **d, window=window, sinks=sinks, scale=case.scale)
    else:
        got = pa.paged_attention_window(**d, window=window, sinks=sinks, scale=case.scale, kernel=int(what == "cuda cores"))
    assert pa.device_error_flags() == pa.PA_DEVERR_BLOCK_ID
    m, n = (30 if chunks else 1), 200
    rows, ref, spread, size = case.oracle()
    for r in range(m):
        at = [j for j in oracle.window.seen_positions(n - m + r, window, sinks) if j // S not in blocks]
        slots = [case.row_of(0, int(j)) for j in at]
        slots = [blk * S + tok for blk, tok in slots]
        rep = lambda x: np.repeat(x[slots], 2, 1)  # noqa: E731
        ref[r], spread[r], plain = oracle.window.attend(case.q[r].double().numpy(), rep(k), rep(v), case.scale)
        size[r] = np.maximum(size[r], plain)
    tol = case.bound(ref, spread, size) if what == "packed" else pool_bound(case, ref, spread, size, what == "cuda cores")
    assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("every", [2, 3])
def test_chunks_between_refused_ones(cuda_lib, every):
    """Items with tiles and without in turn: a sample of the rows that are not refused against the oracle, all of them
    against the CUDA-core kernel."""
    pa, n = cuda_lib, 1200
    good = [b % every == 0 for b in range(n)]
    new = [1 + 97 * b % 270 if ok else 1 + b % 3 for b, ok in enumerate(good)]
    ctx = [m + b % 40 if ok else 0 for b, (m, ok) in enumerate(zip(new, good))]
    case = WindowCase(18, ctx, [m if ok else 0 for m, ok in zip(new, good)], 50, 2, q_heads=2, kv_heads=2, head_dim=64,
                      block_size=16, dtype=BF16)
    d = case.device()
    qsl = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn((int(qsl[-1]), 2, 64), generator=torch.Generator().manual_seed(1)).to(BF16)
    mine = torch.cat([torch.arange(qsl[b], qsl[b + 1]) for b in range(n) if good[b]])
    q[mine] = case.q
    d["q"], d["query_start_loc"] = q.cuda(), int32(qsl).cuda()
    got, cores = (pa.paged_attention_window(**d, window=50, sinks=2, scale=case.scale, kernel=k).cpu() for k in (0, 1))
    assert pa.device_error_flags() == pa.PA_DEVERR_QUERY_LOC  # (nothing timed out)
    other = torch.ones(q.shape[0], dtype=torch.bool)
    other[mine] = False
    assert (got[other] == 0).all() and (cores[other] == 0).all()
    # (values are normal numbers, so the absolute weighted ones are below 6; two kernels, each within its own bound)
    assert (got.float() - cores.float()).abs().max() <= 6 * 2.0 ** -8 * 2 + 6 * 2.0 ** -8
    for b in [b for b in range(n) if good[b]][::37]:
        rows, ref, spread, size = oracle.window.window_attention(q[qsl[b]:qsl[b + 1]], int32([0, new[b]]), case.k, case.v,
                                                                 case.table[b:b + 1], case.ctx[b:b + 1], case.scale, 50, 2)
        off = np.abs(got[qsl[b]:qsl[b + 1]].double().numpy() - ref) - pool_bound(case, ref, spread, size)
        assert (off <= 0).all(), b
