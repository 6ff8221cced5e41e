"""GPU tests of paged_attention_tree at the edges of what its calls allow: refused sequences, tables and pools of
unusual layout, weights and scores at the ends of a type's range."""
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


def refused(pa, case, rows, flag, kernel, **change):
    """The call over a buffer of sevens: zeros in `rows`, the fitting sequences' results elsewhere, sevens in none
    of both."""
    d = case.device()
    good = pa.paged_attention_tree(**d, scale=case.scale, kernel=kernel, workspace=None)
    qsl = change.pop("qsl", case.qsl.tolist())
    kept = change.pop("kept")
    d["query_start_loc"] = torch.tensor(qsl, dtype=torch.int32, device="cuda")
    out = torch.full_like(d["q"], 7.0)
    pa.paged_attention_tree(**d, scale=case.scale, kernel=kernel, out=out, workspace=None, **change)
    assert pa.device_error_flags() == flag
    for r in range(out.shape[0]):
        want = torch.zeros_like(out[r]) if r in rows else good[r] if r in kept else torch.full_like(out[r], 7.0)
        assert torch.equal(out[r], want), r


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_every_row_of_a_refused_sequence_is_zero(cuda_lib, kernel, dtype):
    pa = cuda_lib
    case = TreeCase(15, [64, 100, 3], [5, 7, 4], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype, tail=4)
    first, last = set(range(5)), set(range(12, 16))
    # two nodes more than max_nodes
    refused(pa, case, set(range(5, 12)), pa.PA_DEVERR_QUERY_LOC, kernel, kept=first | last, max_nodes=5)
    # the last sequence reaches past the rows: those that it has
    refused(pa, case, set(range(12, 20)), pa.PA_DEVERR_QUERY_LOC, kernel, kept=first | set(range(5, 12)),
            qsl=[0, 5, 12, 23])
    refused(pa, case, set(range(12, 20)), pa.PA_DEVERR_QUERY_LOC, kernel, kept=first | set(range(5, 12)),
            qsl=[0, 5, 12, 2 ** 31 - 1])
    # the first begins before them, and one that has none of them
    refused(pa, case, first, pa.PA_DEVERR_QUERY_LOC, kernel, kept=set(range(5, 12)) | last, qsl=[-2, 5, 12, 16])
    refused(pa, case, set(), pa.PA_DEVERR_QUERY_LOC, kernel, kept=first | set(range(5, 12)), qsl=[0, 5, 12, -9])


@pytest.mark.parametrize("kernel", [0, 1])
def test_a_tree_wider_than_its_mask_gives_zeros(cuda_lib, kernel):
    pa = cuda_lib
    case = TreeCase(16, [40, 9], [70, 3], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16, words=2)
    d = case.device()
    good = pa.paged_attention_tree(**d, scale=case.scale, kernel=kernel, workspace=None)
    d["tree_mask"] = d["tree_mask"][:, :1].contiguous()
    out = torch.full_like(good, 7.0)
    pa.paged_attention_tree(**d, scale=case.scale, kernel=kernel, out=out, max_nodes=73, workspace=None)
    assert pa.device_error_flags() == pa.PA_DEVERR_TREE
    assert (out[:70] == 0).all() and torch.equal(out[70:], good[70:])


@pytest.mark.parametrize("kernel", [0, 1])
def test_a_sequence_that_straddles_the_token_arrays(cuda_lib, kernel):
    """What build_block_tables leaves of a sequence past its arrays, attention turns into zeros."""
    pa = cuda_lib
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    table[0, :1], table[1, :3], table[2, :1] = i32([0]), i32([1, 2, 3]), i32([4])
    t = pa.build_block_tables(i32([16, 40, 3]), i32([3, 30, 5]), table, i32([1, 3, 1]), i32(list(range(5, 24))),
                              i32([19, 0]), 16, 24, num_tokens=20)
    assert pa.device_error_flags() == pa.PA_DEVERR_QUERY_LOC
    k, v = (torch.randn((24, 16, 2, 64), device="cuda").to(BF16) for _ in range(2))
    q = torch.randn((20, 4, 64), device="cuda").to(BF16)
    out = torch.full_like(q, 7.0)
    pa.paged_attention_tree(q, t.query_start_loc, None, k, v, table, t.context_lens, out=out, kernel=kernel)
    assert pa.device_error_flags() == pa.PA_DEVERR_QUERY_LOC
    assert (out[3:] == 0).all() and torch.isfinite(out).all() and not (out[:3] == 7.0).any() and (out[:3] != 0).any()


def tight_bound(case, ref, spread, size, tensor_cores: bool):
    """tree_cases.bound with two of its terms put right for fp16: a result is off by half a step of its type, and that
    is never less than 2^-25; a weight that tensor cores round is off by half a step of itself, but at least by 2^-32
    of the row's largest (they are formed 2^7 higher, and 2^-25 is the half step of the smallest numbers)."""
    keys, values = int(case.ctx.max()), float(case.v[torch.isfinite(case.v)].abs().max())
    half = torch.finfo(case.dtype).eps / 2
    tol = bound(case.dtype, ref, spread, size, keys, case.q.shape[2], values, False)
    if case.dtype == FP16:
        tol = tol + 2.0 ** -25
    if tensor_cores:
        tol = tol + spread * half * (1 + half) ** 2
        if case.dtype == FP16:
            tol = tol + keys * 2.0 ** -32 * values * (1 + half)
    return tol


def check_tight(pa, case, kernel, **kw):
    got = pa.paged_attention_tree(**case.device(), scale=case.scale, kernel=kernel, **kw)
    rows, ref, spread, size = oracle.tree.paged_tree_attention(case.q, case.qsl, case.mask, case.k, case.v, case.table,
                                                               case.ctx, case.scale)
    tol = tight_bound(case, ref, spread, size, kernel != 1 and case.dtype != FP32)
    off = np.abs(got.cpu().double().numpy()[rows] - ref) - tol
    assert (off <= 0).all(), f"worst excess {off.max()} at {np.unravel_index(off.argmax(), off.shape)}"
    assert pa.device_error_flags() == 0
    return ref


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("strong", [0, 700, 4990])
@pytest.mark.parametrize("part", [0, 8192])
def test_many_weak_keys_next_to_a_strong_one(cuda_lib, kernel, m, strong, part):
    """5,000 weights of 2^-25.5 of the largest, which fp16 numbers below 2^-24 cannot hold, make up the whole result."""
    case = TreeCase(50, [4996], [m], q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=FP16, words=0)
    case.q = torch.ones_like(case.q)
    token = ~torch.isnan(case.k)
    case.k[token], case.v[token] = 0.0, 1.0
    blk, tok = case.row_of(0, strong)
    case.k[blk, tok] = 25.5 / (8 * 1.4426950408889634)  # 64 of them times the scale of 1/8
    case.v[blk, tok] = 0.0
    ref = check_tight(cuda_lib, case, kernel, partition_tokens=part)
    assert (ref[0] > 5e-5).all() and (ref < 3e-4).all()


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("gain,size", [(1.0, 2.0 ** -9), (6.0, 1.0), (30.0, 2.0 ** -12)])
def test_small_results_and_uneven_weights(cuda_lib, kernel, dtype, gain, size):
    case = TreeCase(51, [700, 20, 0], [9, 60, 5], q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=dtype, gain=gain)
    case.v = (case.v.float() * size).to(dtype)
    check_tight(cuda_lib, case, kernel)
    check_tight(cuda_lib, case, kernel, partition_tokens=128)


@pytest.mark.parametrize("m", [9, 60])
def test_fp16_weights_at_their_largest(cuda_lib, m):
    """The maximum grows by almost 2^8 within what moves no stabiliser, 64 keys at a time, under large values."""
    case = TreeCase(52, [640], [m], q_heads=4, kv_heads=1, head_dim=64, block_size=16, dtype=FP16)
    case.q = torch.ones_like(case.q)
    for j in range(640 + m):
        blk, tok = case.row_of(0, j)
        case.k[blk, tok] = 7.9 / (8 * 1.4426950408889634) * (j // 64) / 2
        case.v[blk, tok] = 60000.0
    check_tight(cuda_lib, case, 0)


@pytest.mark.parametrize("kernel,S", [(0, 16), (1, 16), (0, 4)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("part", [0, 64])
def test_a_seen_key_whose_score_is_minus_infinity_has_no_weight(cuda_lib, kernel, S, dtype, part):
    """Results as if no row saw the key, whatever the block size."""
    case = TreeCase(53, [90, 3, 128], [20, 50, 64], q_heads=8, kv_heads=2, head_dim=64, block_size=S, dtype=dtype)
    case.q = case.q.abs() + 0.5
    for b in range(3):
        blk, tok = case.row_of(b, case.hist[b] + 7)
        case.k[blk, tok] = -float("inf")
    sevens = (case.mask[:, 0] >> 7) & 1
    assert sevens.any() and not sevens.all()
    got = cuda_lib.paged_attention_tree(**case.device(), scale=case.scale, kernel=kernel, partition_tokens=part)
    case.mask[:, 0] &= ~(1 << 7)
    case.k = torch.nan_to_num(case.k, neginf=0.0)
    rows, ref, spread, size = oracle.tree.paged_tree_attention(case.q, case.qsl, case.mask, case.k, case.v, case.table,
                                                               case.ctx, case.scale)
    tol = tight_bound(case, ref, spread, size, kernel == 0 and S == 16)
    assert (np.abs(got.cpu().double().numpy()[rows] - ref) <= tol).all()
    assert cuda_lib.device_error_flags() == 0


@pytest.mark.parametrize("kernel", [0, 1])
def test_one_sequence_with_a_transposed_table(cuda_lib, kernel):
    """A [1, n] table is contiguous whatever its first stride says."""
    pa = cuda_lib
    case = TreeCase(54, [300], [9], q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    d = case.device()
    d["block_table"] = d["block_table"][0].clone()[:, None].t()
    assert d["block_table"].stride() == (1, 1) and d["block_table"].shape[1] > 1
    out = pa.paged_attention_tree(**d, scale=case.scale, kernel=kernel)
    assert pa.device_error_flags() == 0
    rows, ref, spread, size = oracle.tree.paged_tree_attention(case.q, case.qsl, case.mask, case.k, case.v, case.table,
                                                               case.ctx, case.scale)
    tol = tight_bound(case, ref, spread, size, kernel == 0)
    assert (np.abs(out.cpu().double().numpy()[rows] - ref) <= tol).all()


def test_one_sequence_with_transposed_tables_in_the_rest_of_the_step(cuda_lib):
    pa = cuda_lib
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = i32([[5], [3], [0], [-1], [-1]]).t()
    assert table.stride() == (1, 1)
    t = pa.build_block_tables(i32([40]), i32([20]), table, i32([3]), i32([1, 2, 4]), i32([3, 0]), 16, 6, num_tokens=20)
    assert table.cpu().tolist() == [[5, 3, 0, 4, -1]]
    p = np.arange(40, 60)
    assert np.array_equal(t.slot_mapping.cpu().numpy(), np.array([5, 3, 0, 4])[p // 16] * 16 + p % 16)
    k, v = (torch.randn((6, 16, 2, 64), device="cuda") for _ in range(2))
    accepted = i32([[2], [9], [18]]).t()
    want = oracle.tree.paged_kv_accept(k.cpu(), v.cpu(), accepted.cpu(), i32([3]).cpu(), i32([40]).cpu(), table.cpu())
    pa.paged_kv_accept(k, v, accepted, i32([3]), i32([40]), table)
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
    assert pa.device_error_flags() == 0


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("m", [2, 70])
def test_the_longest_contexts(cuda_lib, kernel, m):
    """Tables of 2^31 tokens that name the same block over and over, keys all alike, values all 1, so that every sum is a
    whole number and the result 1: 2^31 - 4096 tokens are attended, one more is refused."""
    pa = cuda_lib
    k = torch.ones((1, 256, 1, 64), dtype=BF16, device="cuda")
    q = torch.ones((m, 2, 64), dtype=BF16, device="cuda")
    table = torch.zeros((1, 2 ** 23), dtype=torch.int32, device="cuda")
    qsl = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    for n, flag in ((2 ** 31 - 1, pa.PA_DEVERR_CONTEXT_LEN), (2 ** 31 - 4095, pa.PA_DEVERR_CONTEXT_LEN), (2 ** 31 - 4096, 0)):
        out = torch.full_like(q, 7.0)
        ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
        pa.paged_attention_tree(q, qsl, None, k, k, table, ctx, out=out, kernel=kernel)
        assert pa.device_error_flags() == flag
        assert (out == (0.0 if flag else 1.0)).all()


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("m", [5, 40])
@pytest.mark.parametrize("part", [0, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_far_beyond_the_exponents_range(cuda_lib, kernel, dtype, m, part, sign):
    """Queries and keys that are powers of two times small whole numbers, so that every score is exact in 32 bits and
    two different ones are far more than 2^128 apart: the largest take it all, equal ones in equal parts."""
    case = TreeCase(55, [300, 20], [m, 9], q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    q, k = (2.0 ** 11, 2.0 ** 9) if dtype == FP16 else (2.0 ** 35, 2.0 ** 30)
    rng = np.random.default_rng(int(sign) + m)
    case.q = torch.full_like(case.q, sign * q)
    for b in range(2):
        for j in range(int(case.ctx[b])):
            blk, tok = case.row_of(b, j)
            case.k[blk, tok] = k * float(rng.integers(64, 100))
            if j in (17, 18, 130, 299):  # the largest scores and the smallest ones are met four and two times
                case.k[blk, tok] = k * (120.0 if sign > 0 else 60.0)
    got = cuda_lib.paged_attention_tree(**case.device(), scale=case.scale, kernel=kernel, partition_tokens=part)
    assert cuda_lib.device_error_flags() == 0
    rows, ref, spread, _ = oracle.tree.paged_tree_attention(case.q, case.qsl, case.mask, case.k, case.v, case.table, case.ctx,
                                                            case.scale)
    # weights are 0 or exactly alike, so nothing is rounded but a sum of a few values and the output
    half = torch.finfo(dtype).eps / 2
    tol = half * np.abs(ref) + spread * 8 * 2.0 ** -24 + (2.0 ** -25 if dtype == FP16 else 0.0)
    assert (np.abs(got.cpu().double().numpy()[rows] - ref) <= tol * (1 + half)).all()
