"""GPU parity of the 4-bit cache's calls: what rows are packed to and unpacked to, bit for bit, and attention over it."""
import numpy as np
import pytest
import torch

import oracle
from window_cases import ALL, PackedCase, int32, pack

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _clean(cuda_lib):
    cuda_lib.device_error_flags(clear=True)
    yield
    cuda_lib.set_checked_mode(False)
    cuda_lib.device_error_flags(clear=True)


def same(a, b):
    """Equal bits, NaN scales included."""
    return torch.equal(a.cpu().contiguous().view(torch.int16), b.cpu().contiguous().view(torch.int16))


def rows_of(dtype, T, H, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g)
    x[:, :, ::16] *= 6
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [1, 3, 8])
@pytest.mark.parametrize("T", [1, 7, 150])
def test_rows_are_packed_to_the_bit(cuda_lib, dtype, D, H, T):
    pa = cuda_lib
    k, v = rows_of(dtype, T, H, D, T), rows_of(dtype, T, H, D, T + 1) * 0.01
    S, NB = 16, 12
    slots = torch.randperm(NB * S, generator=torch.Generator().manual_seed(3))[:T]
    slots[::5] = -1
    cache = pa.q4_cache(NB, S, H, D)
    for x in cache:
        x.fill_(3)
    pa.paged_kv_write_q4(k.cuda(), v.cuda(), slots.cuda(), cache)
    keep = slots >= 0
    for x, codes, params in ((k, cache.k_codes, cache.k_params), (v, cache.v_codes, cache.v_params)):
        want_c, want_p = torch.full(codes.shape, 3, dtype=torch.uint8).flatten(0, 1), torch.full(params.shape, 3.0, dtype=BF16).flatten(0, 1)
        c, p = pack(x[keep])
        want_c[slots[keep]], want_p[slots[keep]] = c, p
        assert torch.equal(codes.cpu().flatten(0, 1), want_c) and same(params.flatten(0, 1), want_p)
    assert pa.device_error_flags() == 0


def special_groups(dtype):
    """Groups of 64 whose packing is decided by ties, ends of the range, or nothing at all."""
    fi = torch.finfo(dtype)
    g = torch.Generator().manual_seed(5)
    out = [torch.zeros(64), torch.full((64,), 3.0), torch.full((64,), -3.0), torch.arange(64.0), -torch.arange(64.0),
           torch.arange(64.0) - 20, torch.arange(64) / 64.0, torch.full((64,), fi.tiny), torch.full((64,), fi.max),
           torch.full((64,), -fi.max)]
    half = torch.arange(64) * 0.5  # scale 1: every second value is a tie
    half = half.clamp(max=7.5) - 7.5 + (torch.arange(64) % 16) * 0.5
    half[0], half[1] = -7.5, 7.5
    out += [half, half * 2.0 ** -10, -half]
    x = torch.randint(-15, 16, (64,), generator=g) * 0.5
    x[0], x[1] = -5.0, 10.0
    out.append(x)
    big = torch.randn(64, generator=g)
    big[3], big[4] = fi.max, -fi.max
    out.append(big)
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = torch.randn(64, generator=g)
        y[37] = bad
        out.append(y)
    z = torch.randn(64, generator=g)
    z[5], z[6] = float("inf"), float("nan")
    out.append(z)
    if dtype != FP16:
        out += [torch.randn(64, generator=g) * 1e-38, torch.randn(64, generator=g) * 1e-40, torch.randn(64, generator=g) * 1e37]
    else:
        out += [torch.randn(64, generator=g) * 1e-7]
    return torch.stack(out).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_ties_ends_and_groups_that_are_not_finite(cuda_lib, dtype):
    pa = cuda_lib
    x = special_groups(dtype)[:, None, :]
    n = x.shape[0]
    want_c, want_p = oracle.window.q4_pack(x)
    fast_c, fast_p = pack(x)
    assert np.array_equal(want_c, fast_c.numpy()) and np.array_equal(want_p, fast_p.double().numpy(), equal_nan=True)
    cache = pa.q4_cache(n, 1, 1, 64)
    pa.paged_kv_write_q4(x.cuda(), x.flip(0).contiguous().cuda(), torch.arange(n).cuda(), cache)
    assert np.array_equal(cache.k_codes.cpu().numpy().reshape(n, 1, -1), want_c)
    assert np.array_equal(cache.k_params.cpu().double().numpy().reshape(n, 1, -1), want_p, equal_nan=True)
    assert np.array_equal(cache.v_codes.cpu().numpy().reshape(n, 1, -1)[::-1], want_c)
    # and back: every finite value within its type, the others NaN
    k, v = torch.empty((n, 1, 1, 64), dtype=dtype, device="cuda"), torch.empty((n, 1, 1, 64), dtype=dtype, device="cuda")
    pa.paged_kv_unpack_q4(cache, k, v, torch.stack([torch.arange(n), torch.arange(n)], 1).cuda())
    k = k.cpu().view(n, 64)
    good = torch.isfinite(x.view(n, 64)).all(1)
    assert torch.isfinite(k[good]).all() and torch.isnan(k[~good]).all()
    top = torch.finfo(dtype).max
    exact = np.clip(oracle.window.q4_values(torch.from_numpy(want_c), torch.from_numpy(want_p)).reshape(n, 64), -top, top)
    assert torch.equal(k[good], torch.from_numpy(exact[good.numpy()]).to(dtype))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_a_million_random_values(cuda_lib, dtype):
    """Values next to the borders of their grid, many of them exactly on one."""
    pa = cuda_lib
    g = torch.Generator().manual_seed(6)
    x = torch.randn((16384, 1, 64), generator=g)
    x[:8192] = (x[:8192] * 4).round() / 8  # few significant bits: ties are common
    x[8192:12288] *= torch.exp2(torch.randint(-20, 10, (4096, 1, 1), generator=g).float())
    x = x.to(dtype)
    c, p = pack(x)
    cache = pa.q4_cache(1024, 16, 1, 64)
    pa.paged_kv_write_q4(x.cuda(), x.cuda(), torch.arange(16384).cuda(), cache)
    assert torch.equal(cache.k_codes.cpu().view(16384, 1, 32), c) and same(cache.k_params.view(16384, 1, 2), p)
    assert torch.equal(cache.v_codes, cache.k_codes)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("S,H,D", [(1, 1, 64), (16, 8, 128), (32, 3, 64), (256, 2, 128)])
def test_blocks_are_unpacked_to_the_bit(cuda_lib, dtype, S, H, D):
    pa = cuda_lib
    NB, n = 9, 5
    g = torch.Generator().manual_seed(7)
    cache = pa.q4_cache(NB, S, H, D)
    for i in (0, 1):
        c, p = pack(torch.randn((NB, S, H, D), generator=g))
        cache[i].copy_(c)
        cache[2 + i].copy_(p)
    pool = torch.full((7, 2, S, H, D), 5.0, dtype=dtype, device="cuda")
    src, dst = torch.tensor([8, 0, 3, 3, 7]), torch.tensor([6, 2, 0, 1, 5])
    pa.paged_kv_unpack_q4(cache, *pa.unified_views(pool), torch.stack([src, dst], 1).cuda())
    for i in (0, 1):
        want = torch.full((7, S, H, D), 5.0, dtype=dtype)
        want[dst] = torch.from_numpy(oracle.window.q4_values(cache[i].cpu(), cache[2 + i].cpu()))[src].to(dtype)
        assert torch.equal(pool[:, i].cpu(), want)
    assert pa.device_error_flags() == 0


def test_slots_and_blocks_out_of_range(cuda_lib):
    pa = cuda_lib
    x = rows_of(BF16, 4, 2, 64).cuda()
    cache = pa.q4_cache(3, 16, 2, 64)
    slots = torch.tensor([5, 48, -3, 7]).cuda()
    pa.paged_kv_write_q4(x, x, slots, cache)
    assert pa.device_error_flags() == pa.PA_DEVERR_SLOT
    written = cache.k_params.flatten(0, 1)[:, 0, 0] != 0
    assert written.nonzero().flatten().tolist() == [5, 7]
    k, v = (torch.full((2, 16, 2, 64), 5.0, dtype=BF16, device="cuda") for _ in range(2))
    pairs = torch.tensor([[0, 0], [3, 1], [-1, 1], [1, 2], [1, -1]]).cuda()
    pa.paged_kv_unpack_q4(cache, k, v, pairs)
    assert pa.device_error_flags() == pa.PA_DEVERR_COPY_PAIR
    assert (k[1] == 5).all() and not (k[0] == 5).all()
    pa.set_checked_mode(True)
    for s in ([5, 48, -3, 7], [5, 6, 5, -1]):
        with pytest.raises(pa.PagedAttnError) as e:
            pa.paged_kv_write_q4(x, x, torch.tensor(s).cuda(), cache)
        assert e.value.status == pa.PA_ERANGE
    for p in ([[3, 0]], [[0, 2]], [[0, -1]], [[0, 1], [1, 1]]):
        with pytest.raises(pa.PagedAttnError) as e:
            pa.paged_kv_unpack_q4(cache, k, v, torch.tensor(p).cuda())
        assert e.value.status == pa.PA_ERANGE
    pa.paged_kv_write_q4(x, x, torch.tensor([5, 6, -1, -1]).cuda(), cache)
    pa.paged_kv_unpack_q4(cache, k, v, torch.tensor([[1, 0], [1, 1]]).cuda())


def run(pa, case, **kw):
    return pa.paged_attention_decode_q4(cache=case.cache(pa), **case.device(), window=case.window, sinks=case.sinks,
                                        scale=case.scale, **kw)


def check(pa, case, got, flags=0):
    torch.cuda.synchronize()
    rows, ref, spread, size = case.oracle()
    g = got.cpu().double().numpy()
    assert np.isfinite(g).all()
    off = np.abs(g - ref) - case.bound(ref, spread, size)
    assert (off <= 0).all(), f"worst excess {off.max()} at {np.unravel_index(off.argmax(), off.shape)}"
    assert pa.device_error_flags() == flags


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("H", [1, 2, 3])
def test_attention(cuda_lib, dtype, D, G, H):
    case = PackedCase(10 * G + D, [1, 0, 17, 300, 129, 64, 700], ALL, 0, q_heads=H * G, kv_heads=H, head_dim=D, block_size=16,
                      dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("H", [4, 8, 12, 16])
def test_many_heads(cuda_lib, dtype, H):
    case = PackedCase(H, [5, 0, 333, 90], ALL, 0, q_heads=4 * H, kv_heads=H, head_dim=128, block_size=32, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("S", [1, 2, 4, 8, 16, 64, 256])
def test_block_sizes(cuda_lib, dtype, S):
    case = PackedCase(S, [100, 7, 555], ALL, 0, q_heads=8, kv_heads=4, head_dim=64, block_size=S, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("part", [0, 1, 16, 200, 4096])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_split_contexts(cuda_lib, dtype, part, workspace):
    case = PackedCase(part, [900, 5, 333, 700], ALL, 0, q_heads=16, kv_heads=8, head_dim=128, block_size=16, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case, partition_tokens=part, workspace=workspace))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 3), (100, 0), (100, 40), (5000, 4), (3, 5000)])
def test_behind_a_window(cuda_lib, dtype, window, sinks):
    case = PackedCase(window, [640, 33, 260, 1], window, sinks, q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    check(cuda_lib, case, run(cuda_lib, case))
    cuda_lib.set_checked_mode(True)
    check(cuda_lib, case, run(cuda_lib, case))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("size", [1e-4, 1.0, 1e3])
def test_sizes_of_values(cuda_lib, dtype, size):
    """Scales far from 1 in keys and values: fp16 queries meet them in bf16 weights."""
    case = PackedCase(21, [300, 40], ALL, 0, q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=dtype)
    case.kp[..., 0::2] *= size
    case.vp[..., 0::2] *= size * 0.25
    case.scale /= size
    check(cuda_lib, case, run(cuda_lib, case))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_rows_that_are_not_finite(cuda_lib, dtype):
    """A NaN key leaves nothing of the heads that read it; a NaN group of a value, of its 64 dimensions."""
    case = PackedCase(22, [300, 40, 90], ALL, 0, q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=dtype)
    fine = run(cuda_lib, case)
    case.kp[case.row_of(0, 33)][1, 2] = float("nan")
    case.vp[case.row_of(1, 7)][0, 0] = float("nan")
    got = run(cuda_lib, case)
    assert torch.isnan(got[0, 4:]).all() and torch.equal(got[0, :4], fine[0, :4])
    assert torch.isnan(got[1, :4, :64]).all() and torch.equal(got[1, :4, 64:], fine[1, :4, 64:])
    assert torch.equal(got[1, 4:], fine[1, 4:]) and torch.equal(got[2], fine[2])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_refused_sequences_and_bad_blocks(cuda_lib, dtype):
    pa = cuda_lib
    case = PackedCase(23, [50, 60, 70], ALL, 0, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    d = case.device()
    d["context_lens"] = int32([50, -1, 70]).cuda()
    got = pa.paged_attention_decode_q4(cache=case.cache(pa), **d, scale=case.scale)
    assert (got[1] == 0).all() and pa.device_error_flags() == pa.PA_DEVERR_CONTEXT_LEN
    d = case.device()
    d["block_table"][2] = case.num_blocks
    got = pa.paged_attention_decode_q4(cache=case.cache(pa), **d, scale=case.scale)
    assert (got[2] == 0).all() and pa.device_error_flags() == pa.PA_DEVERR_BLOCK_ID
    pa.set_checked_mode(True)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.paged_attention_decode_q4(cache=case.cache(pa), **d, scale=case.scale)
    assert e.value.status == pa.PA_ERANGE


@pytest.mark.parametrize("batch", [300, 1500])
def test_large_batches(cuda_lib, batch):
    ctx = np.random.default_rng(batch).integers(0, 40, batch).tolist()
    case = PackedCase(batch, ctx, ALL, 0, q_heads=2, kv_heads=1, head_dim=64, block_size=16, dtype=BF16)
    check(cuda_lib, case, run(cuda_lib, case))


def test_blocks_of_the_cache_are_copied_and_swapped(cuda_lib):
    """copy_blocks and swap_blocks take codes and params as two pairs of pools."""
    pa = cuda_lib
    case = PackedCase(24, [100, 60], ALL, 0, q_heads=8, kv_heads=4, head_dim=64, block_size=16, dtype=BF16)
    fine = run(pa, case)
    c, d = case.cache(pa), case.device()
    fork = torch.tensor([[int(case.table[0, 1]), case.num_blocks]]).cuda()
    c = pa.Q4Cache(*(torch.cat([x, torch.zeros_like(x[:1])]) for x in c))
    pa.copy_blocks(c.k_codes, c.v_codes, fork)
    pa.copy_blocks(c.k_params, c.v_params, fork)
    d["block_table"][0, 1] = case.num_blocks
    assert torch.equal(pa.paged_attention_decode_q4(cache=c, **d, scale=case.scale), fine)
    host = pa.Q4Cache(*(torch.zeros_like(x, device="cpu").pin_memory() for x in c))
    back = pa.Q4Cache(*(torch.zeros_like(x) for x in c))
    every = torch.stack([torch.arange(case.num_blocks + 1)] * 2, 1).cuda()
    for a, b in ((c, host), (host, back)):
        pa.swap_blocks(b.k_codes, b.v_codes, a.k_codes, a.v_codes, every)
        pa.swap_blocks(b.k_params, b.v_params, a.k_params, a.v_params, every)
    assert torch.equal(pa.paged_attention_decode_q4(cache=back, **d, scale=case.scale), fine)
