"""Windowed attention and the 4-bit cache at the edges of what they take: refusals of the binding, workspaces, pools and
contexts past 32-bit offsets, captured and overlapping calls, and the calls together as a server makes them."""
import numpy as np
import pytest
import torch

import oracle
from pagedattention_kv_cache_paged_gb300 import _abi
from window_cases import ALL, PackedCase, WindowCase, int32, pack, pool_bound

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _clean(cuda_lib):
    cuda_lib.device_error_flags(clear=True)
    yield
    cuda_lib.set_checked_mode(False)
    cuda_lib.device_error_flags(clear=True)


# ---------------------------------------------------------------------------------------------
# what the binding and the library refuse, one change at a time to calls that succeed
# ---------------------------------------------------------------------------------------------

def window_args(dtype=FP32, S=16):
    case = WindowCase(1, [40, 17], [3, 2], 30, 2, q_heads=4, kv_heads=2, head_dim=64, block_size=S, dtype=dtype)
    return dict(case.device(), window=30, sinks=2)


def one_args(dtype=FP32, S=16):
    case = WindowCase(1, [40, 17], None, 30, 2, q_heads=4, kv_heads=2, head_dim=64, block_size=S, dtype=dtype)
    return dict(case.device(), window=30, sinks=2)


def q4_args(pa):
    case = PackedCase(1, [40, 17], ALL, 0, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    return dict(case.device(), cache=case.cache(pa))


def write_args(pa):
    rows = torch.randn((3, 2, 64), dtype=BF16, device="cuda")
    return dict(k_new=rows, v_new=rows + 1, slot_mapping=torch.tensor([5, -1, 9], device="cuda"), cache=pa.q4_cache(4, 16, 2, 64))


def unpack_args(pa):
    pools = torch.zeros((2, 4, 16, 2, 64), dtype=BF16, device="cuda")
    return dict(cache=pa.q4_cache(4, 16, 2, 64), k_pool=pools[0], v_pool=pools[1], block_pairs=torch.tensor([[0, 3], [2, 1]], device="cuda"))


CALLS = {"paged_attention_window": lambda pa: window_args(), "paged_attention_decode_q4": q4_args,
         "paged_kv_write_q4": write_args, "paged_kv_unpack_q4": unpack_args}
TENSORS = [(call, name) for call, names in
           (("paged_attention_window", "q query_start_loc k_pool v_pool block_table context_lens"),
            ("paged_attention_decode_q4", "q block_table context_lens"), ("paged_kv_write_q4", "k_new v_new slot_mapping"),
            ("paged_kv_unpack_q4", "k_pool v_pool block_pairs"))
           for name in names.split()]


@pytest.mark.parametrize("call", list(CALLS))
def test_the_calls_succeed_as_they_are(cuda_lib, call):
    getattr(cuda_lib, call)(**CALLS[call](cuda_lib))
    torch.cuda.synchronize()
    assert cuda_lib.device_error_flags() == 0


@pytest.mark.parametrize("call,name", TENSORS)
def test_what_is_no_tensor(cuda_lib, call, name):
    args = CALLS[call](cuda_lib)
    for wrong in (args[name].cpu().tolist(), 7):
        with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
            getattr(cuda_lib, call)(**{**args, name: wrong})


@pytest.mark.parametrize("call,name", TENSORS)
def test_tensors_of_another_type_or_place(cuda_lib, call, name):
    args = CALLS[call](cuda_lib)
    with pytest.raises((TypeError, ValueError), match="must be torch|of one dtype|unsupported dtype"):
        getattr(cuda_lib, call)(**{**args, name: args[name].to(torch.float64)})
    with pytest.raises(ValueError, match="must be a CUDA tensor|is on cpu|is on cuda"):
        getattr(cuda_lib, call)(**{**args, name: args[name].cpu()})


@pytest.mark.parametrize("call", ["paged_attention_decode_q4", "paged_kv_write_q4", "paged_kv_unpack_q4"])
@pytest.mark.parametrize("name", ["k_codes", "v_codes", "k_params", "v_params"])
def test_caches_of_another_layout(cuda_lib, call, name):
    args = CALLS[call](cuda_lib)
    t = getattr(args["cache"], name)
    for wrong, error in ((t.to(torch.int32), TypeError), (t.cpu(), ValueError), (strided(t), ValueError), (t[:, :8], ValueError),
                         (t.tolist(), TypeError)):
        with pytest.raises(error):
            getattr(cuda_lib, call)(**{**args, "cache": args["cache"]._replace(**{name: wrong})})


def strided(t):
    return torch.stack([t, t], -1)[..., 0]


@pytest.mark.parametrize("call,change,match", [
    ("paged_attention_window", lambda a: dict(q=a["q"][0]), r"q must be \[total_q"),
    ("paged_attention_window", lambda a: dict(q=a["q"][:, :, :32].contiguous()), r"q must be \[total_q"),
    ("paged_attention_window", lambda a: dict(q=strided(a["q"])), "(q|out) must be contiguous"),
    ("paged_attention_window", lambda a: dict(query_start_loc=None), "one query per sequence"),
    ("paged_attention_window", lambda a: dict(query_start_loc=a["query_start_loc"][:2]), r"query_start_loc must be \[3\]"),
    ("paged_attention_window", lambda a: dict(block_table=a["block_table"][:1]), r"block_table must be \[batch"),
    ("paged_attention_window", lambda a: dict(block_table=strided(a["block_table"])), r"block_table must be \[batch"),
    ("paged_attention_window", lambda a: dict(v_pool=a["v_pool"][:2]), "k_pool and v_pool must both be"),
    ("paged_attention_window", lambda a: dict(k_pool=strided(a["k_pool"])), "k_pool: each block must be contiguous"),
    ("paged_attention_window", lambda a: dict(out=a["q"][:2]), r"out must be \[5, 4, 64\]"),
    ("paged_attention_window", lambda a: dict(out=a["q"].to(BF16)), "out must be torch.float32"),
    ("paged_attention_window", lambda a: dict(window=2 ** 31), "window must fit 32 bits"),
    ("paged_attention_window", lambda a: dict(sinks=2 ** 31), "sinks must fit 32 bits"),
    ("paged_attention_decode_q4", lambda a: dict(q=a["q"][:1]), r"q must be \[batch"),
    ("paged_attention_decode_q4", lambda a: dict(q=a["q"][:, :, :32].contiguous()), r"q must be \[batch"),
    ("paged_attention_decode_q4", lambda a: dict(out=a["q"].float()), "out must be torch.bfloat16"),
    ("paged_attention_decode_q4", lambda a: dict(window=2 ** 31), "window must fit 32 bits"),
    ("paged_kv_write_q4", lambda a: dict(k_new=a["k_new"][:2]), r"k_new must be \[3, 2, 64\]"),
    ("paged_kv_write_q4", lambda a: dict(v_new=a["v_new"].float()), "v_new must be torch.bfloat16"),
    ("paged_kv_write_q4", lambda a: dict(slot_mapping=a["slot_mapping"].int()), "slot_mapping must be torch.int64"),
    ("paged_kv_unpack_q4", lambda a: dict(block_pairs=a["block_pairs"][0]), r"block_pairs must be \[n, 2\]"),
    ("paged_kv_unpack_q4", lambda a: dict(k_pool=a["k_pool"][:, :8], v_pool=a["v_pool"][:, :8]), "blocks of the pools are"),
])
def test_tensors_of_another_layout(cuda_lib, call, change, match):
    args = CALLS[call](cuda_lib)
    with pytest.raises((ValueError, TypeError), match=match):
        getattr(cuda_lib, call)(**{**args, **change(args)})


@pytest.mark.parametrize("make", [window_args, one_args])
@pytest.mark.parametrize("change,status", [
    (dict(kernel=3), "EINVAL"), (dict(kernel=-1), "EINVAL"), (dict(partition_tokens=-1), "EINVAL"),
    (dict(partition_tokens=2 ** 30 + 1), "EINVAL"), (dict(scale=0), "EINVAL"), (dict(scale=-1.0), "EINVAL"),
    (dict(scale=float("nan")), "EINVAL"), (dict(scale=2.4e38), "EINVAL"), (dict(window=0), "EINVAL"), (dict(window=-5), "EINVAL"),
    (dict(sinks=-1), "EINVAL"),
])
def test_options_that_the_library_refuses(cuda_lib, make, change, status):
    with pytest.raises(cuda_lib.PagedAttnError) as e:
        cuda_lib.paged_attention_window(**{**make(), **change})
    assert e.value.status == getattr(_abi, "PA_" + status)


def test_tcgen05_where_the_shape_does_not_allow_it(cuda_lib):
    for dtype, S in ((FP32, 16), (BF16, 8)):
        with pytest.raises(cuda_lib.PagedAttnError) as e:
            cuda_lib.paged_attention_window(**window_args(dtype, S), kernel=2)
        assert e.value.status == cuda_lib.PA_EUNSUPPORTED
    args = window_args(BF16)
    assert torch.equal(cuda_lib.paged_attention_window(**args, kernel=2), cuda_lib.paged_attention_window(**args))


def test_numbers_as_numpy_holds_them(cuda_lib):
    args = one_args()
    want = cuda_lib.paged_attention_window(**args, scale=0.25)
    args.update(window=np.int64(args["window"]), sinks=np.int32(args["sinks"]))
    assert torch.equal(cuda_lib.paged_attention_window(**args, scale=np.float32(0.25)), want)


def test_empty_calls(cuda_lib):
    pa = cuda_lib
    args = one_args()
    none = torch.empty((0, 4, 64), device="cuda")
    got = pa.paged_attention_window(**{**args, "q": none, "block_table": args["block_table"][:0], "context_lens": args["context_lens"][:0]})
    assert got.shape == none.shape
    args = window_args()
    assert pa.paged_attention_window(**{**args, "q": none}).shape == none.shape
    a = q4_args(pa)
    pa.paged_attention_decode_q4(**{**a, "q": none.to(BF16), "block_table": a["block_table"][:0], "context_lens": a["context_lens"][:0]})
    a = write_args(pa)
    pa.paged_kv_write_q4(a["k_new"][:0], a["v_new"][:0], a["slot_mapping"][:0], a["cache"])
    a = unpack_args(pa)
    pa.paged_kv_unpack_q4(a["cache"], a["k_pool"], a["v_pool"], a["block_pairs"][:0])
    torch.cuda.synchronize()
    assert pa.device_error_flags() == 0


# ---------------------------------------------------------------------------------------------
# workspaces
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("packed", [False, True])
def test_a_workspace_of_the_size_it_says(cuda_lib, packed):
    """Exactly as many bytes, nothing written behind them; one less is refused, so is an odd address."""
    pa = cuda_lib
    if packed:
        case = PackedCase(3, [3000, 40], ALL, 0, q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
        call = lambda **kw: pa.paged_attention_decode_q4(cache=case.cache(pa), **case.device(), **kw)  # noqa: E731
        size = pa.decode_q4_workspace_size(2, case.table.shape[1], 16, ALL, 0, 8, 2, 64, BF16)
    else:
        case = WindowCase(3, [3000, 40], None, ALL, 0, q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
        call = lambda **kw: pa.paged_attention_window(**case.device(), window=ALL, **kw)  # noqa: E731
        size = pa.window_workspace_size(2, case.table.shape[1], 16, ALL, 0, 8, 2, 64, BF16)
    assert size > 0
    want = call()
    held = torch.full((size + 64,), 0xa5, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(call(workspace=held[:size]), want)
    assert (held[size:] == 0xa5).all()
    for wrong in (held[:size - 1], held[8:size + 8], held[:16]):
        with pytest.raises(pa.PagedAttnError) as e:
            call(workspace=wrong)
        assert e.value.status == pa.PA_EWORKSPACE
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        call(workspace=torch.zeros((size, 2), dtype=torch.uint8, device="cuda")[:, 0])


def test_sizes_of_short_contexts_are_zero(cuda_lib):
    pa = cuda_lib
    for size in (pa.window_workspace_size, pa.decode_q4_workspace_size):
        assert size(4, 1, 16, ALL, 0, 8, 8, 128, BF16) == 0  # a table of 16 tokens
        assert size(4, 4096, 16, 1, 1, 8, 8, 128, BF16) == 0  # a window of as few
        assert size(4, 4096, 16, 5000, 4, 8, 8, 128, BF16) > 0
        assert size(4, 4096, 24, ALL, 0, 8, 8, 128, BF16) == 0 and size(4, 4096, 16, 0, 0, 8, 8, 128, BF16) == 0


# ---------------------------------------------------------------------------------------------
# large ones
# ---------------------------------------------------------------------------------------------

def repeated(case, n, S=16):
    """Tables of `n` positions that name the blocks of the case's first context again and again, at the pools' far end."""
    used = case.table[0, :case.ctx_list[0] // S]
    return used.repeat(-(-n // (S * used.numel())))[:n // S][None].cuda()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("chunks", [False, True])
def test_blocks_past_32_bits_of_offsets(cuda_lib, dtype, chunks):
    """Pools of more than 2^31 elements (5 GB and more): the blocks in use are their last ones."""
    pa = cuda_lib
    case = WindowCase(5, [300, 64], [40, 64] if chunks else None, 100, 5, q_heads=8, kv_heads=8, head_dim=128, block_size=16,
                      dtype=dtype)
    NB = (2 ** 31 // (16 * 8 * 128)) + 50
    d = case.device()
    far = NB - case.num_blocks
    for name in ("k_pool", "v_pool"):
        big = torch.empty((NB, 16, 8, 128), dtype=dtype, device="cuda")
        big[far:] = d[name]
        d[name] = big
    d["block_table"] = torch.where(d["block_table"] >= 0, d["block_table"] + far, d["block_table"])
    got = pa.paged_attention_window(**d, window=100, sinks=5, scale=case.scale)
    check_pool(pa, case, got)


def check_pool(pa, case, got):
    torch.cuda.synchronize()
    rows, ref, spread, size = case.oracle()
    g = got.cpu().double().numpy()[rows]
    assert np.isfinite(g).all() and (np.abs(g - ref) <= pool_bound(case, ref, spread, size)).all()
    assert pa.device_error_flags() == 0


def check_packed(pa, case, got):
    torch.cuda.synchronize()
    _, ref, spread, size = case.oracle()
    g = got.cpu().double().numpy()
    assert np.isfinite(g).all() and (np.abs(g - ref) <= case.bound(ref, spread, size)).all()
    assert pa.device_error_flags() == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_4_bit_cache_past_32_bits_of_bytes(cuda_lib, dtype):
    """Codes of more than 2^32 bytes: packed, attended to and unpacked at the far end."""
    pa = cuda_lib
    case = PackedCase(6, [200, 33], 90, 4, q_heads=8, kv_heads=8, head_dim=128, block_size=16, dtype=dtype)
    NB = 2 ** 32 // (16 * 8 * 64) + 40
    far = NB - case.num_blocks
    cache = pa.Q4Cache(*(torch.empty((NB, 16, 8, w), dtype=t, device="cuda") for w, t in
                         ((64, torch.uint8), (64, torch.uint8), (4, BF16), (4, BF16))))
    k, v = torch.nan_to_num(case.k), torch.nan_to_num(case.v)
    slots = torch.arange(case.num_blocks * 16) + far * 16
    pa.paged_kv_write_q4(k.flatten(0, 1).cuda(), v.flatten(0, 1).cuda(), slots.cuda(), cache)
    (want_kc, want_kp), (want_vc, _) = pack(k), pack(v)
    assert torch.equal(cache.k_codes[far:].cpu(), want_kc) and torch.equal(cache.k_params[far:].cpu(), want_kp)
    assert torch.equal(cache.v_codes[far:].cpu(), want_vc)
    d = case.device()
    d["block_table"] = torch.where(d["block_table"] >= 0, d["block_table"] + far, d["block_table"])
    got = pa.paged_attention_decode_q4(cache=cache, **d, window=90, sinks=4, scale=case.scale)
    check_packed(pa, case, got)
    pools = torch.empty((2, 2 ** 31 // (16 * 8 * 128) + 9, 16, 8, 128), dtype=BF16, device="cuda")
    last = pools.shape[1] - 1
    pa.paged_kv_unpack_q4(cache, pools[0], pools[1], torch.tensor([[NB - 1, last], [far, last - 1]]).cuda())
    for i, (codes, params) in enumerate(((cache.k_codes, cache.k_params), (cache.v_codes, cache.v_params))):
        want = oracle.window.q4_values(codes[[far, NB - 1]].cpu(), params[[far, NB - 1]].cpu())
        assert torch.equal(pools[i, last - 1:].cpu(), torch.from_numpy(want).to(BF16))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("packed", [False, True])
def test_a_context_of_two_million_tokens(cuda_lib, dtype, packed):
    """32 tokens again and again: the attention over them.  Sums are held to 2^-24 a key, as everywhere."""
    pa, n = cuda_lib, 1 << 21
    kw = dict(q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    case = PackedCase(7, [32], ALL, 0, **kw) if packed else WindowCase(7, [32], None, ALL, 0, **kw)
    d = case.device()
    d["block_table"], d["context_lens"] = repeated(case, n), int32([n]).cuda()
    if packed:
        got = pa.paged_attention_decode_q4(cache=case.cache(pa), **d, scale=case.scale)
    else:
        got = pa.paged_attention_window(**d, window=ALL, scale=case.scale)
    case.most_seen = lambda: n
    (check_packed if packed else check_pool)(pa, case, got)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("what", ["one", "chunk", "packed"])
def test_the_longest_contexts(cuda_lib, dtype, what):
    """A context of 2^31 - 4096 tokens behind a window; one token more is refused."""
    pa, n, S = cuda_lib, 2 ** 31 - 4096, 256
    kw = dict(q_heads=4, kv_heads=2, head_dim=64, block_size=S, dtype=dtype)
    new = 70 if what == "chunk" else 1
    args = dict(window=600, sinks=300)
    # the same visible keys in a short context: 300 sinks, and the last blocks, ending at the same place of a block
    short = 300 + 212 + 4 * S + n % S
    if what == "packed":
        case = PackedCase(8, [short], 600, 300, **kw)
    else:
        case = WindowCase(8, [short], [new] if what == "chunk" else None, 600, 300, **kw)
    d = case.device()
    table = torch.full((1, n // S + 17), -1, dtype=torch.int32, device="cuda")
    k = -(-short // S)
    table[0, :2] = d["block_table"][0, :2]
    table[0, n // S - (k - 2):n // S] = d["block_table"][0, 2:k]
    assert n % S == 0 and short % S == 0
    d["block_table"], d["context_lens"] = table, int32([n]).cuda()
    if what == "packed":
        run = lambda: pa.paged_attention_decode_q4(cache=case.cache(pa), **d, **args, scale=case.scale)  # noqa: E731
    else:
        run = lambda: pa.paged_attention_window(**d, **args, scale=case.scale)  # noqa: E731
    (check_packed if what == "packed" else check_pool)(pa, case, run())
    pa.set_checked_mode(True)
    (check_packed if what == "packed" else check_pool)(pa, case, run())
    pa.set_checked_mode(False)
    d["context_lens"] = int32([n + 1]).cuda()
    assert (run() == 0).all()
    assert pa.device_error_flags() == (pa.PA_DEVERR_QUERY_LOC if what == "chunk" else pa.PA_DEVERR_CONTEXT_LEN)


# ---------------------------------------------------------------------------------------------
# what is not as documented, and overlapping calls
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("qsl", [[0, 60, 30, 120], [-40, 20, 50, 120], [0, 20, 50, 500], [0, 200, 10, 120], [120, 90, 20, 0],
                                 [5, 5, 5, 5]])
def test_query_start_locs_out_of_order(cuda_lib, kernel, qsl):
    """Nothing outside the output is touched, the call ends, and checked mode refuses what is out of order."""
    pa = cuda_lib
    case = WindowCase(9, [90, 60, 100], [20, 30, 70], 30, 2, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    d = case.device()
    d["query_start_loc"] = int32(qsl).cuda()
    held = torch.full((40 + 120 + 40, 4, 64), 7.0, dtype=BF16, device="cuda")
    pa.paged_attention_window(**d, window=30, sinks=2, kernel=kernel, out=held[40:160])
    torch.cuda.synchronize()
    assert (held[:40] == 7).all() and (held[160:] == 7).all()
    assert pa.device_error_flags() & ~(pa.PA_DEVERR_QUERY_LOC | pa.PA_DEVERR_BLOCK_ID) == 0
    pa.set_checked_mode(True)
    if qsl == [5, 5, 5, 5]:
        pa.paged_attention_window(**d, window=30, sinks=2, kernel=kernel, out=held[40:160])
        assert (held == 7).all()
        return
    with pytest.raises(pa.PagedAttnError) as e:
        pa.paged_attention_window(**d, window=30, sinks=2, kernel=kernel)
    assert e.value.status == pa.PA_ERANGE


@pytest.mark.parametrize("every", [0, 2, 5, 40])
def test_many_refused_chunks_in_a_row(cuda_lib, every):
    """More of them than a CTA's pipeline is deep, with chunks that are not refused in between, of one Q tile and of two."""
    pa, n = cuda_lib, 2400
    good = [every > 0 and b % every == 0 for b in range(n)]
    new = [1 + 97 * b % 270 if ok else 1 + b % 3 for b, ok in enumerate(good)]
    ctx = [m + b % 40 if ok else 0 for b, (m, ok) in enumerate(zip(new, good))]
    case = WindowCase(17, ctx, [m if ok else 0 for m, ok in zip(new, good)], 50, 2, q_heads=2, kv_heads=2, head_dim=64,
                      block_size=16, dtype=BF16)
    d = case.device()
    qsl = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn((int(qsl[-1]), 2, 64), generator=torch.Generator().manual_seed(1)).to(BF16)
    mine = torch.cat([torch.arange(qsl[b], qsl[b + 1]) for b in range(n) if good[b]] + [torch.arange(0)])
    q[mine] = case.q
    d["q"], d["query_start_loc"] = q.cuda(), int32(qsl).cuda()
    got = pa.paged_attention_window(**d, window=50, sinks=2, scale=case.scale)
    torch.cuda.synchronize()
    assert pa.device_error_flags() == pa.PA_DEVERR_QUERY_LOC  # (nothing timed out)
    other = torch.ones(q.shape[0], dtype=torch.bool)
    other[mine] = False
    got = got.cpu()
    assert (got[other] == 0).all()
    if every >= 5:
        rows, ref, spread, size = case.oracle()
        assert (np.abs(got[mine].double().numpy()[rows] - ref) <= pool_bound(case, ref, spread, size)).all()
    elif every:
        assert torch.isfinite(got).all() and (got[mine] != 0).any()


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_chunks_whose_every_value_is_nan(cuda_lib, kernel, dtype):
    """A model that has diverged: NaN everywhere, and the call ends as soon as with numbers or so."""
    case = WindowCase(10, [500, 90], [300, 90], 200, 4, q_heads=8, kv_heads=2, head_dim=64, block_size=16, dtype=dtype)
    case.v[:] = float("nan")
    assert torch.isnan(cuda_lib.paged_attention_window(**case.device(), window=200, sinks=4, kernel=kernel)).all()


def test_calls_over_one_cache_on_two_streams_and_one_graph_each(cuda_lib):
    """Graphs of their own over one cache, replayed side by side, each with its own scratch."""
    pa = cuda_lib
    cases = [PackedCase(s, [3000, 700], 1500, 7, q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=BF16) for s in (11, 12)]
    caches, devs = [c.cache(pa) for c in cases], [c.device() for c in cases]
    outs = [torch.empty_like(d["q"]) for d in devs]
    streams, graphs = [torch.cuda.Stream() for _ in cases], [torch.cuda.CUDAGraph() for _ in cases]
    call = lambda i: pa.paged_attention_decode_q4(cache=caches[i], **devs[i], window=1500, sinks=7, scale=cases[i].scale, out=outs[i])  # noqa: E731
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            call(i)
    for o in outs:
        o.fill_(0)
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        check_packed(pa, c, o)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_results_over_the_cache_do_not_change_from_call_to_call(cuda_lib, dtype):
    pa = cuda_lib
    case = PackedCase(13, [3000, 5, 700], ALL, 0, q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=dtype)
    cache = case.cache(pa)
    call = lambda: pa.paged_attention_decode_q4(cache=cache, **case.device(), scale=case.scale)  # noqa: E731
    first = call()
    for _ in range(5):
        assert torch.equal(call(), first)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_results_of_chunks_do_not_change_from_call_to_call(cuda_lib, dtype):
    case = WindowCase(14, [900, 5, 400], [300, 5, 100], 200, 4, q_heads=8, kv_heads=2, head_dim=128, block_size=16, dtype=dtype)
    call = lambda: cuda_lib.paged_attention_window(**case.device(), window=200, sinks=4, scale=case.scale)  # noqa: E731
    first = call()
    for _ in range(5):
        assert torch.equal(call(), first)


def test_views_of_a_cache_and_a_wide_table(cuda_lib):
    """One layer of a cache of several, a table inside a wider one, queries and lengths at an offset."""
    pa = cuda_lib
    case = PackedCase(15, [640, 33, 90], 80, 3, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=BF16)
    d, c = case.device(), case.cache(pa)
    layers = pa.Q4Cache(*(torch.stack([torch.zeros_like(x), x, torch.zeros_like(x)]) for x in c))
    wide = torch.full((3, 100), -7, dtype=torch.int32, device="cuda")
    wide[:, 9:9 + case.table.shape[1]] = d["block_table"]
    d["block_table"] = wide[:, 9:9 + case.table.shape[1]]
    d["context_lens"] = torch.cat([int32([9, 9, 9]).cuda(), d["context_lens"]])[3:]
    d["q"] = torch.cat([d["q"][:1], d["q"]])[1:]
    got = pa.paged_attention_decode_q4(cache=pa.Q4Cache(*(x[1] for x in layers)), **d, window=80, sinks=3, scale=case.scale)
    check_packed(pa, case, got)


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------

class Held(WindowCase):
    """What a server holds, as the cases above have it."""

    def __init__(self, q, qsl, k, v, table, ctx, new, window, sinks):
        self.q, self.qsl, self.k, self.v, self.table = q.cpu(), qsl, k.cpu(), v.cpu(), table.clone()
        self.ctx_list, self.new_list, self.ctx = list(ctx), list(new), int32(list(ctx))
        self.window, self.sinks, self.block_size, self.dtype, self.scale = window, sinks, k.shape[1], q.dtype, q.shape[2] ** -0.5
        low = [max(n - m + 1 - window, 0) for n, m in zip(ctx, new)]
        self.seen = [[j for j in range(n) if j < min(sinks, lo) or j >= lo] for n, lo in zip(ctx, low)]


class HeldPacked(Held, PackedCase):
    def __init__(self, q, cache, table, ctx, window, sinks):
        super().__init__(q, None, cache.k_codes, cache.v_codes, table, ctx, [1] * len(ctx), window, sinks)
        self.kc, self.vc, self.kp, self.vp = (x.cpu() for x in cache)

    oracle, bound = PackedCase.oracle, PackedCase.bound


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_a_server_of_a_windowed_model_with_a_packed_cache(cuda_lib, dtype):
    """Prompts in chunks, the earlier ones' keys and values unpacked for the later ones; then tokens one by one from a
    captured step over the packed cache, blocks before the window given back on the way.  Every output is checked against
    the oracle over what the cache holds, and what it holds against the format."""
    pa = cuda_lib
    S, Hq, Hkv, D, NB, W, sinks = 16, 8, 2, 64, 40, 30, 5
    g = torch.Generator().manual_seed(16)
    rand = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()  # noqa: E731
    cache = pa.q4_cache(NB, S, Hkv, D)
    pools = torch.full((NB, 2, S, Hkv, D), float("nan"), dtype=dtype, device="cuda")  # scratch for prompts
    k_pool, v_pool = pa.unified_views(pools)
    free = list(range(NB))
    table = torch.full((3, 12), -1, dtype=torch.int32)
    ctx = [0, 0, 0]
    rows_of = [[], [], []]  # (k, v) of every token of a request, on the CPU

    def slots_of(b, lo, hi):
        for j in range(lo // S, -(-hi // S)):
            if table[b, j] < 0:
                table[b, j] = free.pop(0)
        return [int(table[b, j // S]) * S + j % S for j in range(lo, hi)]

    # ---- prompts: 70, 20 and 33 tokens; the first in chunks of 37, so its second reads what the cache holds of the first
    for new in ([37, 20, 33], [33, 0, 0]):
        held = [(b, n) for b, n in enumerate(ctx) if n and new[b]]
        pairs = [(int(t), int(t)) for b, n in held for t in table[b, :-(-n // S)]]
        if pairs:
            pools.fill_(float("nan"))
            pa.paged_kv_unpack_q4(cache, k_pool, v_pool, torch.tensor(pairs).cuda())
        slots = sum((slots_of(b, n, n + m) for b, (n, m) in enumerate(zip(ctx, new))), [])
        T = len(slots)
        q, k, v, s = rand(T, Hq, D), rand(T, Hkv, D), rand(T, Hkv, D), torch.tensor(slots).cuda()
        pa.paged_kv_write(k, v, s, k_pool, v_pool)
        ctx = [n + m for n, m in zip(ctx, new)]
        qsl = int32(np.concatenate([[0], np.cumsum(new)]))
        live = [n if m else 0 for n, m in zip(ctx, new)]
        out = pa.paged_attention_window(q, qsl.cuda(), k_pool, v_pool, table.cuda(), int32(live).cuda(), W, sinks)
        check_pool(pa, Held(q, qsl, k_pool, v_pool, table, live, new, W, sinks), out)
        pa.paged_kv_write_q4(k, v, s, cache)
        for b, m in enumerate(new):
            rows_of[b] += [(k[t].cpu(), v[t].cpu()) for t in range(int(qsl[b]), int(qsl[b]) + m)]

    # ---- tokens one by one, a captured step
    q, k, v = rand(3, Hq, D), rand(3, Hkv, D), rand(3, Hkv, D)
    lens, dev_table, s = int32([0, 0, 0]).cuda(), table.cuda(), torch.full((3,), -1, device="cuda")
    out = torch.empty_like(q)

    def step():
        pa.paged_kv_write_q4(k, v, s, cache)
        pa.paged_attention_decode_q4(q, cache, dev_table, lens, W, sinks, out=out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    given_back = 0
    for _ in range(40):
        now = [slots_of(b, n, n + 1)[0] for b, n in enumerate(ctx)]
        ctx = [n + 1 for n in ctx]
        for b, n in enumerate(ctx):  # what lies before the window and holds no sink
            for j in range(-(-sinks // S), max(n - W, 0) // S):
                if table[b, j] >= 0:
                    free.append(int(table[b, j]))
                    table[b, j] = -1
                    given_back += 1
        for x, src in ((q, rand(3, Hq, D)), (k, rand(3, Hkv, D)), (v, rand(3, Hkv, D)), (lens, int32(ctx)), (dev_table, table),
                       (s, torch.tensor(now))):
            x.copy_(src)
        graph.replay()
        for b in range(3):
            rows_of[b].append((k[b].cpu(), v[b].cpu()))
        check_packed(pa, HeldPacked(q, cache, table, ctx, W, sinks), out)
    assert given_back == 5
    case = HeldPacked(q, cache, table, ctx, W, sinks)
    for b in range(3):
        for j in case.seen[b]:
            for row, codes, params in zip(rows_of[b][j], (case.kc, case.vc), (case.kp, case.vp)):
                c, p = pack(row)
                assert torch.equal(codes[case.row_of(b, j)], c) and torch.equal(params[case.row_of(b, j)], p)
