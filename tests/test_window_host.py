"""Refusals of windowed attention and the 4-bit cache before anything is launched, and their oracle's own pins (no GPU)."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
import pagedattention_kv_cache_paged_gb300 as pa
from oracle import window_oracle as WO
from pagedattention_kv_cache_paged_gb300 import _abi
from test_tree_host import P, call, lib  # noqa: F401  (lib: the fixture)
from window_cases import ALL, PackedCase, WindowCase, pack

OPTS = {"stride": dict(kv_block_stride_bytes=16 * 2 * 64 * 2 + 8), "short": dict(kv_block_stride_bytes=16 * 2 * 64 * 2 - 16),
        "kernel": dict(prefill_kernel=3), "part": dict(partition_tokens=-1), "long": dict(partition_tokens=2 ** 30 + 1),
        "wide": dict(kv_block_stride_bytes=2 * 16 * 2 * 64 * 2)}


def status(lib, name, base, change):  # noqa: F811
    change = dict(change)
    if "opts" in change:
        change["opts"] = ctypes.byref(pa.make_opts(**OPTS[change["opts"]]))
    return call(lib, name, list(base), base, **change)


ONE = dict(out=P, q=P, qsl=None, total_q=2, window=64, sinks=4, k=P, v=P, table=P, stride=4, ctx=P, batch=2, blocks=8, bs=16,
           scale=0.125, hq=8, hkv=2, d=64, dt=pa.PA_BF16, ws=None, ws_bytes=0, opts=None, stream=None)
CHUNKS = dict(ONE, qsl=P, total_q=7)
SHARED = [
    (dict(dt=7), "EDTYPE"), (dict(hq=6, hkv=4), "EINVAL"), (dict(hq=64, hkv=2), "EUNSUPPORTED"), (dict(hq=0), "EINVAL"),
    (dict(hq=6, hkv=2), "EUNSUPPORTED"), (dict(d=96), "EUNSUPPORTED"), (dict(bs=12), "EUNSUPPORTED"),
    (dict(bs=512), "EUNSUPPORTED"), (dict(bs=0), "EINVAL"), (dict(batch=-1), "EINVAL"), (dict(window=0), "EINVAL"),
    (dict(window=-1), "EINVAL"), (dict(sinks=-1), "EINVAL"), (dict(scale=0.0), "EINVAL"), (dict(scale=-0.0), "EINVAL"),
    (dict(scale=-1.0), "EINVAL"), (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
    (dict(scale=2.36e38), "EINVAL"), (dict(out=None), "EINVAL"), (dict(q=None), "EINVAL"), (dict(q=P + 2), "EINVAL"),
    (dict(out=P + 8), "EINVAL"), (dict(ctx=None), "EINVAL"), (dict(table=None), "EINVAL"), (dict(stride=0), "EINVAL"),
    (dict(blocks=0), "EINVAL"), (dict(opts="kernel"), "EINVAL"), (dict(opts="part"), "EINVAL"), (dict(opts="long"), "EINVAL"),
]


@pytest.mark.parametrize("chunks", [False, True])
@pytest.mark.parametrize("change,want", SHARED + [
    (dict(k=None), "EINVAL"), (dict(k=P + 8), "EINVAL"), (dict(v=None), "EINVAL"), (dict(v=P + 2), "EINVAL"),
    (dict(total_q=-1), "EINVAL"), (dict(opts="stride"), "EINVAL"), (dict(opts="short"), "EINVAL"),
    (dict(batch=0, total_q=0), "OK"), (dict(batch=0, total_q=0, scale=2.35e38), "OK"), (dict(batch=0, total_q=0, scale=1e-45), "OK"),
    (dict(batch=0, total_q=0, window=ALL, sinks=ALL), "OK"),
])
def test_window_refusals(lib, chunks, change, want):  # noqa: F811
    assert status(lib, "paged_attention_window", CHUNKS if chunks else ONE, change) == getattr(pa, "PA_" + want)


def test_query_rows_and_sequences_that_do_not_fit_each_other(lib):  # noqa: F811
    for total in (0, 1, 3):
        assert status(lib, "paged_attention_window", ONE, dict(total_q=total)) == pa.PA_EINVAL
    assert status(lib, "paged_attention_window", CHUNKS, dict(total_q=2 ** 31)) == pa.PA_EINVAL
    assert status(lib, "paged_attention_window", CHUNKS, dict(total_q=0)) == pa.PA_OK


Q4 = dict(out=P, q=P, kc=P, vc=P, kp=P, vp=P, table=P, stride=4, ctx=P, batch=2, blocks=8, bs=16, window=64, sinks=4,
          scale=0.125, hq=8, hkv=2, d=64, dt=pa.PA_BF16, ws=None, ws_bytes=0, opts=None, stream=None)
CACHE = [(dict([(name, wrong)]), "EINVAL") for name in ("kc", "vc", "kp", "vp") for wrong in (None, P + 8)]


@pytest.mark.parametrize("change,want", SHARED + CACHE + [
    (dict(opts="wide"), "EINVAL"),  # the cache is contiguous
    (dict(blocks=2 ** 27), "EUNSUPPORTED"),  # rows past 32 bits
    (dict(batch=0), "OK"), (dict(batch=0, scale=2.35e38), "OK"), (dict(batch=0, window=ALL, sinks=ALL), "OK"),
])
def test_decode_q4_refusals(lib, change, want):  # noqa: F811
    assert status(lib, "paged_attention_decode_q4", Q4, change) == getattr(pa, "PA_" + want)


WRITE = dict(kn=P, vn=P, slots=P, n=4, kc=P, vc=P, kp=P, vp=P, blocks=8, bs=16, hkv=2, d=64, dt=pa.PA_BF16, stream=None)
SIZES = [(dict(dt=7), "EDTYPE"), (dict(bs=0), "EINVAL"), (dict(bs=24), "EUNSUPPORTED"), (dict(bs=512), "EUNSUPPORTED"),
         (dict(hkv=0), "EINVAL"), (dict(d=0), "EINVAL"), (dict(d=32), "EUNSUPPORTED"), (dict(d=96), "EUNSUPPORTED"),
         (dict(d=256), "EUNSUPPORTED"), (dict(hkv=2 ** 20, d=128), "EUNSUPPORTED")]


@pytest.mark.parametrize("change,want", SIZES + CACHE + [
    (dict(n=-1), "EINVAL"), (dict(n=0), "OK"), (dict(kn=None), "EINVAL"), (dict(vn=None), "EINVAL"), (dict(slots=None), "EINVAL"),
    (dict(kn=P + 8), "EINVAL"), (dict(vn=P + 4), "EINVAL"), (dict(blocks=0), "EINVAL"), (dict(blocks=2 ** 27), "EUNSUPPORTED"),
])
def test_write_q4_refusals(lib, change, want):  # noqa: F811
    assert status(lib, "paged_kv_write_q4", WRITE, change) == getattr(pa, "PA_" + want)


UNPACK = dict(kc=P, vc=P, kp=P, vp=P, from_blocks=8, k=P, v=P, blocks=8, pairs=P, n=3, bs=16, hkv=2, d=64, dt=pa.PA_BF16,
              opts=None, stream=None)


@pytest.mark.parametrize("change,want", SIZES + CACHE + [
    (dict(n=-1), "EINVAL"), (dict(n=0), "OK"), (dict(n=0, opts="wide"), "OK"), (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"),
    (dict(k=P + 8), "EINVAL"), (dict(v=P + 2), "EINVAL"), (dict(pairs=None), "EINVAL"), (dict(blocks=0), "EINVAL"),
    (dict(from_blocks=0), "EINVAL"), (dict(from_blocks=2 ** 27), "EUNSUPPORTED"), (dict(opts="stride"), "EINVAL"),
    (dict(opts="short"), "EINVAL"),
])
def test_unpack_q4_refusals(lib, change, want):  # noqa: F811
    assert status(lib, "paged_kv_unpack_q4", UNPACK, change) == getattr(pa, "PA_" + want)


@pytest.mark.parametrize("name", ["paged_attention_window_workspace_size", "paged_attention_decode_q4_workspace_size"])
def test_workspace_of_bad_sizes_is_zero(lib, name):  # noqa: F811
    good = [2, 512, 16, 4096, 4, 8, 2, 64, pa.PA_BF16]
    for i, wrong in [(i, 0) for i in (0, 1, 2, 3, 5, 6, 7)] + [(4, -1), (5, 7), (5, 64), (7, 96), (2, 24), (2, 512), (8, 9)]:
        bad = list(good)
        bad[i] = wrong
        assert getattr(lib, name)(*bad, None) == 0, (i, wrong)
    for o in OPTS.values():
        if o.get("partition_tokens") or o.get("prefill_kernel"):
            assert getattr(lib, name)(*good, ctypes.byref(pa.make_opts(**o))) == 0


def test_the_binding_refuses_wrong_tensors(lib):  # noqa: F811
    """By type, layout and place; all of these are on the CPU, which the calls refuse too."""
    case = WindowCase(1, [4, 40], [2, 3], 30, 2, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=torch.float32)
    good = dict(q=case.q, query_start_loc=case.qsl, k_pool=case.k, v_pool=case.v, block_table=case.table,
                context_lens=case.ctx, window=30)
    for change in (dict(), dict(q=case.q[0]), dict(q=case.q[..., :32]), dict(block_table=case.table[:1]),
                   dict(v_pool=case.v[:2]), dict(query_start_loc=None), dict(out=case.q[:2]),
                   dict(window=2 ** 31), dict(sinks=2 ** 31), dict(window=-2 ** 31 - 1)):
        with pytest.raises(ValueError):
            pa.paged_attention_window(**{**good, **change})
    for wrong in (2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="window must fit 32 bits"):
            _abi._int32(window=wrong, sinks=0)
    for name in ("q", "query_start_loc", "k_pool", "v_pool", "block_table", "context_lens"):
        with pytest.raises((TypeError, ValueError)):
            pa.paged_attention_window(**{**good, name: [1, 2]})
    packed = PackedCase(1, [4, 40], ALL, 0, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=torch.bfloat16)
    cache = pa.Q4Cache(packed.kc, packed.vc, packed.kp, packed.vp)
    good = dict(q=packed.q, cache=cache, block_table=packed.table, context_lens=packed.ctx)
    for change in (dict(), dict(q=packed.q[0]), dict(q=packed.q[:1]), dict(window=2 ** 31), dict(sinks=-2 ** 31 - 1)):
        with pytest.raises(ValueError):
            pa.paged_attention_decode_q4(**{**good, **change})
    for wrong in (None, cache[:3], (1, 2, 3, 4), packed.kc, cache._replace(k_codes=packed.kc[0])):
        with pytest.raises(TypeError, match="cache must be a Q4Cache"):
            pa.paged_attention_decode_q4(**{**good, "cache": wrong})
        with pytest.raises(TypeError, match="cache must be a Q4Cache"):
            pa.paged_kv_write_q4(packed.k[0], packed.k[0], torch.arange(16), wrong)
    with pytest.raises(ValueError):
        pa.paged_kv_write_q4(packed.k[0], packed.k[0], torch.arange(16), cache)
    for name, wrong in (("k_new", [1]), ("slot_mapping", [1])):
        with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
            pa.paged_kv_write_q4(**{**dict(k_new=packed.k[0], v_new=packed.k[0], slot_mapping=torch.arange(16), cache=cache),
                                    name: wrong})
    for name, wrong in (("k_pool", [1]), ("block_pairs", [[0, 1]])):
        with pytest.raises(TypeError, match=f"{name} must be a torch.Tensor"):
            pa.paged_kv_unpack_q4(**{**dict(cache=cache, k_pool=packed.k, v_pool=packed.v, block_pairs=torch.zeros((1, 2))),
                                     name: wrong})


# ---------------------------------------------------------------------------------------------
# the oracle: windowed attention
# ---------------------------------------------------------------------------------------------

def case64(seed=2, **kw):
    a = dict(window=20, sinks=3, q_heads=4, kv_heads=2, head_dim=64, block_size=16, dtype=torch.float32)
    return WindowCase(seed, [70, 9, 33], [5, 9, 20], **{**a, **kw})


def run(case, **change):
    a = dict(q=case.q, query_start_loc=case.qsl, k_pool=case.k, v_pool=case.v, block_table=case.table, context_lens=case.ctx,
             scale=0.125, window=case.window, sinks=case.sinks)
    return WO.window_attention(**{**a, **change})


def torch_attention(case, mask_of):
    """torch's float64 attention under an explicit mask of positions, sequence by sequence."""
    out, t = [], 0
    for n, m, table in zip(case.ctx_list, case.new_list, case.table):
        at = torch.arange(n)
        blk = table[at // 16].long().clamp(min=0)
        k, v = (torch.nan_to_num(p[blk, at % 16].double()).transpose(0, 1).repeat_interleave(2, 0) for p in (case.k, case.v))
        p = torch.arange(n - m, n)[:, None]
        q = case.q[t:t + m].double().transpose(0, 1)
        res = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], attn_mask=mask_of(p, at[None]),
                                                               scale=0.125)[0]
        out.append(res.transpose(0, 1))
        t += m
    return torch.cat(out).numpy()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (20, 3), (20, 60), (500, 0), (ALL, ALL)])
def test_the_oracle_is_torch_under_the_mask(window, sinks):
    case = case64(window=window, sinks=sinks)
    want = torch_attention(case, lambda p, j: (j <= p) & ((p - j < window) | (j < sinks)))
    assert np.abs(run(case)[1] - want).max() < 1e-12


@pytest.mark.parametrize("mistake", [lambda p, j: (j <= p) & ((p - j <= 20) | (j < 3)), lambda p, j: (j <= p) & ((p - j < 20) | (j <= 3)),
                                     lambda p, j: (j < p) & ((p - j < 20) | (j < 3)) | (j == p - 1) | (j == 0),
                                     lambda p, j: (j <= p) & (p - j < 20)])
def test_planted_masks_are_seen(mistake):
    case = case64()
    assert not np.abs(run(case)[1] - np.nan_to_num(torch_attention(case, mistake))).max() < 1e-3


def test_without_a_window_it_is_the_causal_chunk_and_the_decode():
    case = case64(window=ALL, sinks=0)
    ref = oracle.paged_prefill(case.q, case.qsl, case.k, case.v, case.table, case.ctx, 0.125)
    rows, out, spread, size = run(case)
    assert all(np.abs(out[i] - ref[r]).max() < 1e-12 for i, r in enumerate(rows))
    assert (np.abs(out) <= spread + 1e-12).all() and (size > 0).all()
    q = case.q[:3]
    one = WO.window_attention(q, None, case.k, case.v, case.table, case.ctx, 0.125, ALL, 0)[1]
    assert np.abs(one - oracle.paged_decode(q, case.k, case.v, case.table, case.ctx, 0.125)).max() < 1e-12


def test_a_window_of_one_is_the_value_itself():
    case = case64(window=1, sinks=0)
    rows, out, _, _ = run(case)
    t = 0
    for b, (n, m) in enumerate(zip(case.ctx_list, case.new_list)):
        for j in range(n - m, n):
            assert np.array_equal(out[t], case.v[case.row_of(b, j)].double().repeat_interleave(2, 0).numpy())
            t += 1


# ---------------------------------------------------------------------------------------------
# the oracle: the 4-bit format
# ---------------------------------------------------------------------------------------------

def test_a_group_worked_by_hand():
    """0, 1, .. 15 and back: scale 1, zero 0, the codes themselves; shifted down by 5: zero 5."""
    x = [min(i, 15) for i in range(64)]
    codes, scale, zero = WO.pack_group(x)
    assert codes == x and (scale, zero) == (1.0, 0)
    codes, scale, zero = WO.pack_group([v - 5 for v in x])
    assert codes == x and (scale, zero) == (1.0, 5)
    # halves go to the even number: 0.5 -> 0, 1.5 -> 2, 2.5 -> 2
    codes, _, _ = WO.pack_group([15.0, 0.5, 1.5, 2.5] + [0.0] * 60)
    assert codes[:4] == [15, 0, 2, 2]
    # a byte holds the even dimension in its low half
    c, p = WO.q4_pack(torch.tensor([[15.0, 1.0] + [0.0] * 62]))
    assert c[0, 0] == 15 | 1 << 4 and not c[0, 1:].any() and p.tolist() == [[1.0, 0.0]]


def test_groups_of_nothing_and_of_what_is_not_finite():
    assert WO.pack_group([0.0] * 64) == ([0] * 64, 0.0, 0)
    assert WO.pack_group([2.0 ** -130] * 64) == ([0] * 64, 0.0, 0)
    for bad in (float("nan"), float("inf"), -float("inf")):
        codes, scale, zero = WO.pack_group([1.0] * 63 + [bad])
        assert codes == [0] * 64 and np.isnan(scale) and zero == 0
        c, p = WO.q4_pack(torch.tensor([[1.0] * 63 + [bad]]))
        assert np.isnan(WO.q4_values(torch.from_numpy(c), torch.from_numpy(p))).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_values_come_back_near_where_they_were(dtype):
    """The scale is at most one bf16 half step (2^-9) and a few fp32 ones below (hi - lo) / 15.  Inside the codes' range a
    value moves by half a scale for its own code, and its zero's rounding moves only which codes are cut off: a value next
    to an end lies at most 15 2^-9 + 1/2 of a zero's step outside the middle of the last code, 1/2 + 15/512 + 1/512 of a
    scale and its rounding in all, below 9/16."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn((40, 2, 128), generator=g).to(dtype)
    x[::2] += 1.5
    x[1::4] *= 1e-3
    c, p = WO.q4_pack(x)
    back = WO.q4_values(torch.from_numpy(c), torch.from_numpy(p))
    scale = np.repeat(p[..., 0::2], 64, -1)
    assert (np.abs(back - x.double().numpy()) <= scale * 9 / 16).all()
    fast_c, fast_p = pack(x)
    assert np.array_equal(c, fast_c.numpy()) and np.array_equal(p, fast_p.double().numpy())


def test_every_code_is_the_nearest_point():
    """Against a search of the whole grid, exactly: no point of it lies nearer (ties aside)."""
    g = torch.Generator().manual_seed(10)
    for x in ((torch.randn(64, generator=g) * 4).round() / 4, torch.randn(64, generator=g)):
        codes, scale, zero = WO.pack_group(x)
        for v, c in zip(x.tolist(), codes):
            off = [abs(Fraction(v) - Fraction(scale) * (k - zero)) for k in range(16)]
            assert off[c] == min(off)


@pytest.mark.parametrize("mistake", ["halves", "order", "zero"])
def test_planted_mistakes_of_the_format_are_seen(mistake, monkeypatch):
    x = torch.tensor([[-5.0, 10.0] + [0.5 * i - 4 for i in range(28)] + [0.0] * 34])
    c, p = WO.q4_pack(x)
    if mistake == "halves":
        monkeypatch.setattr(WO, "_nearest", lambda a, s: int((a / s + Fraction(1, 2)) // 1))
    if mistake == "order":
        fine = WO.q4_values
        monkeypatch.setattr(WO, "q4_values", lambda c, p: fine(c, p).reshape(-1, 2)[:, ::-1].reshape(1, -1))
    if mistake == "zero":
        p = p.copy()
        p[..., 1::2] += 1
    bad_c, _ = WO.q4_pack(x)
    back = WO.q4_values(torch.from_numpy(bad_c), torch.from_numpy(p))
    assert not np.array_equal(bad_c, c) or np.abs(back - x.double().numpy()).max() > 0.9
