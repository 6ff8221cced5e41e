"""Long contexts that one CTA goes through alone: sums do not drift with their length."""
import numpy as np
import pytest
import torch

import oracle
from window_cases import ALL, int32, pack

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
BASE = 512  # tokens, seen again and again


@pytest.fixture(autouse=True)
def _clean(cuda_lib):
    cuda_lib.device_error_flags(clear=True)
    yield
    cuda_lib.device_error_flags(clear=True)


def table_of(n, S):
    return (torch.arange(n // S, dtype=torch.int32) % (BASE // S))[None].cuda()


def bound(dtype, q, k, v, times, lost, weight, cut):
    """(output, how far one may be from it), [Hq, D], of queries [Hq, D] over keys and values [BASE, Hq, D], each `times` over.

    Scores: head_dim + 4 half steps of their absolute products (`lost` [Hq]), the exponential's argument one more, the
    exponential 2^-22, in the numerator and in the denominator.  `weight`: relative rounding of a weight for the product with
    V.  Sums: runs of at most 256 steps of 16 tokens, each a rounded addition (32-bit pools) or one of the tensor core's, which
    cuts off up to 2^-23 of the absolute sum `cut` [Hq, D]; then one rounded addition a run and 64 for lanes, warps
    and parts.  Half a step of the output."""
    u32 = 2.0 ** -24
    z = np.einsum("hd,nhd->hn", q, k) * q.shape[1] ** -0.5
    w = np.exp(z - z.max(1, keepdims=True)) * times
    w /= w.sum(1, keepdims=True)
    ref, spread = np.einsum("hn,nhd->hd", w, v), np.einsum("hn,nhd->hd", w, np.abs(v))
    adds = (256 if cut else 16 * 256) + times.sum() / (256 * 16) + 64
    off = spread * (2 * ((q.shape[1] + 4) * u32 * lost[:, None] + 2.0 ** -22 + adds * u32) + weight * (1 + weight))
    if cut:
        off = off + 256 * 2.0 ** -23 * cut(w)
    half = torch.finfo(dtype).eps / 2
    return ref, (off + half * np.abs(ref)) * (1 + half)


def check(pa, got, ref, off):
    assert pa.device_error_flags() == 0
    excess = np.abs(got[0].double().cpu().numpy() - ref) - off
    assert (excess <= 0).all(), f"worst excess {excess.max()} of {np.abs(ref).max()}"


# a context by one CTA for a unit, or in parts of so many tokens
SPLITS = [dict(workspace=None), dict(partition_tokens=200_000)]


@pytest.mark.parametrize("dtype,log_n,window", [(FP16, 21, ALL), (FP16, 20, 2 ** 19 + 5), (BF16, 23, ALL), (FP32, 20, ALL)])
@pytest.mark.parametrize("S", [8, 16])
@pytest.mark.parametrize("group", [1, 16])
@pytest.mark.parametrize("split", SPLITS)
def test_pools(cuda_lib, dtype, log_n, window, S, group, split):
    """Values of one sign, so that whatever sums lose shows."""
    pa, n, D, H = cuda_lib, 1 << log_n, 64, 2
    g = torch.Generator().manual_seed(log_n + group)
    k = torch.randn((BASE // S, S, H, D), generator=g).to(dtype)
    v = (1 + 0.2 * torch.rand((BASE // S, S, H, D), generator=g)).to(dtype)
    q = torch.randn((1, H * group, D), generator=g).to(dtype)
    got = pa.paged_attention_window(q.cuda(), None, k.cuda(), v.cuda(), table_of(n, S), int32([n]).cuda(), window,
                                    **split)
    kf, vf = (np.repeat(x.double().numpy().reshape(BASE, H, D), group, 1) for x in (k, v))
    qf = q[0].double().numpy()
    size = (np.einsum("hd,nhd->hn", np.abs(qf), np.abs(kf)) * D ** -0.5).max(1)
    weight = 0.0 if dtype == FP32 else torch.finfo(dtype).eps / 2
    seen = min(n, window)
    times = np.full(BASE, seen // BASE) + (np.arange(BASE) >= BASE - seen % BASE)
    check(pa, got, *bound(dtype, qf, kf, vf, times, size, weight,
                          None if dtype == FP32 else lambda w: np.einsum("hn,nhd->hd", w, np.abs(vf))))


@pytest.mark.parametrize("dtype,log_n", [(FP16, 20), (FP16, 17), (BF16, 21), (FP32, 20)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,group", [(8, 1), (8, 2), (2, 16), (1, 1)])
@pytest.mark.parametrize("split", SPLITS)
def test_the_4_bit_cache(cuda_lib, dtype, log_n, D, H, group, split):
    """Large codes and small ones, zeros of 0 and of 7: what is summed is larger than what is left."""
    pa, n, S = cuda_lib, 1 << log_n, 16
    g = torch.Generator().manual_seed(log_n + D)
    k = torch.randn((BASE // S, S, H, D), generator=g)
    v = 6 + torch.rand((BASE // S, S, H, D), generator=g)
    v[..., 0::64] = 0
    v[..., 1::2] -= 5.5
    v[..., 3::64] = torch.where(torch.arange(S)[:, None, None] % 2 == 0, -6.0, 0.0).expand(v[..., 3::64].shape)
    (kc, kp), (vc, vp) = pack(k), pack(v)
    q = torch.randn((1, H * group, D), generator=g).to(dtype)
    cache = pa.Q4Cache(*(x.cuda() for x in (kc, vc, kp, vp)))
    got = pa.paged_attention_decode_q4(q.cuda(), cache, table_of(n, S), int32([n]).cuda(), **split)
    kf, vf = (np.repeat(oracle.window.q4_values(c, p).reshape(BASE, H, D), group, 1) for c, p in ((kc, kp), (vc, vp)))
    ks, vs = (np.repeat(p[..., 0::2].double().numpy().reshape(BASE, H, D // 64), group, 1) for p in (kp, vp))
    qf = q[0].double().numpy()
    size = (np.einsum("hg,nhg->nh", np.abs(qf).reshape(qf.shape[0], -1, 64).sum(-1), ks) * 30 * D ** -0.5).max(0)
    cut = None if dtype == FP32 else lambda w: np.repeat(30 * np.einsum("hn,nhg->hg", w, vs), 64, 1)
    ref, off = bound(dtype, qf, kf, vf, np.full(BASE, n // BASE), size, 2.0 ** (-24 if dtype == FP32 else -11), cut)
    if dtype != FP32:  # (fp16's smallest step: 2^-26 of the largest product, BASE tokens of which one has it at least)
        off = off + BASE * 15 * 2.0 ** -26 * vs.max()
    check(pa, got, ref, off)
