"""The 4-bit format's scale: products with fp32(1 / 15), on groups where quotients by 15 give another number."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from window_cases import pack

FP16, FP32 = torch.float16, torch.float32

# (lo, hi) of a group, and its scale by products and by quotients: both from exact fractions below
FP16_PAIR = (-1.7705078125, 2.052734375, 0.255859375, 0.25390625)


def nearest(x: Fraction, bits: int) -> Fraction:
    """x rounded to `bits` significant bits, halves to the even number."""
    if x == 0:
        return x
    step = Fraction(2) ** (abs(x).numerator.bit_length() - abs(x).denominator.bit_length())
    if abs(x) < step:
        step /= 2
    step /= 2 ** (bits - 1)
    return round(x / step) * step


def scale_of(lo, hi, products: bool) -> float:
    r = nearest(Fraction(1, 15), 24)
    part = lambda v: nearest(Fraction(v) * r if products else Fraction(v) / 15, 24)  # noqa: E731
    return float(nearest(nearest(part(hi) - part(lo), 24), 8))


def groups(dtype, n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((n, 1, 64), generator=g).to(dtype)


def test_a_group_where_the_two_rules_differ():
    lo, hi, by_products, by_quotients = FP16_PAIR
    assert scale_of(lo, hi, True) == by_products and scale_of(lo, hi, False) == by_quotients
    x = torch.linspace(lo, hi, 64).to(FP16)[None, None]
    assert x.min() == lo and x.max() == hi
    assert float(pack(x)[1][..., 0]) == by_products and oracle.window.q4_pack(x)[1][..., 0] == by_products


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP16, FP32])
def test_scales_by_exact_fractions(dtype):
    x = groups(dtype, 300, 1)
    want = [scale_of(float(v.min()), float(v.max()), True) for v in x[:, 0]]
    assert pack(x)[1][..., 0].double().flatten().tolist() == want
    assert oracle.window.q4_pack(x[:40])[1][..., 0].flatten().tolist() == want[:40]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,some", [(torch.bfloat16, False), (FP16, True), (FP32, True)])
def test_tensor_operations_on_the_gpu_pack_alike(cuda_lib, dtype, some):
    """(hi / 15 - lo / 15) of tensors on the GPU is the stored scale; the same on the CPU is not always."""
    pa, n = cuda_lib, 400_000
    x = groups(dtype, n, 2)
    x[0, 0] = torch.linspace(FP16_PAIR[0], FP16_PAIR[1], 64).to(dtype)
    cache = pa.q4_cache(n // 16, 16, 1, 64)
    pa.paged_kv_write_q4(x.cuda(), x.cuda(), torch.arange(n).cuda(), cache)

    def scale(t):
        v = t.float()
        return (v.amax((1, 2)).clamp(min=0) / 15 - v.amin((1, 2)).clamp(max=0) / 15).to(torch.bfloat16)

    stored = cache.k_params.view(n, 2)[:, 0]
    assert torch.equal(stored, scale(x.cuda()))
    apart = int((stored.cpu() != scale(x)).sum())
    assert (0 < apart < n // 300) if some else apart == 0
    if dtype == FP16:
        assert np.isclose(float(stored[0]), FP16_PAIR[2], rtol=0)
