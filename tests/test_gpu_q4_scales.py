"""Attention over a 4-bit cache whose scales lie far apart: what a token of little weight costs the others."""
import numpy as np
import pytest
import torch

import oracle
from window_cases import int32, pack

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _clean(cuda_lib):
    cuda_lib.device_error_flags(clear=True)
    yield
    cuda_lib.device_error_flags(clear=True)


class Case:
    """One sequence of `n` tokens in blocks of 16; `weight` {token: log2 of its weight against the others'}, `scale`
    {token: log2 of what the scales of its values are multiplied by}."""

    def __init__(self, seed, n, dtype, weight, scale, *, kv_heads=2, group=4, head_dim=128):
        g = torch.Generator().manual_seed(seed)
        self.n, self.dtype, D = n, dtype, head_dim
        blocks = -(-n // 16)
        # queries with one large dimension, which alone decides the weights that are given
        self.q = 0.25 * torch.randn((1, kv_heads * group, D), generator=g)
        self.q[..., 3] = 8.0
        self.q = self.q.to(dtype)
        k = torch.randn((blocks * 16, kv_heads, D), generator=g)
        k[..., 3] = 0.0
        for t, w in weight.items():
            k[t] = 0.0
            k[t, :, 3] = w * np.log(2.0) * D ** 0.5 / 8.0
        rows = (blocks, 16, kv_heads)
        self.kc, self.kp = (x.view(rows + x.shape[2:]) for x in pack(k))
        self.vc, self.vp = (x.view(rows + x.shape[2:]) for x in pack(torch.randn((blocks * 16, kv_heads, D), generator=g)))
        for t, e in scale.items():
            self.vp[t // 16, t % 16, :, 0::2] *= 2.0 ** e
        self.table = torch.arange(blocks, dtype=torch.int32)[None]
        self.group = group

    def run(self, pa, **kw):
        cache = pa.Q4Cache(*(x.cuda() for x in (self.kc, self.vc, self.kp, self.vp)))
        return pa.paged_attention_decode_q4(self.q.cuda(), cache, self.table.cuda(), int32([self.n]).cuda(), **kw)

    def oracle(self):
        """(output, how far one may be from it) in 64 bits, [Hq, D].

        Every key by itself.  Its score: sums of products in 32 bits, head_dim + 4 half steps of their absolute values
        (query values times codes, and times zeros), the exponential's argument one more and the exponential 2^-22; its
        weight is off by that, in the numerator and in the denominator.  Weight times scale: half a step of fp16 (2^-11),
        at least half of 2^-25 of the largest product of the head and the group (bf16 and fp16 queries), or 2^-24 (fp32);
        a weight below 2^-126 of the largest may be left out.  Sums of codes of up to 15, and of zeros times codes' weights:
        a tensor core's, cut off at 2^-23 a step of 16 tokens.  Then half a step of the output's type."""
        D, u32 = self.q.shape[2], 2.0 ** -24
        k, v = (oracle.window.q4_values(c, p).reshape(-1, *c.shape[2:3], D)[:self.n] for c, p in ((self.kc, self.kp), (self.vc, self.vp)))
        ks, vs = (p[..., 0::2].double().numpy().reshape(-1, p.shape[2], D // 64)[:self.n] for p in (self.kp, self.vp))
        rep = lambda x: np.repeat(x, self.group, 1)  # noqa: E731
        k, v, ks, vs = rep(k), rep(v), rep(ks), rep(vs)
        q = self.q[0].double().numpy()
        z = np.einsum("hd,nhd->nh", q, k) * D ** -0.5
        size = np.einsum("hg,nhg->nh", np.abs(q).reshape(q.shape[0], -1, 64).sum(-1), ks) * 30 * D ** -0.5
        w = np.exp(z - z.max(0))
        raw = w.copy()
        w /= w.sum(0)
        ref = np.einsum("nh,nhd->hd", w, v)
        rel = (D + 4) * u32 * size + 2.0 ** -22 + u32 * np.abs(z - z.max(0))
        wide = lambda x: np.repeat(x, 64, -1)  # noqa: E731 (a group's number for each of its dimensions)
        products = w[:, :, None] * vs                                        # [n, h, group]
        step = 2.0 ** -24 if self.dtype == FP32 else 2.0 ** -11
        off = np.einsum("nh,nhd->hd", w * (rel + step), np.abs(v)) + np.abs(ref) * np.einsum("nh,nh->h", w, rel)[:, None]
        if self.dtype != FP32:
            off += wide(self.n * 15 * 2.0 ** -26 * products.max(0))
        off += wide(np.where(raw < 2.0 ** -125, 15 * products.transpose(2, 0, 1), 0).sum(1).T)
        off += wide((self.n / 16 + 16) * 2.0 ** -23 * 30 * products.sum(0)) + 2 * (self.n + 16) * u32 * np.abs(ref)
        half = torch.finfo(self.dtype).eps / 2
        return ref, (off + half * np.maximum(np.abs(ref), torch.finfo(self.dtype).tiny)) * (1 + half)

    def check(self, pa, **kw):
        ref, off = self.oracle()
        got = self.run(pa, **kw)[0].double().cpu().numpy()
        assert np.isfinite(got).all()
        excess = np.abs(got - ref) - off
        assert (excess <= 0).all(), f"worst excess {excess.max()} of {np.abs(ref).max()}"
        assert pa.device_error_flags() == 0


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where", [0, 300, 512])
@pytest.mark.parametrize("far", [8, 24, 32, 60, 100])
def test_a_large_scale_of_little_weight(cuda_lib, dtype, D, where, far):
    """Its product is 2^-8 of the others'; they keep their bits, whatever its scale."""
    Case(far, 513, dtype, {where: -far - 8}, {where: far}, head_dim=D).check(cuda_lib)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("group", [1, 16])
@pytest.mark.parametrize("workspace", ["auto", None])
def test_scales_of_every_size(cuda_lib, dtype, group, workspace):
    """Every eighth token has a scale of its own, up to 2^90 over the others', and a weight that outweighs it."""
    far = {t: 3 * (7 * t // 8 % 31) for t in range(0, 500, 8)}
    Case(3, 500, dtype, {t: -e - 5 for t, e in far.items()}, far, group=group).check(cuda_lib, workspace=workspace)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("weight", [20, 60, 100])
def test_a_late_token_of_all_the_weight(cuda_lib, dtype, weight):
    """The first tokens' products are the largest until a token comes whose weight takes theirs to nothing, with a small
    scale; then others like it."""
    late = {t: weight for t in (200, 201, 320)}
    Case(4, 400, dtype, late, {**{t: 10 for t in range(0, 190, 3)}, **{t: -12 for t in late}}).check(cuda_lib)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_a_scale_near_the_largest_without_weight(cuda_lib, dtype):
    """A weight of 0 in 32 bits, times whatever scale, is 0."""
    Case(5, 300, dtype, {7: -300.0, 170: -300.0, 290: -300.0}, {7: 120, 170: 125, 290: 60}).check(cuda_lib)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("power", [-110, 110])
def test_scales_near_the_ends_of_the_range(cuda_lib, dtype, power):
    scale = {t: power + t % 5 for t in range(400)}
    Case(6, 400, dtype, {t: t % 7 - 3.0 for t in range(0, 400, 9)}, scale).check(cuda_lib)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("largest", [1.0, 2.0 ** -12, 30000.0])
def test_small_values_of_a_query(cuda_lib, dtype, D, largest):
    """A head's largest value meets keys of 0 and the others are 2^-12 to 2^-30 of it: each enters by itself, rounded by 2^-35
    of the largest at most, and only below 2^-27 (bf16) or 2^-24 (fp16)."""
    pa, n, H = cuda_lib, 64, 2
    g = torch.Generator().manual_seed(D)
    size = torch.exp2(-12 - 18 * torch.rand((1, H, D), generator=g))
    q = (size * torch.randn((1, H, D), generator=g)).clamp(-2.0 ** -9, 2.0 ** -9)
    q[..., ::16] = 1.0
    q = (q * largest).to(dtype)
    k = torch.rand((n // 16, 16, H, D), generator=g)
    k[..., ::16] = 0.0
    (kc, kp), (vc, vp) = pack(k), pack(torch.randn(k.shape, generator=g))
    assert (kp[..., 1::2] == 0).all()  # (so that the largest value is multiplied by nothing but codes of 0)
    scale = 2.0 ** 10 / largest
    got = pa.paged_attention_decode_q4(q.cuda(), pa.Q4Cache(*(x.cuda() for x in (kc, vc, kp, vp))),
                                       torch.arange(n // 16, dtype=torch.int32)[None].cuda(), int32([n]).cuda(), scale=scale)
    kf, vf = (oracle.window.q4_values(c, p).reshape(n, H, D) for c, p in ((kc, kp), (vc, vp)))
    qf, u32 = q[0].double().numpy(), 2.0 ** -24
    z = scale * np.einsum("hd,nhd->nh", qf, kf)
    w = np.exp(z - z.max(0))
    w /= w.sum(0)
    ref, spread = np.einsum("nh,nhd->hd", w, vf), np.einsum("nh,nhd->hd", w, np.abs(vf))
    top = np.abs(qf).max(1)[:, None]
    small = np.abs(qf) < top * (2.0 ** -27 if dtype == BF16 else 2.0 ** -24)
    assert small.any() and not small.all()
    lost = scale * (np.einsum("hd,nhd->nh", small * top * 2.0 ** -35, kf) + (D + 4) * u32 * np.einsum("hd,nhd->nh", np.abs(qf) * (qf != top), kf)).max(0)
    rel = 2 * (lost + 2.0 ** -22 + u32 * np.abs(z).max(0)) + 2 * (n + 16) * u32 + 2.0 ** -11
    off = spread * rel[:, None] + n * 15 * 2.0 ** -26 * vp[..., 0::2].double().numpy().max()
    half = torch.finfo(dtype).eps / 2
    assert (np.abs(got[0].double().cpu().numpy() - ref) <= (off + half * np.abs(ref)) * (1 + half)).all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 16, 64, 700])
@pytest.mark.parametrize("gain", [1.0, 3.0])
def test_dimensions_of_zeros(cuda_lib, dtype, D, n, gain):
    """Values of 0 are code = zero: two sums that are taken from one another.  With fp32 queries the difference is formed
    first, and is 0; else 16 products and a sum are each cut off at 2^-14 of a step's largest product of weight and scale, in
    units of a code, and the largest of the steps, summed, are at most the sum of all weights."""
    pa, H, S = cuda_lib, 4, 16
    g = torch.Generator().manual_seed(n)
    rows = (-(-n // S), S, H, D)
    k, v = gain * torch.randn(rows, generator=g), torch.zeros(rows)
    v[..., 0::64] = -0.5 - 4 * torch.rand(v[..., 0::64].shape, generator=g)
    v[..., 1::64] = 0.5 + 4 * torch.rand(v[..., 1::64].shape, generator=g)
    (kc, kp), (vc, vp) = pack(k), pack(v)
    q = torch.randn((1, 4 * H, D), generator=g).to(dtype)
    got = pa.paged_attention_decode_q4(q.cuda(), pa.Q4Cache(*(x.cuda() for x in (kc, vc, kp, vp))),
                                       torch.arange(rows[0], dtype=torch.int32)[None].cuda(), int32([n]).cuda())
    zeros = got[0].float().cpu().unflatten(-1, (-1, 64))[..., 2:].abs().max()
    assert zeros <= (0.0 if dtype == FP32 else 17 * 2.0 ** -14 * float(vp[..., 0::2].float().max()))
