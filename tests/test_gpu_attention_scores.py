"""GPU tests of attention where scores are far from those of normed heads: so large that one key takes all the
weight, beyond fp32 once they are scaled, or so far apart that most keys have next to none."""
import pytest
import torch

import attention_ref as ref
from test_gpu_attention import rand
from vla_action_head_b200 import nvfp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _probe():
    nvfp4.probe()


def winners(B, T, S, H, D, at, size):
    """Queries and keys along one direction u of signs, with a quarter of noise: key `at` is 2 u, the others are
    in [-u, u], so its scores (about 2 size D) exceed every other by 0.8 size D at least."""
    g = torch.Generator().manual_seed(S)
    u = (torch.randint(0, 2, (1, 1, 1, D), generator=g) * 2 - 1).float()
    a = torch.rand(B, S, H, 1, generator=g) * 2 - 1
    a[:, at] = 2.0
    k = (a * u + 0.05 * torch.randn(B, S, H, D, generator=g)).bfloat16()
    q = (size * (u + 0.25 * torch.rand(B, T, H, D, generator=g))).bfloat16()
    return q, k


@pytest.mark.parametrize("size", [1e3, 1e7, 1e9, 1e11, 1e13])
@pytest.mark.parametrize("B,T,S,H,D", [(1, 1, 300, 2, 128), (1, 1, 9000, 1, 256), (1, 9, 300, 1, 128), (1, 50, 300, 2, 128),
                                       (2, 150, 700, 2, 64), (1, 300, 200, 4, 48), (1, 70, 3000, 1, 256), (40, 140, 260, 8, 128),
                                       (1, 12, 4000, 1, 64)])
def test_one_key_takes_all(B, T, S, H, D, size):
    """Finite scores up to 1e16, one key far ahead of the others in every row: its weight is exactly 1 and the
    others' 0, so the output is that key's value, bit for bit, with bf16 keys and over the cache; wherever the
    key lies, so that the reference is found first, in between or last."""
    v = rand(B, S, H, D, seed=3)
    for at in (0, S // 2, S - 1):
        q, k = (t.cuda() for t in winners(B, T, S, H, D, at, size))
        c = nvfp4.empty_kv_cache(B, S, H, D)
        nvfp4.kv_write(c, k, v.cuda())
        kc, vc = nvfp4.kv_read(c)
        # the gap that the docstring claims, in 64 bits, for the keys as they are and as the cache holds them
        for kk in (k, kc):
            s = torch.einsum("bthd,bshd->bhts", q[:, :1].double(), kk.double())
            top = s[..., at].clone()
            s[..., at] = -float("inf")
            assert (top - s.amax(-1) > 0.5 * size * D).all()
        got = nvfp4.attention(q, k, v.cuda())
        assert torch.equal(got, v[:, at:at + 1].expand(B, T, H, D).cuda()), at
        got = nvfp4.attention(q, cache=c)
        assert torch.equal(got, vc[:, at:at + 1].expand(B, T, H, D)), at
    nvfp4.device_status()


@pytest.mark.parametrize("B", [1, 160])
@pytest.mark.parametrize("T,Hq", [(1, 1), (1, 8), (50, 1), (20, 8)])
def test_many_cached_keys_of_next_to_no_weight(B, T, Hq):
    """2^18 keys of weight 2^-25.4 beside one of weight 1 and value 0: all of the result, which is 0.58 % of the
    largest value.  (160 sequences: a CTA has the keys of a whole sequence, so the others' reference is that key.)

    Bound: the weights' roundings as in attention_ref.attention_ref, but off by 2^-32 each below fp16's normal range,
    as the largest is brought to 2^7 at least; scores are sums of 16 exact products; the sums are chains of 16 keys
    a step at least."""
    N, D = 1 << 18, 16
    c = nvfp4.empty_kv_cache(B, N, 1, D)
    c.k_codes[:, 0, 0], c.k_sf[:, 0, 0] = 0x22, 0x38  # 1.0 times a scale of 1
    c.v_codes[:, 0, 1:], c.v_sf[:, 0, 1:] = 0x22, 0x38
    q = torch.full((B, T, Hq, D), 1.1).bfloat16().cuda()
    x = 16 * float(q[0, 0, 0, 0])
    tail = (N - 1) * torch.exp(-torch.tensor(x, dtype=torch.float64))
    want = (tail / (1 + tail)).expand(B, T, Hq, D)
    rel = ref.BF16 + 2 * (2 * (D + 4) * ref.F32 * x) + 2 * ref.F32 * (2 * x + 8) + 4 * (N // 16 + 64) * ref.F32
    bound = ref.BF16 * want + 1.01 * rel * want + N * 2.0 ** -32
    ref.check(nvfp4.attention(q, cache=c, scale=1.0), want, bound)
    # the same with the key of weight 1 somewhere else, and behind a length
    for t in (c.k_codes, c.k_sf, c.v_codes, c.v_sf):
        t[:, 0, [0, N - 9]] = t[:, 0, [N - 9, 0]]
    n = torch.full((B,), N - 5, dtype=torch.int32).cuda()
    ref.check(nvfp4.attention(q, cache=c, kv_len=n, scale=1.0), want, bound + 5.0 / N * want)


@pytest.mark.parametrize("B,T,S,Hq,D", [(1, 1, 300, 1, 64), (1, 1, 9000, 8, 256), (150, 1, 700, 2, 128), (1, 50, 1500, 1, 64),
                                        (1, 9, 2000, 1, 256), (1, 50, 3000, 8, 256), (1, 300, 5000, 1, 128), (160, 20, 900, 1, 64)])
@pytest.mark.parametrize("large", [16, 20, 21, 22])
def test_parts_of_large_exact_scores(orc, B, T, S, Hq, D, large):
    """Scores 2^large + n / 4 (exact in fp32, as the sum of two exact products) with n rising along the keys, so that
    every part of the keys has another reference: their weights differ by exp(n / 4) all the same.

    Bound: no error in the scores; the weights' and the output's rounding to bf16 (fp16 is closer), the sums of S
    weights and products, 2^-32 a weight (cache), and the exponent: its difference of scores is exact, below 4 / ln 2
    = 5.8 in size, times a factor off by 2^-24 twice (scale log2(e) and the product), and 2^y off by 2^-22 as
    documented; each once in a key's weight and once in its part's.  From 2^22 on the sum is not exact: 2^22 to 2^-2
    are 25 bits, fp32 holds multiples of 1/2 there, and a score is off by less than that (cut or rounded): a weight
    by less than a factor of e^(1/2), and so is the sum that divides it."""
    n = (1 + torch.arange(S) * 15 // S).clamp(max=15)
    q, k = torch.zeros(B, T, Hq, D), torch.zeros(B, S, 1, D)
    q[..., 0], q[..., 16] = 2.0 ** large, 0.25
    k[..., 0], k[..., 16] = 1.0, n.float()[None, :, None]
    q, k, v = q.bfloat16().cuda(), k.bfloat16().cuda(), rand(1, S, 1, D, seed=4).cuda().expand(B, S, 1, D)
    c = nvfp4.empty_kv_cache(B, S, 1, D)
    nvfp4.kv_write(c, k, v)
    # a key's two blocks hold 1 and n: codes of 1 with scales of 1 and n
    for t in (c.k_codes, c.k_sf):
        t.zero_()
    c.k_codes[..., 0] = 2
    c.k_codes[..., 8] = 2
    c.k_sf[..., 0] = 0x38
    c.k_sf[:, :, :S, 1] = n.float().cuda().to(torch.float8_e4m3fn).view(torch.uint8)
    kr, vr = nvfp4.kv_read(c)
    assert torch.equal(kr, k)
    p = torch.softmax(n.double() / 4, 0)
    for got, val, cached in ((nvfp4.attention(q, k, v, scale=1.0), v, 0), (nvfp4.attention(q, cache=c, scale=1.0), vr, 1)):
        x = val[0, :, 0].double().cpu()
        want, A = p @ x, p @ x.abs()
        rel = ref.BF16 + 2 * (2 * 5.8 * ref.F32 + 2.0 ** -22) + 4 * (S + 64) * ref.F32
        rel += 2.72 - 1 if large >= 22 else 0.0
        bound = ref.BF16 * want.abs() + 1.01 * rel * A + cached * S * 2.0 ** -32 * x.abs().amax()
        ref.check(got, want.expand(B, T, Hq, D), bound.expand(B, T, Hq, D), cached)
    nvfp4.device_status()


@pytest.mark.parametrize("scale", [1e-20, 1e25, 3e38])
@pytest.mark.parametrize("T,S,H,D", [(1, 300, 2, 128), (1, 9000, 1, 256), (50, 300, 2, 128), (70, 3000, 1, 256), (12, 4000, 1, 64)])
def test_scaled_scores_beyond_fp32(T, S, H, D, scale):
    """Scores of 1e15 to 1e16 that fp32 holds, and does not hold once they are scaled; and scaled to next to nothing:
    all keys weigh the same within what the weights resolve."""
    q, k = (t.cuda() for t in winners(1, T, S, H, D, S // 3, 1e13))
    v = rand(1, S, H, D, seed=3).cuda()
    c = nvfp4.empty_kv_cache(1, S, H, D)
    nvfp4.kv_write(c, k, v)
    for f, x in ((lambda: nvfp4.attention(q, k, v, scale=scale), v), (lambda: nvfp4.attention(q, cache=c, scale=scale), nvfp4.kv_read(c)[1])):
        if scale > 1:
            assert torch.equal(f(), x[:, S // 3:S // 3 + 1].expand(1, T, H, D))
            continue
        want, A = x.double().mean(1, keepdim=True), x.double().abs().mean(1, keepdim=True)
        # scores below 1e-3: weights within 2e-3 of each other, in the weight and in the sum; roundings as elsewhere
        bound = ref.BF16 * want.abs() + 1.01 * (ref.BF16 + 2 * 2e-3 + 4 * (S + 64) * ref.F32) * A
        ref.check(f(), want.expand(1, T, H, D).cpu(), bound.expand(1, T, H, D).cpu(), scale)
    nvfp4.device_status()
