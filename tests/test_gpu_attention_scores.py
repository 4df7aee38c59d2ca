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
