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
