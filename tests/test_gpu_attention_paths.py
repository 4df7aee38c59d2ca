"""GPU tests of the ways that the attention-side kernels divide their work: second row tiles that are partly
filled, key ranges in parts (joined in a cluster or through the workspace, some of them without keys),
CTAs dealt out by lengths, groups of heads; each against the 64-bit form or, bit for bit, against the
same work done another way, and repeated, as what goes wrong there goes wrong now and then."""
import pytest
import torch

import attention_ref as ref
from test_gpu_attention import cache_values, rand, rand_cache, run_bf16, run_cache
from vla_action_head_b200 import nvfp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _probe():
    nvfp4.probe()


PARTS = [
    # B, T, S, Hq, Hkv, D
    (1, 130, 5000, 1, 1, 128), (2, 255, 1500, 1, 1, 64), (1, 257, 2100, 1, 1, 128), (3, 129, 129, 2, 1, 48),
    (1, 9, 4000, 1, 1, 64), (2, 16, 1030, 2, 2, 256), (1, 41, 301, 32, 32, 48), (1, 64, 900, 1, 1, 64),
    (1, 50, 20000, 8, 1, 256), (4, 33, 3000, 8, 1, 128), (160, 12, 140, 1, 1, 128),
]


@pytest.mark.parametrize("size", PARTS, ids=str)
def test_parts(orc, size):
    run_bf16(*size)
    run_cache(orc, *size)


@pytest.mark.parametrize("T,Hq,Hkv,D", [(130, 1, 1, 128), (9, 1, 1, 64), (16, 2, 2, 256), (50, 8, 1, 256), (41, 4, 4, 48)])
def test_parts_without_keys(orc, T, Hq, Hkv, D):
    """Lengths that end in the first part, at its border, in the last one, or nowhere."""
    S = 2300
    n = torch.tensor([0, 1, 128, 300, 1152, 2299, 2300], dtype=torch.int32)
    m = torch.rand(len(n), S, generator=torch.Generator().manual_seed(8)) > 0.5
    m[3, :256] = False
    m[6, 128:2200] = False
    for B in (1, len(n)):
        for kw in (dict(kv_len=n[-B:]), dict(kv_len=n[-B:], key_mask=m[-B:]), dict(kv_len=n[:B])):
            run_bf16(B, T, S, Hq, Hkv, D, **kw)
            run_cache(orc, B, T, S, Hq, Hkv, D, **kw)


@pytest.mark.parametrize("size", [(8, 300, 700, 4, 2, 128), (2, 9, 3000, 2, 2, 64), (1, 50, 1018, 8, 1, 256),
                                  (6, 200, 1100, 8, 1, 256), (1, 41, 301, 32, 32, 48), (8, 1, 5000, 8, 1, 256)], ids=str)
def test_every_run_is_the_same(size):
    """Runs back to back, with another call's traffic between them."""
    B, T, S, Hq, Hkv, D = size
    q, k, v = rand(B, T, Hq, D).cuda(), rand(B, S, Hkv, D, seed=1).cuda(), rand(B, S, Hkv, D, seed=2).cuda()
    c = rand_cache(B, Hkv, S, D)
    m = (torch.rand(B, S, generator=torch.Generator().manual_seed(1)) > 0.2).cuda()
    calls = [lambda: nvfp4.attention(q, k, v), lambda: nvfp4.attention(q, cache=c),
             lambda: nvfp4.attention(q, k, v, key_mask=m), lambda: nvfp4.attention(q, cache=c, key_mask=m)]
    first = [f() for f in calls]
    side = torch.cuda.Stream()
    for i in range(40):
        with torch.cuda.stream(side):
            calls[i % 4]()
        for f, want in zip(calls, first):
            assert torch.equal(f(), want)
    torch.cuda.synchronize()
    nvfp4.device_status()


@pytest.mark.parametrize("B,Hq,Hkv,D", [(40, 8, 1, 256), (70, 4, 2, 64), (3, 8, 1, 128), (33, 1, 1, 80)])
def test_single_tokens_over_unequal_lengths(orc, B, Hq, Hkv, D):
    """More sequences than a warp has lanes, many of them short or without keys, one long."""
    S = 4100
    g = torch.Generator().manual_seed(B)
    n = torch.randint(0, 200, (B,), generator=g, dtype=torch.int32)
    n[::5] = 0
    n[B // 2] = S
    n[-1] = 17
    run_bf16(B, 1, S, Hq, Hkv, D, kv_len=n)
    run_cache(orc, B, 1, S, Hq, Hkv, D, kv_len=n)
    run_cache(orc, B, 1, S, Hq, Hkv, D, kv_len=torch.zeros(B, dtype=torch.int32))


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 8, 1, 256), (60, 4, 2, 128), (150, 2, 1, 64)])
def test_a_bad_query_stays_in_its_row(T, Hq, Hkv, D):
    """NaN or infinity in one query changes no bit of the others."""
    B, S = 2, 400
    q, k, v = rand(B, T, Hq, D), rand(B, S, Hkv, D, seed=1).cuda(), rand(B, S, Hkv, D, seed=2).cuda()
    c = rand_cache(B, Hkv, S, D)
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[1, T // 2, Hq - 1, 3] = bad
        for f in (lambda x: nvfp4.attention(x, k, v), lambda x: nvfp4.attention(x, cache=c)):
            a, b = f(q.cuda()), f(q2.cuda())
            assert torch.isnan(b[1, T // 2, Hq - 1]).all()
            b[1, T // 2, Hq - 1] = a[1, T // 2, Hq - 1]
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 50])
@pytest.mark.parametrize("power", [-100, -20, 20, 100])
def test_cache_queries_of_any_size(orc, T, power):
    """Queries times 2^n with the scale times 2^-n: the same scores, out of fp16's range."""
    B, S, Hq, Hkv, D = 2, 300, 8, 1, 256
    q, c = rand(B, T, Hq, D), rand_cache(B, Hkv, S, D)
    k, v = cache_values(orc, c)
    scale = ref.default_scale(D)
    want, bound = ref.attention_ref(q.double(), k, v, scale)
    big = (q.double() * 2.0 ** power).bfloat16()
    ref.check(nvfp4.attention(big.cuda(), cache=c, scale=scale * 2.0 ** -power), want, bound)


@pytest.mark.parametrize("pairs", ["half", "inter"])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(9, 3, 128, 128), (8, 1, 256, 256), (4, 4, 64, 32), (5, 6, 96, 96)])
def test_groups_of_heads_change_no_bit(Hq, Hkv, D, R, pairs):
    """Many tokens (groups of several heads, the last ones partly filled) against a few at a time."""
    B, T = 24, 500
    q, k, v = (rand(B, T, h, D, seed=i).cuda() for i, h in enumerate((Hq, Hkv, Hkv)))
    qg, kg = rand(D, seed=5, mean=1.0, std=0.2).cuda(), rand(D, seed=6, mean=1.0, std=0.2).cuda()
    table = nvfp4.rope_table(2 * T, R)
    pos = torch.randint(0, 2 * T, (B, T), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    count = torch.randint(0, T + 1, (B,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    kw = dict(table=table, pairs=pairs)
    a, b = nvfp4.qk_norm_rope(q, k, qg, kg, positions=pos, **kw)
    whole = nvfp4.empty_kv_cache(B, T, Hkv, D, k_scale=0.01, v_scale=0.01)
    some = nvfp4.empty_kv_cache(B, T, Hkv, D, k_scale=0.01, v_scale=0.01)
    qa = torch.full_like(q, 3.0)
    qb = torch.full_like(q, 3.0)
    nvfp4.qk_norm_rope(q, k, qg, kg, positions=pos, v=v, cache=whole, count=count, q_out=qa, **kw)
    for i in range(B):
        s = slice(i, i + 1)
        a1, b1 = nvfp4.qk_norm_rope(q[s, :40], k[s, :40], qg, kg, positions=pos[s, :40].contiguous(), **kw)
        assert torch.equal(a1, a[s, :40]) and torch.equal(b1, b[s, :40])
        one = nvfp4.KVCache(*[t[s] for t in (some.k_codes, some.k_sf, some.v_codes, some.v_sf)], 0.01, 0.01, T)
        nvfp4.qk_norm_rope(q[s], k[s], qg, kg, positions=pos[s].contiguous(), v=v[s], cache=one, count=count[s],
                           q_out=qb[s], **kw)
    assert torch.equal(qa, qb)
    for x, y in ((whole.k_codes, some.k_codes), (whole.k_sf, some.k_sf), (whole.v_codes, some.v_codes), (whole.v_sf, some.v_sf)):
        assert torch.equal(x, y)
    nvfp4.device_status()


@pytest.mark.parametrize("many", [False, True])
def test_norm_of_extreme_rows(many):
    """Zeros, subnormals, the largest values and infinities, with an eps that does not count: the root and
    the products of the formula in 64 and 32 bits, whichever way the heads are grouped."""
    D, eps = 128, 0.0
    rows = [torch.full((D,), x, dtype=torch.float64) for x in (1e-40, 2e-38, 1e-20, 1.0, 1e20, 3e38)]
    rows += [r * torch.linspace(0.5, 1, D, dtype=torch.float64) for r in rows]
    mixed = torch.zeros(D, dtype=torch.float64)
    mixed[5] = 1.0
    x = torch.stack(rows + [mixed]).bfloat16()
    n = x.shape[0]
    q = x[None, :, None].expand(1, n, 8, D).contiguous()
    if many:
        q = q.repeat(1, 600, 1, 1)
    got, _ = nvfp4.qk_norm_rope(q.cuda(), None, eps=eps)
    x64 = x.double()
    r = (1.0 / (x64.square().mean(-1, keepdim=True) + eps).sqrt()).float()
    want = (x.float() * r).bfloat16()
    got = got.cpu().view(-1, n, 8, D)
    # subnormal inputs and roots that pass fp32 may be taken as zero or infinite: those rows are not compared
    fine = (x.float().abs().amax(-1) > 1.2e-38) & torch.isfinite(r[:, 0]) & (r[:, 0] > 1.2e-38)
    assert int(fine.sum()) >= 9
    for h in range(8):
        assert torch.equal(got[0, fine, h], want[fine])
    assert torch.equal(got[:, fine], got[:1, fine, :1].expand_as(got[:, fine]))
    # a zero row with an eps is zero; an infinity gives 0 in the finite places (x r with r = 0) and NaN in its own
    z = torch.zeros(1, 1, 1, D).bfloat16()
    assert (nvfp4.qk_norm_rope(z.cuda(), None, eps=1e-6)[0] == 0).all()
    z[..., 3] = float("inf")
    z[..., 4] = 1.0
    y = nvfp4.qk_norm_rope(z.cuda(), None, eps=1e-6)[0].cpu()[0, 0, 0]
    assert torch.isnan(y[3]) and (y[4:] == 0).all() and (y[:3] == 0).all()


@pytest.mark.parametrize("T", [1, 50])
def test_scales_at_the_ends_of_fp32(T):
    """Products of scales that fp32 cannot hold, with whole tiles left out before the first key: equal
    weights, as the scores are equal to within what the weights resolve."""
    B, S, Hq, Hkv, D = 2, 400, 8, 1, 256
    m = torch.ones(B, S, dtype=torch.bool)
    m[0, :260] = False
    c = rand_cache(B, Hkv, S, D, k_scale=1e-30)
    q = rand(B, T, Hq, D)
    _, v = nvfp4.kv_read(c)
    v = v.double().cpu()
    for x, scale in ((q, 1e-30), (q * 2.0 ** -100, 1e-15), (torch.zeros_like(q), 3e38)):
        out = nvfp4.attention(x.cuda(), cache=c, key_mask=m.cuda(), scale=scale)
        for b in range(B):
            at = v[b, m[b], 0]
            want, A = at.mean(0), at.abs().mean(0)
            # the sum of 400 equal weights and its division, the output's rounding; kv_read's own
            bound = ref.BF16 * want.abs() + (ref.BF16 + 4 * (S + 64) * ref.F32) * A
            assert ((out[b].double().cpu() - want).abs() <= bound).all()
    k, w = rand(B, S, Hkv, D, seed=1).cuda(), rand(B, S, Hkv, D, seed=2).cuda()
    out = nvfp4.attention(torch.zeros_like(q).cuda(), k, w, key_mask=m.cuda(), scale=3e38)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("T", [1, 4, 70])
@pytest.mark.parametrize("D", [8, 72, 136, 144, 168, 192, 200])
def test_nothing_is_read_behind_a_head(T, D):
    """Head sizes that do not fill the kernels' blocks, after a call that left NaN and infinity on every SM."""
    B, S, H = 2, 46, 8
    bad = [torch.full((16, n, 16, 256), x, dtype=torch.bfloat16, device="cuda") for n, x in ((T, 1.0), (600, float("nan")))]
    q, k, v = rand(B, T, H, D), rand(B, S, H, D, seed=1), rand(B, S, H, D, seed=2)
    want, bound = ref.attention_ref(q.double(), k.double(), v.double(), ref.default_scale(D))
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    for x in (float("nan"), float("inf")):
        bad[1].fill_(x)
        nvfp4.attention(bad[0], bad[1], bad[1])
        ref.check(nvfp4.attention(q, k, v), want, bound, (T, D, x))


@pytest.mark.parametrize("T", [1, 4, 70])
@pytest.mark.parametrize("D", [16, 48, 80, 112, 144, 208, 240])
def test_nothing_is_read_behind_a_cached_head(orc, T, D):
    """The same over a cache."""
    q = torch.full((16, T, 16, 256), 1.0, dtype=torch.bfloat16, device="cuda")
    for x in (float("nan"), float("inf")):
        k = torch.full((16, 600, 16, 256), x, dtype=torch.bfloat16, device="cuda")
        nvfp4.attention(q, k, k)
        run_cache(orc, 2, T, 46, 8, 8, D)


@pytest.mark.parametrize("T", [1, 20, 150])
def test_keys_beyond_32_bits(orc, T):
    """bf16 keys and values whose elements pass 2^32 along the keys, and along the batch together with the queries'
    and the output's; a cache whose planes pass 2^32 bytes, under the tile kernel too."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    S, n, D, Hq = 17000000, 300, 256, 2
    q = rand(2, T, Hq, D)
    k, v = rand(2, n, 1, D, seed=1), rand(2, n, 1, D, seed=2)
    want, bound = ref.attention_ref(q.double(), k.double(), v.double(), ref.default_scale(D))
    mask = torch.zeros(1, S, dtype=torch.bool, device="cuda")
    mask[0, S - n:] = True
    long = [torch.zeros(1, S, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert long[0].numel() > 1 << 32
    for t, x in zip(long, (k, v)):
        t[0, S - n:] = x[1].cuda()
    out = nvfp4.attention(q[1:].cuda(), long[0], long[1], key_mask=mask)
    ref.check(out, want[1:], bound[1:], "keys")
    # two sequences, the second at the far end of the same memory
    far = (S - n) * D
    for t, x in zip(long, (k, v)):
        t[0, :n] = x[0].cuda()
    views = [t.as_strided((2, n, 1, D), (far, D, D, 1)) for t in long]
    queries = torch.zeros(S * D, dtype=torch.bfloat16, device="cuda").as_strided((2, T, Hq, D), (far, Hq * D, D, 1))
    queries.copy_(q)
    ref.check(nvfp4.attention(queries, *views, out=queries), want, bound, "batch")
    del long, views, queries
    c = nvfp4.KVCache(*[torch.zeros((1, 1, 2 * S, D // m), dtype=torch.uint8, device="cuda") for m in (2, 16, 2, 16)])
    assert c.k_codes.numel() > 1 << 32
    small = rand_cache(1, 1, n, D)
    for t, x in zip((c.k_codes, c.k_sf, c.v_codes, c.v_sf), (small.k_codes, small.k_sf, small.v_codes, small.v_sf)):
        t[:, :, 2 * S - n:] = x[:, :, :n]
    mask = torch.zeros(1, 2 * S, dtype=torch.bool, device="cuda")
    mask[0, 2 * S - n:] = True
    want, bound = ref.attention_ref(q[:1].double(), *cache_values(orc, small), ref.default_scale(D))
    ref.check(nvfp4.attention(q[:1].cuda(), cache=c, key_mask=mask), want, bound, "cache")
    nvfp4.device_status()


def test_heads_beyond_32_bits():
    """Norm + rotation in place, and a cache read, over sequences that lie 2^32 elements apart."""
    T, D, far = 40, 128, (1 << 32) + 1024
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    big = torch.zeros(far + T * 6 * D, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, T, 6, D), (far, 6 * D, D, 1))
    x.copy_(rand(2, T, 6, D))
    small, table = x.contiguous(), nvfp4.rope_table(T, D)
    a, b = nvfp4.qk_norm_rope(small[:, :, :4], small[:, :, 4:], table=table)
    c = nvfp4.empty_kv_cache(2, T, 2, D)
    nvfp4.kv_write(c, small[:, :, 4:], small[:, :, 4:])
    d = nvfp4.empty_kv_cache(2, T, 2, D)
    nvfp4.kv_write(d, x[:, :, 4:], x[:, :, 4:])
    assert torch.equal(c.k_codes, d.k_codes) and torch.equal(c.v_sf, d.v_sf)
    nvfp4.qk_norm_rope(x[:, :, :4], x[:, :, 4:], table=table, q_out=x[:, :, :4], k_out=x[:, :, 4:])
    assert torch.equal(x[:, :, :4], a) and torch.equal(x[:, :, 4:], b)
    k, v = nvfp4.kv_read(c)
    nvfp4.kv_read(c, k_out=x[:, :, :2], v_out=x[:, :, 2:4])
    assert torch.equal(x[:, :, :2], k) and torch.equal(x[:, :, 2:4], v)
    nvfp4.device_status()
