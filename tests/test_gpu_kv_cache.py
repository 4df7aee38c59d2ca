"""GPU tests of the per-head norm + rotation and of the NVFP4 cache: bf16 results against fp32
steps evaluated on the CPU, codes and scales bit for bit against the oracle's quantizer."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from vla_action_head_b200 import nvfp4

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _probe():
    nvfp4.probe()
    nvfp4.device_status()


def rand(*shape, seed=0, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).bfloat16()


def dev(t):
    return None if t is None else t.cuda()


def expect(orc, x, gamma, eps, norm, table, pos, R, pairs):
    n = ref.normed(orc, x, gamma, eps) if norm else x.float().numpy()
    return ref.rotated(n, table, pos, R, pairs) if R else n


def as_bf16(y):
    return torch.from_numpy(np.ascontiguousarray(y, np.float32)).bfloat16()


SHAPES = [  # B, T, Hq, Hkv, D, R
    (1, 1, 8, 1, 256, 256), (2, 50, 8, 1, 256, 256), (1, 41, 32, 32, 48, 48), (3, 7, 12, 4, 80, 80),
    (1, 5, 3, 1, 96, 32), (2, 33, 4, 2, 128, 64), (1, 129, 2, 2, 16, 16), (1, 3, 5, 5, 240, 224), (1, 968, 8, 1, 256, 256),
    (4, 2, 16, 8, 128, 128), (1, 9, 1, 1, 32, 0), (2, 3, 6, 3, 208, 16),
]


@pytest.mark.parametrize("pairs", ["half", "inter"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm_and_rotation(orc, shape, pairs):
    """Bit for bit: the fp32 steps are the oracle's norm and single products and sums."""
    B, T, Hq, Hkv, D, R = shape
    q, k = rand(B, T, Hq, D), rand(B, T, Hkv, D, seed=1, std=3.0)
    qg, kg = rand(D, seed=2, std=0.1, mean=1.0), rand(D, seed=3, std=0.1, mean=1.0)
    table = ref.table_np(2000, R) if R else None
    pos = np.random.default_rng(4).integers(0, 2000, (B, T)).astype(np.int32)
    a, b = nvfp4.qk_norm_rope(q.cuda(), k.cuda(), qg.cuda(), kg.cuda(), table=dev(torch.from_numpy(table) if R else None),
                              positions=torch.from_numpy(pos).cuda() if R else None, eps=EPS, pairs=pairs)
    for got, x, g in ((a, q, qg), (b, k, kg)):
        want = as_bf16(expect(orc, x, g, EPS, True, table, pos, R, pairs))
        assert torch.equal(got.cpu(), want)
    nvfp4.device_status()


def test_against_64_bits():
    """The whole formula in 64 bits: half a bf16 step and a few fp32 roundings of each term."""
    B, T, H, D, R = 2, 60, 4, 128, 128
    q = rand(B, T, H, D, std=2.0)
    g = rand(D, seed=2, std=0.1, mean=1.0)
    table = nvfp4.rope_table(40000, R)
    pos = torch.randint(0, 40000, (B, T), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    got, none = nvfp4.qk_norm_rope(q.cuda(), None, g.cuda(), table=table, positions=pos.cuda(), eps=EPS)
    assert none is None
    x = q.double()
    n = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * g.double()
    f = 10000.0 ** (-torch.arange(0, R, 2).double() / R)
    ang = pos.double()[..., None, None] * f
    a, b = n[..., :64], n[..., 64:]
    want = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    terms = torch.cat([a.abs() + b.abs()] * 2, -1)
    # the norm: 3 roundings (statistic, two products); the turn: table, product, sum
    ref.check(got, want, ref.BF16 * want.abs() + 8 * ref.F32 * terms)


def test_variants(orc):
    """No gamma, no norm, no rotation, q or k alone, in place, slices of a QKV output, positions
    from start, fewer tokens than rows, zero rows and rows of extreme values."""
    B, T, Hq, Hkv, D = 2, 11, 4, 2, 64
    qkv = rand(B, T, Hq + 2 * Hkv, D)
    qkv[0, 3] = 0
    qkv[1, 2] = 1e4
    qkv[1, 3] = 1e-4
    table = ref.table_np(100, D)
    tab = torch.from_numpy(table).cuda()
    start = np.array([5, 60], np.int32)
    pos = start[:, None] + np.arange(T)[None]
    g = rand(D, seed=2, std=0.1, mean=1.0)
    for norm, gamma, R in ((True, None, D), (False, None, D), (True, g, 0), (False, None, 0)):
        x = qkv.cuda()
        q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
        kw = dict(norm=norm, table=tab if R else None, start=torch.from_numpy(start).cuda(), eps=EPS)
        a, b = nvfp4.qk_norm_rope(q, k, dev(gamma), dev(gamma), **kw)
        wq = as_bf16(expect(orc, qkv[:, :, :Hq], gamma, EPS, norm, table, pos, R, "half"))
        wk = as_bf16(expect(orc, qkv[:, :, Hq:Hq + Hkv], gamma, EPS, norm, table, pos, R, "half"))
        assert torch.equal(a.cpu(), wq) and torch.equal(b.cpu(), wk)
        a1, _ = nvfp4.qk_norm_rope(q, None, dev(gamma), **kw)
        _, b1 = nvfp4.qk_norm_rope(None, k, None, dev(gamma), **kw)
        assert torch.equal(a1, a) and torch.equal(b1, b)
        # in place, only the first tokens of each sequence
        count = torch.tensor([4, 0], dtype=torch.int32).cuda()
        nvfp4.qk_norm_rope(q, k, dev(gamma), dev(gamma), q_out=q, k_out=k, count=count, **kw)
        want = qkv.clone()
        want[0, :4, :Hq], want[0, :4, Hq:Hq + Hkv] = wq[0, :4], wk[0, :4]
        assert torch.equal(x.cpu(), want)
    nvfp4.device_status()


@pytest.mark.parametrize("scales", [(1.0, 1.0), (0.37, 20.0)])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_cache_write_is_the_oracle_quantizer(orc, shape, scales):
    """Keys (normed, turned, quantized from fp32) and values bit for bit; q as without a cache; the
    rows around the written ones stay; reading back gives the codes' values."""
    B, T, Hq, Hkv, D, R = shape
    q, k, v = rand(B, T, Hq, D), rand(B, T, Hkv, D, seed=1), rand(B, T, Hkv, D, seed=2, std=4.0)
    v[0, 0] = 0
    k[0, 0, 0, :16] = 0
    kg = rand(D, seed=3, std=0.1, mean=1.0)
    table = ref.table_np(T + 40, R) if R else None
    tab = torch.from_numpy(table).cuda() if R else None
    start = np.random.default_rng(5).integers(0, 40, B).astype(np.int32)
    c = nvfp4.empty_kv_cache(B, T + 45, Hkv, D, k_scale=scales[0], v_scale=scales[1])
    for t in (c.k_codes, c.k_sf, c.v_codes, c.v_sf):
        t.fill_(0x55)
    st = torch.from_numpy(start).cuda()
    a, same = nvfp4.qk_norm_rope(q.cuda(), k.cuda(), None, kg.cuda(), table=tab, eps=EPS, v=v.cuda(), cache=c, start=st)
    assert same is c
    pos = start[:, None] + np.arange(T)[None]
    assert torch.equal(a.cpu(), as_bf16(expect(orc, q, None, EPS, True, table, pos, R, "half")))
    for got_c, got_s, y, g in ((c.k_codes, c.k_sf, expect(orc, k, kg, EPS, True, table, pos, R, "half"), scales[0]),
                               (c.v_codes, c.v_sf, v.float().numpy(), scales[1])):
        wc, ws = ref.codes_of(orc, y, g)
        want_c, want_s = (np.full(t.shape, 0x55, np.uint8) for t in (got_c, got_s))
        for b in range(B):
            want_c[b, :, start[b]:start[b] + T] = wc[b].transpose(1, 0, 2)
            want_s[b, :, start[b]:start[b] + T] = ws[b].transpose(1, 0, 2)
        assert np.array_equal(got_c.cpu().numpy(), want_c) and np.array_equal(got_s.cpu().numpy(), want_s)
    kr, vr = nvfp4.kv_read(c, start=st, length=T)
    for got, cc, ss, g in ((kr, c.k_codes, c.k_sf, scales[0]), (vr, c.v_codes, c.v_sf, scales[1])):
        full = ref.values_of(orc, cc.cpu().numpy(), ss.cpu().numpy(), 1.0)
        for b in range(B):
            want = full[b, :, start[b]:start[b] + T].transpose(1, 0, 2).astype(np.float32) * np.float32(g)
            assert torch.equal(got[b].cpu(), as_bf16(want))
    nvfp4.device_status()


def test_plain_write_and_read_views(orc):
    """kv_write without norm or rotation; reads of all rows, of one plane's views, of a length
    that ends inside the cache; counts."""
    B, T, H, D = 2, 30, 3, 48
    k, v = rand(B, T, H, D), rand(B, T, H, D, seed=1)
    c = nvfp4.empty_kv_cache(B, 61, H, D)
    count = torch.tensor([30, 12], dtype=torch.int32).cuda()
    nvfp4.kv_write(c, k.cuda(), v.cuda(), start=torch.tensor([31, 0], dtype=torch.int32).cuda(), count=count)
    kr, vr = nvfp4.kv_read(c)
    assert kr.shape == (B, 61, H, D)
    for got, x in ((kr, k), (vr, v)):
        codes, sf = ref.codes_of(orc, x.float().numpy(), 1.0)
        val = as_bf16(ref.values_of(orc, codes, sf, 1.0))
        assert torch.equal(got[0, 31:].cpu(), val[0]) and (got[0, :31] == 0).all()
        assert torch.equal(got[1, :12].cpu(), val[1, :12]) and (got[1, 12:] == 0).all()
    big = torch.full((B, 70, 2 * H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    nvfp4.kv_read(c, k_out=big[:, 4:65, :H], v_out=big[:, 4:65, H:])
    assert torch.equal(big[:, 4:65, :H], kr) and torch.equal(big[:, 4:65, H:], vr)
    assert (big[:, :4] == 3).all() and (big[:, 65:] == 3).all()
    nvfp4.device_status()


def test_places_that_do_not_exist():
    """A token whose position or row does not exist is left out, the others are done, and the
    device status says so once."""
    B, T, H, D = 2, 6, 2, 32
    x = rand(B, T, H, D).cuda()
    tab = nvfp4.rope_table(10, D)
    pos = torch.tensor([[0, 1, 2, 10, 3, -1]] * 2, dtype=torch.int32).cuda()
    out = torch.full_like(x, 9.0)
    nvfp4.qk_norm_rope(x, None, table=tab, positions=pos, q_out=out)
    with pytest.raises(nvfp4.NVFP4Error) as e:
        nvfp4.device_status()
    assert e.value.status == 1
    nvfp4.device_status()
    ok = [0, 1, 2, 4]
    want, _ = nvfp4.qk_norm_rope(x[:, ok], None, table=tab, positions=pos[:, ok].contiguous())
    assert torch.equal(out[:, ok], want) and (out[:, [3, 5]] == 9).all()
    nvfp4.device_status()
    c = nvfp4.empty_kv_cache(B, 8, H, D)  # capacity 16, rows 8
    nvfp4.kv_write(c, x, x, start=torch.tensor([4, -2], dtype=torch.int32).cuda())
    with pytest.raises(nvfp4.NVFP4Error):
        nvfp4.device_status()
    k, v = nvfp4.kv_read(c)
    full = nvfp4.empty_kv_cache(B, 8, H, D)
    nvfp4.kv_write(full, x, x)
    kf, _ = nvfp4.kv_read(full)
    assert torch.equal(k[0, 4:], kf[0, :4]) and (k[0, :4] == 0).all()
    assert torch.equal(k[1, :4], kf[1, 2:6]) and (k[1, 4:] == 0).all()
    assert (c.k_codes[:, :, 8:] == 0).all() and (c.v_sf[:, :, 8:] == 0).all()
    nvfp4.device_status()
    far = torch.tensor([2 ** 31 - 1, 5], dtype=torch.int32).cuda()
    k, v = nvfp4.kv_read(full, start=far, length=5)
    with pytest.raises(nvfp4.NVFP4Error):
        nvfp4.device_status()
    assert (k[0] == 0).all() and (k[1, 3:] == 0).all() and torch.equal(k[1, :3], kf[1, 5:8])


def test_quantizer_extremes(orc):
    """Ties, signed zeros, saturated and subnormal scales go through the cache as through the
    oracle."""
    rng = np.random.default_rng(0)
    rows = []
    for s in (1e-6, 2.0 ** -12, 0.01, 1.0, 448.0, 3000.0, 1e6):
        rows.append(rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -5.0, -0.0, 0.0], (6, 64)) * s)
    x = as_bf16(np.concatenate(rows)).reshape(1, -1, 1, 64)
    c = nvfp4.empty_kv_cache(1, x.shape[1], 1, 64)
    nvfp4.kv_write(c, x.cuda(), x.cuda())
    codes, sf = ref.codes_of(orc, x.float().numpy(), 1.0)
    n = x.shape[1]
    assert np.array_equal(c.k_codes[0, 0, :n].cpu().numpy(), codes[0, :, 0])
    assert np.array_equal(c.v_sf[0, 0, :n].cpu().numpy(), sf[0, :, 0])


def test_stream_graph_and_no_tokens():
    c = nvfp4.empty_kv_cache(1, 64, 1, 256)
    x = rand(1, 10, 1, 256).cuda()
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    nvfp4.kv_write(c, x, x, start=start)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nvfp4.kv_write(c, x, x, start=start)
        kr, _ = nvfp4.kv_read(c)
    start.fill_(20)
    x.copy_(rand(1, 10, 1, 256, seed=8).cuda())
    g.replay()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c2 = nvfp4.empty_kv_cache(1, 64, 1, 256)
        nvfp4.kv_write(c2, x, x, start=start)
        k2, _ = nvfp4.kv_read(c2)
    st.synchronize()
    assert torch.equal(kr[:, 20:], k2[:, 20:])
    # nothing to do
    e = rand(1, 0, 1, 256).cuda()
    nvfp4.kv_write(c, e, e)
    a, b = nvfp4.qk_norm_rope(rand(0, 4, 2, 64).cuda(), rand(0, 4, 1, 64).cuda())
    assert a.shape == (0, 4, 2, 64) and b.shape == (0, 4, 1, 64)
    assert nvfp4.kv_read(c, length=0)[0].shape == (1, 0, 1, 256)
    nvfp4.device_status()


@pytest.mark.parametrize("R,D,pairs,B", [(32, 32, "half", 2), (16, 48, "half", 2), (128, 128, "inter", 3), (128, 128, "half", 400)])
def test_a_token_that_does_not_exist_keeps_all_its_places(R, D, pairs, B):
    """q, k, v, table and cache in one call: a token whose table row or whose cache row does not exist leaves q_out,
    here q itself, and all four planes as they were; the other tokens are done."""
    T, Hq, H, rows, table_rows = 8, 6, 2, 20, 30
    table = nvfp4.rope_table(table_rows, R)
    start = torch.tensor(([4, 16, -3] * B)[:B], dtype=torch.int32)
    pos = torch.tensor([[0, 29, 30, 5, -1, 6, 7, 2 ** 31 - 1]] * B, dtype=torch.int32)
    row = start[:, None] + torch.arange(T, dtype=torch.int32)
    good = (pos >= 0) & (pos < table_rows) & (row >= 0) & (row < rows)
    q, k, v = (rand(B, T, h, D, seed=i).cuda() for i, h in enumerate((Hq, H, H)))
    c = nvfp4.empty_kv_cache(B, rows, H, D)
    for t in (c.k_codes, c.k_sf, c.v_codes, c.v_sf):
        t.fill_(0x55)
    want_q, _ = nvfp4.qk_norm_rope(q, None, table=table, pairs=pairs, positions=pos.clamp(0, table_rows - 1).cuda())
    want_q = torch.where(good.cuda()[:, :, None, None], want_q, q)
    want_k, _ = nvfp4.qk_norm_rope(k, None, table=table, pairs=pairs, positions=pos.clamp(0, table_rows - 1).cuda())
    nvfp4.device_status()
    nvfp4.qk_norm_rope(q, k, table=table, pairs=pairs, positions=pos.cuda(), v=v, cache=c, start=start.cuda(), q_out=q)
    with pytest.raises(nvfp4.NVFP4Error) as e:
        nvfp4.device_status()
    assert e.value.status == 1
    assert torch.equal(q, want_q)
    written = torch.zeros(B, c.k_codes.shape[2], dtype=torch.bool)
    for b in range(min(B, 3)):
        written[b, row[b, good[b]].long()] = True
    for t in (c.k_codes, c.k_sf, c.v_codes, c.v_sf):
        assert (t[:3].cpu()[~written[:3, None].expand(-1, H, -1)] == 0x55).all()
    # the good tokens' values are there, and their keys within a code's step of the bf16 keys
    kr, vr = nvfp4.kv_read(nvfp4.KVCache(c.k_codes, c.k_sf, c.v_codes, c.v_sf))
    other = nvfp4.empty_kv_cache(B, T, H, D)
    nvfp4.kv_write(other, k, v)
    _, vo = nvfp4.kv_read(other)
    for b in range(min(B, 3)):
        at = good[b].nonzero()[:, 0]
        assert torch.equal(vr[b, row[b, at].long().cuda()], vo[b, at.cuda()])
        top = want_k[b, at.cuda()].abs().amax()
        assert ((kr[b, row[b, at].long().cuda()] - want_k[b, at.cuda()]).abs() <= 0.3 * top).all()
    nvfp4.device_status()
