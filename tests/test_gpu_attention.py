"""GPU tests of the attention-side operators against plain 64-bit forms: attention over bf16 keys
and over the NVFP4 cache (lengths from none to long, head groups, masks, strides, streams,
graphs).  Bounds are derived in attention_ref.attention_ref."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from vla_action_head_b200 import nvfp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _probe():
    nvfp4.probe()


def rand(*shape, seed=0, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).bfloat16()


def rand_cache(B, H, rows, D, seed=0, k_scale=1.0, v_scale=1.0, garbage=False):
    """A cache with random codes and scales around 1; garbage: rows behind `rows` hold the bytes
    0x7F and 0xFF (NaN scales)."""
    g = torch.Generator().manual_seed(seed)
    cap = (rows + 15) // 16 * 16
    bufs = []
    for _ in range(2):
        bufs.append(torch.randint(0, 256, (B, H, cap, D // 2), generator=g, dtype=torch.uint8))
        bufs.append(torch.randint(0x18, 0x38, (B, H, cap, D // 16), generator=g, dtype=torch.uint8))
    if garbage:
        for t in bufs:
            t[:, :, rows:] = 0x7F
    return nvfp4.KVCache(*[t.cuda() for t in bufs], k_scale, v_scale, rows)


def cache_values(orc, c):
    """fp64 (k, v), each [B, rows, H, D]."""
    out = []
    for codes, sf, g in ((c.k_codes, c.k_sf, c.k_scale), (c.v_codes, c.v_sf, c.v_scale)):
        x = ref.values_of(orc, codes[:, :, :c.rows()].cpu().numpy(), sf[:, :, :c.rows()].cpu().numpy(), g)
        out.append(torch.from_numpy(x).transpose(1, 2))
    return out


def run_bf16(B, T, S, Hq, Hkv, D, seed=1, std=1.0, **kw):
    q, k, v = rand(B, T, Hq, D, seed=seed, std=std), rand(B, S, Hkv, D, seed=seed + 1), rand(B, S, Hkv, D, seed=seed + 2)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in kw.items()}
    scale = kw.get("scale") or ref.default_scale(D)
    out = nvfp4.attention(q.cuda(), k.cuda(), v.cuda(), **dev)
    want, bound = ref.attention_ref(q.double(), k.double(), v.double(), scale, kw.get("kv_len"), kw.get("key_mask"))
    return ref.check(out, want, bound, (B, T, S, Hq, Hkv, D))


def run_cache(orc, B, T, S, Hq, Hkv, D, seed=1, garbage=True, k_scale=1.0, v_scale=1.0, **kw):
    q = rand(B, T, Hq, D, seed=seed)
    c = rand_cache(B, Hkv, S, D, seed, k_scale, v_scale, garbage)
    k, v = cache_values(orc, c)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in kw.items()}
    scale = kw.get("scale") or ref.default_scale(D)
    out = nvfp4.attention(q.cuda(), cache=c, **dev)
    want, bound = ref.attention_ref(q.double(), k, v, scale, kw.get("kv_len"), kw.get("key_mask"))
    return ref.check(out, want, bound, ("cache", B, T, S, Hq, Hkv, D))


SIZES = [
    # B, T, S, Hq, Hkv, D
    (1, 1, 1, 1, 1, 64), (1, 1, 7, 8, 1, 256), (2, 1, 128, 8, 1, 256), (1, 1, 129, 4, 2, 128),
    (3, 1, 1000, 8, 1, 256), (1, 1, 5003, 8, 1, 256), (2, 2, 300, 8, 2, 128), (1, 3, 65, 6, 2, 96),
    (1, 41, 301, 32, 32, 48), (1, 50, 1018, 8, 1, 256), (2, 17, 127, 12, 4, 80), (1, 128, 128, 1, 1, 64),
    (1, 129, 257, 2, 1, 128), (1, 300, 968, 8, 1, 256), (1, 5, 2500, 3, 1, 256), (2, 100, 640, 4, 4, 64),
    (1, 43, 200, 3, 1, 128), (1, 200, 64, 5, 1, 16), (1, 7, 1111, 24, 1, 128), (1, 1000, 33, 2, 2, 32),
]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_bf16_sizes(size):
    run_bf16(*size)


@pytest.mark.parametrize("D", [8, 24, 40, 72, 104, 136, 200, 248])
def test_bf16_odd_head_sizes(D):
    run_bf16(2, 9, 150, 4, 2, D)
    run_bf16(1, 1, 150, 4, 2, D)


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_cache_sizes(orc, size):
    run_cache(orc, *size)


@pytest.mark.parametrize("D", [16, 48, 112, 144, 208, 240])
def test_cache_head_sizes_and_scales(orc, D):
    run_cache(orc, 2, 9, 150, 4, 2, D, k_scale=0.37, v_scale=5.5)
    run_cache(orc, 1, 1, 150, 4, 2, D, k_scale=3.0, v_scale=0.01)


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 8, 1, 256), (40, 8, 2, 64), (3, 4, 4, 128), (70, 8, 1, 256)])
def test_lengths(orc, T, Hq, Hkv, D):
    """None, one, tile edges, all, and lengths outside [0, S], which are clamped."""
    S = 333
    n = torch.tensor([0, 1, 64, 127, 128, 129, 333, 9999, -5], dtype=torch.int32)
    run_bf16(len(n), T, S, Hq, Hkv, D, kv_len=n)
    run_cache(orc, len(n), T, S, Hq, Hkv, D, kv_len=n)


@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 8, 1, 256), (41, 4, 2, 48), (130, 2, 1, 128), (70, 8, 1, 256)])
def test_masks(orc, dtype, T, Hq, Hkv, D):
    """Random masks, whole tiles left out, everything left out, together with lengths."""
    B, S = 5, 700
    m = torch.rand(B, S, generator=torch.Generator().manual_seed(3)) > 0.3
    m[1, 64:520] = False
    m[2] = False
    m[3] = True
    m[4, :690] = False
    n = torch.tensor([700, 650, 700, 130, 691], dtype=torch.int32)
    for kw in (dict(key_mask=m.to(dtype)), dict(key_mask=m.to(dtype), kv_len=n)):
        run_bf16(B, T, S, Hq, Hkv, D, **kw)
        run_cache(orc, B, T, S, Hq, Hkv, D, **kw)
    # a mask whose sequences are rows of a wider tensor
    wide = torch.zeros(B, S + 37, dtype=dtype)
    wide[:, :S] = m
    q, k, v = rand(B, T, Hq, D), rand(B, S, Hkv, D, seed=1), rand(B, S, Hkv, D, seed=2)
    out = nvfp4.attention(q.cuda(), k.cuda(), v.cuda(), key_mask=wide.cuda()[:, :S])
    want, bound = ref.attention_ref(q.double(), k.double(), v.double(), ref.default_scale(D), None, m)
    ref.check(out, want, bound, "wide mask")


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 8, 1, 256), (1, 2, 2, 64), (41, 4, 2, 48), (150, 2, 1, 128), (70, 8, 1, 256)])
def test_left_out_places_hold_anything(orc, T, Hq, Hkv, D):
    """Infinities, NaN and the type's extremes in left-out keys and values change no bit."""
    B, S = 3, 500
    q, k, v = rand(B, T, Hq, D), rand(B, S, Hkv, D, seed=1), rand(B, S, Hkv, D, seed=2)
    n = torch.tensor([500, 201, 65], dtype=torch.int32)
    m = torch.rand(B, S, generator=torch.Generator().manual_seed(3)) > 0.2
    a = nvfp4.attention(q.cuda(), k.cuda(), v.cuda(), kv_len=n.cuda(), key_mask=m.cuda())
    out_of = ~m | (torch.arange(S)[None] >= n[:, None])
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min):
        k2, v2 = k.clone(), v.clone()
        k2[out_of], v2[out_of] = bad, bad
        b = nvfp4.attention(q.cuda(), k2.cuda(), v2.cuda(), kv_len=n.cuda(), key_mask=m.cuda())
        assert torch.equal(a, b), bad
    # the cache: NaN scales (0x7F) in left-out rows
    c = rand_cache(B, Hkv, S, D)
    a = nvfp4.attention(q.cuda(), cache=c, kv_len=n.cuda(), key_mask=m.cuda())
    at = out_of.cuda()[:, None, :].expand(B, Hkv, S)
    cap = c.k_codes.shape[2]
    full = torch.ones(B, Hkv, cap, dtype=torch.bool, device="cuda")
    full[:, :, :S] = at
    for t in (c.k_codes, c.k_sf, c.v_codes, c.v_sf):
        t[full] = 0x7F
    b = nvfp4.attention(q.cuda(), cache=c, kv_len=n.cuda(), key_mask=m.cuda())
    assert torch.equal(a, b)
    assert torch.isfinite(b).all()


def test_values_reach_the_output_unchanged():
    """A NaN or infinity in a key's value that is attended to reaches its columns."""
    q, k, v = rand(1, 20, 2, 128), rand(1, 300, 2, 128, seed=1), rand(1, 300, 2, 128, seed=2)
    v[0, 200, 1, 5] = float("inf")
    v[0, 100, 0, 7] = float("nan")
    out = nvfp4.attention(q.cuda(), k.cuda(), v.cuda()).float().cpu()
    assert torch.isinf(out[0, :, 1, 5]).all() and torch.isnan(out[0, :, 0, 7]).all()
    out[0, :, 1, 5] = 0
    out[0, :, 0, 7] = 0
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("T", [1, 60])
def test_large_scores_and_growing_maximum(T):
    """Scores that rise along the keys (the running maximum is replaced in every tile), scores of
    hundreds, and a row where one key outweighs all others."""
    B, S, H, D = 1, 900, 2, 128
    q, v = rand(B, T, H, D, std=1.0), rand(B, S, H, D, seed=2)
    base = rand(1, 1, 1, D, seed=5)
    for slope in (0.02, -0.02, 0.3):
        q1 = (base.float() + 0.1 * q.float()).bfloat16()
        k = (base.float() * slope * torch.arange(S)[None, :, None, None] / 8 + 0.1 * rand(B, S, H, D, seed=6).float()).bfloat16()
        out = nvfp4.attention(q1.cuda(), k.cuda(), v.cuda(), scale=0.5)
        want, bound = ref.attention_ref(q1.double(), k.double(), v.double(), 0.5)
        ref.check(out, want, bound, slope)


def test_scale_argument(orc):
    run_bf16(1, 33, 200, 2, 1, 64, scale=1.7)
    run_bf16(1, 1, 200, 2, 1, 64, scale=0.001)
    run_cache(orc, 1, 33, 200, 2, 1, 64, scale=0.3)


def test_views():
    """Slices of a QKV output, head-major storage, a broadcast batch and broadcast heads, and an
    output inside a larger tensor whose other places stay."""
    B, T, S, Hq, Hkv, D = 2, 37, 190, 4, 2, 64
    want = None
    q, k, v = rand(B, T, Hq, D), rand(1, S, 1, D, seed=1), rand(1, S, Hkv, D, seed=2)
    kk, vv = k.expand(B, S, Hkv, D), v.expand(B, S, Hkv, D)
    want, bound = ref.attention_ref(q.double(), kk.double(), vv.double(), ref.default_scale(D))
    ref.check(nvfp4.attention(q.cuda(), k.cuda().expand(B, S, Hkv, D), v.cuda().expand(B, S, Hkv, D)), want, bound)
    ref.check(nvfp4.attention(q[:, :1].cuda(), k.cuda().expand(B, S, Hkv, D), v.cuda().expand(B, S, Hkv, D)),
              want[:, :1], bound[:, :1])
    # head-major q, k, v
    hm = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    ref.check(nvfp4.attention(hm(q.cuda()), hm(kk.contiguous().cuda()), hm(vv.contiguous().cuda())), want, bound)
    # q, k, v side by side in one row; the output in the middle of a larger tensor
    x = torch.zeros(B, S, Hq + 2 * Hkv, D, dtype=torch.bfloat16)
    x[:, :T, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:] = q, kk, vv
    x = x.cuda()
    big = torch.full((B + 1, T + 2, Hq + 3, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[:B, 1:T + 1, 2:2 + Hq]
    nvfp4.attention(x[:, :T, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], out=out)
    ref.check(out, want, bound)
    rest = big.clone()
    rest[:B, 1:T + 1, 2:2 + Hq] = 7.0
    assert (rest == 7.0).all()


def test_out_may_not_be_needed(orc):
    """No sequences, no queries, no keys."""
    for B, T, S in ((0, 5, 9), (2, 0, 9), (2, 5, 0)):
        q, k = rand(B, T, 4, 64).cuda(), rand(B, S, 2, 64).cuda()
        out = nvfp4.attention(q, k, k)
        assert out.shape == (B, T, 4, 64) and (out == 0).all()
    c = nvfp4.empty_kv_cache(2, 0, 2, 64)
    assert (nvfp4.attention(rand(2, 5, 4, 64).cuda(), cache=c) == 0).all()
    # an untouched cache holds zeros
    c = nvfp4.empty_kv_cache(2, 40, 2, 64)
    assert (nvfp4.attention(rand(2, 5, 4, 64).cuda(), cache=c) == 0).all()


def test_two_runs_are_equal():
    """Split keys are joined in a fixed order."""
    q, k, v = rand(2, 50, 8, 256).cuda(), rand(2, 1018, 1, 256, seed=1).cuda(), rand(2, 1018, 1, 256, seed=2).cuda()
    a = nvfp4.attention(q, k, v)
    for _ in range(5):
        assert torch.equal(a, nvfp4.attention(q, k, v))
    c = rand_cache(4, 1, 9000, 256)
    q1 = rand(4, 1, 8, 256).cuda()
    a = nvfp4.attention(q1, cache=c)
    for _ in range(5):
        assert torch.equal(a, nvfp4.attention(q1, cache=c))


@pytest.mark.parametrize("T,S", [(1, 3000), (50, 1018)])
def test_streams_and_graphs(T, S):
    """On a stream of its own; captured and replayed with new inputs; two graphs at a time."""
    q, k, v = rand(1, T, 8, 256).cuda(), rand(1, S, 1, 256, seed=1).cuda(), rand(1, S, 1, 256, seed=2).cuda()
    want = nvfp4.attention(q, k, v)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = nvfp4.attention(q, k, v)
    st.synchronize()
    assert torch.equal(want, got)
    graphs = []
    for i in range(2):
        qi = q.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            oi = nvfp4.attention(qi, k, v)
        graphs.append((g, qi, oi))
    q2 = rand(1, T, 8, 256, seed=9).cuda()
    want2 = nvfp4.attention(q2, k, v)
    graphs[0][1].copy_(q)
    graphs[1][1].copy_(q2)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (g, _, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][2], want) and torch.equal(graphs[1][2], want2)
    nvfp4.device_status()


def test_workspace_is_reused():
    ws = nvfp4.Workspace()
    for T, S, Hq in ((1, 9000, 8), (3, 5000, 2), (50, 3000, 8), (1, 200, 8)):
        q, k, v = rand(1, T, Hq, 256).cuda(), rand(1, S, 1, 256, seed=1).cuda(), rand(1, S, 1, 256, seed=2).cuda()
        assert torch.equal(nvfp4.attention(q, k, v), nvfp4.attention(q, k, v, workspace=ws))


def test_offsets_beyond_32_bits(orc):
    """The last sequence of a cache whose planes pass 2^32 bytes, and keys whose elements do."""
    B, H, S, D = 2, 1, 20000000, 256
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    bufs = [torch.zeros((B, H, S, D // n), dtype=torch.uint8, device="cuda") for n in (2, 16, 2, 16)]
    n = 300
    small = rand_cache(1, H, n, D)
    c = nvfp4.KVCache(*bufs)
    at = S - n
    mask = torch.zeros(B, S, dtype=torch.bool, device="cuda")
    mask[1, at:] = True
    for t, s in zip(bufs, (small.k_codes, small.k_sf, small.v_codes, small.v_sf)):
        t[1, :, at:] = s[0, :, :n]
    q = rand(B, 2, 2, D).cuda()
    out = nvfp4.attention(q, cache=c, key_mask=mask)
    k, v = cache_values(orc, small)
    want, bound = ref.attention_ref(q[1:].double().cpu(), k, v, ref.default_scale(D))
    ref.check(out[1:], want, bound)
    assert (out[0] == 0).all()
    start = torch.tensor([0, at], dtype=torch.int32, device="cuda")
    kr, vr = nvfp4.kv_read(c, start=start, length=n)
    assert torch.equal(kr[1].double().cpu(), k[0]) and torch.equal(vr[1].double().cpu(), v[0])
    assert np.all(kr[0].float().cpu().numpy() == 0)


@pytest.mark.parametrize("T,S,Hq", [(1, 9000, 8), (50, 1018, 8), (50, 6000, 8)])
def test_one_workspace_for_gemms_and_attention(T, S, Hq):
    """GEMMs that reduce through the workspace and attention in parts, in turn on one workspace, eager and in a graph:
    bit for bit what each gives on one of its own."""
    q, k, v = rand(1, T, Hq, 256).cuda(), rand(1, S, 1, 256, seed=1).cuda(), rand(1, S, 1, 256, seed=2).cuda()
    gemms = []
    for M, N, K, splits in ((41, 1536, 6144, -1), (50, 1024, 4096, -1), (968, 2048, 16384, 0)):
        a = nvfp4.quantize_norm(rand(M, K, seed=3).cuda(), "none")
        w = nvfp4.quantize_weight(rand(N, K, seed=4, std=0.02).cuda())
        assert nvfp4.lib().nvfp4_gemm_workspace_bytes_ex(M, N, K, 0, splits) > 16384
        gemms.append(lambda ws, a=a, w=w, splits=splits: nvfp4.gemm(a, w, workspace=ws, splits=splits))
    calls = [f for g in gemms for f in (g, lambda ws: nvfp4.attention(q, k, v, workspace=ws))]
    want = [f(nvfp4.Workspace()) for f in calls]
    ws = nvfp4.Workspace()
    for _ in range(3):
        got = [f(ws) for f in calls]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert not ws.buf[:16384].any()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = [f(ws) for f in calls]
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    nvfp4.device_status()
