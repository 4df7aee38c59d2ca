"""Refusals of the attention-side entry points, on the CPU: the C ABI checks its arguments before
it touches a device, the binding its tensors before it calls the library."""
import ctypes as C
import weakref

import pytest
import torch

from vla_action_head_b200 import build, layers, nvfp4

INVALID, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 4
NO_DEVICE = (5, 6)


@pytest.fixture(scope="module")
def L():
    build.build()
    return nvfp4.lib()


def heads(ptr=0x10000, sb=1 << 20, st=4096, sh=256):
    return nvfp4._Heads(ptr, sb, st, sh)


def cache(**kw):
    d = dict(k_codes=0x1000, k_sf=0x2000, v_codes=0x3000, v_sf=0x4000, k_scale=1.0, v_scale=1.0, B=2, H=1,
             capacity=64, D=256, length=50)
    d.update(kw)
    return nvfp4._KVCache(*[d[f[0]] for f in nvfp4._KVCache._fields_])


def qk(**kw):
    d = dict(B=2, T=4, Hq=8, Hkv=1, D=256, R=256, pairs=0, norm=1, eps=1e-6, q=heads(), k=heads(), v=heads(),
             q_out=heads(), k_out=heads(), table=0x5000, table_rows=100)
    d.update(kw)
    return nvfp4._QkArgs(**d)


def at(**kw):
    d = dict(B=2, T=4, S=50, Hq=8, Hkv=1, D=256, scale=0.1, q=heads(), k=heads(), v=heads(), out=heads())
    d.update(kw)
    return nvfp4._AttentionArgs(**d)


def test_qk_refusals(L):
    f = lambda **kw: L.nvfp4_qk_norm_rope(C.byref(qk(**kw)), None)  # noqa: E731
    assert L.nvfp4_qk_norm_rope(None, None) == INVALID
    for kw in (dict(B=-1), dict(T=-1), dict(Hq=-1), dict(Hkv=-1), dict(D=0), dict(R=-16), dict(R=272), dict(pairs=2),
               dict(norm=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(norm=0, q_gamma=0x1000), dict(table=None), dict(table_rows=0), dict(q=heads(None)),
               dict(k=heads(None)), dict(q_out=heads(None)), dict(k_out=heads(None)), dict(q=heads(sb=-8)),
               dict(q_out=heads(sh=128)), dict(k_out=heads(st=0)), dict(q=heads(sb=1 << 40))):
        assert f(**kw) == INVALID, kw
    for kw in (dict(D=72, R=16), dict(D=272), dict(R=24), dict(B=1 << 20, T=1 << 20)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(q=heads(0x10008)), dict(q=heads(st=4100)), dict(k_gamma=0x1008), dict(table=0x5004),
               dict(positions=0x1002), dict(start=0x1001), dict(count=0x1003)):
        assert f(**kw) == MISALIGNED, kw
    # nothing to do: no pointer is read
    assert f(B=0, q=heads(None), k=heads(None)) == 0 and f(Hq=0, Hkv=0) == 0
    assert f() in NO_DEVICE
    assert f(cached=2) == INVALID
    # with a cache
    g = lambda c, **kw: f(cache=c, cached=1, **kw)  # noqa: E731
    assert g(cache(), v=heads(None)) == INVALID
    assert g(cache(), Hkv=0) == INVALID
    assert g(cache(), k_out=heads(None)) in NO_DEVICE
    for kw in (dict(B=3), dict(H=2), dict(D=128), dict(length=65), dict(length=-1), dict(k_codes=None),
               dict(v_sf=None), dict(capacity=-16), dict(k_scale=0.0), dict(v_scale=float("nan")), dict(k_scale=float("inf"))):
        assert g(cache(**kw)) == INVALID, kw
    assert g(cache(capacity=63)) == SHAPE
    for kw in (dict(k_codes=0x1008), dict(v_sf=0x4001)):
        assert g(cache(**kw)) == MISALIGNED, kw


def test_kv_read_refusals(L):
    f = lambda c=cache(), start=None, n=10, k=heads(), v=heads(): L.nvfp4_kv_read(  # noqa: E731
        C.byref(nvfp4._KvReadArgs(c, start, n, k, v)), None)
    assert L.nvfp4_kv_read(None, None) == INVALID
    assert f(n=-1) == INVALID and f(n=1 << 31) == INVALID and f(cache(length=99)) == INVALID
    assert f(cache(D=264)) == SHAPE and f(cache(capacity=60)) == SHAPE
    assert f(k=heads(0x10002)) == MISALIGNED and f(v=heads(sb=8)) == INVALID and f(start=0x1001) == MISALIGNED
    assert f(n=0) == 0 and f(k=heads(None), v=heads(None)) == 0
    assert f(k=heads(None)) in NO_DEVICE


def test_attention_refusals(L):
    f = lambda **kw: L.nvfp4_attention(C.byref(at(**kw)), 0x100000, 1 << 40, None)  # noqa: E731
    assert L.nvfp4_attention(None, None, 0, None) == INVALID
    assert f(cached=2) == INVALID
    for kw in (dict(B=-1), dict(T=-1), dict(S=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=heads(None)),
               dict(k=heads(None)), dict(v=heads(None)), dict(out=heads(None)), dict(k=heads(st=-8)),
               dict(out=heads(sh=8)), dict(key_mask=0x100, mask_stride=-1), dict(key_mask=0x100, mask_stride=49)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(Hq=8, Hkv=3), dict(D=12), dict(D=264), dict(T=1 << 28)):
        assert f(**kw) == SHAPE, kw
    for kw in (dict(q=heads(0x10008)), dict(k=heads(st=260)), dict(out=heads(sb=(1 << 20) + 4)), dict(kv_len=0x1002)):
        assert f(**kw) == MISALIGNED, kw
    assert f(B=0) == 0 and f(T=0) == 0
    assert f() in NO_DEVICE
    g = lambda c, **kw: f(cache=c, cached=1, k=heads(None), v=heads(None), **kw)  # noqa: E731
    assert g(cache()) in NO_DEVICE
    assert g(cache(), S=51) == INVALID
    assert g(cache(H=2)) == INVALID and g(cache(B=1)) == INVALID
    assert g(cache(D=24), D=24) == SHAPE


def test_workspace_query(L):
    """Asked without a device; a call that needs scratch refuses a smaller one."""
    big = at(T=1, S=40000, B=1)
    need = L.nvfp4_attention_workspace_bytes(C.byref(big))
    assert L.nvfp4_attention_workspace_bytes(C.byref(at(T=1, S=1))) == 0
    assert L.nvfp4_attention_workspace_bytes(C.byref(at(D=7))) == 0
    assert need > 0
    assert L.nvfp4_attention(C.byref(big), 0x100000, need - 1, None) == WORKSPACE
    assert L.nvfp4_attention(C.byref(big), None, need, None) == WORKSPACE
    assert L.nvfp4_attention(C.byref(big), 0x100008, need, None) == MISALIGNED
    assert L.nvfp4_attention(C.byref(big), 0x100000, need, None) in NO_DEVICE


def test_binding_refusals():
    b = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16)
    c = nvfp4.empty_kv_cache(2, 10, 2, 64, device="cpu")
    bad = [
        lambda: nvfp4.qk_norm_rope(None, None),
        lambda: nvfp4.qk_norm_rope(b[0], k),
        lambda: nvfp4.qk_norm_rope(b, k[:, :3]),
        lambda: nvfp4.qk_norm_rope(b.float(), k),
        lambda: nvfp4.qk_norm_rope(b, k, pairs="other"),
        lambda: nvfp4.qk_norm_rope(b, k, v=k),
        lambda: nvfp4.qk_norm_rope(b, k, cache=c),
        lambda: nvfp4.qk_norm_rope(b, k, v=k, cache=c, k_out=k),
        lambda: nvfp4.qk_norm_rope(b, k, q_gamma=torch.zeros(64)),
        lambda: nvfp4.qk_norm_rope(b, k, positions=torch.zeros(2, 4, dtype=torch.int64)),
        lambda: nvfp4.qk_norm_rope(b, k, start=torch.zeros(3, dtype=torch.int32)),
        lambda: nvfp4.qk_norm_rope(b[..., ::2], k[..., :32]),
        lambda: nvfp4.attention(b, k),
        lambda: nvfp4.attention(b, k, k, cache=c),
        lambda: nvfp4.attention(b[0], k, k),
        lambda: nvfp4.attention(b, k, k[:, :3]),
        lambda: nvfp4.attention(b, k, k, kv_len=torch.zeros(2, dtype=torch.int64)),
        lambda: nvfp4.attention(b, k, k, key_mask=torch.zeros(2, 5, dtype=torch.bool)),
        lambda: nvfp4.attention(b, k, k, key_mask=torch.zeros(2, 4)),
        lambda: nvfp4.attention(b, k, k, key_mask=torch.zeros(2, 8, dtype=torch.bool)[:, ::2]),
        lambda: nvfp4.attention(b, k, k),  # tensors on the CPU
        lambda: nvfp4.kv_read(nvfp4.KVCache(c.k_codes, c.k_sf[:, :, :5], c.v_codes, c.v_sf)),
        lambda: nvfp4.kv_read(nvfp4.KVCache(c.k_codes.float(), c.k_sf, c.v_codes, c.v_sf)),
        lambda: nvfp4.kv_read(c),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print(i)
    assert c.rows() == 10 and c.k_codes.shape == (2, 2, 16, 32)


def test_rope_table():
    t = nvfp4.rope_table(5, 8, device="cpu")
    assert t.shape == (5, 8) and torch.equal(t[0], torch.tensor([1.0] * 4 + [0.0] * 4))
    assert abs(float(t[3, 1]) - 0.955336489) < 1e-6  # cos(3 / 10)


def test_kv_read_counts_rows_in_31_bits(L):
    """The last CTA's rows, those behind the last one included, must not pass 2^31: their count is signed, and a
    row that came back below 0 would be written in front of the output."""
    def f(D, n):
        c = cache(B=1, D=D)
        h = heads(sb=1 << 38, st=D, sh=D)
        return L.nvfp4_kv_read(C.byref(nvfp4._KvReadArgs(c, None, n, h, heads(None))), None)

    for D in range(16, 257, 16):
        per = 4 * (256 // (D // 8))
        last = 2 ** 31 // per * per
        for n in (2 ** 31 - 1, last, last + 1, last - 1):
            if n < 2 ** 31:
                top = (n + per - 1) // per * per - 1  # the largest row that a lane counts
                assert f(D, n) == SHAPE if top >= 2 ** 31 else f(D, n) in NO_DEVICE, (D, n)


def test_a_workspace_keeps_the_buffers_it_outgrew():
    """A graph that was captured with one holds its address; and many small steps do not pile up."""
    ws = nvfp4.Workspace("cpu")
    assert ws.get(0) == (None, 0)
    first = ws.get(1000)[0]
    at, alive = first.data_ptr(), weakref.ref(first)
    assert ws.get(first.numel())[0] is first
    del first
    total = 0
    for need in range(1 << 20, 12 << 20, 1 << 18):
        buf, n = ws.get(need)
        assert n >= need and not buf.any()
        total = sum(b.numel() for b in [buf] + ws.replaced)
    assert total < 2 * buf.numel() and buf.numel() < 2 * need
    assert alive() is not None and alive().data_ptr() == at and not alive().any()


@pytest.mark.parametrize("kw", [dict(T=1, S=40000, B=1), dict(T=50, S=9000, B=1), dict(T=200, S=3000, B=2, D=128)], ids=str)
def test_parts_lie_behind_the_counters_of_gemms(L, kw):
    """A workspace is 16 KiB of GEMM counters, then whole parts: D sums and four numbers more a row."""
    D = kw.get("D", 256)
    need = L.nvfp4_attention_workspace_bytes(C.byref(at(**kw)))
    assert need > 16384 and (need - 16384) % (4 * (D + 4)) == 0


def test_a_workspace_of_another_device_is_refused(L):
    q, k = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 40000, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="workspace is on meta"):
        nvfp4.attention(q, k, k, workspace=nvfp4.Workspace("meta"))


def test_a_layer_without_context_or_attend_says_so():
    with pytest.raises(ValueError, match="attend"):
        layers._CacheAttention(4, 8, 1, 256, "cpu")(torch.zeros(4, 2560, dtype=torch.bfloat16), None)


def test_the_keys_of_a_layer_end_with_its_own_tokens(monkeypatch):
    """Without a kv_len: not with the cache's last row, which may never have been written."""
    seen = []
    monkeypatch.setattr(nvfp4, "qk_norm_rope", lambda *a, **kw: None)
    monkeypatch.setattr(nvfp4, "attention", lambda q, **kw: seen.append(kw["kv_len"]))
    start = torch.tensor([7], dtype=torch.int32)
    c = nvfp4.empty_kv_cache(1, 60, 1, 256, device="cpu")
    step = layers._CacheAttention(4, 8, 1, 256, "cpu")
    step(torch.zeros(4, 2560, dtype=torch.bfloat16), layers.Attend(c, start, None))
    given = torch.tensor([9], dtype=torch.int32)
    step(torch.zeros(4, 2560, dtype=torch.bfloat16), layers.Attend(c, start, None, given))
    assert seen[0].tolist() == [11] and seen[0].dtype is torch.int32 and seen[1] is given
