"""GPU tests of the layers that attend themselves: prompt layer -> cache -> action-expert layer, and
DiT cross attention, each step against its 64-bit form on the inputs the layer gave it, and the whole
layer against itself with the same context supplied by the caller."""
import numpy as np
import pytest
import torch

import attention_ref as ref
from vla_action_head_b200 import layers, nvfp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _probe():
    nvfp4.probe()


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


P, M = 130, 50  # prompt and chunk


@pytest.fixture(scope="module")
def prompt():
    lay = layers.PrefillLayer(M=P, H=512, F=1024)
    att = layers.Attend(nvfp4.empty_kv_cache(1, P + M, 1, 256), torch.zeros(1, dtype=torch.int32, device="cuda"),
                        nvfp4.rope_table(P + M, 256))
    x, y, y0 = rand(P, 512), torch.empty(P, 512, dtype=torch.bfloat16, device="cuda"), None
    lay.forward(x, None, y, attend=att)
    y0 = torch.empty_like(y)
    lay.forward(x, None, y0)
    assert torch.equal(y, y0)  # filling the cache changes nothing else
    return lay, att


def turned(x, start):
    table = ref.table_np(P + M, 256)
    pos = start + np.arange(x.shape[1])[None]
    return ref.rotated(x.float().cpu().numpy(), table, pos, 256, "half")


def test_prompt_fills_the_cache(orc, prompt):
    lay, att = prompt
    qkv = lay.qkv_out.view(1, P, 10, 256).cpu()
    for x, codes, sf in ((turned(qkv[:, :, 8:9], 0), att.cache.k_codes, att.cache.k_sf),
                         (qkv[:, :, 9:].float().numpy(), att.cache.v_codes, att.cache.v_sf)):
        # the layer's table comes from the device's cos and sin: codes may differ next to a border
        c, s = ref.codes_of(orc, x, 1.0)
        same = (codes[0, 0, :P].cpu().numpy() == c[0, :, 0]).mean(), (sf[0, 0, :P].cpu().numpy() == s[0, :, 0]).mean()
        assert same[0] > 0.9995 and same[1] > 0.9995, same
        assert (codes[0, 0, P:P + M].cpu() == 0).all()


def expert_context(lay, att, start):
    """The 64-bit context of the layer's own queries over the cache as it stands."""
    q = torch.from_numpy(turned(lay.qkv_out.view(1, M, 10, 256)[:, :, :8].cpu(), start)).bfloat16()
    k, v = nvfp4.kv_read(att.cache, length=start + M)
    # queries may differ by a bf16 step where the tables differ: a relative 2^-7 of a score's terms is left out
    # by taking the layer's own
    own = lay.attention.q.cpu()
    assert (own.float() - q.float()).abs().max() <= 2.0 ** -7 * q.float().abs().max()
    return ref.attention_ref(own.double(), k.cpu().double(), v.cpu().double(), 1 / 16.0)


@pytest.mark.parametrize("kind", [layers.ActionExpertLayer, layers.GatedActionExpertLayer])
def test_action_expert_attends_to_prompt_and_chunk(prompt, kind):
    _, filled = prompt
    c = filled.cache
    cache = nvfp4.KVCache(c.k_codes.clone(), c.k_sf.clone(), c.v_codes.clone(), c.v_sf.clone(), length=P + M)
    att = layers.Attend(cache, torch.tensor([P], dtype=torch.int32, device="cuda"), filled.table,
                        torch.tensor([P + M], dtype=torch.int32, device="cuda"))
    lay = kind(M=M)
    x, y = rand(M, 1024, seed=3), torch.empty(M, 1024, dtype=torch.bfloat16, device="cuda")

    def run(context, attend):
        if kind is layers.ActionExpertLayer:
            return lay.forward(x, context, y, attend=attend).clone()
        return lay.forward(x.clone(), None, None, context, attend=attend)[0].clone()

    got = run(None, att)
    want, bound = expert_context(lay, att, P)
    ref.check(lay.attention.context, want, bound, kind.__name__)
    # the same context from the caller: the same layer output
    assert torch.equal(got, run(lay.attention.context.view(M, -1).clone(), None))
    # the prompt's rows stayed
    assert torch.equal(cache.k_codes[:, :, :P], c.k_codes[:, :, :P])
    # captured: another chunk into the same rows
    run(None, att)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(None, att)
    x.copy_(rand(M, 1024, seed=5))
    g.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    assert torch.equal(replayed, run(None, att)) and not torch.equal(replayed, got)
    nvfp4.device_status()


def test_dit_attends_to_an_encoder_and_to_itself():
    S = 77
    lay = layers.DiTLayer()
    x = rand(41, 1536)
    y = torch.empty_like(x)
    # the encoder's K and V projections of one grouped launch, as two tensors
    states = nvfp4.quantize_norm(rand(S, 1536, seed=1), "none")
    kv = [torch.empty(S, 1536, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    w = [nvfp4.quantize_weight((rand(1536, 1536, seed=2 + i).float() * 0.03).bfloat16()) for i in range(2)]
    nvfp4.GroupedGemm([(states, wi, o) for wi, o in zip(w, kv)]).run()
    k, v = (t.view(1, S, 32, 48) for t in kv)
    mask = torch.rand(1, S, generator=torch.Generator().manual_seed(4)) > 0.3
    for enc, m in (((k, v), mask), ((k, v), None), (None, None)):
        got = lay.forward(x, None, y, encoder=enc, key_mask=None if m is None else m.cuda()).clone()
        qkv = lay.qkv_out.view(1, 41, 96, 48).cpu().double()
        kk, vv = (t.cpu().double() for t in enc) if enc else (qkv[:, :, 32:64], qkv[:, :, 64:])
        want, bound = ref.attention_ref(qkv[:, :, :32], kk, vv, 48 ** -0.5, None, m)
        ref.check(lay.context, want, bound)
        assert torch.equal(got, lay.forward(x, lay.context.view(41, 1536).clone(), y))


@pytest.mark.parametrize("kind", [layers.ActionExpertLayer, layers.GatedActionExpertLayer])
def test_a_captured_layer_outlives_a_longer_cache(kind):
    """A graph per cache length, captured from one layer: a call over a longer cache in between, and what the
    allocator then gives out, change nothing in the first graph's replay, and its replay writes only where it may."""
    lay = kind(M=M)
    x, y = rand(M, 1024, seed=3), torch.empty(M, 1024, dtype=torch.bfloat16, device="cuda")

    def cache(rows, seed):
        c = nvfp4.empty_kv_cache(1, rows, 1, 256)
        nvfp4.kv_write(c, rand(1, rows, 1, 256, seed=seed), rand(1, rows, 1, 256, seed=seed + 1))
        return layers.Attend(c, torch.tensor([rows - M], dtype=torch.int32, device="cuda"),
                             nvfp4.rope_table(rows, 256), torch.tensor([rows], dtype=torch.int32, device="cuda"))

    def run(attend):
        if kind is layers.ActionExpertLayer:
            return lay.forward(x, None, y, attend=attend)
        return lay.forward(x.clone(), None, None, None, attend=attend)[0]

    def need(rows):
        a = nvfp4._AttentionArgs(B=1, T=M, S=rows, Hq=8, Hkv=1, D=256, scale=0.1, q=nvfp4._Heads(16, 0, 2048, 256),
                                 out=nvfp4._Heads(16, 0, 2048, 256), cached=1,
                                 cache=nvfp4._KVCache(16, 16, 16, 16, 1.0, 1.0, 1, 1, rows, 256, rows))
        return nvfp4.lib().nvfp4_attention_workspace_bytes(nvfp4.C.byref(a))

    # (the case would show nothing if the second call did not need a larger workspace)
    assert need(8000) > 2 * need(1024) > 2 << 20
    short, long = cache(1024, 5), cache(8000, 7)
    want = run(short).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(short)
    run(long)
    torch.cuda.synchronize()
    # whatever was released is given out again
    taken = [torch.full((n,), 7.0, dtype=torch.float32, device="cuda") for n in [1 << 18] * 40 + [1 << 20] * 8 + [need(1024) // 4]]
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(bool((t == 7).all()) for t in taken)
    nvfp4.device_status()


def test_rows_behind_the_chunk_are_not_attended_to(prompt):
    """An Attend without kv_len, over a cache that is longer than prompt and chunk and holds an older prompt's rows."""
    _, filled = prompt
    c = nvfp4.empty_kv_cache(1, P + M + 500, 1, 256)
    old = rand(1, P + M + 500, 1, 256, seed=9)
    nvfp4.kv_write(c, old, old)
    for new, t in zip((c.k_codes, c.k_sf, c.v_codes, c.v_sf),
                      (filled.cache.k_codes, filled.cache.k_sf, filled.cache.v_codes, filled.cache.v_sf)):
        new[:, :, :P] = t[:, :, :P]
    start = torch.tensor([P], dtype=torch.int32, device="cuda")
    table = nvfp4.rope_table(P + M, 256)
    lay = layers.ActionExpertLayer(M=M)
    x, y = rand(M, 1024, seed=3), torch.empty(M, 1024, dtype=torch.bfloat16, device="cuda")
    want = lay.forward(x, None, y, attend=layers.Attend(c, start, table, start + M)).clone()
    got = lay.forward(x, None, y, attend=layers.Attend(c, start, table)).clone()
    assert torch.equal(got, want)
    everything = torch.tensor([P + M + 500], dtype=torch.int32, device="cuda")
    assert not torch.equal(lay.forward(x, None, y, attend=layers.Attend(c, start, table, everything)), want)
    nvfp4.device_status()


def test_prompt_fills_the_cache_to_the_code(orc, prompt):
    """Every code and scale, with the layer's own table."""
    lay, att = prompt
    qkv = lay.qkv_out.view(1, P, 10, 256).cpu()
    k = ref.rotated(qkv[:, :, 8:9].float().numpy(), att.table.cpu().numpy(), np.arange(P)[None], 256, "half")
    for x, codes, sf in ((k, att.cache.k_codes, att.cache.k_sf),
                         (qkv[:, :, 9:].float().numpy(), att.cache.v_codes, att.cache.v_sf)):
        c, s = ref.codes_of(orc, x, 1.0)
        assert np.array_equal(codes[0, 0, :P].cpu().numpy(), c[0, :, 0])
        assert np.array_equal(sf[0, 0, :P].cpu().numpy(), s[0, :, 0])


def test_a_prompt_layer_turns_no_queries(orc, prompt):
    """Filling the cache is all that `attend` asks of it: the same codes, and the place for queries stays."""
    lay, att = prompt
    before = [t.clone() for t in (att.cache.k_codes, att.cache.k_sf, att.cache.v_codes, att.cache.v_sf)]
    c = nvfp4.empty_kv_cache(1, P + M, 1, 256)
    lay.attention.q.fill_(7.0)
    lay.forward(rand(P, 512), None, torch.empty(P, 512, dtype=torch.bfloat16, device="cuda"),
                attend=layers.Attend(c, att.start, att.table))
    assert (lay.attention.q == 7.0).all()
    assert all(torch.equal(a, b) for a, b in zip(before, (c.k_codes, c.k_sf, c.v_codes, c.v_sf)))
