"""Plain forms of the attention-side operators in numpy / 64-bit torch on the CPU, with the error
bounds the GPU results are held to.  Shared by the CPU and the GPU tests."""
import math

import numpy as np
import torch

BF16 = 2.0 ** -8   # half a step relative to the value: finfo(bfloat16).eps / 2
F32 = 2.0 ** -24


def bf16_np(t):
    """bf16 tensor -> its bit patterns."""
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def normed(orc, x, gamma, eps):
    """bf16 [..., D] -> the fp32 normed rows, bit for bit as the oracle's RMSNorm."""
    D = x.shape[-1]
    y = orc.norm_rows(bf16_np(x).reshape(-1, D), "rmsnorm", gamma=None if gamma is None else bf16_np(gamma), eps=eps)
    return np.asarray(y, np.float32).reshape(x.shape)


def rotated(n, table, pos, R, pairs):
    """fp32 [B, T, H, D] turned by table rows pos [B, T]: single fp32 operations in order."""
    y = n.copy()
    if R:
        c, s = table[pos][:, :, None, :R // 2], table[pos][:, :, None, R // 2:]
        i = np.arange(R // 2)
        a, b = (i, i + R // 2) if pairs == "half" else (2 * i, 2 * i + 1)
        y[..., a] = n[..., a] * c - n[..., b] * s
        y[..., b] = n[..., b] * c + n[..., a] * s
    return y


def codes_of(orc, y, g):
    """fp32 [..., D] -> codes [..., D/2], scale bytes [..., D/16] of the oracle's quantizer."""
    D = y.shape[-1]
    rows = int(np.prod(y.shape[:-1]))
    codes, sf = orc.quantize_rows(np.ascontiguousarray(y, np.float32).reshape(rows, D), g)
    r, b = np.arange(rows)[:, None], np.arange(D // 16)[None]
    at = (r // 128 * ((D + 63) // 64) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4  # the atoms' layout
    assert at[-1, -1] == orc.sf_offset(rows - 1, D // 16 - 1, D)
    return codes.reshape(*y.shape[:-1], D // 2), np.asarray(sf, np.uint8)[at].reshape(*y.shape[:-1], D // 16)


def values_of(orc, codes, sf, g):
    """Codes and scale bytes [..., D/2], [..., D/16] -> fp64 values."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    return (np.asarray(orc.e2m1_decode(c), np.float64).reshape(c.shape) *
            np.repeat(np.asarray(orc.e4m3_decode(sf), np.float64).reshape(sf.shape), 16, -1) * g)


def attention_ref(q, k, v, scale, kv_len=None, mask=None):
    """fp64 attention and the bound on each output of the kernels: q [B, T, Hq, D], k, v
    [B, S, Hkv, D] fp64 on the CPU -> (out, bound), both [B, T, Hq, D].

    With p = softmax, A = sum_j p_j |v_j| and x = the largest sum_d |q_d k_jd| * scale of the row:
      - the output's rounding to bf16: 2^-8 |out|;
      - the weights' rounding to bf16 (fp16 is closer): 2^-8 A;
      - scores: a sum of D fp32 products, each sum off by at most 2 half steps of the running
        magnitude (the tensor core may cut instead of round): 2 (D + 4) 2^-24 x absolute, once in
        the weight and once in the sum that divides it; the fp32 scaled difference to the
        reference and its 2^y: 2^-24 (2 x + 8);
      - the S weights' sum and the S products' sum in fp32: 2 (S + 64) 2^-24 A each;
      - weights below fp16's normal range (cache): off by 2^-25 each where the largest is at
        least 1: S 2^-25 max |v|."""
    B, T, Hq, D = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for b in range(B):
        n = S if kv_len is None else max(0, min(S, int(kv_len[b])))
        at = torch.arange(n)
        if mask is not None:
            at = at[mask[b, :n].bool()]
        if len(at) == 0:
            continue
        for h in range(Hq):
            kk, vv = k[b, at, h // (Hq // Hkv)], v[b, at, h // (Hq // Hkv)]
            s = q[b, :, h] @ kk.T * scale
            p = torch.softmax(s, -1)
            o = p @ vv
            A = p @ vv.abs()
            x = (q[b, :, h].abs() @ kk.abs().T * scale).amax(-1, keepdim=True)
            rel = BF16 + 2 * (2 * (D + 4) * F32 * x) + 2 * F32 * (2 * x + 8) + 4 * (len(at) + 64) * F32
            out[b, :, h] = o
            bound[b, :, h] = (BF16 * o.abs() + 1.01 * rel * A + len(at) * 2.0 ** -25 * vv.abs().amax() + 1e-30)
    return out, bound


def check(got, want, bound, what=""):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), (what, "not finite")
    off = (got - want).abs() / bound.clamp(min=1e-300)
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 1.0, (what, worst, int(off.argmax()))
    return worst


def table_np(rows, R, base=10000.0):
    f = float(base) ** (-np.arange(0, R, 2) / R)
    a = np.arange(rows)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def default_scale(D):
    return 1.0 / math.sqrt(D)
