// qk_norm_rope.cu — per-head norm and position rotation of queries and keys in one pass, and
// the NVFP4 cache write of keys and values in the same launch.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = (x r) gamma          (per head of D elements)
//   pair (a, b) at angle i:  (a cos_i - b sin_i,  b cos_i + a sin_i)
//   -> bf16, or per 16 elements the block quantizer of quant.cuh -> cache row start[b] + t
//
// One head of one token is held by a group of LPH lanes, 8 elements (16 bytes) a lane, from the
// load to the store: read once, written once.  The sum of squares is fp64 (order-independent
// after its one rounding to fp32, so the quantized keys do not depend on LPH); every later step
// is a single fp32 operation in a fixed order.  A pair's other half sits R / 16 lanes away (or
// in the same lane for adjacent pairs): its packed bf16 words come by shuffle and its norm is
// redone, which costs half the shuffles of exchanging normed fp32 values.
#include <cuda_runtime.h>

#include <atomic>

#include "attention.h"
#include "gemm.h"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16lo(w[j]);
        x[2 * j + 1] = bf16hi(w[j]);
    }
}

// Half a 16-element block per lane; the other half is in lane ^ 1.  The steps of
// quantize_block16.  Returns this lane's four code bytes; *scale is the block's scale byte.
__device__ __forceinline__ uint32_t quantize_half16(const float (&y)[8], float g, uint32_t *scale) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(y[i]));
    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
    const uint32_t s = cvt_e4m3_rn_satfinite(__fdiv_rn(a, __fmul_rn(6.0f, g)));
    const float ds = e4m3_to_f32(s);
    *scale = s;
    if (ds == 0.0f) return 0u;
    const float r = __frcp_rn(__fmul_rn(ds, g));
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(y[i], r);
    return cvt_e2m1x8(v);
}

template <int LPH>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const QkArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int l = threadIdx.x & (LPH - 1);
    const int e0 = 8 * l;
    const int heads = p.Hq + p.Hkv + (p.cached ? p.Hkv : 0);
    const long long item = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / LPH;
    const long long token = item / heads;
    const int h = static_cast<int>(item - token * heads);
    const int b = static_cast<int>(token / p.T), t = static_cast<int>(token - static_cast<long long>(b) * p.T);
    const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
    const int hh = is_q ? h : is_v ? h - p.Hq - p.Hkv : h - p.Hq;

    bool on = b < p.B;
    if (on && p.count != nullptr) on = t < __ldg(p.count + b);
    const long long row = (on && p.start != nullptr ? static_cast<long long>(__ldg(p.start + b)) : 0ll) + t;
    long long pos = row;
    if (on && p.positions != nullptr) pos = __ldg(p.positions + token);
    const bool turns = p.R > 0 && !is_v, stores = p.cached && !is_q;
    if (on && ((turns && (pos < 0 || pos >= p.table_rows)) || (stores && (row < 0 || row >= p.cache.length)))) {
        if (l == 0) atomicCAS(p.status, static_cast<uint32_t>(kStatusOk), static_cast<uint32_t>(kStatusBadIndex));
        on = false;
    }
    on = on && e0 < p.D;

    const Heads in = is_q ? p.q : is_v ? p.v : p.k;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (on) raw = __ldcg(reinterpret_cast<const uint4 *>(in.ptr + b * in.sb + t * in.st + hh * in.sh + e0));
    float n[8];
    unpack8(raw, n);

    // ---- norm ----
    const uint16_t *gamma = is_q ? p.q_gamma : p.k_gamma;
    float r = 1.0f;
    if (p.norm) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = __fma_rn(static_cast<double>(n[i]), static_cast<double>(n[i]), s);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        r = static_cast<float>(1.0 / sqrt(s / p.D + static_cast<double>(p.eps)));
    }
    const bool normed = p.norm && !is_v;
    auto apply_norm = [&](float (&x)[8], int at) {
        if (!normed) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], r);
        if (gamma != nullptr && on) {
            float ga[8];
            unpack8(__ldg(reinterpret_cast<const uint4 *>(gamma + at)), ga);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], ga[i]);
        }
    };
    apply_norm(n, e0);

    // ---- rotation ----
    if (p.R > 0) {
        const float *cs = p.table + (on && turns ? pos : 0) * p.R;
        if (p.inter) {
            if (turns && on && e0 < p.R) {
                const float4 c = __ldg(reinterpret_cast<const float4 *>(cs + e0 / 2));
                const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + p.R / 2 + e0 / 2));
                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = n[2 * i], y = n[2 * i + 1];
                    n[2 * i] = __fsub_rn(__fmul_rn(x, cc[i]), __fmul_rn(y, ss[i]));
                    n[2 * i + 1] = __fadd_rn(__fmul_rn(y, cc[i]), __fmul_rn(x, ss[i]));
                }
            }
        } else {
            const int half = p.R / 2;
            const bool first = e0 < half;
            const int src = (threadIdx.x & 31 & ~(LPH - 1)) | ((first ? l + half / 8 : l - half / 8) & (LPH - 1));
            uint4 o;
            o.x = __shfl_sync(0xffffffffu, raw.x, src);
            o.y = __shfl_sync(0xffffffffu, raw.y, src);
            o.z = __shfl_sync(0xffffffffu, raw.z, src);
            o.w = __shfl_sync(0xffffffffu, raw.w, src);
            if (turns && on && e0 < p.R) {
                float m[8];
                unpack8(o, m);
                apply_norm(m, first ? e0 + half : e0 - half);
                const float *c0 = cs + (first ? e0 : e0 - half);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 c = __ldg(reinterpret_cast<const float4 *>(c0) + j);
                    const float4 s = __ldg(reinterpret_cast<const float4 *>(c0 + half) + j);
                    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float own = __fmul_rn(n[4 * j + i], cc[i]), other = __fmul_rn(m[4 * j + i], ss[i]);
                        n[4 * j + i] = first ? __fsub_rn(own, other) : __fadd_rn(own, other);
                    }
                }
            }
        }
    }

    // ---- store ----
    if (p.cached) {
        const CachePlane c = is_v ? p.cache.v : p.cache.k;
        uint32_t sc;
        const uint32_t codes = quantize_half16(n, c.g, &sc);
        if (stores) {
            if (on) {
                const size_t at = (static_cast<size_t>(b) * p.Hkv + hh) * p.cache.C + row;
                *reinterpret_cast<uint32_t *>(c.codes + at * (p.D >> 1) + 4 * l) = codes;
                if ((l & 1) == 0) c.sf[at * (p.D >> 4) + (l >> 1)] = static_cast<uint8_t>(sc);
            }
            return;
        }
    }
    if (on) {
        const Heads out = is_q ? p.q_out : p.k_out;
        *reinterpret_cast<uint4 *>(out.ptr + b * out.sb + t * out.st + hh * out.sh + e0) =
            make_uint4(pack_bf16x2_rn(n[0], n[1]), pack_bf16x2_rn(n[2], n[3]), pack_bf16x2_rn(n[4], n[5]),
                       pack_bf16x2_rn(n[6], n[7]));
    }
}

template <int LPH>
cudaError_t launch_lph(const QkArgs &a, cudaStream_t s) {
    const long long heads = a.Hq + static_cast<long long>(a.Hkv) * (a.cached ? 2 : 1);
    const long long ctas = (heads * a.B * a.T * LPH + kThreads - 1) / kThreads;
    if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, qk_norm_rope_kernel<LPH>, a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t s) {
    const int lanes = a.D / 8;  // 2 .. 32, D % 16 == 0
    if (lanes <= 2) return launch_lph<2>(a, s);
    if (lanes <= 4) return launch_lph<4>(a, s);
    if (lanes <= 8) return launch_lph<8>(a, s);
    if (lanes <= 16) return launch_lph<16>(a, s);
    return launch_lph<32>(a, s);
}

}  // namespace nvfp4
