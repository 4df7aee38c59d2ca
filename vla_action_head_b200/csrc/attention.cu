// attention.cu — attention of queries to keys and values of another length, in bf16 or in the
// NVFP4 cache:  out = sum_j softmax_j(scale q . k_j) v_j  over the keys that kv_len and the mask
// leave.  One pass over the keys with the running maximum and sum.
#include <cuda_runtime.h>

#include "attention.h"
#include "gemm.h"
#include "kv_decode.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 128;

// 8 elements of row j of key head h of sequence b.
template <bool CACHED>
__device__ __forceinline__ void load8(const AttnArgs &p, const Heads &x, const CachePlane &c, int b, int h, int j,
                                      int e0, float (&y)[8]) {
    if constexpr (CACHED) {
        const size_t at = (static_cast<size_t>(b) * p.Hkv + h) * p.cache.C + j;
        decode_e2m1x8(__ldcg(reinterpret_cast<const uint32_t *>(c.codes + at * (p.D >> 1)) + (e0 >> 3)), y);
        const float s = e4m3_to_f32(__ldcg(c.sf + at * (p.D >> 4) + (e0 >> 4)));
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= s;
    } else {
        const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(x.ptr + b * x.sb + j * x.st + h * x.sh + e0));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = bf16lo(w[i]);
            y[2 * i + 1] = bf16hi(w[i]);
        }
    }
}

// A warp per query row, 8 elements a lane.
template <bool CACHED>
__global__ void __launch_bounds__(kThreads) attention_kernel(const AttnArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, e0 = 8 * lane;
    const long long row = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.B) * p.T * p.Hq) return;
    const int h = static_cast<int>(row % p.Hq);
    const long long bt = row / p.Hq;
    const int t = static_cast<int>(bt % p.T), b = static_cast<int>(bt / p.T);
    const int hk = h / p.G;
    const bool on = e0 < p.D;
    float q[8] = {}, o[8] = {}, y[8] = {};
    if (on) load8<false>(p, p.q, p.cache.k, b, h, t, e0, q);
    int n = p.S;
    if (p.kv_len != nullptr) n = min(max(__ldg(p.kv_len + b), 0), p.S);
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < n; ++j) {
        if (p.mask != nullptr && p.mask[b * p.mask_stride + j] == 0) continue;
        float s = 0.0f;
        if (on) {
            load8<CACHED>(p, p.k, p.cache.k, b, hk, j, e0, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(q[i], y[i], s);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s);
        const float f = mn == -INFINITY ? 1.0f : exp2f(m - mn), w = mn == -INFINITY ? 0.0f : exp2f(s - mn);
        m = mn;
        l = l * f + w;
        if (on) {
            load8<CACHED>(p, p.v, p.cache.v, b, hk, j, e0, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = o[i] * f + w * y[i];
        }
    }
    if (!on) return;
    const float f = l != 0.0f ? (CACHED ? p.cache.v.g : 1.0f) / l : 0.0f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2_rn(o[2 * i] * f, o[2 * i + 1] * f);
    *reinterpret_cast<uint4 *>(p.out.ptr + b * p.out.sb + t * p.out.st + h * p.out.sh + e0) =
        make_uint4(w[0], w[1], w[2], w[3]);
}

// Joins the parts of a split key range: with M the largest reference of the parts that have a sum,
// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s (references in units of log2), in the order of s.  A warp a row.
__global__ void __launch_bounds__(kThreads) attention_join_kernel(const AttnArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.B) * p.T * p.Hq) return;
    const int rows = p.T * p.G;
    const int r = static_cast<int>(row % rows), bh = static_cast<int>(row / rows);
    const int hk = bh % p.Hkv, b = bh / p.Hkv, t = r / p.G, h = hk * p.G + r % p.G;
    const float2 *ml = p.part_ml + static_cast<size_t>(row) * p.splits;
    float M = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) {
        const float2 x = __ldcg(ml + s);
        if (x.y != 0.0f) M = fmaxf(M, x.x);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    const int e0 = 8 * lane;
    const float *po = p.part_o + static_cast<size_t>(row) * p.splits * p.D;
    float l = 0.0f, o[8] = {};
    for (int s = 0; s < p.splits; ++s) {
        const float2 x = __ldcg(ml + s);
        if (x.y == 0.0f) continue;
        const float f = exp2f(x.x - M);
        l = fmaf(f, x.y, l);
        if (e0 < p.D) {
            const float4 a = __ldcg(reinterpret_cast<const float4 *>(po + static_cast<size_t>(s) * p.D + e0));
            const float4 c = __ldcg(reinterpret_cast<const float4 *>(po + static_cast<size_t>(s) * p.D + e0 + 4));
            const float y[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(f, y[i], o[i]);
        }
    }
    if (e0 >= p.D) return;
    const float f = l != 0.0f ? (p.cached ? p.cache.v.g : 1.0f) / l : 0.0f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2_rn(o[2 * i] * f, o[2 * i + 1] * f);
    *reinterpret_cast<uint4 *>(p.out.ptr + b * p.out.sb + t * p.out.st + h * p.out.sh + e0) =
        make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace

cudaError_t launch_attention_join(const AttnArgs &a, cudaStream_t s) {
    const long long rows = static_cast<long long>(a.B) * a.T * a.Hq;
    const long long ctas = (rows + kThreads / 32 - 1) / (kThreads / 32);
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
    return cudaLaunchKernelEx(&cfg, attention_join_kernel, a);
}

cudaError_t launch_attention(const AttnArgs &a, cudaStream_t s) {
    const long long rows = static_cast<long long>(a.B) * a.T * a.Hq;
    const long long ctas = (rows + kThreads / 32 - 1) / (kThreads / 32);
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
    return a.cached ? cudaLaunchKernelEx(&cfg, attention_kernel<true>, a)
                    : cudaLaunchKernelEx(&cfg, attention_kernel<false>, a);
}

cudaError_t probe_attention() {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, attention_kernel<false>);
}

}  // namespace nvfp4
