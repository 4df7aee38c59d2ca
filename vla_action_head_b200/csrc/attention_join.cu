// attention_join.cu — the last step of attention over a key range that was split among CTAs.
#include <cuda_runtime.h>

#include "attention.h"
#include "gemm.h"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 128;

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

cudaError_t probe_attention() {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, attention_join_kernel);
}

}  // namespace nvfp4
