// attention_join.cu — the last step of attention over a key range that was split among CTAs.
//
// Few bytes and a chain of loads: bound by latency, so eight parts' statistics and sums are asked for together,
// before it is known which count.  (8 parts of 400 rows of 256: 5.8 us behind the tile kernel with the sums
// loaded after the statistics, 3 so; 18 parts of 64 rows of 256: 2 us less.)
#include <cuda_runtime.h>

#include "attention.h"
#include "attention_share.cuh"
#include "gemm.h"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 128;  // also the rows of a tile

// With M the largest reference of the parts that have a sum,
// out = sum_s 2^(c (m_s - M)) O_s / sum_s 2^(c (m_s - M)) l_s, in the order of s.

// The tile kernel's parts: a thread a row and 8 columns; adjacent rows lie side by side.
__global__ void __launch_bounds__(kThreads) attention_join_tiles_kernel(const AttnArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int rows = p.T * p.G, tiles = p.row_tiles(), pr = p.part_rows(), groups = p.D >> 3;
    const int cg = static_cast<int>(blockIdx.x % groups), id = static_cast<int>(blockIdx.x / groups);
    const int tile = id % tiles, bh = id / tiles, hk = bh % p.Hkv, b = bh / p.Hkv;
    const int r = static_cast<int>(threadIdx.x), row = tile * 128 + r;
    if (row >= rows) return;
    const float4 *ml = p.part_ml + static_cast<size_t>(id) * p.splits * pr + r;
    const size_t step = static_cast<size_t>(p.D >> 2) * pr;  // from a part to the next, in float4
    const float4 *po = reinterpret_cast<const float4 *>(p.part_o) + id * p.splits * step + 2 * static_cast<size_t>(cg) * pr + r;
    // eight parts at a time, all their loads in flight together
    constexpr int kParts = 8;
    float M = -INFINITY, l = 0.0f, c = 0.0f, o[8] = {};
    for (int s0 = 0; s0 < p.splits; s0 += kParts) {
        float4 x[kParts];
        float4 u[kParts], v[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            const int s = min(s0 + i, p.splits - 1);
            x[i] = __ldcg(ml + static_cast<size_t>(s) * pr);
            u[i] = __ldcg(po + s * step);
            v[i] = __ldcg(po + s * step + pr);
            if (s0 + i >= p.splits) x[i].y = 0.0f;
        }
        const float before = M;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            if (x[i].y != 0.0f) M = fmaxf(M, x[i].x), c = x[i].z;
        const float g = before == -INFINITY ? 0.0f : exp2f((before - M) * c);
        l *= g;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] *= g;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
            if (x[i].y != 0.0f) {  // a part without keys may hold anything
                const float f = exp2f((x[i].x - M) * c);
                l = fmaf(f, x[i].y, l);
                const float y[8] = {u[i].x, u[i].y, u[i].z, u[i].w, v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = fmaf(f, y[k], o[k]);
            }
    }
    const float f = l != 0.0f ? (p.cached ? p.cache.v.g : 1.0f) / l : 0.0f;
    const int t = row / p.G, h = hk * p.G + row - t * p.G;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2_rn(o[2 * i] * f, o[2 * i + 1] * f);
    *reinterpret_cast<uint4 *>(p.out.ptr + b * p.out.sb + t * p.out.st + h * p.out.sh + 8 * cg) =
        make_uint4(w[0], w[1], w[2], w[3]);
}

// The row kernel's pieces: a warp a row.
// The factors are found 32 parts at a time, a part a lane; the sums' loads do not wait for one another.
__global__ void __launch_bounds__(kThreads) attention_join_kernel(const AttnArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.B) * p.T * p.Hq) return;
    const int rows = p.T * p.G;
    const int r = static_cast<int>(row % rows), bh = static_cast<int>(row / rows);
    const int hk = bh % p.Hkv, b = bh / p.Hkv, t = r / p.G, h = hk * p.G + r % p.G;
    // the row's parts: first index, number, and the step to the next
    int len;
    const int steps = key_steps(p, b, &len), piece = key_piece(p), parts = (steps + piece - 1) / piece;
    const size_t first = static_cast<size_t>(first_piece(p, b, hk, piece, steps)) * rows + r, step = rows;
    const float4 *ml = p.part_ml + first;
    float M = -INFINITY;
    for (int s = lane; s < parts; s += 32) {
        const float4 x = __ldcg(ml + s * step);
        if (x.y != 0.0f) M = fmaxf(M, x.x);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    const int e0 = 8 * lane;
    const float *po = p.part_o + first * p.D + e0;
    float l = 0.0f, o[8] = {};
    for (int s0 = 0; s0 < parts; s0 += 32) {
        float f = 0.0f;
        if (s0 + lane < parts) {
            const float4 x = __ldcg(ml + (s0 + lane) * step);
            if (x.y != 0.0f) f = exp2f((x.x - M) * x.z);
            l = fmaf(f, x.y, l);
        }
        const int n = min(32, parts - s0);
        for (int s1 = 0; s1 < n; s1 += 8) {
            float4 u[8], v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 *q = reinterpret_cast<const float4 *>(po + (s0 + min(s1 + i, n - 1)) * step * p.D);
                u[i] = v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (e0 < p.D) u[i] = __ldcg(q), v[i] = __ldcg(q + 1);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float fs = s1 + i < n ? __shfl_sync(0xffffffffu, f, s1 + i) : 0.0f;
                if (fs != 0.0f) {  // a part without keys may hold anything
                    const float y[8] = {u[i].x, u[i].y, u[i].z, u[i].w, v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = fmaf(fs, y[k], o[k]);
                }
            }
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
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
    const long long ctas = a.share > 0 ? (rows + kThreads / 32 - 1) / (kThreads / 32)
                                       : static_cast<long long>(a.B) * a.Hkv * a.row_tiles() * (a.D >> 3);
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
    return cudaLaunchKernelEx(&cfg, a.share > 0 ? attention_join_kernel : attention_join_tiles_kernel, a);
}

cudaError_t probe_attention() {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, attention_join_tiles_kernel);
    return e != cudaSuccess ? e : cudaFuncGetAttributes(&fa, attention_join_kernel);
}

}  // namespace nvfp4
