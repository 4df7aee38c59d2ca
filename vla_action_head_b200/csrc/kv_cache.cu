// kv_cache.cu — the NVFP4 key/value cache read back to bf16.
//
//   y = bf16( val(code) dec(sf) g )      (the product of code and scale is exact in fp32)
//
// A lane turns 8 codes (4 bytes) and their block's scale into 16 bytes of bf16, so a warp's
// stores are whole lines; bound by memory (0.5625 bytes read, 2 written per element).
#include <cuda_runtime.h>

#include "attention.h"
#include "gemm.h"
#include "kv_decode.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int units = p.D >> 3;
    const long long per = static_cast<long long>(p.B) * p.L * p.H * units;
    const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= per) return;
    const bool is_v = blockIdx.y == 1 || p.k_out.ptr == nullptr;
    const Heads out = is_v ? p.v_out : p.k_out;
    const CachePlane c = is_v ? p.cache.v : p.cache.k;
    const int u = static_cast<int>(i % units);
    long long j = i / units;
    const int h = static_cast<int>(j % p.H);
    j /= p.H;
    const int t = static_cast<int>(j % p.L), b = static_cast<int>(j / p.L);
    const long long row = (p.start != nullptr ? static_cast<long long>(__ldg(p.start + b)) : 0ll) + t;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (row >= 0 && row < p.cache.length) {
        const size_t at = (static_cast<size_t>(b) * p.H + h) * p.cache.C + row;
        const uint32_t codes = __ldcg(reinterpret_cast<const uint32_t *>(c.codes + at * (p.D >> 1)) + u);
        const float s = e4m3_to_f32(__ldcg(c.sf + at * (p.D >> 4) + (u >> 1)));
        float y[8];
        decode_e2m1x8(codes, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * s * c.g;
        w = make_uint4(pack_bf16x2_rn(y[0], y[1]), pack_bf16x2_rn(y[2], y[3]), pack_bf16x2_rn(y[4], y[5]),
                       pack_bf16x2_rn(y[6], y[7]));
    } else if (u == 0) {
        atomicCAS(p.status, static_cast<uint32_t>(kStatusOk), static_cast<uint32_t>(kStatusBadIndex));
    }
    *reinterpret_cast<uint4 *>(out.ptr + b * out.sb + t * out.st + h * out.sh + 8 * u) = w;
}

}  // namespace

cudaError_t launch_kv_read(const ReadArgs &a, cudaStream_t s) {
    const long long per = static_cast<long long>(a.B) * a.L * a.H * (a.D >> 3);
    const long long ctas = (per + kThreads - 1) / kThreads;
    if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), a.k_out.ptr != nullptr && a.v_out.ptr != nullptr ? 2 : 1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kv_read_kernel, a);
}

}  // namespace nvfp4
