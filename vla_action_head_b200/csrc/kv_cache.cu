// kv_cache.cu — the NVFP4 key/value cache read back to bf16.
//
//   y = bf16( val(code) dec(sf) g )      (the product of code and scale is exact in fp32)
//
// A lane turns 8 codes (4 bytes) and their block's scale into 16 bytes of bf16, so a warp's
// stores are whole lines, four such pieces at a time, loads first.  Bound by memory (0.5625 bytes
// read, 2 written per element) once the indexes cost no 64-bit divisions: 8 x 16384 rows of 256,
// keys and values, 65 -> XX us (172 MB).
#include <cuda_runtime.h>

#include "attention.h"
#include "gemm.h"
#include "kv_decode.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;  // pieces of 8 elements a lane, kThreads apart

__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const bool is_v = blockIdx.y == 1 || p.k_out.ptr == nullptr;
    const Heads out = is_v ? p.v_out : p.k_out;
    const CachePlane c = is_v ? p.cache.v : p.cache.k;
    uint32_t codes[kUnits] = {}, scale[kUnits] = {};
    uint16_t *to[kUnits];
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
        const uint32_t i = (blockIdx.x * kUnits + q) * kThreads + threadIdx.x;
        to[q] = nullptr;
        if (i < p.units) {
            uint32_t j = p.by_units.div(i);
            const int u = static_cast<int>(i - j * p.by_units.d);
            const uint32_t bt = p.by_h.div(j);
            const int h = static_cast<int>(j - bt * p.by_h.d);
            const int b = static_cast<int>(p.by_l.div(bt)), t = static_cast<int>(bt - b * p.by_l.d);
            const long long row = (p.start != nullptr ? static_cast<long long>(__ldg(p.start + b)) : 0ll) + t;
            to[q] = out.ptr + b * out.sb + t * out.st + h * out.sh + 8 * u;
            if (row >= 0 && row < p.cache.length) {
                const size_t at = (static_cast<size_t>(b) * p.H + h) * p.cache.C + row;
                codes[q] = __ldcg(reinterpret_cast<const uint32_t *>(c.codes + at * (p.D >> 1)) + u);
                scale[q] = __ldcg(c.sf + at * (p.D >> 4) + (u >> 1));
            } else if (u == 0) {
                atomicCAS(p.status, static_cast<uint32_t>(kStatusOk), static_cast<uint32_t>(kStatusBadIndex));
            }
        }
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q)
        if (to[q] != nullptr) {
            float y[8];
            decode_e2m1x8(codes[q], y);
            const float s = e4m3_to_f32(scale[q]);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = y[e] * s * c.g;
            *reinterpret_cast<uint4 *>(to[q]) =
                make_uint4(pack_bf16x2_rn(y[0], y[1]), pack_bf16x2_rn(y[2], y[3]), pack_bf16x2_rn(y[4], y[5]),
                           pack_bf16x2_rn(y[6], y[7]));
        }
}

}  // namespace

cudaError_t launch_kv_read(const ReadArgs &args, cudaStream_t s) {
    ReadArgs a = args;
    a.units = static_cast<uint32_t>(a.B) * a.L * a.H * (a.D >> 3);
    a.by_units = FastDiv(a.D >> 3);
    a.by_h = FastDiv(a.H);
    a.by_l = FastDiv(a.L);
    const uint32_t ctas = (a.units + kThreads * kUnits - 1) / (kThreads * kUnits);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, a.k_out.ptr != nullptr && a.v_out.ptr != nullptr ? 2 : 1);
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
