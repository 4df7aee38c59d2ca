// kv_cache.cu — the NVFP4 key/value cache read back to bf16.
//
//   y = bf16( val(code) dec(sf) g )      (the product of code and scale is exact in fp32)
//
// A lane turns 8 codes (4 bytes) and their block's scale into 16 bytes of bf16, so a warp's
// stores are whole lines, and does so for four rows, loads first.  Bound by memory (0.5625 bytes
// read, 2 written per element) once a piece's index costs no divisions: 8 x 16384 rows of 256,
// keys and values (172 MB), 65 us with 64-bit divisions, 43 with multiplications, 35 with the rows
// of a lane a fixed step apart (75 % of the rate that a copy reaches).
#include <cuda_runtime.h>

#include "attention.h"
#include "gemm.h"
#include "kv_decode.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;  // rows a lane

__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const bool is_v = blockIdx.y == 1 || p.k_out.ptr == nullptr;
    const Heads out = is_v ? p.v_out : p.k_out;
    const CachePlane c = is_v ? p.cache.v : p.cache.k;
    // a CTA: kSteps x `rows` rows of one sequence's head; a lane: the same 8 elements of every rows-th
    const uint32_t plane = p.by_chunks.div(blockIdx.x);
    const int chunk = static_cast<int>(blockIdx.x - plane * p.by_chunks.d);
    const int b = static_cast<int>(p.by_h.div(plane)), h = static_cast<int>(plane - b * p.by_h.d);
    const int units = p.D >> 3, rows = kThreads / units;
    const int r = static_cast<int>(threadIdx.x) / units, u = static_cast<int>(threadIdx.x) - r * units;
    if (r >= rows) return;
    const long long row0 = p.start != nullptr ? __ldg(p.start + b) : 0;
    const int t0 = chunk * kSteps * rows + r;
    const size_t at = static_cast<size_t>(plane) * p.cache.C;
    uint32_t codes[kSteps], scale[kSteps];
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
        const int t = t0 + q * rows;
        const long long row = row0 + t;
        codes[q] = scale[q] = 0u;
        if (t < p.L) {
            if (row >= 0 && row < p.cache.length) {
                codes[q] = __ldcg(reinterpret_cast<const uint32_t *>(c.codes + (at + row) * (p.D >> 1)) + u);
                scale[q] = __ldcg(c.sf + (at + row) * (p.D >> 4) + (u >> 1));
            } else if (u == 0) {
                atomicCAS(p.status, static_cast<uint32_t>(kStatusOk), static_cast<uint32_t>(kStatusBadIndex));
            }
        }
    }
    uint16_t *to = out.ptr + b * out.sb + h * out.sh + t0 * out.st + 8 * u;
#pragma unroll
    for (int q = 0; q < kSteps; ++q, to += rows * out.st)
        if (t0 + q * rows < p.L) {
            uint32_t w[4];
            decode_e2m1x8_f16(codes[q], w);
            const uint32_t s = scale_f16x2(scale[q]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // code times scale is exact in fp16
                const uint32_t y = mul_f16x2(w[e], s);
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y));
                w[e] = pack_bf16x2_rn(f.x * c.g, f.y * c.g);
            }
            *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        }
}

}  // namespace

int kv_read_rows(int D) { return kSteps * (kThreads / (D >> 3)); }

cudaError_t launch_kv_read(const ReadArgs &args, cudaStream_t s) {
    ReadArgs a = args;
    const int per = kv_read_rows(a.D);
    const uint32_t chunks = static_cast<uint32_t>((a.L + static_cast<long long>(per) - 1) / per);
    a.by_chunks = FastDiv(chunks);
    a.by_h = FastDiv(a.H);
    const unsigned long long ctas = static_cast<unsigned long long>(chunks) * a.B * a.H;
    if (ctas > 0x7FFFFFFFull) return cudaErrorInvalidValue;
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
