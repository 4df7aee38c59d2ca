// qk_norm_rope.cu — per-head norm and position rotation of queries and keys in one pass, and
// the NVFP4 cache write of keys and values in the same launch.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = (x r) gamma          (per head of D elements)
//   pair (a, b) at angle i:  (a cos_i - b sin_i,  b cos_i + a sin_i)
//   -> bf16, or per 16 elements the block quantizer of quant.cuh -> cache row start[b] + t
//
// One head of one token is held by a group of LPH lanes from the load to the store: read once,
// written once.  The sum of squares is fp64 (order-independent after its one rounding to fp32, so
// the quantized keys do not depend on LPH); every later step is a single fp32 operation in a fixed
// order.  Two kernels by how a lane's elements lie:
//   both_halves  elements 8l and D/2 + 8l: the other half of a pair (i, i + D/2) is in the same
//                lane.  Wherever that holds: whole heads (R = D or 0) or adjacent pairs, D % 32 == 0.
//   one_run      8 elements a lane; a pair's other half sits R / 16 lanes away: its packed bf16 words
//                come by shuffle and its norm is redone.  Partial rotations by halves, D % 32 == 16.
// Bound by instructions before memory (66-69 % of the issue slots).  16 x 968 tokens of 24 heads of 128 (190 MB):
// 93 us with 64-bit index divisions and fp64 division and root; 47 us with indexes by multiplication, the root by
// Newton steps and both halves in a lane; 39 us with packed fp32 pairs and four heads a group, which is 74 % of
// the rate that a copy reaches.  The cache write of 16 x 968 tokens of 8 + 1 + 1 heads of 256 and its read back:
// 102, 56, 46 us; the write alone 41.  one_run, 64 of 128 elements turned by halves, 24 heads: 91 us, with a head's
// 16 bytes a lane on their way and gamma and the angles fetched for every head.
#include <cuda_runtime.h>

#include <atomic>

#include "attention.h"
#include "gemm.h"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // of a group, where there is work for all SMs

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

// A group's heads of a token: up to U of q, of k or of v.  Tokens before heads, so that the groups of a warp
// do alike.
struct Item {
    int b, t, h0, n;  // n heads from h0; 0: no work
    bool is_q, is_v, turns, stores;
    long long row;  // cache row
    uint32_t pos;   // table row
};
template <int U>
__device__ __forceinline__ Item item_of(const QkArgs &p, uint32_t item, bool first_lane) {
    Item x;
    const bool any = item < p.items;
    if (!any) item = 0;
    int c = static_cast<int>(p.by_tokens.div(item));
    const uint32_t token = item - static_cast<uint32_t>(c) * p.by_tokens.d;
    x.b = static_cast<int>(p.by_t.div(token));
    x.t = static_cast<int>(token - static_cast<uint32_t>(x.b) * p.by_t.d);
    const int nq = (p.Hq + U - 1) / U, nk = (p.Hkv + U - 1) / U;
    x.is_q = c < nq;
    x.is_v = c >= nq + nk;
    if (!x.is_q) c -= x.is_v ? nq + nk : nq;
    x.h0 = c * U;
    x.n = any ? min(U, (x.is_q ? p.Hq : p.Hkv) - x.h0) : 0;
    if (p.count != nullptr && x.t >= __ldg(p.count + x.b)) x.n = 0;
    x.row = (p.start != nullptr ? static_cast<long long>(__ldg(p.start + x.b)) : 0ll) + x.t;
    const long long pos = p.positions != nullptr ? static_cast<long long>(__ldg(p.positions + token)) : x.row;
    x.turns = p.R > 0 && !x.is_v;
    x.stores = p.cached && !x.is_q;
    // a token's q, k and v are all left alone if its table row or its cache row does not exist
    if (x.n > 0 && ((p.R > 0 && (pos < 0 || pos >= p.table_rows)) ||
                    (p.cached && (x.row < 0 || x.row >= p.cache.length)))) {
        if (first_lane) atomicCAS(p.status, static_cast<uint32_t>(kStatusOk), static_cast<uint32_t>(kStatusBadIndex));
        x.n = 0;
    }
    x.pos = x.n > 0 && x.turns ? static_cast<uint32_t>(pos) : 0u;
    return x;
}

// 1 / sqrt(m) in fp64, rounded to fp32: two Newton steps from the fp32 estimate where fp32 holds m.
__device__ __forceinline__ float rsqrt_f64(double m) {
    if (!(m > 1e-30 && m < 1e30)) return static_cast<float>(1.0 / sqrt(m));
    double y = static_cast<double>(rsqrtf(static_cast<float>(m)));
    const double h = -0.5 * m;
#pragma unroll
    for (int i = 0; i < 2; ++i) y = y * __fma_rn(h * y, y, 1.5);
    return static_cast<float>(y);
}
__device__ __forceinline__ double squares(const float (&x)[8]) {
    double s[2] = {};  // two chains
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i & 1] = __fma_rn(static_cast<double>(x[i]), static_cast<double>(x[i]), s[i & 1]);
    return s[0] + s[1];
}
// The quantized half block of lane l into its cache row.
__device__ __forceinline__ void store_half16(const CachePlane &c, size_t at, int D, int e, uint32_t codes,
                                             uint32_t scale) {
    *reinterpret_cast<uint32_t *>(c.codes + at * (D >> 1) + (e >> 1)) = codes;
    if ((e & 8) == 0) c.sf[at * (D >> 4) + (e >> 4)] = static_cast<uint8_t>(scale);
}
__device__ __forceinline__ uint4 pack8(const float (&n)[8]) {
    return make_uint4(pack_bf16x2_rn(n[0], n[1]), pack_bf16x2_rn(n[2], n[3]), pack_bf16x2_rn(n[4], n[5]),
                      pack_bf16x2_rn(n[6], n[7]));
}
// (x r) gamma; without a gamma its words are ones, and a product with 1 changes no bit.
__device__ __forceinline__ void scale8(float (&n)[8], float r, const uint4 &gamma) {
    float ga[8];
    unpack8(gamma, ga);
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = __fmul_rn(__fmul_rn(n[i], r), ga[i]);
}
__device__ __forceinline__ uint4 load_gamma(const uint16_t *gamma, bool on) {
    const uint32_t one = 0x3F803F80u;
    return gamma != nullptr && on ? __ldg(reinterpret_cast<const uint4 *>(gamma)) : make_uint4(one, one, one, one);
}
// Four adjacent pairs by the angles cc and ss.
__device__ __forceinline__ void turn_adjacent(float (&n)[8], const float *cc, const float *ss) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = n[2 * i], y = n[2 * i + 1];
        n[2 * i] = __fsub_rn(__fmul_rn(x, cc[i]), __fmul_rn(y, ss[i]));
        n[2 * i + 1] = __fadd_rn(__fmul_rn(y, cc[i]), __fmul_rn(x, ss[i]));
    }
}

// Sums and differences of pairs are fma2(a, s, b) with s = 1 or -1, which is one rounding.  s comes with the launch: a packed product and
// a sum (or one that is seen to be a sum) are compiled into one operation, and with one rounding fewer some
// results fall on the other side of a bf16 border.
struct Eight {
    uint64_t x[4];
};
__device__ __forceinline__ Eight pairs_of(const uint4 &u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    Eight e;
#pragma unroll
    for (int j = 0; j < 4; ++j) e.x[j] = pair(bf16lo(w[j]), bf16hi(w[j]));
    return e;
}
__device__ __forceinline__ double squares(const Eight &e) {
    double s[2] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = halves(e.x[j]);
        s[0] = __fma_rn(static_cast<double>(v.x), static_cast<double>(v.x), s[0]);
        s[1] = __fma_rn(static_cast<double>(v.y), static_cast<double>(v.y), s[1]);
    }
    return s[0] + s[1];
}
__device__ __forceinline__ void scale8(Eight &n, uint64_t rr, const Eight &gamma) {
#pragma unroll
    for (int j = 0; j < 4; ++j) n.x[j] = mul2(mul2(n.x[j], rr), gamma.x[j]);
}
__device__ __forceinline__ void turn_adjacent(Eight &n, const uint64_t *cc, const uint64_t *ss, float one) {  // 4 angles
    const uint64_t sign = pair(-one, one);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = halves(n.x[i]), c2 = halves(cc[i >> 1]), s2 = halves(ss[i >> 1]);
        const float c = i & 1 ? c2.y : c2.x, s = i & 1 ? s2.y : s2.x;
        n.x[i] = fma2(mul2(pair(v.y, v.x), pair(s, s)), sign, mul2(n.x[i], pair(c, c)));
    }
}
__device__ __forceinline__ uint4 pack8(const Eight &n) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = halves(n.x[j]);
        w[j] = pack_bf16x2_rn(v.x, v.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void unpack8(const Eight &n, float (&y)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = halves(n.x[j]);
        y[2 * j] = v.x;
        y[2 * j + 1] = v.y;
    }
}

template <int LPH, int U, bool CACHED>
__global__ void __launch_bounds__(kThreads, 4) qk_both_halves_kernel(const QkArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int l = threadIdx.x & (LPH - 1);
    const Item x = item_of<U>(p, blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH, l == 0);
    const bool lane_on = 16 * l < p.D && x.n > 0;
    const int half = p.D >> 1, ea = 8 * l, eb = half + 8 * l;
    const Heads in = x.is_q ? p.q : x.is_v ? p.v : p.k;
    const uint16_t *src = in.ptr + x.b * in.sb + x.t * in.st + x.h0 * in.sh + ea;
    uint4 ua, ub;
    auto load = [&](int u) {
        ua = ub = make_uint4(0u, 0u, 0u, 0u);
        if (lane_on && u < x.n) {
            ua = __ldcg(reinterpret_cast<const uint4 *>(src));
            ub = __ldcg(reinterpret_cast<const uint4 *>(src + half));
        }
        src += in.sh;
    };
    load(0);
    // what the heads share: gamma and the angles
    const uint16_t *gamma = x.is_q ? p.q_gamma : p.k_gamma;
    uint4 ga = load_gamma(gamma + ea, gamma != nullptr && lane_on);
    uint4 gb = load_gamma(gamma + eb, gamma != nullptr && lane_on);
    const bool turn_a = x.turns && lane_on && (!p.inter || ea < p.R), turn_b = x.turns && lane_on && p.inter && eb < p.R;
    uint64_t ca[4] = {}, sa[4] = {};  // halves: the 8 angles of a and b; adjacent: a's 4, then b's 4
    {
        const float *cs = p.table + static_cast<size_t>(x.pos) * p.R, *sn = cs + (p.R >> 1);
        const int i0 = p.inter ? ea >> 1 : ea, i1 = p.inter ? eb >> 1 : ea + 4;
        auto four = [&](uint64_t *to, const float *from) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(from));
            to[0] = pair(f.x, f.y);
            to[1] = pair(f.z, f.w);
        };
        if (turn_a) {
            four(ca, cs + i0);
            four(sa, sn + i0);
        }
        if (p.inter ? turn_b : turn_a) {
            four(ca + 2, cs + i1);
            four(sa + 2, sn + i1);
        }
    }
    const Heads out = x.is_q ? p.q_out : p.k_out;
    uint16_t *to = out.ptr + x.b * out.sb + x.t * out.st + x.h0 * out.sh + ea;
#pragma unroll 1
    for (int u = 0; u < U && __any_sync(0xffffffffu, u < x.n); ++u) {
        const bool on = lane_on && u < x.n;
        // (gamma stays packed: kept in fp32 its 16 registers would spill)
        asm volatile("" : "+r"(ga.x), "+r"(ga.y), "+r"(ga.z), "+r"(ga.w), "+r"(gb.x), "+r"(gb.y), "+r"(gb.z), "+r"(gb.w));
        Eight a = pairs_of(ua), b = pairs_of(ub);
        if (u + 1 < U) load(u + 1);  // on its way under this head's work
        if (p.norm) {
            double s = squares(a) + squares(b);
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            const float r = rsqrt_f64(__fma_rn(s, p.inv_d, static_cast<double>(p.eps)));
            if (!x.is_v) {
                scale8(a, pair(r, r), pairs_of(ga));
                scale8(b, pair(r, r), pairs_of(gb));
            }
        }
        if (p.inter) {
            if (turn_a) turn_adjacent(a, ca, sa, p.one);
            if (turn_b) turn_adjacent(b, ca + 2, sa + 2, p.one);
        } else if (turn_a) {  // R = D
            const uint64_t plus = pair(p.one, p.one), minus = pair(-p.one, -p.one);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t y = a.x[i], z = b.x[i];
                a.x[i] = fma2(mul2(z, sa[i]), minus, mul2(y, ca[i]));
                b.x[i] = fma2(mul2(y, sa[i]), plus, mul2(z, ca[i]));
            }
        }
        if (CACHED && __any_sync(0xffffffffu, x.stores)) {
            const CachePlane c = x.is_v ? p.cache.v : p.cache.k;
            uint32_t fa, fb;
            float ya[8], yb[8];
            unpack8(a, ya);
            unpack8(b, yb);
            const uint32_t qa = quantize_half16(ya, c.g, &fa), qb = quantize_half16(yb, c.g, &fb);
            if (x.stores && on) {
                const size_t at = (static_cast<size_t>(x.b) * p.Hkv + x.h0 + u) * p.cache.C + x.row;
                store_half16(c, at, p.D, ea, qa, fa);
                store_half16(c, at, p.D, eb, qb, fb);
            }
        }
        if (!(CACHED && x.stores) && on) {
            *reinterpret_cast<uint4 *>(to) = pack8(a);
            *reinterpret_cast<uint4 *>(to + half) = pack8(b);
        }
        to += out.sh;
    }
}

template <int LPH>
__global__ void __launch_bounds__(kThreads) qk_one_run_kernel(const QkArgs p) {
    pdl_launch_dependents();
    pdl_wait();
    const int l = threadIdx.x & (LPH - 1);
    const int e0 = 8 * l;
    const Item x = item_of<1>(p, blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH, l == 0);
    const bool on = x.n > 0 && e0 < p.D, is_q = x.is_q, is_v = x.is_v, turns = x.turns, stores = x.stores;
    const int b = x.b, t = x.t, hh = x.h0;
    const Heads in = is_q ? p.q : is_v ? p.v : p.k;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (on) raw = __ldcg(reinterpret_cast<const uint4 *>(in.ptr + b * in.sb + t * in.st + hh * in.sh + e0));
    float n[8];
    unpack8(raw, n);

    // ---- norm ----
    const uint16_t *gamma = is_q ? p.q_gamma : p.k_gamma;
    float r = 1.0f;
    if (p.norm) {
        double s = squares(n);
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        r = rsqrt_f64(__fma_rn(s, p.inv_d, static_cast<double>(p.eps)));
    }
    auto apply_norm = [&](float (&y)[8], int at) {
        if (p.norm && !is_v) scale8(y, r, load_gamma(gamma + at, gamma != nullptr && on));
    };
    apply_norm(n, e0);

    // ---- rotation ----
    if (p.R > 0) {
        const float *cs = p.table + static_cast<size_t>(x.pos) * p.R;
        if (p.inter) {
            if (turns && on && e0 < p.R) {
                float cc[4], ss[4];
                *reinterpret_cast<float4 *>(cc) = __ldg(reinterpret_cast<const float4 *>(cs + e0 / 2));
                *reinterpret_cast<float4 *>(ss) = __ldg(reinterpret_cast<const float4 *>(cs + p.R / 2 + e0 / 2));
                turn_adjacent(n, cc, ss);
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
            if (on) store_half16(c, (static_cast<size_t>(b) * p.Hkv + hh) * p.cache.C + x.row, p.D, e0, codes, sc);
            return;
        }
    }
    if (on) {
        const Heads out = is_q ? p.q_out : p.k_out;
        *reinterpret_cast<uint4 *>(out.ptr + b * out.sb + t * out.st + hh * out.sh + e0) = pack8(n);
    }
}

// U heads of a token a group (both_halves), which share the angles and gamma, the next head's loads under this
// head's work; 1 where four would leave SMs without work (below three times the lanes that the SMs hold).  1, 2, 4
// and 8 heads a group for 24 heads of 128 of B x 968 tokens: 4.7, 5.7, 7.9, 9.4 us (B = 1), 11.9, 10.7, 10.0, 14.6
// (3), 27.9, 23.8, 21.6, 24.0 (8), and 47 (1), 44, 39.8, 39.3 (16).
template <int LPH, int U, bool BOTH>
cudaError_t launch_lph(QkArgs a, cudaStream_t s) {
    const uint32_t q = static_cast<uint32_t>((a.Hq + U - 1) / U), k = static_cast<uint32_t>((a.Hkv + U - 1) / U);
    const uint32_t heads = q + k * (a.cached ? 2 : 1);
    a.items = heads * static_cast<uint32_t>(a.B) * static_cast<uint32_t>(a.T);
    a.by_tokens = FastDiv(static_cast<uint32_t>(a.B) * static_cast<uint32_t>(a.T));
    a.by_t = FastDiv(static_cast<uint32_t>(a.T));
    a.inv_d = 1.0 / a.D;
    a.one = 1.0f;
    // groups of a launch: below 2^32 / LPH threads
    const unsigned long long ctas = (static_cast<unsigned long long>(a.items) * LPH + kThreads - 1) / kThreads;
    if (ctas > 0x7FFFFFFFull) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    if constexpr (BOTH)
        return cudaLaunchKernelEx(&cfg, a.cached ? qk_both_halves_kernel<LPH, U, true> : qk_both_halves_kernel<LPH, U, false>, a);
    else
        return cudaLaunchKernelEx(&cfg, qk_one_run_kernel<LPH>, a);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t s) {
    if (a.D % 32 == 0 && (a.inter || a.R == 0 || a.R == a.D)) {
        const int lanes = a.D / 16;  // 2 .. 16
        const double threads = static_cast<double>(a.B) * a.T * (a.Hq + (a.cached ? 2 : 1) * a.Hkv) * lanes;
        const bool many = threads > 3.0 * a.sms * 1024;
#define NVFP4_LANES(N) \
    if (lanes <= N) return many ? launch_lph<N, kHeads, true>(a, s) : launch_lph<N, 1, true>(a, s);
        NVFP4_LANES(2) NVFP4_LANES(4) NVFP4_LANES(8) NVFP4_LANES(16)
#undef NVFP4_LANES
    }
    const int lanes = a.D / 8;  // 2 .. 32
    if (lanes <= 2) return launch_lph<2, 1, false>(a, s);
    if (lanes <= 4) return launch_lph<4, 1, false>(a, s);
    if (lanes <= 8) return launch_lph<8, 1, false>(a, s);
    if (lanes <= 16) return launch_lph<16, 1, false>(a, s);
    return launch_lph<32, 1, false>(a, s);
}

}  // namespace nvfp4
