// attention_rows.cu — attention for few query rows per key head (single tokens): up to 8 (query,
// head) pairs share a key head's keys, and the keys are read once, straight into registers.
//
//   S^T = K Q^T,  p = 2^(c S - c m),  l = sum p,  O^T += V^T P^T,  out = O / l,   c = scale log2(e)
//
// The work is the stream of keys and values, so the matrix instruction is the one that takes its
// operands from registers (m16n8k16): 16 keys (or 16 elements of V) are its rows, the 8 query
// rows its columns.  A contraction may take
// its elements in any order as long as both sides do, so every thread takes runs of adjacent
// elements: of a key the quarter of its lane % 4 (k of S^T), of a value row the eighth of its
// lane / 4 (the rows of O^T), which makes 16-byte loads of plain rows.  The weights turn from S^T's
// accumulator into the next operand by one 8 x 8 transposition in registers (movmatrix).
//
// Cache: codes become fp16 (exact: 2-bit significand times 4-bit scale; the weights are then fp16
// too, closer than bf16).  Query rows are scaled by a power of two into fp16's range, which changes no bit of them.
//
// The loads are asynchronous copies, kStages - 1 steps of 16 keys ahead, and each thread copies just
// what it will read itself into a place of its own: no barrier in the loop, conflict-free shared
// memory, and 100 KB and more on their way per SM (loads into registers left one step in flight:
// 71 us instead of XX for 8 sequences of 32701 cached keys, 256-wide heads).
//
// The warps of a CTA take turns at the steps and are joined through shared memory; one CTA takes a
// range of keys, and the ranges of a long sequence are joined by attention_join_kernel.
// The reference m of a row is replaced only when a score outgrows it by 2^8, found by one vote a
// step, so the steps carry no reductions; l stays per thread until the end.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attention.h"
#include "gemm.h"
#include "kv_decode.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kRows = 8;
constexpr float kLazy = 8.0f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool HALF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, bool on) {
    const uint32_t n = on ? BYTES : 0u;  // 0: zeros
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the newest N groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// A run of N adjacent elements of a row (from e0) as it passes through this thread's places of a
// stage: kBytes per lane, the lanes' pieces of a copy side by side.
//   copy: global -> shared, zeros for rows that do not exist and elements past D
//   load: shared -> registers;  keep = 0 makes the run zero whatever its bytes are
//   pairs(i): elements 8i .. 8i + 7 as four 16-bit pairs
template <int N, bool FULL>
struct CodeRun {  // NVFP4; FULL: D fills the kernel's width, so rows are aligned as runs are
    static constexpr int kWords = N / 8, kScales = N >= 16 ? N / 16 : 1;
    static constexpr int kPiece = N / 2 < 8 ? 4 : FULL && N / 2 >= 16 ? 16 : 8, kPieces = N / 2 / kPiece;
    static constexpr int kScaleWords = FULL || kScales == 1 ? 1 : 2;  // a run's bytes may cross a word
    static constexpr int kBytes = N / 2 + 4 * kScaleWords;
    uint32_t w[kWords], s[kScales];

    __device__ __forceinline__ static void copy(uint32_t dst, int lane, const CachePlane &c, size_t row, int e0, int D,
                                                bool on) {
        const uint8_t *codes = c.codes + row * (D >> 1) + (e0 >> 1);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const bool in = on && e0 + 2 * kPiece * i < D;
            copy_async<kPiece>(dst + i * 32 * kPiece + lane * kPiece, in ? codes + i * kPiece : c.codes, in);
        }
        // whole words that hold the scale bytes (the plane's size is a multiple of 16 bytes)
        const size_t at = row * (D >> 4) + (e0 >> 4);
        const int last = static_cast<int>(at & 3) + kScales - 1;
        const bool in = on && e0 < D;
        copy_async<4>(dst + 16 * N + lane * 4, in ? c.sf + (at & ~size_t(3)) : c.sf, in);
        if constexpr (kScaleWords == 2) {
            const bool two = in && last >= 4 && e0 + 16 * (4 - static_cast<int>(at & 3)) < D;
            copy_async<4>(dst + 16 * N + 128 + lane * 4, two ? c.sf + (at & ~size_t(3)) + 4 : c.sf, two);
        }
    }
    __device__ __forceinline__ void load(uint32_t src, int lane, size_t row, int e0, int D, bool keep) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint32_t a = src + i * 32 * kPiece + lane * kPiece;
            if constexpr (kPiece == 16) {
                const uint4 u = lds16(a);
                w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
            } else if constexpr (kPiece == 8) {
                const uint2 u = lds8(a);
                w[2 * i] = u.x, w[2 * i + 1] = u.y;
            } else {
                w[0] = lds4(a);
            }
        }
        const uint32_t off = 8u * static_cast<uint32_t>((FULL ? (e0 >> 4) : static_cast<int>(row * (D >> 4) + (e0 >> 4))) & 3);
        uint32_t x = lds4(src + 16 * N + lane * 4);
        if constexpr (kScaleWords == 2) x = __funnelshift_r(x, lds4(src + 16 * N + 128 + lane * 4), off);
        else x >>= off;
        if (!keep) x = 0u;
#pragma unroll
        for (int i = 0; i < kScales; ++i) s[i] = (FULL || e0 + 16 * i < D) ? (x >> (8 * i)) & 255u : 0u;
    }
    __device__ __forceinline__ void pairs(int i, uint32_t (&h)[4]) const {
        decode_e2m1x8_f16(w[i], h);
        const uint32_t sc = scale_f16x2(s[i / 2]);
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = mul_f16x2(h[q], sc);
    }
};
template <int N>
struct WideRun {  // bf16
    static constexpr int kBytes = 2 * N;
    uint4 u[N / 8];
    __device__ __forceinline__ static void copy(uint32_t dst, int lane, const uint16_t *row, int e0, int D, bool on) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            const bool in = on && e0 + 8 * i < D;
            copy_async<16>(dst + i * 512 + lane * 16, in ? row + e0 + 8 * i : row, in);
        }
    }
    __device__ __forceinline__ void load(uint32_t src, int lane, size_t, int, int, bool keep) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            u[i] = lds16(src + i * 512 + lane * 16);
            if (!keep) u[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __device__ __forceinline__ void load_global(const uint16_t *row, int e0, int D, bool on) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            u[i] = make_uint4(0u, 0u, 0u, 0u);
            if (on && e0 + 8 * i < D) u[i] = __ldcg(reinterpret_cast<const uint4 *>(row + e0) + i);
        }
    }
    __device__ __forceinline__ void pairs(int i, uint32_t (&h)[4]) const {
        h[0] = u[i].x, h[1] = u[i].y, h[2] = u[i].z, h[3] = u[i].w;
    }
};
template <int N, bool FULL, bool CACHED>
struct RunOf {
    using type = CodeRun<N, FULL>;
};
template <int N, bool FULL>
struct RunOf<N, FULL, false> {
    using type = WideRun<N>;
};

template <int DP, bool FULL, bool CACHED>
struct Cfg {
    using KRun = typename RunOf<DP / 4, FULL, CACHED>::type;  // of 2 keys
    using VRun = typename RunOf<DP / 8, FULL, CACHED>::type;  // of 4 keys
    static constexpr int kKBytes = 32 * KRun::kBytes, kVBytes = 32 * VRun::kBytes;
    static constexpr int kStage = 2 * kKBytes + 4 * kVBytes;  // of a warp: 16 KB (bf16) or 5 KB at DP = 256
    static constexpr int kWarps = !CACHED && DP == 256 ? 4 : 8, kThreads = 32 * kWarps;
    static constexpr int kStages = !CACHED && DP >= 128 ? 3 : 4;
    static constexpr int kRing = kWarps * kStages * kStage, kJoin = kWarps * kRows * DP * 4;
    static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
    static_assert(kSmem + 1024 <= 232448, "shared memory");
};

template <int DP, bool FULL, bool CACHED>
__global__ void __launch_bounds__(Cfg<DP, FULL, CACHED>::kThreads, 1) attention_rows_kernel(const AttnArgs p) {
    using C = Cfg<DP, FULL, CACHED>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
    constexpr int kKRun = DP / 4, kVRun = DP / 8;  // adjacent elements of a thread
    constexpr int kTiles = DP / 16;                // k steps of S^T, row tiles of O^T
    extern __shared__ __align__(16) float smem_o[];  // the warps' stages, then [kWarps][kRows][DP]
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int rest = static_cast<int>(blockIdx.x);
    const int split = rest % p.splits;
    rest /= p.splits;
    const int hk = rest % p.Hkv, b = rest / p.Hkv;
    const int rows = p.T * p.G;  // <= kRows
    int len = p.S;
    if (p.kv_len != nullptr) len = min(max(__ldcg(p.kv_len + b), 0), p.S);
    // whole steps of 16 keys to the splits, in turn to the warps
    const int steps = (len + 15) >> 4, per = (steps + p.splits - 1) / p.splits;
    const int step0 = split * per, step1 = min(steps, step0 + per);

    // Q: row g, elements of the quarter t
    uint32_t q[kTiles][2];
    float c = p.scale_log2;
    {
        const bool on = g < rows;
        const int tq = on ? g / p.G : 0, hq = hk * p.G + (on ? g - tq * p.G : 0);
        WideRun<kKRun> r;
        r.load_global(p.q.ptr + b * p.q.sb + tq * p.q.st + hq * p.q.sh, t * kKRun, p.D, on);
        if constexpr (CACHED) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < kKRun / 8; ++i) {
                uint32_t h[4];
                r.pairs(i, h);
#pragma unroll
                for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(bf16lo(h[k])), fabsf(bf16hi(h[k]))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float up = f16_row_factor(top);
#pragma unroll
            for (int i = 0; i < kKRun / 8; ++i) {
                uint32_t h[4];
                r.pairs(i, h);
#pragma unroll
                for (int k = 0; k < 4; ++k) q[2 * i + k / 2][k & 1] = pack_f16x2(bf16lo(h[k]) * up, bf16hi(h[k]) * up);
            }
            // this thread's score columns are rows 2t and 2t + 1: their factors come below
            sm_m[warp][g] = 1.0f / up;  // 4 equal writes
        } else {
#pragma unroll
            for (int i = 0; i < kKRun / 8; ++i) {
                uint32_t h[4];
                r.pairs(i, h);
#pragma unroll
                for (int k = 0; k < 4; ++k) q[2 * i + k / 2][k & 1] = h[k];
            }
        }
    }
    float cr[2] = {c, c};
    if constexpr (CACHED) {
        __syncwarp();
        cr[0] = c * sm_m[warp][2 * t];
        cr[1] = c * sm_m[warp][2 * t + 1];
        __syncwarp();
    }

    const uint8_t *mask = p.mask != nullptr ? p.mask + b * p.mask_stride : nullptr;
    const size_t plane = (static_cast<size_t>(b) * p.Hkv + hk) * p.cache.C;
    const uint16_t *kbase = p.k.ptr + b * p.k.sb + hk * p.k.sh, *vbase = p.v.ptr + b * p.v.sb + hk * p.v.sh;
    const uint32_t ring = smem_u32(smem_o) + warp * C::kStages * C::kStage;
    // a step's keys: g, g + 8 for the scores; 2t, 2t + 1, 2t + 8, 2t + 9 for the values
    auto copy_step = [&](int st, int slot) {
        const uint32_t at = ring + slot * C::kStage;
        if (st < step1) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = 16 * st + g + 8 * i;
                if constexpr (CACHED) C::KRun::copy(at + i * C::kKBytes, lane, p.cache.k, plane + j, t * kKRun, p.D, j < len);
                else C::KRun::copy(at + i * C::kKBytes, lane, j < len ? kbase + j * p.k.st : kbase, t * kKRun, p.D, j < len);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 16 * st + 2 * t + (i & 1) + 8 * (i >> 1);
                const uint32_t to = at + 2 * C::kKBytes + i * C::kVBytes;
                if constexpr (CACHED) C::VRun::copy(to, lane, p.cache.v, plane + j, g * kVRun, p.D, j < len);
                else C::VRun::copy(to, lane, j < len ? vbase + j * p.v.st : vbase, g * kVRun, p.D, j < len);
            }
        }
        copy_commit();
    };
    // lane's key of a step, 1 if it is attended to; asked for one step ahead
    auto key_on = [&](int st) -> uint32_t {
        const int j = 16 * st + (lane & 15);
        if (st >= step1 || j >= len) return 0u;
        return mask == nullptr ? 1u : __ldcg(mask + j) != 0 ? 1u : 0u;
    };

    float o[kTiles][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // rows 2t, 2t + 1; m in units of log2
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) copy_step(step0 + warp + i * kWarps, i);
    uint32_t key = key_on(step0 + warp);
    int slot = 0;
    for (int st = step0 + warp; st < step1; st += kWarps) {
        copy_wait<C::kStages - 2>();
        copy_step(st + (C::kStages - 1) * kWarps, slot == 0 ? C::kStages - 1 : slot - 1);
        const uint32_t keys = __ballot_sync(0xffffffffu, key != 0u);
        key = key_on(st + kWarps);
        const uint32_t at = ring + slot * C::kStage;
        slot = slot + 1 == C::kStages ? 0 : slot + 1;
        const bool ok[2] = {((keys >> g) & 1u) != 0u, ((keys >> (g + 8)) & 1u) != 0u};
        typename C::KRun kr[2];
        typename C::VRun vr[4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            kr[i].load(at + i * C::kKBytes, lane, plane + 16 * st + g + 8 * i, t * kKRun, p.D, true);
        float s[4] = {};
#pragma unroll
        for (int i = 0; i < kKRun / 8; ++i) {
            uint32_t h0[4], h1[4];
            kr[0].pairs(i, h0);
            kr[1].pairs(i, h1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t a[4] = {h0[2 * k], h1[2 * k], h0[2 * k + 1], h1[2 * k + 1]};
                mma16816<CACHED>(s, a, q[2 * i + k][0], q[2 * i + k][1]);
            }
        }
        // scores in units of log2; left-out keys are -inf whatever their bytes gave
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ok[i >> 1] ? s[i] * cr[i & 1] : -INFINITY;
        const float top[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
        const bool grow = (top[0] > m[0] && !(top[0] - m[0] <= kLazy)) || (top[1] > m[1] && !(top[1] - m[1] <= kLazy));
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float n = fmaxf(m[i], top[i]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
                const float f = n > m[i] ? ex2(m[i] - n) : 1.0f;
                m[i] = n;
                l[i] *= f;
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    o[j][i] *= f;
                    o[j][2 + i] *= f;
                }
            }
        }
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = ex2(x[i] - (m[i & 1] == -INFINITY ? 0.0f : m[i & 1]));
            l[i & 1] += w[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 2 * t + (i & 1) + 8 * (i >> 1);
            vr[i].load(at + 2 * C::kKBytes + i * C::kVBytes, lane, plane + 16 * st + j, g * kVRun, p.D,
                       mask == nullptr || ((keys >> j) & 1u) != 0u);
        }
        uint32_t pb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            pb[i] = transpose8x8(CACHED ? pack_f16x2(w[2 * i], w[2 * i + 1]) : pack_bf16x2_rn(w[2 * i], w[2 * i + 1]));
#pragma unroll
        for (int i = 0; i < kVRun / 8; ++i) {
            uint32_t h[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) vr[k].pairs(i, h[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // pair (e, e + 1): rows g and g + 8 of tile 4i + k
                const uint32_t a[4] = {__byte_perm(h[0][k], h[1][k], 0x5410), __byte_perm(h[0][k], h[1][k], 0x7632),
                                       __byte_perm(h[2][k], h[3][k], 0x5410), __byte_perm(h[2][k], h[3][k], 0x7632)};
                mma16816<CACHED>(o[4 * i + k], a, pb[0], pb[1]);
            }
        }
    }

    // ---- join the warps (in the place of the stages) ----
    copy_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        if (g == 0) {
            sm_m[warp][2 * t + i] = m[i];
            sm_l[warp][2 * t + i] = l[i];
        }
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
            *reinterpret_cast<float2 *>(smem_o + (warp * kRows + 2 * t + i) * DP + g * kVRun + 2 * j) =
                make_float2(o[j][i], o[j][2 + i]);
    }
    __syncthreads();
    constexpr int kPer = kRows * DP / kThreads;  // 2, 4, 8 or 16 adjacent elements a thread
    const int r = threadIdx.x * kPer / DP, e0 = threadIdx.x * kPer % DP;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (sm_l[w][r] != 0.0f) M = fmaxf(M, sm_m[w][r]);
    float sum = 0.0f, acc[kPer] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (sm_l[w][r] == 0.0f) continue;
        const float f = ex2(sm_m[w][r] - M);
        sum = fmaf(f, sm_l[w][r], sum);
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(f, smem_o[(w * kRows + r) * DP + e0 + e], acc[e]);
    }
    if (r >= rows) return;
    if (p.splits > 1) {
        const size_t at = ((static_cast<size_t>(b) * p.Hkv + hk) * rows + r) * p.splits + split;
        if (e0 == 0) p.part_ml[at] = make_float2(M, sum);
        if (sum != 0.0f) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (e0 + e < p.D) p.part_o[at * p.D + e0 + e] = acc[e];
        }
    } else {
        const float f = sum != 0.0f ? (CACHED ? p.cache.v.g : 1.0f) / sum : 0.0f;
        const int tq = r / p.G, hq = hk * p.G + r - tq * p.G;
        uint16_t *to = p.out.ptr + b * p.out.sb + tq * p.out.st + hq * p.out.sh + e0;
#pragma unroll
        for (int e = 0; e < kPer; e += 2)
            if (e0 + e < p.D) *reinterpret_cast<uint32_t *>(to + e) = pack_bf16x2_rn(acc[e] * f, acc[e + 1] * f);
    }
}

template <int DP, bool FULL, bool CACHED>
cudaError_t launch_rows(const AttnArgs &a, cudaStream_t s) {
    static std::atomic<bool> attr_set[kMaxDevices];
    auto *kernel = attention_rows_kernel<DP, FULL, CACHED>;
    using C = Cfg<DP, FULL, CACHED>;
    cudaError_t e = set_smem_limit_once(reinterpret_cast<const void *>(kernel), C::kSmem, attr_set);
    if (e != cudaSuccess) return e;
    const long long ctas = static_cast<long long>(a.B) * a.Hkv * a.splits;
    if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <int DP>
cudaError_t launch_rows_dp(const AttnArgs &a, cudaStream_t s) {
    if (!a.cached) return launch_rows<DP, false, false>(a, s);
    return a.D == DP ? launch_rows<DP, true, true>(a, s) : launch_rows<DP, false, true>(a, s);
}

}  // namespace

cudaError_t launch_attention_rows(const AttnArgs &a, cudaStream_t s) {
    if (a.D <= 64) return launch_rows_dp<64>(a, s);
    if (a.D <= 128) return launch_rows_dp<128>(a, s);
    return launch_rows_dp<256>(a, s);
}

cudaError_t probe_attention_rows() {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, attention_rows_kernel<256, true, true>);
}

}  // namespace nvfp4
