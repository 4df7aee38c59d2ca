// attention_rows.cu — attention for few query rows per key head (single tokens): up to 8 (query,
// head) pairs share a key head's keys, which are read once.
//
//   S^T = K Q^T,  p = 2^(c (S - m)),  l = sum p,  O^T += V^T P^T,  out = O / l,   c = scale log2(e)
//
// The work is the stream of keys and values, so the matrix instruction is the one that takes its
// operands from registers (m16n8k16): 16 keys (or 16 elements of V) are its rows, the 8 query
// rows its columns.  (On tcgen05 the 8 rows would be 8 of a tile's 128, and a cache's numbers would pass
// through shared memory once more.)  A contraction may take its elements in any order as long as both sides do, so every thread takes runs of adjacent
// elements: of a key the quarter of its lane % 4 (k of S^T), of a value row the eighth of its
// lane / 4 (the rows of O^T), which makes 16-byte loads of plain rows.  The weights turn from S^T's
// accumulator into the next operand by one 8 x 8 transposition in registers (movmatrix).
//
// Cache: codes become fp16 (exact: 2-bit significand times 4-bit scale; the weights are then fp16
// too, closer than bf16).  Query rows are scaled by a power of two into fp16's range, which keeps every bit of an
// element down to 2^-31 of the row's largest; smaller ones are off by 2^-39 of it at most.
//
// Every warp takes steps of 16 keys of its own: its lane 0 asks the copy engine for the next step's
// rows (a tensor copy whose 128-byte swizzle makes the reads above free of bank conflicts; plain
// bulk copies where a cache row is no multiple of 16 bytes), and the warp waits on its own barrier.
// No barrier of the CTA in the loop, a few instructions a step for the loads.  (8 sequences of 32701
// cached keys, 256-wide heads: 71 us with loads into registers, 46 with cp.async by every thread, 34 so,
// 31 with the CTAs dealt out by the lengths, 29.1 with the pieces joined eight at a time, 29.5 with weights that
// reach down to 2^-32.  Bound by the instructions that turn codes into numbers, and by about 4 us of start and join.
// The same over bf16 keys: 45 us, 76 % of the rate that a copy reaches.)
//
// The warps of a CTA are joined through shared memory.  A CTA takes a whole key head, or (long keys,
// few heads) a piece of one, dealt out by the sequences' lengths (attention_share.cuh); the pieces are
// joined by attention_join_kernel.
// The reference m of a row is replaced only when a score outgrows it by 2^8, found by one vote a
// step, so the steps carry no reductions; l stays per thread until the end.
#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.h"
#include "attention_share.cuh"
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

__device__ __forceinline__ uint32_t lds2(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t a) {
    uint16_t v;
    asm volatile("{\n\t.reg .u32 x;\n\tld.shared.u8 x, [%1];\n\tcvt.u16.u32 %0, x;\n\t}" : "=h"(v) : "r"(a));
    return v;
}

// A stage of a warp holds 16 rows of K and of V.  bf16: 64-element blocks of 16 rows x 128 bytes,
// swizzled.  Cache: 16 rows of codes (FULL, D = DP: swizzled over the row's 128, 64 or 32 bytes; else as
// they are in the cache, D / 2 bytes a row), then the rows' D / 16 scale bytes.
template <int DP, bool FULL, bool CACHED>
struct Cfg {
    static constexpr int kCodes = CACHED ? 16 * DP / 2 : 16 * DP * 2;  // bytes of K's rows, and of V's
    static constexpr int kScale = CACHED ? 16 * DP / 16 : 0;
    static constexpr int kOffV = kCodes, kOffKs = 2 * kCodes, kOffVs = kOffKs + kScale;
    static constexpr int kStage = (2 * (kCodes + kScale) + 1023) / 1024 * 1024;  // swizzle atoms
    // cache: 16 warps, as turning codes into numbers is what keeps the SM busy; bf16: as many as leave
    // two steps on their way
    static constexpr int kWarps = CACHED ? 16 : DP == 256 ? 4 : 8, kThreads = 32 * kWarps;
    static constexpr int kStages = CACHED ? (DP == 256 ? 2 : 3) : DP >= 128 ? 3 : 4;
    static constexpr int kQ = DP / 16 * 256;  // Q: a step's pair of operand words per lane
    static constexpr int kPitch = DP + 4;     // floats of a row in the join: lanes on different banks
    static constexpr int kRing = kWarps * kStages * kStage, kJoin = kWarps * kRows * kPitch * 4;
    static constexpr int kSmem = kQ + (kRing > kJoin ? kRing : kJoin);
    // elements taken at a time: 16 bytes, or what a thread has of a row
    static constexpr int kKBlock = CACHED ? (DP / 4 < 32 ? DP / 4 : 32) : 8, kKBlocks = DP / 4 / kKBlock;
    static constexpr int kVBlock = CACHED ? DP / 8 : 8, kVBlocks = DP / 8 / kVBlock;
    static_assert(kOffKs >= 0 && kOffVs + kScale <= kStage, "a stage's parts");
    static_assert(kQ % 1024 == 0 && kSmem + 2048 <= 232448, "shared memory");
    // first element of a thread's block, and of pair x of the rows of O^T
    __device__ static int k_element(int t, int i) {
        return CACHED ? t * (DP / 4) + i * kKBlock : (i >> 1) * 64 + (2 * t + (i & 1)) * 8;
    }
    __device__ static int v_element(int g, int i) { return CACHED ? g * (DP / 8) : i * 64 + g * 8; }
    __device__ static int o_element(int g, int x) {
        return CACHED ? g * (DP / 8) + 2 * x : (x >> 2) * 64 + g * 8 + 2 * (x & 3);
    }
};

// 16-byte unit c of row r in rows of BYTES (a power of two) under the copy engine's swizzle of that span.
template <int BYTES>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    if constexpr (BYTES == 128) return r * 128 + ((c ^ (r & 7)) << 4);
    else if constexpr (BYTES == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    else return r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}

// N elements (from e) of row r of a stage: their codes and scale bytes (zeros past D).
template <int DP, bool FULL, int N>
__device__ __forceinline__ void load_codes(uint32_t codes, uint32_t sf, int r, int e, int D, uint32_t (&w)[N / 8],
                                           uint32_t &s) {
    s = 0u;
    if constexpr (FULL) {
        const uint32_t a = codes + swizzled<DP / 2>(r, e >> 5) + ((e >> 1) & 15);
        if constexpr (N == 32) {
            const uint4 u = lds16(a);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
            s = lds2(sf + r * (DP / 16) + (e >> 4));
        } else if constexpr (N == 16) {
            const uint2 u = lds8(a);
            w[0] = u.x, w[1] = u.y;
            s = lds1(sf + r * (DP / 16) + (e >> 4));
        } else {
            w[0] = lds4(a);
            s = lds1(sf + r * (DP / 16) + (e >> 4));
        }
    } else {
        const uint32_t a = codes + r * (D >> 1) + (e >> 1), b = sf + r * (D >> 4) + (e >> 4);
        if constexpr (N >= 16) {
#pragma unroll
            for (int i = 0; i < N / 16; ++i) {
                w[2 * i] = w[2 * i + 1] = 0u;
                if (e + 16 * i < D) {
                    const uint2 u = lds8(a + 8 * i);
                    w[2 * i] = u.x, w[2 * i + 1] = u.y;
                    s |= lds1(b + i) << (8 * i);
                }
            }
        } else {
            w[0] = 0u;
            if (e < D) {
                w[0] = lds4(a);
                s = lds1(b);
            }
        }
    }
}
// The same -> fp16 pairs of adjacent elements.
template <int DP, bool FULL, int N>
__device__ __forceinline__ void codes_f16(uint32_t codes, uint32_t sf, int r, int e, int D, uint32_t (&h)[N / 2]) {
    uint32_t w[N / 8], s, sc[2];
    load_codes<DP, FULL, N>(codes, sf, r, e, D, w, s);
    scale2_f16x2(s, sc[0], sc[1]);
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
        uint32_t d[4];
        decode_e2m1x8_f16(w[q], d);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[4 * q + k] = mul_f16x2(d[k], sc[q >> 1]);
    }
}
// N elements (from e) of rows r and r + 1 of a stage's codes -> fp16 pairs (row r, row r + 1): lo[i] of
// element 2i, hi[i] of 2i + 1, the matrix operand as it is.  The codes are paired by nibbles before they
// are decoded, which is half the work of transposing decoded pairs.  `on`, `on1`: as above.
template <int DP, bool FULL, int N>
__device__ __forceinline__ void codes_f16_rows(uint32_t codes, uint32_t sf, int r, int e, int D, bool on, bool on1,
                                               uint32_t (&lo)[N / 2], uint32_t (&hi)[N / 2]) {
    uint32_t w[2][N / 8], s[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        load_codes<DP, FULL, N>(codes, sf, r + x, e, D, w[x], s[x]);
        if (!(x == 0 ? on : on1)) s[x] = 0u;
    }
    const uint32_t ss = __byte_perm(s[0], s[1], 0x5140);  // scale bytes of block 0 of both rows, then of block 1
    uint32_t sc[2];
    sc[0] = scales_f16x2(ss);
    sc[1] = N > 16 ? scales_f16x2(ss >> 16) : 0u;
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
        const uint32_t a = w[0][q], b = w[1][q];
        uint32_t d[4];
        decode_e2m1x8_f16((a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u), d);
#pragma unroll
        for (int k = 0; k < 4; ++k) lo[4 * q + k] = mul_f16x2(d[k], sc[q >> 1]);
        decode_e2m1x8_f16(((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u), d);
#pragma unroll
        for (int k = 0; k < 4; ++k) hi[4 * q + k] = mul_f16x2(d[k], sc[q >> 1]);
    }
}
// 8 elements: 16-byte unit c of row r of a 64-element block.
__device__ __forceinline__ void wide_pairs(uint32_t block, int r, int c, bool on, uint32_t (&h)[4]) {
    const uint4 u = lds16(block + swizzled<128>(r, c));
    h[0] = on ? u.x : 0u, h[1] = on ? u.y : 0u, h[2] = on ? u.z : 0u, h[3] = on ? u.w : 0u;
}

template <int DP, bool FULL, bool CACHED>
__global__ void __launch_bounds__(Cfg<DP, FULL, CACHED>::kThreads, 1)
    attention_rows_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                          const AttnArgs p) {
    using C = Cfg<DP, FULL, CACHED>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
    constexpr int kTiles = DP / 16;  // k steps of S^T, row tiles of O^T
    extern __shared__ __align__(1024) uint8_t smem[];  // Q, then the warps' stages, then their [kRows][kPitch]
    float *smem_o = reinterpret_cast<float *>(smem + C::kQ);
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows], sm_q[kRows];
    __shared__ __align__(8) uint64_t sm_bar[kWarps][C::kStages];
    __shared__ int sm_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t bar = smem_u32(&sm_bar[warp][0]);
    if (lane == 0) {
        for (int i = 0; i < C::kStages; ++i) mbar_init(bar + 8 * i, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) sm_abort = 0;
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();
    const int rows = p.T * p.G;  // <= kRows
    const uint32_t sq = smem_u32(smem), ring = sq + C::kQ + warp * C::kStages * C::kStage;
    const int kc = (p.D + 63) >> 6;
    const uint64_t policy = policy_evict_first();
    int slot = 0;
    uint32_t phase = 0u;

    KeyRange range;
    if (!key_range(p, range)) return;  // the whole CTA
    const int b = range.b, hk = range.hk, len = range.len, step0 = range.step0, step1 = range.step1;

    // Q (warp 0): row g, the thread's elements of each block of K
    constexpr int kQUnits = DP / 32;  // 8 elements each
    uint4 qu[kQUnits];
    if (warp == 0) {
        const bool on = g < rows;
        const int tq = on ? g / p.G : 0, hq = hk * p.G + (on ? g - tq * p.G : 0);
        const uint16_t *src = p.q.ptr + b * p.q.sb + tq * p.q.st + hq * p.q.sh;
#pragma unroll
        for (int i = 0; i < kQUnits; ++i) {
            const int e = C::k_element(t, i * 8 / C::kKBlock) + i * 8 % C::kKBlock;
            qu[i] = make_uint4(0u, 0u, 0u, 0u);
            if (on && e < p.D) qu[i] = __ldcg(reinterpret_cast<const uint4 *>(src + e));
        }
    }

    const uint8_t *mask = p.mask != nullptr ? p.mask + b * p.mask_stride : nullptr;
    const size_t plane = (static_cast<size_t>(b) * p.Hkv + hk) * p.cache.C;
    auto ask = [&](int st, int slot) {  // lane 0
        const uint32_t to = ring + slot * C::kStage, on = bar + 8 * slot;
        if constexpr (CACHED) {
            const size_t row = plane + 16 * static_cast<size_t>(st);
            const uint32_t bytes = FULL ? C::kCodes : 8 * p.D;
            mbar_arrive_expect_tx(on, 2 * bytes + 2 * p.D);
            if constexpr (FULL) {
                tma_load_2d(to, &map_k, 0, static_cast<int>(row), on, policy);
                tma_load_2d(to + C::kOffV, &map_v, 0, static_cast<int>(row), on, policy);
            } else {
                bulk_load(to, p.cache.k.codes + row * (p.D >> 1), bytes, on, policy);
                bulk_load(to + C::kOffV, p.cache.v.codes + row * (p.D >> 1), bytes, on, policy);
            }
            bulk_load(to + C::kOffKs, p.cache.k.sf + row * (p.D >> 4), p.D, on, policy);
            bulk_load(to + C::kOffVs, p.cache.v.sf + row * (p.D >> 4), p.D, on, policy);
        } else {
            mbar_arrive_expect_tx(on, 2 * kc * 2048);
            for (int e = 0; e < kc; ++e) {
                tma_load_4d(to + 2048 * e, &map_k, 64 * e, p.k_mul_h * hk, 16 * st, p.k_mul_b * b, on, policy);
                tma_load_4d(to + C::kOffV + 2048 * e, &map_v, 64 * e, p.v_mul_h * hk, 16 * st, p.v_mul_b * b, on,
                            policy);
            }
        }
    };
    if (lane == 0)
        for (int i = 0, to = slot; i < C::kStages; ++i) {
            if (step0 + warp + i * kWarps < step1) ask(step0 + warp + i * kWarps, to);
            to = to + 1 == C::kStages ? 0 : to + 1;
        }
    // lane's key of a step, 1 if it is attended to; asked for one step ahead
    auto key_on = [&](int st) -> uint32_t {
        const int j = 16 * st + (lane & 15);
        if (st >= step1 || j >= len) return 0u;
        return mask == nullptr ? 1u : __ldcg(mask + j) != 0 ? 1u : 0u;
    };
    uint32_t key = key_on(step0 + warp);

    if (warp == 0) {  // Q as the operand words of each step of 16 elements
        float up = 1.0f, down = 1.0f;
        if constexpr (CACHED) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < kQUnits; ++i) {
                const uint32_t w[4] = {qu[i].x, qu[i].y, qu[i].z, qu[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(bf16lo(w[k])), fabsf(bf16hi(w[k]))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            up = f16_row_factor(top, &down);
        }
        if (t == 0) sm_q[g] = down;
#pragma unroll
        for (int i = 0; i < kQUnits; ++i) {
            uint32_t w[4] = {qu[i].x, qu[i].y, qu[i].z, qu[i].w};
            if constexpr (CACHED) {
#pragma unroll
                for (int k = 0; k < 4; ++k) w[k] = pack_f16x2(bf16lo(w[k]) * up, bf16hi(w[k]) * up);
            }
            uint2 *to = reinterpret_cast<uint2 *>(smem) + lane;
            to[(2 * i) * 32] = make_uint2(w[0], w[1]);
            to[(2 * i + 1) * 32] = make_uint2(w[2], w[3]);
        }
    }
    __syncthreads();
    const float cr[2] = {score_factor(p.scale_log2, sm_q[2 * t]), score_factor(p.scale_log2, sm_q[2 * t + 1])};  // of rows 2t, 2t + 1

    float o[kTiles][4] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // rows 2t, 2t + 1
    for (int st = step0 + warp; st < step1; st += kWarps) {
        const uint32_t keys = __ballot_sync(0xffffffffu, key != 0u);
        key = key_on(st + kWarps);
        const bool landed = mbar_wait(bar + 8 * slot, phase, &sm_abort, p.status, kStatusTimeoutFull);
        if (!__all_sync(0xffffffffu, landed)) {
            // leave no copy in flight behind
            int dummy = 0;
            for (int i = 0; i < C::kStages && st + i * kWarps < step1; ++i) {
                mbar_wait(bar + 8 * slot, phase, &dummy, p.status, kStatusTimeoutDrain);
                if (++slot == C::kStages) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            break;
        }
        const uint32_t at = ring + slot * C::kStage, vat = at + C::kOffV;
        const bool ok[2] = {((keys >> g) & 1u) != 0u, ((keys >> (g + 8)) & 1u) != 0u};
        float sa[2][4] = {};  // two chains
#pragma unroll
        for (int i = 0; i < C::kKBlocks; ++i) {
            if (!CACHED && (i >> 1) >= kc) break;  // blocks past the head were not brought: they hold anything
            uint32_t h0[C::kKBlock / 2], h1[C::kKBlock / 2];
            if constexpr (CACHED) {
                codes_f16<DP, FULL, C::kKBlock>(at, at + C::kOffKs, g, C::k_element(t, i), p.D, h0);
                codes_f16<DP, FULL, C::kKBlock>(at, at + C::kOffKs, g + 8, C::k_element(t, i), p.D, h1);
            } else {
                wide_pairs(at + (i >> 1) * 2048, g, 2 * t + (i & 1), true, h0);
                wide_pairs(at + (i >> 1) * 2048, g + 8, 2 * t + (i & 1), true, h1);
            }
#pragma unroll
            for (int k = 0; k < C::kKBlock / 4; ++k) {
                const uint32_t a[4] = {h0[2 * k], h1[2 * k], h0[2 * k + 1], h1[2 * k + 1]};
                const uint2 q = lds8(sq + (i * (C::kKBlock / 4) + k) * 256 + lane * 8);
                mma16816<CACHED>(sa[k & 1], a, q.x, q.y);
            }
        }
        const float s[4] = {sa[0][0] + sa[1][0], sa[0][1] + sa[1][1], sa[0][2] + sa[1][2], sa[0][3] + sa[1][3]};
        // scores; left-out keys are -inf whatever their bytes gave
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ok[i >> 1] ? s[i] : -INFINITY;
        const float top[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
        const bool grow = (top[0] > m[0] && !((top[0] - m[0]) * cr[0] <= kLazy)) ||
                          (top[1] > m[1] && !((top[1] - m[1]) * cr[1] <= kLazy));
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float n = fmaxf(m[i], top[i]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
                const float f = n > m[i] ? ex2((m[i] - n) * cr[i]) : 1.0f;
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
            const float d = x[i] - (m[i & 1] == -INFINITY ? 0.0f : m[i & 1]);
            w[i] = ex2(CACHED ? fmaf(d, cr[i & 1], kF16WeightBits) : d * cr[i & 1]);
            l[i & 1] += w[i];
        }
        uint32_t pb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            pb[i] = transpose8x8(CACHED ? pack_f16x2(w[2 * i], w[2 * i + 1]) : pack_bf16x2_rn(w[2 * i], w[2 * i + 1]));
        // keys 2t, 2t + 1, 2t + 8, 2t + 9; zeros for the left-out ones (whatever their bytes are)
#pragma unroll
        for (int i = 0; i < C::kVBlocks; ++i) {
            if (!CACHED && i >= kc) break;
            // pairs of keys (2t, 2t + 1) and (2t + 8, 2t + 9): element 2x in lo[x], 2x + 1 in hi[x]
            uint32_t lo[2][C::kVBlock / 2], hi[2][C::kVBlock / 2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int j = 2 * t + 8 * k;
                const bool on = ((keys >> j) & 1u) != 0u, on1 = ((keys >> (j + 1)) & 1u) != 0u;
                if constexpr (CACHED) {
                    codes_f16_rows<DP, FULL, C::kVBlock>(vat, at + C::kOffVs, j, C::v_element(g, i), p.D, on, on1, lo[k],
                                                         hi[k]);
                } else {
                    uint32_t h0[4], h1[4];
                    wide_pairs(vat + i * 2048, j, g, on, h0);
                    wide_pairs(vat + i * 2048, j + 1, g, on1, h1);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        lo[k][x] = __byte_perm(h0[x], h1[x], 0x5410);
                        hi[k][x] = __byte_perm(h0[x], h1[x], 0x7632);
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < C::kVBlock / 2; ++x) {  // rows g and g + 8 of a tile: elements 2x and 2x + 1
                const uint32_t a[4] = {lo[0][x], hi[0][x], lo[1][x], hi[1][x]};
                mma16816<CACHED>(o[i * (C::kVBlock / 2) + x], a, pb[0], pb[1]);
            }
        }
        __syncwarp();  // every lane has read the stage
        if (lane == 0 && st + C::kStages * kWarps < step1) ask(st + C::kStages * kWarps, slot);
        if (++slot == C::kStages) {
            slot = 0;
            phase ^= 1u;
        }
    }

    // ---- join the warps (in the place of the stages; every copy asked for has been waited for) ----
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
            *reinterpret_cast<float2 *>(smem_o + (warp * kRows + 2 * t + i) * C::kPitch + 16 * j + 2 * g) =
                make_float2(o[j][i], o[j][2 + i]);
    }
    __syncthreads();
    // each warp's factor against the row's largest reference, and the row's sum
    for (int r = warp; r < rows; r += kWarps) {
        const float c = score_factor(p.scale_log2, sm_q[r]);
        const float lw = lane < kWarps ? sm_l[lane][r] : 0.0f, mw = lane < kWarps && lw != 0.0f ? sm_m[lane][r] : -INFINITY;
        float M = mw;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        const float f = lw != 0.0f ? ex2((sm_m[lane][r] - M) * c) : 0.0f;
        float sum = f * lw;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane < kWarps) sm_l[lane][r] = f;
        if (lane == 0) sm_q[r] = sum;
        if (lane == 0 && p.share > 0) p.part_ml[static_cast<size_t>(blockIdx.x) * rows + r] = make_float4(M, sum, c, 0.0f);
    }
    __syncthreads();
    // a thread: every kThreads-th pair of elements of the rows
    for (int x = threadIdx.x; x < rows * (DP / 2); x += kThreads) {
        const int r = x / (DP / 2), pair = x % (DP / 2), e = C::o_element(pair & 7, pair >> 3);
        if (e >= p.D) continue;
        float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            // (a warp without keys has a factor of 0, and sums of 0)
            const float f = sm_l[w][r];
            const float2 v = *reinterpret_cast<const float2 *>(smem_o + (w * kRows + r) * C::kPitch + 2 * pair);
            a0 = fmaf(f, v.x, a0);
            a1 = fmaf(f, v.y, a1);
        }
        const float sum = sm_q[r];
        if (p.share > 0) {
            *reinterpret_cast<float2 *>(p.part_o + (static_cast<size_t>(blockIdx.x) * rows + r) * p.D + e) = make_float2(a0, a1);
        } else {
            const float f = sum != 0.0f ? (CACHED ? p.cache.v.g : 1.0f) / sum : 0.0f;
            const int tq = r / p.G, hq = hk * p.G + r - tq * p.G;
            *reinterpret_cast<uint32_t *>(p.out.ptr + b * p.out.sb + tq * p.out.st + hq * p.out.sh + e) =
                pack_bf16x2_rn(a0 * f, a1 * f);
        }
    }
}

template <int DP, bool FULL, bool CACHED>
cudaError_t launch_rows(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, cudaStream_t s) {
    static std::atomic<bool> attr_set[kMaxDevices];
    auto *kernel = attention_rows_kernel<DP, FULL, CACHED>;
    using C = Cfg<DP, FULL, CACHED>;
    cudaError_t e = set_smem_limit_once(reinterpret_cast<const void *>(kernel), C::kSmem, attr_set);
    if (e != cudaSuccess) return e;
    const long long ctas = a.share > 0 ? a.share : static_cast<long long>(a.B) * a.Hkv;
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
    return cudaLaunchKernelEx(&cfg, kernel, mk, mv, a);
}
template <int DP>
cudaError_t launch_rows_dp(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, cudaStream_t s) {
    if (!a.cached) return launch_rows<DP, false, false>(mk, mv, a, s);
    return attention_rows_mapped(a) ? launch_rows<DP, true, true>(mk, mv, a, s)
                                    : launch_rows<DP, false, true>(mk, mv, a, s);
}

}  // namespace

bool attention_rows_mapped(const AttnArgs &a) {
    return (a.D == 64 || a.D == 128 || a.D == 256) &&
           static_cast<long long>(a.B) * a.Hkv * a.cache.C < 0x7FFFFFFFLL;
}

int attention_rows_warps(bool cached, int D) { return cached ? 16 : D > 128 ? 4 : 8; }

cudaError_t launch_attention_rows(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, cudaStream_t s) {
    if (a.D <= 64) return launch_rows_dp<64>(mk, mv, a, s);
    if (a.D <= 128) return launch_rows_dp<128>(mk, mv, a, s);
    return launch_rows_dp<256>(mk, mv, a, s);
}

cudaError_t probe_attention_rows() {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, attention_rows_kernel<256, true, true>);
}

}  // namespace nvfp4
