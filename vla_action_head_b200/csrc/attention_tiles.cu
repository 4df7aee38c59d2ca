// attention_tiles.cu — attention in tiles of 128 query rows x 128 keys on the tensor cores.
//
//   S = Q K^T (fp32, tensor memory);  p = 2^(c S - c m) with the running reference m;
//   l = sum p;  O += P V;  out = O / l,                  c = scale log2(e)
//
// The rows of a tile are the (query, head) pairs that share a key head, query-major, so a group of
// G heads reads its keys once.  One CTA takes one row tile and a range of key tiles (the whole
// sequence, or one of `splits` parts whose O, m and l are joined by attention_join_kernel).
//
// Roles (192 threads; cache: 384): warp 5 brings K and V through a ring of 16 KB chunks by TMA (a K chunk is 128
// keys x 64 elements, a V chunk all elements of 16384 / (2 DP) keys: both are what one step of
// the MMA loop eats), warp 4 issues the MMAs, warps 0-3 own a row a thread: scores from tensor
// memory, softmax, P back to tensor memory as the A operand of P V, where it overwrites its own
// scores.  With 256-wide heads O takes half of the tensor memory and two score tiles the rest, so
// Q K^T of the next tile runs under the softmax of this one; narrower heads keep one score tile
// and half of the tensor and shared memory, and two CTAs share an SM and fill each other's gaps.
//
// O is rescaled only where the row maximum outgrew the reference by more than 2^8 (the weights
// stay below 2^8, l and O are fp32; the final division cancels the reference).
//
// Cache: warps 5-11 take TMA's place: they load codes and scales, several pieces ahead, and write
// fp16 (code times scale is exact there) into the same ring; queries and weights are fp16 too.
//
// Left-out keys: their scores become -inf whatever they hold, and their V rows are zeroed in
// shared memory before the product, as 0 x inf is not 0.
#include <cuda.h>
#include <cuda_runtime.h>

#include "attention.h"
#include "gemm.h"
#include "kv_decode.cuh"
#include "quant.cuh"
#include "sm100.cuh"

namespace nvfp4 {

namespace {

constexpr int kChunk = 16384;
constexpr float kLazy = 8.0f;  // log2 of the growth of the maximum that forces a rescale
constexpr int kDequant = 7;    // cache: warps that turn codes into fp16
constexpr int kAhead = 4;      // cache: loads of a dequantizing warp on their way

template <int DP, bool CACHED>
struct Cfg {
    static constexpr bool kBig = CACHED || DP == 256;        // one CTA per SM, two score tiles
    static constexpr int kThreads = CACHED ? 32 * (5 + kDequant) : 192;
    static constexpr int kScores = kBig ? 2 : 1;             // score tiles in tensor memory
    static constexpr int kRing = kBig ? 10 : 5;              // chunks
    static constexpr int kVC = DP / 64;                      // V chunks of a tile
    static constexpr int kKeysPerV = 128 / kVC;              // keys of a V chunk
    static constexpr int kQBytes = 128 * DP * 2;
    static constexpr int kOffRing = kQBytes;
    static constexpr int kOffBar = kOffRing + kRing * kChunk;
    // full[kRing], empty[kRing], s_full[2], p_ready[2], o_done, all_done, q_ready
    static constexpr int kOffMisc = kOffBar + (2 * kRing + 8) * 8;
    static constexpr int kOffRow = kOffMisc + 16;            // cache: a score factor per row
    static constexpr int kSmem = kOffRow + (CACHED ? 512 : 0);
    static constexpr int kTmemCols = kBig ? 512 : 256;
    static constexpr int kColS = kBig ? 256 : 128;           // O at 0, then the score tiles
    static constexpr int kCtas = kBig ? 1 : 2;               // per SM
    static constexpr bool kKeep = DP == 256 && !CACHED;      // a softmax thread has registers for its 128 scores
};
static_assert(Cfg<256, false>::kSmem <= 232448 && Cfg<256, true>::kSmem <= 232448 &&
                  2 * (Cfg<128, false>::kSmem + 1024) <= 233472,
              "shared memory");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Ring positions of a tile's first K and V chunk.  The MMA loop's order is K0 K1 V0 K2 V1 ... with
// two score tiles, K0 V0 K1 V1 ... with one.
template <int SCORES>
__device__ __forceinline__ int k_pos(int i, int kc, int vc) {
    if constexpr (SCORES == 1) return i * (kc + vc);
    return i == 0 ? 0 : kc + (i - 1) * (kc + vc);
}
template <int SCORES>
__device__ __forceinline__ int v_pos(int i, int n, int kc, int vc) {
    if constexpr (SCORES == 1) return i * (kc + vc) + kc;
    return i < n - 1 ? 2 * kc + i * (kc + vc) : n * kc + i * vc;
}

// Cache: a dequantizing warp's piece of a chunk is 32 rows (keys) of one 64-element block: per lane
// 32 bytes of codes and 4 scale bytes (zeros for keys that are left out and elements past D).
struct Codes {
    uint32_t w[8], s;
};
__device__ __forceinline__ Codes load_codes(const CachePlane &c, size_t row, int e0, int D, bool on) {
    Codes x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.w[i] = 0u;
    x.s = 0u;
    if (!on) return x;
    const uint8_t *codes = c.codes + row * (D >> 1) + (e0 >> 1), *sf = c.sf + row * (D >> 4) + (e0 >> 4);
    if ((D & 63) == 0) {  // whole blocks, aligned
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(codes) + i);
            x.w[4 * i] = u.x, x.w[4 * i + 1] = u.y, x.w[4 * i + 2] = u.z, x.w[4 * i + 3] = u.w;
        }
        x.s = __ldcg(reinterpret_cast<const uint32_t *>(sf));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (e0 + 16 * i < D) {
                const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(codes) + i);
                x.w[2 * i] = u.x, x.w[2 * i + 1] = u.y;
                x.s |= static_cast<uint32_t>(__ldcg(sf + i)) << (8 * i);
            }
    }
    return x;
}
// Row r (128 bytes, swizzled) of a 64-element block at `base`: code times scale in fp16, exact.
__device__ __forceinline__ void store_f16(uint8_t *base, int r, const Codes &x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t h[4];
        decode_e2m1x8_f16(x.w[i], h);
        const uint32_t sc = scale_f16x2((x.s >> (8 * (i >> 1))) & 255u);
        *reinterpret_cast<uint4 *>(base + r * 128 + ((i ^ (r & 7)) << 4)) =
            make_uint4(mul_f16x2(h[0], sc), mul_f16x2(h[1], sc), mul_f16x2(h[2], sc), mul_f16x2(h[3], sc));
    }
}

template <int DP, bool CACHED>
__global__ void __launch_bounds__(Cfg<DP, CACHED>::kThreads, Cfg<DP, CACHED>::kCtas)
    attention_tiles_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                           const AttnArgs p) {
    using C = Cfg<DP, CACHED>;
    extern __shared__ __align__(1024) uint8_t smem[];  // 128-byte swizzle atoms
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + C::kOffBar, bar_empty = bar_full + 8 * C::kRing;
    const uint32_t bar_s = bar_empty + 8 * C::kRing, bar_p = bar_s + 16, bar_o = bar_p + 16, bar_all = bar_o + 8, bar_q = bar_all + 8;
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + C::kOffMisc);  // TMEM base, abort
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    float *row_factor = reinterpret_cast<float *>(smem + C::kOffRow);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the CTA's place: split fastest, then row tile, key head, sequence
    int rest = static_cast<int>(blockIdx.x);
    const int split = rest % p.splits;
    rest /= p.splits;
    const int rows = p.T * p.G;
    const int row_tiles = (rows + 127) >> 7;
    const int row0 = (rest % row_tiles) << 7;
    rest /= row_tiles;
    const int hk = rest % p.Hkv, b = rest / p.Hkv;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(bar_full + 8 * i, CACHED ? 4 : 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        mbar_init(bar_s, 1);
        mbar_init(bar_s + 8, 1);
        mbar_init(bar_p, 128);
        mbar_init(bar_p + 8, 128);
        mbar_init(bar_o, 1);
        mbar_init(bar_all, 1);
        mbar_init(bar_q, 128);
        misc[1] = 0;
        fence_mbar_init();
    }
    if (warp == 4) {
        tmem_alloc(smem_u32(const_cast<uint32_t *>(misc)), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    pdl_launch_dependents();
    pdl_wait();  // q, k, v and kv_len may come from the previous kernel
    int len = p.S;
    if (p.kv_len != nullptr) len = min(max(__ldcg(p.kv_len + b), 0), p.S);
    const int all_tiles = (len + 127) >> 7, per = (all_tiles + p.splits - 1) / p.splits;
    const int tile0 = split * per, n = max(0, min(per, all_tiles - tile0));
    const int kc = (p.D + 63) >> 6;  // 64-element blocks of a head
    constexpr int vc = C::kVC;

    if (CACHED && warp >= 5) {
        // ------------------------------ dequantizers ------------------------------
        // the chunks' pieces in the order of the ring, in turn to the warps
        const uint8_t *mask = p.mask != nullptr ? p.mask + b * p.mask_stride : nullptr;
        const size_t plane = (static_cast<size_t>(b) * p.Hkv + hk) * p.cache.C;
        const int pieces = 4 * n * (kc + vc);
        // piece -> is it V's, tile, chunk, block of elements, first key
        struct Piece {
            bool is_v;
            int row, e0, at;  // key row in the cache, element, byte offset of the block in its chunk
        };
        auto piece_of = [&](int x) {
            int pos = x >> 2, tile, c;
            const int part = x & 3;
            bool is_v;
            // K0 K1 V0 K2 V1 .. V(n-1)
            if (pos < kc) {
                is_v = false, tile = 0, c = pos;
            } else {
                pos -= kc;
                const int pair = pos / (kc + vc), in = pos - pair * (kc + vc);
                if (pair < n - 1) is_v = in >= kc, tile = is_v ? pair : pair + 1, c = is_v ? in - kc : in;
                else is_v = true, tile = n - 1, c = in;
            }
            constexpr int groups = C::kKeysPerV / 32;  // pieces of a block of a V chunk
            const int j0 = (tile0 + tile) << 7;
            if (!is_v) return Piece{false, j0 + 32 * part, 64 * c, 32 * part * 128};
            const int e = part / groups, r = part % groups;
            return Piece{true, j0 + c * C::kKeysPerV + 32 * r, 64 * e, (e * C::kKeysPerV + 32 * r) * 128};
        };
        auto fetch = [&](int x) {
            if (x >= pieces) return Codes{};
            const Piece f = piece_of(x);
            const int j = f.row + lane;
            bool on = j < len && f.e0 < p.D;
            if (on && f.is_v && mask != nullptr) on = __ldcg(mask + j) != 0;
            return load_codes(f.is_v ? p.cache.v : p.cache.k, plane + j, f.e0, p.D, on);
        };
        Codes q[kAhead];
        const int x0 = warp - 5;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) q[i] = fetch(x0 + i * kDequant);
        bool ok = true;
        for (int x = x0; x < pieces && ok; x += kAhead * kDequant) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int y = x + i * kDequant;
                if (y < pieces && ok) {
                    const int pos = y >> 2, slot = pos % C::kRing, use = pos / C::kRing;
                    if (use > 0) ok = mbar_wait(bar_empty + 8 * slot, (use - 1) & 1, abort_flag, p.status, kStatusTimeoutEmpty);
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok) {
                        store_f16(smem + C::kOffRing + slot * kChunk + piece_of(y).at, lane, q[i]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_full + 8 * slot);
                    }
                    q[i] = fetch(y + kAhead * kDequant);
                }
            }
        }
    } else if (warp == 5) {
        if (elect_one()) {
            // ------------------------------ producer ------------------------------
            const uint64_t pol = policy_evict_last();
            int pos = 0;
            bool ok = true;
            auto take = [&](uint32_t bytes) -> uint32_t {  // the next chunk, free and expecting `bytes`
                const int slot = pos % C::kRing, use = pos / C::kRing;
                if (use > 0) ok = ok && mbar_wait(bar_empty + 8 * slot, (use - 1) & 1, abort_flag, p.status,
                                                  kStatusTimeoutEmpty);
                if (ok) mbar_arrive_expect_tx(bar_full + 8 * slot, bytes);
                return static_cast<uint32_t>(slot);
            };
            const int zh = p.k_mul_h * hk, zb = p.k_mul_b * b, vh = p.v_mul_h * hk, vb = p.v_mul_b * b;
            auto load_k = [&](int i) {
                for (int c = 0; c < kc && ok; ++c, ++pos) {
                    const uint32_t slot = take(kChunk);
                    if (!ok) break;
                    tma_load_4d(sbase + C::kOffRing + slot * kChunk, &map_k, 64 * c, zh, (tile0 + i) << 7, zb,
                                bar_full + 8 * slot, pol);
                }
            };
            auto load_v = [&](int i) {
                for (int c = 0; c < vc && ok; ++c, ++pos) {
                    const uint32_t slot = take(kc * C::kKeysPerV * 128);
                    if (!ok) break;
                    for (int e = 0; e < kc; ++e)
                        tma_load_4d(sbase + C::kOffRing + slot * kChunk + e * C::kKeysPerV * 128, &map_v, 64 * e, vh,
                                    ((tile0 + i) << 7) + c * C::kKeysPerV, vb, bar_full + 8 * slot, pol);
                }
            };
            if (n > 0) load_k(0);
            for (int i = 0; i < n && ok; ++i) {
                if (C::kScores == 2 && i + 1 < n) load_k(i + 1);
                load_v(i);
                if (C::kScores == 1 && i + 1 < n) load_k(i + 1);
            }
            // leave no copy in flight behind
            int dummy = 0;
            for (int q = max(0, pos - C::kRing); q < pos; ++q)
                mbar_wait(bar_full + 8 * (q % C::kRing), (q / C::kRing) & 1, &dummy, p.status, kStatusTimeoutDrain);
        }
    } else if (warp == 4) {
        if (n > 0 && elect_one()) {
            // ------------------------------ MMA issuer ------------------------------
            constexpr uint32_t idesc_s = idesc_f16(128, 128, !CACHED, false);
            const uint32_t idesc_o = idesc_f16(128, (p.D + 15) & ~15, !CACHED, true);
            const int ksteps = (p.D + 15) >> 4;
            bool ok = mbar_wait(bar_q, 0, abort_flag, p.status, kStatusTimeoutFull);
            auto full = [&](int pos) {
                ok = ok && mbar_wait(bar_full + 8 * (pos % C::kRing), (pos / C::kRing) & 1, abort_flag, p.status,
                                     kStatusTimeoutFull);
                tc_fence_after();
                return sbase + C::kOffRing + (pos % C::kRing) * kChunk;
            };
            auto qk = [&](int i) {
                const int pos = k_pos<C::kScores>(i, kc, vc), buf = i % C::kScores;
                const uint32_t d = tmem + C::kColS + buf * 128;
                uint32_t on = 0u;
                for (int c = 0; c < kc && ok; ++c) {
                    const uint32_t kb = full(pos + c);
                    if (!ok) break;
                    // a step of 16 elements is 32 bytes on: 2 in the descriptors' address field
                    const uint64_t qd = desc_kmajor_sw128(sbase + c * kChunk), kd = desc_kmajor_sw128(kb);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (4 * c + k < ksteps) {
                            tc_mma_f16_ss(d, qd + 2 * k, kd + 2 * k, idesc_s, on);
                            on = 1u;
                        }
                    tc_commit(bar_empty + 8 * ((pos + c) % C::kRing));
                }
                tc_commit(bar_s + 8 * buf);
            };
            qk(0);
            for (int i = 0; i < n && ok; ++i) {
                if (C::kScores == 2 && i + 1 < n) qk(i + 1);
                ok = ok && mbar_wait(bar_p + 8 * (i % C::kScores), (i / C::kScores) & 1, abort_flag, p.status,
                                     kStatusTimeoutSoftmax);
                if (!ok) break;
                tc_fence_after();
                const int pos = v_pos<C::kScores>(i, n, kc, vc);
                const uint32_t pt = tmem + C::kColS + (i % C::kScores) * 128;
                uint32_t on = i > 0 ? 1u : 0u;
#pragma unroll
                for (int c = 0; c < vc; ++c) {
                    const uint32_t v = full(pos + c);
                    if (!ok) break;
                    const uint64_t vd = desc_mnmajor_sw128(v, C::kKeysPerV * 128);
                    constexpr int steps = C::kKeysPerV / 16;
#pragma unroll
                    for (int k = 0; k < steps; ++k) {  // 16 keys: 2048 bytes of V, 8 columns of P
                        tc_mma_f16_ts(tmem, pt + 8 * (c * steps + k), vd + 128 * k, idesc_o, on);
                        on = 1u;
                    }
                    tc_commit(bar_empty + 8 * ((pos + c) % C::kRing));
                }
                tc_commit(i + 1 < n ? bar_o : bar_all);
                if (C::kScores == 1 && i + 1 < n) qk(i + 1);
            }
        }
    } else {
        // ------------------------------ Q ------------------------------
        // rows into K-major swizzled tiles (zeros past D and past the last row), all copies in flight at once
        if (n > 0) {
            constexpr int kUnits = DP / 8, kStep = 128 / kUnits;  // rows of a pass of the 128 threads
            const int c = threadIdx.x % kUnits, r0 = threadIdx.x / kUnits;
            const uint16_t *base = p.q.ptr + b * p.q.sb + static_cast<long long>(hk) * p.G * p.q.sh + 8 * c;
            // row -> (query, head of the group), stepped without a division
            const int dt = kStep / p.G, dg = kStep - dt * p.G;
            int t = (row0 + r0) / p.G, g = row0 + r0 - t * p.G;
            if constexpr (CACHED) {
                // bf16 -> fp16: a row times the power of two that brings its largest element to
                // [2^14, 2^15) (no bit is lost that matters: what falls below fp16's range is 2^-39 of
                // that element), the inverse goes into the row's score factor
                constexpr int kBatch = 128 / kStep < 8 ? 128 / kStep : 8;
                for (int rb = r0; rb < 128; rb += kBatch * kStep) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const bool in = row0 + rb + i * kStep < rows && 8 * c < p.D;
                        v[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (in) v[i] = __ldcg(reinterpret_cast<const uint4 *>(base + t * p.q.st + g * p.q.sh));
                        t += dt;
                        g += dg;
                        if (g >= p.G) {
                            g -= p.G;
                            ++t;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const int r = rb + i * kStep;
                        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                        float top = 0.0f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(bf16lo(w[k])), fabsf(bf16hi(w[k]))));
#pragma unroll
                        for (int d = kUnits / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const float up = f16_row_factor(top);
                        uint32_t h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) h[k] = pack_f16x2(bf16lo(w[k]) * up, bf16hi(w[k]) * up);
                        *reinterpret_cast<uint4 *>(smem + (c >> 3) * kChunk + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                            make_uint4(h[0], h[1], h[2], h[3]);
                        if (c == 0) row_factor[r] = 1.0f / up;
                    }
                }
            } else {
#pragma unroll 8
                for (int r = r0; r < 128; r += kStep) {
                    const bool in = row0 + r < rows && 8 * c < p.D;
                    cp_async16(sbase + (c >> 3) * kChunk + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                               in ? base + t * p.q.st + g * p.q.sh : p.q.ptr, in ? 16u : 0u);
                    t += dt;
                    g += dg;
                    if (g >= p.G) {
                        g -= p.G;
                        ++t;
                    }
                }
                cp_async_wait_all();
            }
            fence_proxy_async_smem();
            if (CACHED) asm volatile("bar.sync 1, 128;" ::: "memory");  // the row factors
            mbar_arrive(bar_q);
        }

        // ------------------------------ softmax, a row a thread ------------------------------
        const bool warp_on = row0 + warp * 32 < rows;  // some row of this warp exists
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const float c = CACHED && n > 0 ? p.scale_log2 * row_factor[threadIdx.x] : p.scale_log2;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            ok = mbar_wait(bar_s + 8 * (i % C::kScores), (i / C::kScores) & 1, abort_flag, p.status,
                           kStatusTimeoutAccum);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const int j0 = (tile0 + i) << 7;
            const bool part = p.mask != nullptr || j0 + 128 > len;
            uint32_t keep[4];
            if (part) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int j = j0 + 32 * w + lane;
                    bool in = j < len;
                    if (in && p.mask != nullptr) in = __ldcg(p.mask + b * p.mask_stride + j) != 0;
                    keep[w] = __ballot_sync(0xffffffffu, in);
                }
            }
            if (warp_on) {
                const uint32_t ts = lane_base + C::kColS + (i % C::kScores) * 128;
                // the scores stay in registers where a thread may have 255, else they are read twice
                constexpr bool kKeep = C::kKeep;
                uint32_t s[kKeep ? 4 : 2][32];
                auto load = [&](uint32_t (&x)[32], int w) { tmem_ld_32x32b_x32(ts + 32 * w, x); };
                auto leave_out = [&](uint32_t (&x)[32], int w) {
                    if (part) {
                        const uint32_t k = w == 0 ? keep[0] : w == 1 ? keep[1] : w == 2 ? keep[2] : keep[3];
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (((k >> j) & 1u) == 0u) x[j] = 0xFF800000u;
                    }
                };
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto top_of = [&](const uint32_t (&x)[32]) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(x[j]));
                };
                if constexpr (kKeep) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) load(s[w], w);
                    tmem_ld_wait();
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        leave_out(s[w], w);
                        top_of(s[w]);
                    }
                } else {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        load(s[0], 2 * half);
                        load(s[1], 2 * half + 1);
                        tmem_ld_wait();
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            leave_out(s[w], 2 * half + w);
                            top_of(s[w]);
                        }
                    }
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                // the reference: the first maximum, then only one that outgrew it
                const bool grow = top > m && !((top - m) * c <= kLazy);
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2((m - top) * c) : 1.0f;
                    if (grow) m = top;
                    if (i > 0) {
                        ok = mbar_wait(bar_o, (i - 1) & 1, abort_flag, p.status, kStatusTimeoutAccum);
                        if (!__all_sync(0xffffffffu, ok)) break;
                        tc_fence_after();
                        l *= f;
                        for (int e = 0; e < p.D; e += 32) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(lane_base + e, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st_32x32b_x32(lane_base + e, o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.0f : m * c;
                float sum[4] = {};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pk[32];
                    if constexpr (!kKeep) {  // P of this half overwrites scores already read
                        load(s[0], 2 * half);
                        load(s[1], 2 * half + 1);
                        tmem_ld_wait();
                        leave_out(s[0], 2 * half);
                        leave_out(s[1], 2 * half + 1);
                    }
#pragma unroll
                    for (int w = 0; w < 2; ++w)
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const uint32_t *sw = s[kKeep ? 2 * half + w : w];
                            const float x = ex2(fmaf(__uint_as_float(sw[j]), c, -mc));
                            const float y = ex2(fmaf(__uint_as_float(sw[j + 1]), c, -mc));
                            sum[2 * w] += x;
                            sum[2 * w + 1] += y;
                            pk[16 * w + j / 2] = CACHED ? pack_f16x2(x, y) : pack_bf16x2_rn(x, y);
                        }
                    tmem_st_32x32b_x32(ts + 32 * half, pk);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_st_wait();
            }
            if (part && !CACHED) {
                // this thread's key row of V: zeros if the key is left out.  Once the previous product is
                // done every chunk before V's has landed, so the phase waited for is V's own.
                if (((keep[warp] >> lane) & 1u) == 0u) {
                    if (i > 0) ok = mbar_wait(bar_o, (i - 1) & 1, abort_flag, p.status, kStatusTimeoutAccum);
                    const int key = threadIdx.x, pos = v_pos<C::kScores>(i, n, kc, vc) + key / C::kKeysPerV;
                    ok = ok && mbar_wait(bar_full + 8 * (pos % C::kRing), (pos / C::kRing) & 1, abort_flag,
                                         p.status, kStatusTimeoutFull);
                    uint8_t *v = smem + C::kOffRing + (pos % C::kRing) * kChunk + (key % C::kKeysPerV) * 128;
                    if (ok)
                        for (int e = 0; e < kc; ++e)
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<uint4 *>(v + e * C::kKeysPerV * 128 + ((q ^ (lane & 7)) << 4)) =
                                    make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                if (!__all_sync(0xffffffffu, ok)) break;
            }
            tc_fence_before();
            // one barrier per score tile: a warp may be a tile ahead of another
            mbar_arrive(bar_p + 8 * (i % C::kScores));
        }

        // ------------------------------ output ------------------------------
        // (on a barrier of its own: the one before the last may still be running, or have been done long ago)
        if (ok && n > 0) ok = mbar_wait(bar_all, 0, abort_flag, p.status, kStatusTimeoutAccum);
        tc_fence_after();
        if (__all_sync(0xffffffffu, ok) && warp_on) {
            // through shared memory (the ring is idle now), so that a warp stores whole rows: a row a thread
            // would touch 32 lines per instruction
            const float f = l != 0.0f ? (CACHED ? p.cache.v.g : 1.0f) / l : 0.0f;
            const size_t row_g = (static_cast<size_t>(b) * p.Hkv + hk) * rows + row0 + warp * 32;
            const int live = min(32, rows - row0 - warp * 32);
            if (p.splits > 1) {
                constexpr int kPitch = DP * 4;
                uint8_t *st = smem + C::kOffRing + warp * 32 * kPitch;
                if (lane < live) p.part_ml[(row_g + lane) * p.splits + split] = make_float2(m * c, l);
                if (n > 0) {
                    for (int e = 0; e < p.D; e += 32) {
                        uint32_t o[32];
                        tmem_ld_32x32b_x32(lane_base + e, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4 *>(st + lane * kPitch + (((e >> 2) + j) ^ (lane & 7)) * 16) =
                                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                    __syncwarp();
                    const int units = p.D >> 2, lanes = units < 32 ? 32 / units : 1;  // rows an instruction
                    const int r0 = units < 32 ? lane / units : 0, c0 = units < 32 ? lane % units : lane;
                    for (int r = r0; r < live && r0 < lanes; r += lanes)
                        for (int c = c0; c < units; c += 32)
                            *reinterpret_cast<uint4 *>(p.part_o + ((row_g + r) * p.splits + split) * p.D + 4 * c) =
                                *reinterpret_cast<const uint4 *>(st + r * kPitch + (c ^ (r & 7)) * 16);
                }
            } else {
                constexpr int kPitch = DP * 2;
                uint8_t *st = smem + C::kOffRing + warp * 32 * kPitch;
                for (int e = 0; e < p.D; e += 32) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(lane_base + e, o);
                    tmem_ld_wait();
                    if (l == 0.0f) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = 0u;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            w[q] = pack_bf16x2_rn(__uint_as_float(o[8 * j + 2 * q]) * f,
                                                  __uint_as_float(o[8 * j + 2 * q + 1]) * f);
                        *reinterpret_cast<uint4 *>(st + lane * kPitch + (((e >> 3) + j) ^ (lane & 7)) * 16) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
                const int units = p.D >> 3, lanes = 32 / units;  // units <= 32
                const int r0 = lane / units, c = lane % units;
                uint16_t *to = p.out.ptr + b * p.out.sb + static_cast<long long>(hk) * p.G * p.out.sh + 8 * c;
                const int dt = lanes / p.G, dg = lanes - dt * p.G;
                int t = (row0 + warp * 32 + r0) / p.G, g = row0 + warp * 32 + r0 - t * p.G;
                for (int r = r0; r < live && r0 < lanes; r += lanes) {
                    *reinterpret_cast<uint4 *>(to + t * p.out.st + g * p.out.sh) =
                        *reinterpret_cast<const uint4 *>(st + r * kPitch + (c ^ (r & 7)) * 16);
                    t += dt;
                    g += dg;
                    if (g >= p.G) {
                        g -= p.G;
                        ++t;
                    }
                }
            }
        }
    }

    // teardown
    __syncwarp();
    if (*abort_flag) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

template <int DP, bool CACHED>
cudaError_t launch_dp(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, cudaStream_t s) {
    using C = Cfg<DP, CACHED>;
    static std::atomic<bool> attr_set[kMaxDevices];
    auto *kernel = attention_tiles_kernel<DP, CACHED>;
    cudaError_t e = set_smem_limit_once(reinterpret_cast<const void *>(kernel), C::kSmem, attr_set);
    if (e != cudaSuccess) return e;
    const long long tiles = (static_cast<long long>(a.T) * a.G + 127) / 128;
    const long long ctas = tiles * a.B * a.Hkv * a.splits;
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

}  // namespace

int attention_v_box_rows(int D) { return D <= 64 ? 128 : D <= 128 ? 64 : 32; }

cudaError_t launch_attention_tiles(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, cudaStream_t s) {
    if (a.D <= 64) return a.cached ? launch_dp<64, true>(mk, mv, a, s) : launch_dp<64, false>(mk, mv, a, s);
    if (a.D <= 128) return a.cached ? launch_dp<128, true>(mk, mv, a, s) : launch_dp<128, false>(mk, mv, a, s);
    return a.cached ? launch_dp<256, true>(mk, mv, a, s) : launch_dp<256, false>(mk, mv, a, s);
}

cudaError_t probe_attention_tiles() {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, attention_tiles_kernel<256, false>);
}

}  // namespace nvfp4
