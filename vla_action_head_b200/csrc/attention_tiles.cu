// attention_tiles.cu — attention in tiles of 128 query rows x 128 keys on the tensor cores.
//
//   S = Q K^T (fp32, tensor memory);  p = 2^(c (S - m)) with the running reference m;
//   l = sum p;  O += P V;  out = O / l,                  c = scale log2(e)
//
// The rows of a tile are the (query, head) pairs that share a key head, query-major, so a group of
// G heads reads its keys once.  One CTA takes one row tile (cache, or heads wider than 128) or two, and a
// range of key tiles: the whole sequence, or one of `splits` parts, whose O, m and l are joined in the
// shared memory of a cluster (up to 8 parts of 16 KB) or through the workspace (attention_join.cu).
//
// Roles: eight warps per row tile own half a row a thread (64 keys; the halves exchange their maxima):
// scores from tensor memory, softmax, P back to tensor memory as the A operand of P V, where it
// overwrites scores.  The next warp issues the MMAs, the last brings K and V through a ring of 16 KB
// chunks by TMA (a K chunk is 128 keys x 64 elements, a V chunk all elements of 16384 / (2 DP) keys: both
// are what one step of the MMA loop eats).  Tensor memory holds the row tiles' O (256 columns) and two
// score tiles.  Two row tiles read each chunk of K and V once, and one's products run under the other's
// softmax.  One row tile uses the score tiles in turn: Q K^T of the next keys runs under the softmax of these.
// (8 x 2048 queries of 16 heads over 4096 keys of 4 heads of 128: 650 us with two CTAs per SM of one row tile
// each and a row a thread, 551 with one CTA of two row tiles and half a row a thread, 541 with scores and sums in
// fp32 pairs.  A tile's chain of softmax (2600 cycles) and products (1800) is what it waits for then: the matrix
// and the exponential units are both busy 47 % of the time.  These are nine calls in a row from an idle GPU, at
// 1965 MHz; without a pause the power limit takes the clock to 1760 MHz, and a call 597-606 us.)
//
// O is rescaled only where the row maximum outgrew the reference by more than 2^8 (the weights
// stay below 2^8, l and O are fp32; the final division cancels the reference).
//
// Cache: seven warps take TMA's place: they load codes and scales, several pieces ahead, and write
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
    static constexpr int kTiles = !CACHED && DP <= 128 ? 2 : 1;  // row tiles of a CTA
    static constexpr int kSoftmax = 8 * kTiles;              // warps; then the MMA warp, then the producers
    static constexpr int kThreads = 32 * (kSoftmax + 1 + (CACHED ? kDequant : 1));
    static constexpr int kVC = DP / 64;                      // V chunks of a key tile
    static constexpr int kKeysPerV = 128 / kVC;              // keys of a V chunk
    static constexpr int kRing = kTiles == 2 && DP == 128 ? 9 : 10;  // chunks
    static constexpr int kQTile = 128 * DP * 2;
    static constexpr int kOffRing = kTiles * kQTile;
    static constexpr int kOffBar = kOffRing + kRing * kChunk;
    // full[kRing], empty[kRing], s_full[2], p_ready[2], o_done[2], all_done, q_ready
    static constexpr int kOffMisc = kOffBar + (2 * kRing + 8) * 8;
    static constexpr int kOffMax = kOffMisc + 16;            // exchanged: [parity][half][row]
    static constexpr int kOffRow = kOffMax + kTiles * 2048;  // cache: a score factor per row
    static constexpr int kSmem = kOffRow + (CACHED ? 512 : 0);
    // O of the row tiles (128 or 256 columns in all), then two score tiles
    static constexpr int kTmemCols = 512, kColS = 256;
    // a row on its way out, padded so that the rows of a warp's lanes lie on different banks
    static constexpr int kOutPitch = DP * 4 + 16;
    static_assert(kTiles * 128 * kOutPitch <= kRing * kChunk, "staging of the output rows in the ring");
    static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Ring positions of a key tile's first K and V chunk.  The MMA loop's order is K0 V0 K1 V1 ... with two
// row tiles, K0 K1 V0 K2 V1 ... with one (whose two score tiles then take turns).
__device__ __forceinline__ int k_pos(bool two, int i, int kc, int vc) {
    return two ? i * (kc + vc) : i == 0 ? 0 : kc + (i - 1) * (kc + vc);
}
__device__ __forceinline__ int v_pos(bool two, int i, int n, int kc, int vc) {
    return two ? i * (kc + vc) + kc : i < n - 1 ? 2 * kc + i * (kc + vc) : n * kc + i * vc;
}

// Cache: a dequantizing warp's piece of a chunk is 32 rows (keys) of one 64-element block: per lane
// 32 bytes of codes and 4 scale bytes (zeros for keys that are left out and elements past D).
struct Codes {
    uint32_t w[8], s;
    int at;  // where it goes: byte offset of the 64-element block in its chunk
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
__global__ void __launch_bounds__(Cfg<DP, CACHED>::kThreads, 1)
    attention_tiles_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                           const AttnArgs p) {
    using C = Cfg<DP, CACHED>;
    extern __shared__ __align__(1024) uint8_t smem[];  // 128-byte swizzle atoms
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_full = sbase + C::kOffBar, bar_empty = bar_full + 8 * C::kRing;
    const uint32_t bar_s = bar_empty + 8 * C::kRing, bar_p = bar_s + 16, bar_o = bar_p + 16;
    const uint32_t bar_all = bar_o + 16, bar_q = bar_all + 8;
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + C::kOffMisc);  // TMEM base, abort
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    float *row_factor = reinterpret_cast<float *>(smem + C::kOffRow);
    float *maxima = reinterpret_cast<float *>(smem + C::kOffMax);
    float4 *part_ml = reinterpret_cast<float4 *>(smem);  // in a cluster, where Q was: as in p.part_ml
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the CTA's place: split fastest, then row tile, key head, sequence
    int rest = static_cast<int>(blockIdx.x);
    const int split = rest % p.splits;
    rest /= p.splits;
    const int rows = p.T * p.G;
    const int row_tiles = (rows + 128 * C::kTiles - 1) / (128 * C::kTiles);
    const int row0 = (rest % row_tiles) * (128 * C::kTiles);
    rest /= row_tiles;
    const bool two = C::kTiles == 2 && row0 + 128 < rows;  // both row tiles have rows
    const int hk = rest % p.Hkv, b = rest / p.Hkv;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(bar_full + 8 * i, CACHED ? 4 : 1);
            mbar_init(bar_empty + 8 * i, 1);
        }
        mbar_init(bar_s, 1);
        mbar_init(bar_s + 8, 1);
        mbar_init(bar_p, 8);
        mbar_init(bar_p + 8, 8);
        mbar_init(bar_o, 1);
        mbar_init(bar_o + 8, 1);
        mbar_init(bar_all, 1);
        mbar_init(bar_q, two ? 512 : 256);
        misc[1] = 0;
        fence_mbar_init();
    }
    if (warp == C::kSoftmax) {
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

    // Cache: the chunks' pieces in the order of the ring, in turn to the dequantizing warps
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
        Codes got = load_codes(f.is_v ? p.cache.v : p.cache.k, plane + j, f.e0, p.D, on);
        got.at = f.at;
        return got;
    };
    Codes codes[CACHED ? kAhead : 1];
    const int x0 = warp - C::kSoftmax - 1;
    if (CACHED && warp > C::kSoftmax) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) codes[CACHED ? i : 0] = fetch(x0 + i * kDequant);
    }
    if (CACHED && warp > C::kSoftmax) {
        // ------------------------------ dequantizers ------------------------------
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
                        store_f16(smem + C::kOffRing + slot * kChunk + codes[CACHED ? i : 0].at, lane, codes[CACHED ? i : 0]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_full + 8 * slot);
                    }
                    codes[CACHED ? i : 0] = fetch(y + kAhead * kDequant);
                }
            }
        }
    } else if (warp > C::kSoftmax) {
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
                if (!two && i + 1 < n) load_k(i + 1);
                load_v(i);
                if (two && i + 1 < n) load_k(i + 1);
            }
            // leave no copy in flight behind
            int dummy = 0;
            for (int q = max(0, pos - C::kRing); q < pos; ++q)
                mbar_wait(bar_full + 8 * (q % C::kRing), (q / C::kRing) & 1, &dummy, p.status, kStatusTimeoutDrain);
        }
    } else if (warp == C::kSoftmax) {
        if (n > 0 && elect_one()) {
            // ------------------------------ MMA issuer ------------------------------
            constexpr uint32_t idesc_s = idesc_f16(128, 128, !CACHED, false);
            const uint32_t idesc_o = idesc_f16(128, (p.D + 15) & ~15, !CACHED, true);
            const int ksteps = (p.D + 15) >> 4;
            bool ok = mbar_wait(bar_q, 0, abort_flag, p.status, kStatusTimeoutFull);
            auto chunk = [&](int pos) { return sbase + C::kOffRing + (pos % C::kRing) * kChunk; };
            auto full = [&](int pos) {
                ok = ok && mbar_wait(bar_full + 8 * (pos % C::kRing), (pos / C::kRing) & 1, abort_flag, p.status,
                                     kStatusTimeoutFull);
                tc_fence_after();
            };
            // With two row tiles the first waits for a chunk, the second gives it back.
            auto qk = [&](int tile, int i) {
                const int pos = k_pos(two, i, kc, vc), buf = two ? tile : i & 1;
                const uint32_t d = tmem + C::kColS + buf * 128;
                uint32_t on = 0u;
                for (int c = 0; c < kc && ok; ++c) {
                    if (tile == 0) full(pos + c);
                    if (!ok) break;
                    // a step of 16 elements is 32 bytes on: 2 in the descriptors' address field
                    const uint64_t qd = desc_kmajor_sw128(sbase + tile * C::kQTile + c * kChunk),
                                   kd = desc_kmajor_sw128(chunk(pos + c));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (4 * c + k < ksteps) {
                            tc_mma_f16_ss(d, qd + 2 * k, kd + 2 * k, idesc_s, on);
                            on = 1u;
                        }
                    if (!two || tile == 1) tc_commit(bar_empty + 8 * ((pos + c) % C::kRing));
                }
                tc_commit(bar_s + 8 * buf);
            };
            auto pv = [&](int tile, int i) {
                const int buf = two ? tile : i & 1, pos = v_pos(two, i, n, kc, vc);
                ok = ok && mbar_wait(bar_p + 8 * buf, (two ? i : i >> 1) & 1, abort_flag, p.status,
                                     kStatusTimeoutSoftmax);
                if (!ok) return;
                tc_fence_after();
                const uint32_t pt = tmem + C::kColS + buf * 128;
                uint32_t on = i > 0 ? 1u : 0u;
#pragma unroll
                for (int c = 0; c < vc; ++c) {
                    if (tile == 0) full(pos + c);
                    if (!ok) break;
                    const uint64_t vd = desc_mnmajor_sw128(chunk(pos + c), C::kKeysPerV * 128);
                    constexpr int steps = C::kKeysPerV / 16;
#pragma unroll
                    for (int k = 0; k < steps; ++k) {  // 16 keys: 2048 bytes of V, 8 columns of P
                        tc_mma_f16_ts(tmem + tile * 128, pt + 8 * (c * steps + k), vd + 128 * k, idesc_o, on);
                        on = 1u;
                    }
                    if (!two || tile == 1) tc_commit(bar_empty + 8 * ((pos + c) % C::kRing));
                }
                if (i + 1 < n) tc_commit(bar_o + 8 * tile);
                else if (!two || tile == 1) tc_commit(bar_all);
            };
            qk(0, 0);
            if (two) qk(1, 0);
            for (int i = 0; i < n && ok; ++i) {
                if (!two && i + 1 < n) qk(0, i + 1);
                pv(0, i);
                if (two) {
                    if (i + 1 < n) qk(0, i + 1);
                    pv(1, i);
                    if (i + 1 < n) qk(1, i + 1);
                }
            }
        }
    } else {
        // ------------------------------ Q ------------------------------
        // rows into K-major swizzled tiles (zeros past D and past the last row)
        if constexpr (CACHED) if (n > 0) {
            // bf16 -> fp16 (while the other warps decode the first keys), a row times the power of two that
            // brings its largest element to [2^14, 2^15) (what falls below fp16's range is 2^-39 of that
            // element); the inverse goes into the row's score factor.  kUnits lanes a row, several rows in flight.
            constexpr int kUnits = DP / 8, kStep = 256 / kUnits, kBatch = 128 / kStep < 8 ? 128 / kStep : 8;
            const int c = threadIdx.x % kUnits, r0 = threadIdx.x / kUnits;
            const uint16_t *base = p.q.ptr + b * p.q.sb + static_cast<long long>(hk) * p.G * p.q.sh + 8 * c;
            static_assert(128 % (kBatch * kStep) == 0 && kBatch % 2 == 0, "whole batches");
            const int dt = kStep / p.G, dg = kStep - dt * p.G;
            int t = (row0 + r0) / p.G, g = row0 + r0 - t * p.G;
            for (int rb = r0; rb < 128; rb += kBatch * kStep) {
                uint4 v[kBatch];
                uint32_t top[kBatch];  // magnitudes as bf16 bits, which order as integers
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int row = row0 + rb + i * kStep;
                    v[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (row < rows && 8 * c < p.D)
                        v[i] = __ldcg(reinterpret_cast<const uint4 *>(base + t * p.q.st + g * p.q.sh));
                    t += dt;
                    g += dg;
                    if (g >= p.G) {
                        g -= p.G;
                        ++t;
                    }
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const uint32_t m2 = __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                                 __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
                    top[i] = max(m2 & 0xFFFFu, m2 >> 16);
                }
#pragma unroll
                for (int i = 0; i < kBatch; i += 2) {  // two rows a shuffle
                    uint32_t two = top[i] | (top[i + 1] << 16);
#pragma unroll
                    for (int d = kUnits / 2; d > 0; d >>= 1) two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, d));
                    top[i] = two << 16;
                    top[i + 1] = two & 0xFFFF0000u;
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int r = rb + i * kStep;
                    float down;
                    const float up = f16_row_factor(__uint_as_float(top[i]), &down);
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[k] = pack_f16x2(bf16lo(w[k]) * up, bf16hi(w[k]) * up);
                    *reinterpret_cast<uint4 *>(smem + (c >> 3) * kChunk + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                    if (c == 0) row_factor[r] = down;
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(bar_q);
            mbar_wait(bar_q, 0, abort_flag, p.status, kStatusTimeoutFull);  // the row factors
            __syncwarp();
        }
        const int tile = warp >> 3;
        if (!CACHED && n > 0 && (tile == 0 || two)) {
            constexpr int kUnits = DP / 8, kStep = 256 / kUnits;  // rows of a pass of the tile's 256 threads
            const int c = threadIdx.x % kUnits, r0 = (threadIdx.x & 255) / kUnits;
            const int first = row0 + 128 * tile;
            const uint16_t *base = p.q.ptr + b * p.q.sb + static_cast<long long>(hk) * p.G * p.q.sh + 8 * c;
            // row -> (query, head of the group), stepped without a division
            const int dt = kStep / p.G, dg = kStep - dt * p.G;
            int t = (first + r0) / p.G, g = first + r0 - t * p.G;
#pragma unroll
            for (int r = r0; r < 128; r += kStep) {
                const bool in = first + r < rows && 8 * c < p.D;
                cp_async16(sbase + tile * C::kQTile + (c >> 3) * kChunk + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           in ? base + t * p.q.st + g * p.q.sh : p.q.ptr, in ? 16u : 0u);
                t += dt;
                g += dg;
                if (g >= p.G) {
                    g -= p.G;
                    ++t;
                }
            }
            cp_async_wait_all();
            fence_proxy_async_smem();
            mbar_arrive(bar_q);
        }

        // ------------------------------ softmax, half a row a thread ------------------------------
        const int quarter = warp & 3, half = (warp >> 2) & 1;  // rows 32 * quarter + lane; keys 64 * half + 0 .. 63
        const int row = quarter * 32 + lane, first = row0 + 128 * tile;
        const bool warp_on = first + quarter * 32 < rows;  // some row of this warp exists
        const int tiles = tile == 0 || two ? n : 0;  // key tiles of this row tile
        float *const places = maxima + tile * 512;
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t o_base = lane_base + tile * 128;
        const float c = CACHED && n > 0 ? score_factor(p.scale_log2, row_factor[row]) : p.scale_log2;
        // The two warps of the same rows meet (each as often as the other: no wait that gave up skips a meeting,
        // so this one needs no limit of its own), and the other half's value at the i-th meeting (a place per
        // half and parity of i: no half can be two meetings ahead).
        auto meet = [&]() {
            __syncwarp();
            asm volatile("bar.sync %0, 64;" ::"r"(1 + 4 * tile + quarter) : "memory");
        };
        auto exchange = [&](float v, int i) {
            float *ex = places + (i & 1) * 256 + row;
            ex[half * 128] = v;
            meet();
            return ex[(half ^ 1) * 128];
        };
        float m = -INFINITY, l = 0.0f;
        for (int i = 0; i < tiles; ++i) {
            const int sb = two ? tile : i & 1;  // score tile
            // (a wait that gave up leaves no warp behind at a meeting: the loop goes on, and every later wait
            // sees the abort flag)
            mbar_wait(bar_s + 8 * sb, (two ? i : i >> 1) & 1, abort_flag, p.status, kStatusTimeoutAccum);
            __syncwarp();
            tc_fence_after();
            const int j0 = (tile0 + i) << 7;
            const bool part = p.mask != nullptr || j0 + 128 > len;
            uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
            if (part) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int j = j0 + 64 * half + 32 * w + lane;
                    bool in = j < len;
                    if (in && p.mask != nullptr) in = __ldcg(p.mask + b * p.mask_stride + j) != 0;
                    keep[w] = __ballot_sync(0xffffffffu, in);
                }
            }
            if (warp_on) {
                const uint32_t buf = lane_base + C::kColS + sb * 128;
                uint32_t s[2][32];
                tmem_ld_32x32b_x32(buf + 64 * half, s[0]);
                tmem_ld_32x32b_x32(buf + 64 * half + 32, s[1]);
                tmem_ld_wait();
                if (part) {
#pragma unroll
                    for (int w = 0; w < 2; ++w)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (((keep[w] >> j) & 1u) == 0u) s[w][j] = 0xFF800000u;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(s[w][j]));
                // the row's maximum over both halves (which also orders the other half's reads of its scores
                // before this half's weights overwrite some of them)
                const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const float top = fmaxf(mine, exchange(mine, i));
                // the reference: the first maximum, then only one that outgrew it
                const bool grow = top > m && !((top - m) * c <= kLazy);
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2((m - top) * c) : 1.0f;
                    if (grow) m = top;
                    if (i > 0) {
                        mbar_wait(bar_o + 8 * tile, (i - 1) & 1, abort_flag, p.status, kStatusTimeoutAccum);
                        __syncwarp();
                        tc_fence_after();
                        l *= f;
                        for (int e = 16 * half; e < p.D; e += 32) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(o_base + e, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st_32x32b_x16(o_base + e, o);
                        }
                    }
                }
                // (s - m) c, not s c - m c: the rounding of a large m c would shift every weight of the row, by a
                // factor beyond fp16 or fp32 from |m c| of 2^27 on
                const float ref = m == -INFINITY ? 0.0f : m;
                const uint64_t c2 = pair(c, c), shift = pair(-ref, -ref), up = pair(kF16WeightBits, kF16WeightBits);
                uint64_t sum[2] = {};
                uint32_t pk[32];
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const uint64_t d = add2(pair(__uint_as_float(s[w][j]), __uint_as_float(s[w][j + 1])), shift);
                        const float2 e = halves(CACHED ? fma2(d, c2, up) : mul2(d, c2));
                        const float x = ex2(e.x), y = ex2(e.y);
                        sum[w] = add2(sum[w], pair(x, y));
                        pk[16 * w + j / 2] = CACHED ? pack_f16x2(x, y) : pack_bf16x2_rn(x, y);
                    }
                tmem_st_32x32b_x32(buf + 32 * half, pk);
                const float2 l0 = halves(sum[0]), l1 = halves(sum[1]);
                l += (l0.x + l0.y) + (l1.x + l1.y);
                tmem_st_wait();
            }
            if (part && !CACHED && tile == 0) {
                // a thread's key row of V (this half's keys, 64 of them): zeros if the key is left out.  Once
                // the previous product is done every chunk before V's has landed, so the phase waited for is V's own.
                const int key = 64 * half + 32 * (quarter & 1) + lane;
                if (quarter < 2 && ((keep[quarter & 1] >> lane) & 1u) == 0u) {
                    if (i > 0) mbar_wait(bar_o, (i - 1) & 1, abort_flag, p.status, kStatusTimeoutAccum);
                    const int pos = v_pos(two, i, n, kc, vc) + key / C::kKeysPerV;
                    mbar_wait(bar_full + 8 * (pos % C::kRing), (pos / C::kRing) & 1, abort_flag,
                                         p.status, kStatusTimeoutFull);
                    uint8_t *v = smem + C::kOffRing + (pos % C::kRing) * kChunk + (key % C::kKeysPerV) * 128;
                    for (int e = 0; e < kc; ++e)
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            *reinterpret_cast<uint4 *>(v + e * C::kKeysPerV * 128 + ((q ^ (lane & 7)) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                }
                __syncwarp();
            }
            tc_fence_before();
            // one barrier per score tile: a warp may be a tile ahead of another
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_p + 8 * sb);
        }

        // ------------------------------ output ------------------------------
        // (of both row tiles, as the ring is used for the way out; on a barrier of its own: the product before
        // the last may still be running, or have been done long ago)
        if (tiles > 0) mbar_wait(bar_all, 0, abort_flag, p.status, kStatusTimeoutAccum);
        __syncwarp();
        tc_fence_after();
        if (warp_on) {
            // the row's sum of weights
            const float o = exchange(l, n);
            l = half == 0 ? l + o : o + l;  // the same sum in both
            // (cluster, or no parts) rows into shared memory (the ring is idle now): stored from here, a thread's
            // own row, an instruction would touch 32 lines
            const float f = l != 0.0f ? (CACHED ? p.cache.v.g : 1.0f) / l : 0.0f;
            const int live = min(32, rows - first - quarter * 32);
            const int pitch = p.D * (p.splits > 1 ? 4 : 2) + 16;
            uint8_t *st = smem + C::kOffRing + (tile * 4 + quarter) * 32 * C::kOutPitch + lane * pitch;
            if (p.splits > 1) {
                // through the workspace: four columns of adjacent rows are adjacent, so a warp's store is 512 bytes
                // in a row as it comes out of tensor memory
                const int pr = p.part_rows();
                const size_t part = ((static_cast<size_t>(b) * p.Hkv + hk) * p.row_tiles() + (first >> 7)) * p.splits + split;
                float4 *to = reinterpret_cast<float4 *>(p.part_o) + part * (p.D >> 2) * pr + row;
                if (half == 0 && p.cluster) part_ml[first - row0 + row] = make_float4(m, l, c, 0.0f);
                else if (half == 0 && lane < live) p.part_ml[part * pr + row] = make_float4(m, l, c, 0.0f);
                for (int e = 32 * half; e < p.D && n > 0; e += 64) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(o_base + e, o);
                    tmem_ld_wait();
                    if (!p.cluster) {
                        if (lane < live && *abort_flag == 0) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (e + 4 * j < p.D)
                                    to[static_cast<size_t>(e / 4 + j) * pr] =
                                        make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                                    __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
                        }
                        __syncwarp();
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (e + 4 * j < p.D)
                            *reinterpret_cast<uint4 *>(st + (e + 4 * j) * 4) =
                                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
            } else {
                for (int e = 32 * half; e < p.D; e += 64) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(o_base + e, o);
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
                        if (e + 8 * j < p.D)
                            *reinterpret_cast<uint4 *>(st + (e + 8 * j) * 2) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            // and from there a row by one bulk copy (16 rows a warp)
            if (p.splits == 1) {
                fence_proxy_async_smem();
                meet();
                if (lane / 16 == half && lane < live && *abort_flag == 0) {
                    const int t = (first + row) / p.G, g = first + row - t * p.G;
                    bulk_store(p.out.ptr + b * p.out.sb + t * p.out.st + (static_cast<long long>(hk) * p.G + g) * p.out.sh,
                               smem_u32(st), p.D * 2);
                    bulk_store_wait();
                }
            }
        }
    }

    __syncwarp();
    if (p.cluster) {
        // The parts of a row tile are the CTAs of a cluster: each joins its share of the rows out of all parts'
        // shared memory, 8 columns a thread, all loads in flight together.  (Few bytes a part only: remote
        // reads ran at 4-8 bytes a cycle.)
        cluster_sync_all();
        const int share = (128 * C::kTiles + p.splits - 1) / p.splits, units = p.D >> 3;
        const int r0 = split * share, r1 = min(min(r0 + share, 128 * C::kTiles), rows - row0);
        for (int x = threadIdx.x; x < (r1 - r0) * units; x += C::kThreads) {
            const int r = r0 + x / units, e = x % units * 8;
            const uint32_t ml = smem_u32(part_ml + r);
            const uint32_t at = sbase + C::kOffRing + (r >> 5) * 32 * C::kOutPitch + (r & 31) * (p.D * 4 + 16) + e * 4;
            float2 part[kAttentionCluster];
            float4 y0[kAttentionCluster], y1[kAttentionCluster];
            // (the first part has keys if any has, and so the row's factor)
            float M = -INFINITY;
            const float c = CACHED ? ld_dsmem_f2(mapa_shared(ml + 8, 0)).x : p.scale_log2;
#pragma unroll
            for (int q = 0; q < kAttentionCluster; ++q) {
                part[q] = make_float2(-INFINITY, 0.0f);
                if (q < p.splits) {
                    part[q] = ld_dsmem_f2(mapa_shared(ml, q));
                    y0[q] = ld_dsmem_f4(mapa_shared(at, q));
                    y1[q] = ld_dsmem_f4(mapa_shared(at + 16, q));
                }
            }
#pragma unroll
            for (int q = 0; q < kAttentionCluster; ++q)
                if (part[q].y != 0.0f) M = fmaxf(M, part[q].x);
            float sum = 0.0f, o[8] = {};
#pragma unroll
            for (int q = 0; q < kAttentionCluster; ++q)
                if (part[q].y != 0.0f) {  // a part without keys holds nothing
                    const float f = ex2((part[q].x - M) * c);
                    sum = fmaf(f, part[q].y, sum);
                    const float y[8] = {y0[q].x, y0[q].y, y0[q].z, y0[q].w, y1[q].x, y1[q].y, y1[q].z, y1[q].w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = fmaf(f, y[k], o[k]);
                }
            const float f = sum != 0.0f ? (CACHED ? p.cache.v.g : 1.0f) / sum : 0.0f;
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2_rn(o[2 * k] * f, o[2 * k + 1] * f);
            const int t = (row0 + r) / p.G, g = row0 + r - t * p.G;
            *reinterpret_cast<uint4 *>(p.out.ptr + b * p.out.sb + t * p.out.st +
                                       (static_cast<long long>(hk) * p.G + g) * p.out.sh + e) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
        cluster_sync_all();  // no CTA leaves while its memory is read
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
    if (warp == C::kSoftmax) {
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
    const long long tiles = (static_cast<long long>(a.T) * a.G + 128 * C::kTiles - 1) / (128 * C::kTiles);
    const long long ctas = tiles * a.B * a.Hkv * a.splits;
    if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int attrs = 0;
    if (pdl_enabled()) {
        attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[attrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (a.cluster) {
        attr[attrs].id = cudaLaunchAttributeClusterDimension;
        attr[attrs].val.clusterDim.x = static_cast<unsigned>(a.splits);
        attr[attrs].val.clusterDim.y = 1;
        attr[attrs++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = attrs;
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
