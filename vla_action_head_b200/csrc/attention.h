// attention.h — internal interface between the C ABI (api.cu) and the attention-side kernels
// (qk_norm_rope.cu, kv_cache.cu, attention_*.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace nvfp4 {

// A bf16 [B, T, H, D] view (strides in elements).
struct Heads {
    uint16_t *ptr;
    long long sb, st, sh;
};

// Exact division of 32-bit numbers below 2^31 by a fixed divisor: a multiplication and shifts.
struct FastDiv {
    uint32_t d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t n) : d(n), mul(0), shift(0) {
        while (shift < 32 && (1ull << shift) < n) ++shift;
        mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - n)) / n + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
#endif
};

// The two planes of an NVFP4 cache tensor: codes [B, H, C, D/2], scales [B, H, C, D/16].
struct CachePlane {
    uint8_t *codes, *sf;
    float g;
};
struct Cache {
    CachePlane k, v;
    int H, C, length;
};

struct QkArgs {
    int B, T, Hq, Hkv, D, R;
    int inter;  // pairs (2i, 2i + 1) instead of (i, i + R/2)
    int norm;
    float eps;
    Heads q, k, v, q_out, k_out;
    const uint16_t *q_gamma, *k_gamma;
    const float *table;
    int table_rows;
    const int *positions, *start, *count;
    int cached;
    Cache cache;
    uint32_t *status;
    int sms;                  // of the device
    FastDiv by_tokens, by_t;  // set by the launcher
    uint32_t items;          // groups of lanes: below 2^31
    double inv_d;
    float one;               // 1, which the compiler does not know
};
cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t s);

struct ReadArgs {
    int B, L, H, D;
    const int *start;
    Heads k_out, v_out;  // ptr NULL: not read
    Cache cache;
    uint32_t *status;
    FastDiv by_chunks, by_h;  // set by the launcher
};
int kv_read_rows(int D);  // rows of a CTA
cudaError_t launch_kv_read(const ReadArgs &a, cudaStream_t s);

struct AttnArgs {
    int B, T, S, Hq, Hkv, D, G;  // G = Hq / Hkv
    float scale_log2;            // scale * log2(e) (* the key cache's global scale)
    Heads q, k, v, out;
    const int *kv_len;
    const uint8_t *mask;
    long long mask_stride;
    int cached;
    Cache cache;
    int k_mul_h, k_mul_b, v_mul_h, v_mul_b;  // 0: that dimension is broadcast, its tensor-map size 1
    int splits;      // tile kernel: parts of the key range
    int cluster;     // tile kernel: 1: the parts are a cluster, which joins them; 0: from part_o and part_ml
    int share;       // row kernel: > 0: CTAs dealt out by the lengths, joined; 0: a CTA a key head
    int warps;       // row kernel: of a CTA
    // unnormalized sums; per row its reference score, its sum of weights and its score factor (one value in
    // all parts).  (Not the product of the first and the last: its rounding would weigh the parts of large scores
    // differently than a part weighs its keys.)
    // tile kernel: [key heads, row tiles, splits, D / 4, part_rows(), 4] and [.., splits, part_rows()], so that
    // rows in a warp's lanes are adjacent; row kernel: [CTAs, rows of a key head] (x D)
    float *part_o;
    float4 *part_ml;
    uint32_t *status;
    __host__ __device__ int row_tiles() const { return (T * G + 127) >> 7; }
    __host__ __device__ int part_rows() const { return T * G >= 128 ? 128 : (T * G + 31) & ~31; }
};
cudaError_t launch_attention_join(const AttnArgs &a, cudaStream_t s);
cudaError_t probe_attention();

// Tensor-core tiles of 128 rows x 128 keys; maps over k and v [d, head, key, sequence] with boxes of
// 64 x 1 x 128 x 1 and 64 x 1 x attention_v_box_rows x 1 elements.
constexpr int kAttentionCluster = 8;  // parts that a cluster joins
int attention_v_box_rows(int D);
cudaError_t launch_attention_tiles(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, cudaStream_t s);
cudaError_t probe_attention_tiles();

// Up to kAttentionRows (query, head) pairs per key head, keys streamed through registers.
// Maps (steps of 16 keys): over bf16 k and v as above with boxes of 64 x 1 x 16 x 1; over a cache's
// codes [D / 2 bytes, row], a box of 16 whole rows swizzled over their span, where attention_rows_mapped.
constexpr int kAttentionRows = 8;
bool attention_rows_mapped(const AttnArgs &a);
int attention_rows_warps(bool cached, int D);
cudaError_t launch_attention_rows(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, cudaStream_t s);
cudaError_t probe_attention_rows();

}  // namespace nvfp4
