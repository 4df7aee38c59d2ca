// attention_share.cuh — which steps of 16 keys a CTA of the row kernel takes, and which parts the kernel
// that joins them finds.
//
// With p.share = 0 a CTA takes a whole segment (a key head of a sequence).  Else the p.share CTAs, more than
// there are segments, are dealt out by the lengths on the device: a piece is at most `piece` steps, the least
// with which all segments' pieces fit the CTAs, so uneven lengths keep all SMs at work; no CTA has more than one
// segment.  The pieces are numbered along the segments: a CTA's number is its part's place in the workspace.
#pragma once

#include "attention.h"

namespace nvfp4 {

__device__ __forceinline__ int key_steps(const AttnArgs &p, int b, int *len) {
    *len = p.S;
    if (p.kv_len != nullptr) *len = min(max(__ldcg(p.kv_len + b), 0), p.S);
    return (*len + 15) >> 4;
}
// Sums over the sequences [0, b) of f(steps); the whole warp, b uniform.
template <class F>
__device__ __forceinline__ long long key_sum(const AttnArgs &p, int b, F f) {
    int len;
    if (p.kv_len == nullptr) return b > 0 ? static_cast<long long>(b) * f(key_steps(p, 0, &len)) : 0;
    long long s = 0;
    for (int i = threadIdx.x & 31; i < b; i += 32) s += f(key_steps(p, i, &len));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
}
// Steps of a piece: sum over segments of ceil(steps / piece) <= total / piece + segments <= p.share; a piece
// has a step for each of the CTA's `warps` at least.
__device__ __forceinline__ int key_piece(const AttnArgs &p) {
    const long long total = key_sum(p, p.B, [](int n) { return n; }) * p.Hkv;
    const long long free = p.share - static_cast<long long>(p.B) * p.Hkv;
    return static_cast<int>(max((total + free - 1) / free, static_cast<long long>(p.warps)));
}
// The first piece of segment (b, hk).
__device__ __forceinline__ int first_piece(const AttnArgs &p, int b, int hk, int piece, int steps) {
    const auto pieces = [=](int n) { return (n + piece - 1) / piece; };
    return static_cast<int>(key_sum(p, b, pieces) * p.Hkv) + hk * pieces(steps);
}

struct KeyRange {
    int b, hk, len, step0, step1;
};

// This CTA's steps; the whole warp.  False: a CTA without any (then its part is of no segment).
__device__ __forceinline__ bool key_range(const AttnArgs &p, KeyRange &x) {
    const int c = static_cast<int>(blockIdx.x);
    if (p.share == 0) {
        x.b = c / p.Hkv;
        x.hk = c - x.b * p.Hkv;
        x.step0 = 0;
        x.step1 = key_steps(p, x.b, &x.len);
        return true;
    }
    const int piece = key_piece(p), lane = threadIdx.x & 31;
    // the sequence: 32 at a time, the first whose pieces reach beyond c
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        int len = 0, steps = 0;
        if (b0 + lane < p.B) steps = key_steps(p, b0 + lane, &len);
        const int mine = (steps + piece - 1) / piece * p.Hkv;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        const uint32_t holds = __ballot_sync(0xffffffffu, c < before + upto);
        if (holds != 0u) {
            const int l = __ffs(static_cast<int>(holds)) - 1;
            const int at = c - before - __shfl_sync(0xffffffffu, upto - mine, l);
            const int each = __shfl_sync(0xffffffffu, mine, l) / p.Hkv;
            steps = __shfl_sync(0xffffffffu, steps, l);
            x.len = __shfl_sync(0xffffffffu, len, l);
            x.b = b0 + l;
            x.hk = at / each;
            const int size = (steps + each - 1) / each;  // the segment's pieces alike
            x.step0 = (at - x.hk * each) * size;
            x.step1 = min(x.step0 + size, steps);
            return true;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

}  // namespace nvfp4
