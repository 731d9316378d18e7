// attn_tiles.cuh -- what the prompt kernels share: which query rows a CTA works
// on, and a row computed from its own keys alone.
#pragma once

#include <stdint.h>

#include "attn_common.cuh"
#include "launch.h"

namespace gbe {

// A piece of one packed sequence.
struct SeqPiece {
    int begin;  // the sequence's first row in the packed buffers
    int len;    // its length
    int index;  // which of its pieces; < 0: no such piece
};

// Piece `index` of the packed sequences, a sequence of n rows being cut into
// count(n) pieces of which, under the causal mask, each takes longer than the
// one before.  Up to 128 sequences: the pieces are counted from the largest
// down, so that the longest work is handed out first; more: from the last
// sequence's last piece.  Sequence b holds rows starts[b] .. starts[b + 1] - 1;
// starts are brought into [0, T] and a sequence that would end before it begins
// is empty, so no row outside the buffers is reached whatever starts holds.
// Run by one whole warp.
template <typename Count>
__device__ __forceinline__ SeqPiece find_piece(const int32_t* starts, int n_seqs, int T, uint32_t index,
                                               Count count) {
    const int lane = threadIdx.x & 31;
    SeqPiece r = {0, 0, -1};
    auto sequence = [&](int b, int& s, int& n) {
        s = n = 0;
        if (b >= 0 && b < n_seqs) {
            s = min(max(starts[b], 0), T);
            n = max(min(max(starts[b + 1], 0), T) - s, 0);
        }
    };
    if (n_seqs <= 128) {
        int s[4], n[4];
        uint32_t c[4], most = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            sequence(x * 32 + lane, s[x], n[x]);
            c[x] = n[x] > 0 ? count(n[x]) : 0;
            most = max(most, c[x]);
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        auto from = [&](uint32_t level) {  // pieces that are their sequence's number `level` or a later one
            uint32_t k = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) k += c[x] > level ? c[x] - level : 0;
            return __reduce_add_sync(0xFFFFFFFFu, k);
        };
        if (index >= from(0)) return r;
        uint32_t lo = 0, hi = most;  // from(lo) > index >= from(hi)
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) / 2;
            if (from(mid) > index)
                lo = mid;
            else
                hi = mid;
        }
        uint32_t skip = index - from(lo + 1);  // of the sequences that have a piece number `lo`
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t has = __ballot_sync(0xFFFFFFFFu, c[x] > lo);
            const uint32_t k = __popc(has);
            if (r.index < 0) {
                if (skip < k) {
                    const int who = __fns(has, 0, (int)skip + 1);
                    r.begin = __shfl_sync(0xFFFFFFFFu, s[x], who);
                    r.len = __shfl_sync(0xFFFFFFFFu, n[x], who);
                    r.index = (int)lo;
                } else {
                    skip -= k;
                }
            }
        }
        return r;
    }
    // (64 bits: starts that go back and forth may name more pieces than 32 bits count)
    unsigned long long before = 0;  // pieces of the sequences behind the ones looked at
    for (int top = n_seqs; top > 0; top -= 32) {
        int s, n;
        sequence(top - 1 - lane, s, n);
        unsigned long long sum = n > 0 ? count(n) : 0;  // inclusive scan over the lanes
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xFFFFFFFFu, sum, x);
            if (lane >= x) sum += y;
        }
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, index < before + sum);
        if (hit) {
            const int who = __ffs((int)hit) - 1;
            const unsigned long long upto = __shfl_sync(0xFFFFFFFFu, before + sum, who);
            r.begin = __shfl_sync(0xFFFFFFFFu, s, who);
            r.len = __shfl_sync(0xFFFFFFFFu, n, who);
            r.index = (int)(upto - 1 - index);
            return r;
        }
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    return r;
}

// Four consecutive values, aligned to their size, widened to f32.
template <int DT>
__device__ __forceinline__ float4 load4(const void* base, int64_t i) {
    if constexpr (DT == kF32) {
        return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xFFFF0000u));
    }
}

// One row in f32 from its own keys alone, by a whole warp, for D <= 128 and rows
// on the 16-byte grid: 32 keys at a time, a lane a key for the logits, a lane
// four entries for the output.  The tensor-core kernels call it for rows that
// came out not finite, since there a weight of zero meets an infinity or a NaN
// behind the mask.
template <int DT>
__device__ __noinline__ void exact_row(const PromptArgs& a, int begin, int row, int head) {
    const int lane = threadIdx.x & 31, D = (int)a.D, kvh = head / (int)(a.Hq / a.Hkv);
    const float c = a.scale * kLog2e;
    float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f), o = q;
    if (lane * 4 < D) q = load4<DT>(a.q, (begin + (int64_t)row) * a.q_stride + (int64_t)head * D + lane * 4);
    float m = -INFINITY, l = 0.0f;
    for (int k0 = 0; k0 <= row; k0 += 32) {
        const int j = k0 + lane;
        const bool seen = j <= row;
        const int64_t k_at = (begin + (int64_t)(seen ? j : row)) * a.k_stride + (int64_t)kvh * D;
        float s = 0.0f;
        for (int d = 0; d < D; d += 4) {
            const float4 k = load4<DT>(a.k, k_at + d);
            s = fmaf(__shfl_sync(0xFFFFFFFFu, q.x, d >> 2), k.x, s);
            s = fmaf(__shfl_sync(0xFFFFFFFFu, q.y, d >> 2), k.y, s);
            s = fmaf(__shfl_sync(0xFFFFFFFFu, q.z, d >> 2), k.z, s);
            s = fmaf(__shfl_sync(0xFFFFFFFFu, q.w, d >> 2), k.w, s);
        }
        s *= c;
        // a NaN logit leaves a finite maximum, so that its NaN weight reaches the result
        float mx = seen ? fmaxf(m, s == s ? s : -3.0e38f) : m;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
        const float r = m == -INFINITY ? 0.0f : ex2(m - mx);
        const float p = !seen || s == -INFINITY ? 0.0f : ex2(s - mx);
        m = mx;
        float sum = p;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        l = fmaf(l, r, sum);
        o.x *= r, o.y *= r, o.z *= r, o.w *= r;
        const int keys = min(32, row + 1 - k0);
        for (int t = 0; t < keys; ++t) {
            const float w = __shfl_sync(0xFFFFFFFFu, p, t);
            if (lane * 4 < D) {
                const float4 v =
                    load4<DT>(a.v, (begin + (int64_t)k0 + t) * a.v_stride + (int64_t)kvh * D + lane * 4);
                o.x = fmaf(w, v.x, o.x);
                o.y = fmaf(w, v.y, o.y);
                o.z = fmaf(w, v.z, o.z);
                o.w = fmaf(w, v.w, o.w);
            }
        }
    }
    if (lane * 4 < D) {
        const float y[4] = {o.x, o.y, o.z, o.w};
        const int64_t at = (begin + (int64_t)row) * a.out_stride + (int64_t)head * D + lane * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) Store<DT>::store1(a.out, at + e, m == -INFINITY ? 0.0f : y[e] / l);
    }
}

}  // namespace gbe
