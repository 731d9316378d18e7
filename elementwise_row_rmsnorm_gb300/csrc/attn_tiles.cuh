// attn_tiles.cuh -- which query rows a CTA of the prompt kernels works on.
#pragma once

#include <stdint.h>

#include "attn_common.cuh"

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
                if (skip < k) {  // the lane that has one and `skip` such lanes before it
                    const bool it = c[x] > lo && __popc(has & ((1u << lane) - 1u)) == (int)skip;
                    const int who = __ffs((int)__ballot_sync(0xFFFFFFFFu, it)) - 1;
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

}  // namespace gbe
