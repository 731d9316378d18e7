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
// down, so that the longest work is handed out first.  More: sequence b, which
// begins at row s, has the indexes from first(s, min(b, s)) on, so that it is
// found by a search over b, 32 places at a time, five steps for 2^24 sequences.
// min(b, s) is no less than the number of sequences before b that are not empty,
// and first has to grow by count(n) at least with n rows and one more of these.
// Indexes between are of no piece, which leaves some CTAs with more work than
// others; counted step by step, as long as there are sequences, all would have a
// piece (bf16, 32 heads of 128: 200 prompts of up to 100 tokens 107 us, counted
// 104; 300 of up to 300 311 and 341 us, 1000 of up to 30 462 and 798 us, 4000 of
// up to 8 1.7 and 8.4 ms; both at once in one kernel cost 2 to 4 % of either).
// Sequence b holds rows starts[b] .. starts[b + 1] - 1; starts are brought into
// [0, T] and a sequence that would end before it begins is empty, so no row
// outside the buffers is reached whatever starts holds.  Run by one whole warp.
template <typename Count, typename First>
__device__ __forceinline__ SeqPiece find_piece(const int32_t* starts, int n_seqs, int T, uint32_t index, Count count,
                                               First first) {
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
    int lo = 0, hi = n_seqs;  // the last sequence whose indexes begin at `index` or before is one of these
    for (bool begun = false; !begun || hi - lo > 1; begun = true) {
        const int step = (hi - lo + 31) / 32, b = lo + lane * step;
        bool before = false;
        if (b < hi) {
            const int s = min(max(starts[b], 0), T);
            before = first((uint32_t)s, (uint32_t)min(b, s)) <= index;
        }
        const uint32_t set = __ballot_sync(0xFFFFFFFFu, before);
        if (set == 0) return r;
        lo += (31 - __clz((int)set)) * step;
        hi = min(hi, lo + step);
    }
    int s, n;
    sequence(lo, s, n);
    const uint32_t pieces = n > 0 ? count(n) : 0, at = index - first((uint32_t)s, (uint32_t)min(lo, s));
    if (at < pieces) r = {s, n, (int)(pieces - 1 - at)};
    return r;
}

}  // namespace gbe
