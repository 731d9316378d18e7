// attn_tiles.cuh -- which query rows a CTA of the prompt kernels works on.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace gbe {

// A tile of consecutive query rows of one packed sequence.
struct SeqTile {
    int begin;   // the sequence's first row in the packed buffers
    int len;     // its length
    int row;     // the tile's first row within the sequence; < 0: no such tile
};

// Tile `index` of the packed sequences cut into tiles of M rows, counted from
// the last sequence's last tile, so that under a causal mask the tiles with
// the most keys are handed out first.  Sequence b holds rows starts[b] ..
// starts[b + 1] - 1; starts are brought into [0, T] and a sequence that would
// end before it begins is empty, so no row outside the buffers is reached
// whatever starts holds.  Run by one whole warp.
__device__ __forceinline__ SeqTile find_tile(const int32_t* starts, int n_seqs, int T, int M, uint32_t index) {
    const int lane = threadIdx.x & 31;
    SeqTile r = {0, 0, -1};
    uint32_t before = 0;  // tiles of the sequences behind the ones looked at
    for (int top = n_seqs; top > 0; top -= 32) {
        const int b = top - 1 - lane;
        int s = 0, n = 0;
        if (b >= 0) {
            s = min(max(starts[b], 0), T);
            n = max(min(max(starts[b + 1], 0), T) - s, 0);
        }
        const uint32_t tiles = (uint32_t)((n + M - 1) / M);
        uint32_t sum = tiles;  // inclusive scan over the lanes
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, sum, x);
            if (lane >= x) sum += y;
        }
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, index < before + sum);
        if (hit) {
            const int who = __ffs((int)hit) - 1;
            const uint32_t upto = __shfl_sync(0xFFFFFFFFu, before + sum, who);
            r.begin = __shfl_sync(0xFFFFFFFFu, s, who);
            r.len = __shfl_sync(0xFFFFFFFFu, n, who);
            r.row = (int)(upto - 1 - index) * M;  // index counts from the sequence's last tile
            return r;
        }
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    return r;
}

}  // namespace gbe
