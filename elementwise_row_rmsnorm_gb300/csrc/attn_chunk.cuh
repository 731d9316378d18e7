// attn_chunk.cuh -- what the kernels of new rows behind a cached prefix share:
// which keys a tile of rows sees, how the work is cut, and how it is found.
//
// Sequence s holds n new rows and `len` keys, the rows' own keys last: row i is
// at place p = len - n + i and sees the keys
//
//   j <= p,  and under a window  j > p - window  or  j < sinks.
//
// Query heads that share a kv head share its keys, so a tile of rows is made of
// tokens and heads: row r is token r / heads, head r % heads.  A unit, one or two
// tiles, walks the list of the blocks of keys that its rows see.
//
// Where a sequence's units are few, or do not fill the GPU's last round, each
// unit's list is cut into as many splits as would be done soonest; their partial
// results are joined in order.  How many is a function of the sequence and the
// call's sizes alone -- a sequence is taken to have the GPU for itself --, so that
// a row's bits do not depend on the batch.
#pragma once

#include <stdint.h>

#include "attn_common.cuh"
#include "gbe_elementwise.h"
#include "launch.h"
#include "patience.h"

namespace gbe {
namespace chunk {

constexpr int kWave = 152;       // items at a time, which a sequence's splits are to fill
constexpr int kRounds = 8;       // once at least, and at most as often
// Keys of a split at least; twice as many where a sequence has more rows of a kv head than kFewRows, for every split
// writes and reads partial results of all of them.  A sequence alone is best cut short, a batch best left whole
// (bf16, 32 heads over 8 of 128): 24 sequences of up to 200 behind up to 8000 264 us with 1024 for all and 222 with
// 2048, 16 of 60 behind 8000 182 and 163, one of 100 behind 4000 33 and 42; 64 of 5 behind 8000 411 and 390, but one
// of 5 25 and 38, where so few rows are a user who waits.
constexpr int kLeast = 1024, kFewRows = 128;
constexpr int kEnds = 4;         // what an item's first copies, last rows and join cost, in blocks of 128 keys
constexpr int kUnitRows = 256;   // at most
constexpr int kPacked = -1;      // the type of keys that are not in a cache

struct Args {
    ChunkArgs a;
    int group;             // query heads of a kv head
    int heads, parts;      // of a tile, and tiles that a group is cut into
    int tokens;            // of a tile
    int tiles;             // of a unit
    int width;             // keys of a block
    int window, sinks;     // a's
    int most;              // splits at most; 1: nothing is cut
    uint32_t patience;     // of waits that may last for an item
    int64_t per_seq;       // places for each sequence's; 0: `most` for each row
    float* part_o;         // [places, D]
    float2* part_ml;       // [places]: running maximum (base 2), running sum
};

// The geometry of units of `tiles` tiles of `rows` rows.
inline Args make_args(const ChunkArgs& a, int rows, int tiles, int width) {
    Args g = {};
    g.a = a;
    g.group = (int)(a.Hq / a.Hkv);
    g.heads = g.group < rows ? g.group : rows;
    g.parts = (g.group + g.heads - 1) / g.heads;
    g.tokens = rows / g.heads;
    g.tiles = tiles;
    g.width = width;
    g.patience = patience_for((a.packed ? a.T : a.max_pages * a.c.page_size) / width);
    g.window = (int)a.window, g.sinks = (int)a.sinks;  // (2^30 at most)
    const int64_t keys = a.packed ? 0 : a.max_pages * a.c.page_size;
    const ChunkRoom r = chunk_room(a.n_seqs, a.T, a.Hq, a.Hkv, keys, a.window, a.sinks);
    g.most = r.most;
    g.per_seq = r.per_seq;
    g.part_o = static_cast<float*>(a.workspace);
    g.part_ml = reinterpret_cast<float2*>(g.part_o + (r.most > 1 ? r.entries * a.D : 0));
    return g;
}

struct Seq {
    int begin, n, len;  // first row in the packed buffers, rows, keys
};

// starts are brought into [0, T] and lens into the table's capacity, so that no
// row and no page outside the buffers is reached whatever they hold.
__host__ __device__ __forceinline__ Seq sequence(const ChunkArgs& a, int64_t b) {
    Seq s = {0, 0, 0};
    if (b >= a.n_seqs) return s;
    s.begin = (int)min(max((int64_t)a.starts[b], (int64_t)0), a.T);
    s.n = (int)max(min(max((int64_t)a.starts[b + 1], (int64_t)0), a.T) - s.begin, (int64_t)0);
    s.len = a.packed ? s.n : (int)min(max((int64_t)a.lens[b], (int64_t)0), a.max_pages * a.c.page_size);
    return s;
}

// How a sequence is cut: its units, and the splits of each.
struct Cut {
    int units, splits;
};
static __device__ __noinline__ Cut cut_of(const Args& g, const Seq& s) {
    const ChunkArgs& a = g.a;
    const int Hkv = (int)a.Hkv;
    Cut c = {0, 1};
    if (s.n == 0) return c;
    c.units = ((s.n + g.tokens - 1) / g.tokens * g.parts + g.tiles - 1) / g.tiles;
    if (g.most == 1 || c.units >= kWave * kRounds) return c;
    int64_t keys = s.len;
    if (a.window > 0) keys = min(keys, a.window + a.sinks + min(s.n, g.tiles * g.tokens));
    const int blocks = (int)((keys + 127) / 128), all = c.units * Hkv;
    const int cap = min(g.most, blocks / (kLeast / 128 * ((int64_t)s.n * g.group > kFewRows ? 2 : 1)));
    if (all >= kWave * kRounds || cap < 2) return c;
    // what one round, two, ... make possible; worth it from a 16th on
    float cost = (float)((all + kWave - 1) / kWave * (blocks + kEnds)) * 0.9375f;
#pragma unroll 1
    for (int w = kWave; w <= kRounds * kWave; w += kWave) {
        const int n = min(cap, w / all), rounds = (all * n + kWave - 1) / kWave;
        const float t = (float)rounds * (__fdividef((float)blocks, (float)n) + kEnds);
        if (n > 1 && t < cost) cost = t, c.splits = n;
    }
    return c;
}

// A unit, or a split of it.
struct Item {
    Seq s;
    int seq, tile, tiles;  // its tiles: tile, tile + 1, ...
    int split, splits;
};

// The items of a CTA, one behind the other, by one whole warp: pieces blockIdx.x,
// blockIdx.x + gridDim.x, ... of all; `zigzag`: every other step in the other
// direction.  A lane looks up a piece, 32 at a time, in sequences of which a lane
// holds one, the next 32 when a piece is past these.  (The code is short on
// purpose: it runs while much else does, and is fetched again each time.)
class Source {
  public:
    __device__ __forceinline__ Source(const Args& g, bool zigzag) : g_(g), zigzag_(zigzag) {}

    __device__ __forceinline__ bool next(Item& it, int& kvh) {
        const int from = turn_ & 31;
        if (from == 0) look_up();
        ++turn_;
        it.splits = __shfl_sync(0xFFFFFFFFu, splits_, from);
        if (it.splits == 0) return false;
        it.s.begin = __shfl_sync(0xFFFFFFFFu, s_.begin, from);
        it.s.n = __shfl_sync(0xFFFFFFFFu, s_.n, from);
        it.s.len = __shfl_sync(0xFFFFFFFFu, s_.len, from);
        it.seq = __shfl_sync(0xFFFFFFFFu, seq_, from);
        it.tile = __shfl_sync(0xFFFFFFFFu, unit_, from) * g_.tiles;
        it.tiles = min(g_.tiles, (it.s.n + g_.tokens - 1) / g_.tokens * g_.parts - it.tile);
        it.split = __shfl_sync(0xFFFFFFFFu, split_, from);
        kvh = __shfl_sync(0xFFFFFFFFu, kvh_, from);
        return true;
    }

  private:
    // The lane's piece; splits_ 0: there is none, nor any behind it.
    __device__ __noinline__ void look_up() {
        const int lane = threadIdx.x & 31, round = turn_ + lane;
        const uint64_t index =
            (uint64_t)round * gridDim.x + (zigzag_ && (round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        splits_ = 0;
        for (;;) {
            const uint32_t total = __shfl_sync(0xFFFFFFFFu, upto_, 31);
            const bool here = splits_ == 0 && index >= base_ && index - base_ < total;
            const uint32_t at = here ? (uint32_t)(index - base_) : 0u;
            int who = 0;  // the first lane whose sequences' pieces go up to more than `at`
#pragma unroll
            for (int step = 16; step >= 1; step >>= 1)
                if (__shfl_sync(0xFFFFFFFFu, upto_, who + step - 1) <= at) who += step;
            who = min(who, 31);
            const uint32_t before = __shfl_sync(0xFFFFFFFFu, upto_, who == 0 ? 0 : who - 1);
            const Seq s = {__shfl_sync(0xFFFFFFFFu, group_.begin, who), __shfl_sync(0xFFFFFFFFu, group_.n, who),
                           __shfl_sync(0xFFFFFFFFu, group_.len, who)};
            const int units = __shfl_sync(0xFFFFFFFFu, cut_.units, who);
            const int splits = __shfl_sync(0xFFFFFFFFu, cut_.splits, who);
            if (here) {
                // kv heads innermost, then units, the last rows, which see the most, first; splits outermost, so that
                // what runs at a time reads the same keys
                const uint32_t x = at - (who == 0 ? 0u : before), y = x / (uint32_t)g_.a.Hkv;
                kvh_ = (int)(x - y * (uint32_t)g_.a.Hkv);
                split_ = (int)(y / (uint32_t)max(units, 1));
                unit_ = max(units, 1) - 1 - (int)(y - (uint32_t)split_ * (uint32_t)max(units, 1));
                split_ = min(split_, splits - 1);  // (starts that decrease may have more pieces than 32 bits count)
                s_ = s, splits_ = splits, seq_ = (int)first_ + who;
            }
            const bool past = splits_ == 0 && index >= base_ + total;
            if (!__any_sync(0xFFFFFFFFu, past) || first_ + 32 >= g_.a.n_seqs) return;
            first_ += 32;
            base_ += total;
            group_ = sequence(g_.a, first_ + lane);
            cut_ = cut_of(g_, group_);
            upto_ = (uint32_t)cut_.units * (uint32_t)cut_.splits * (uint32_t)g_.a.Hkv;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto_, d);
                if (lane >= d) upto_ += y;
            }
        }
    }
    const Args& g_;
    const bool zigzag_;
    // of the sequences at hand, first_ + lane: this one, and the pieces up to it
    int64_t first_ = -32;
    uint64_t base_ = 0;
    Seq group_ = {0, 0, 0};
    Cut cut_ = {0, 1};
    uint32_t upto_ = 0;
    int turn_ = 0;  // pieces taken so far
    // the lane's piece
    Seq s_;
    int seq_, kvh_, unit_, split_, splits_;
};

// An item's walk over the list: blocks that hold a sink, then from the first one
// under the window to the last row's place.
struct Walk {
    int first_place, last_place;  // of the item's rows
    int sinks;                    // blocks of sinks ahead of the window
    int window;                   // the window's first block
    int from, to;                 // the split's part of the list
    __device__ __forceinline__ int block(int i) const { return i < sinks ? i : window + (i - sinks); }
};
__device__ __forceinline__ Walk walk(const Args& g, const Item& it) {
    Walk w;
    const int last_tile = it.tile + it.tiles - 1;
    w.first_place = it.s.len - it.s.n + it.tile / g.parts * g.tokens;
    w.last_place = it.s.len - it.s.n + min(it.s.n, (last_tile / g.parts + 1) * g.tokens) - 1;
    const int end = w.last_place < 0 ? 0 : w.last_place / g.width + 1;
    w.window = w.sinks = 0;
    if (g.window > 0) {
        w.window = min(max(w.first_place - g.window + 1, 0) / g.width, end);
        w.sinks = min((max(min(g.sinks, w.last_place + 1), 0) + g.width - 1) / g.width, w.window);
    }
    const int n = w.sinks + end - w.window;
    w.from = 0, w.to = n;
    if (it.splits > 1) {
        w.from = (int)((int64_t)n * it.split / it.splits);
        w.to = (int)((int64_t)n * (it.split + 1) / it.splits);
    }
    return w;
}

// Where a row's partial results lie, one behind the other, and where the item's is.
__device__ __forceinline__ int64_t parts_at(const Args& g, const Item& it, int token, int head) {
    if (g.per_seq > 0) return it.seq * g.per_seq + ((int64_t)token * g.a.Hq + head) * it.splits;
    return ((int64_t)(it.s.begin + token) * g.a.Hq + head) * g.most;
}
__device__ __forceinline__ int64_t part_at(const Args& g, const Item& it, int token, int head) {
    return parts_at(g, it, token, head) + it.split;
}

// The tensor-core form: bf16 rows and, where there is a cache, one of a page at
// least; D <= 128, rows, the cache's too, on the 16-byte grid, all in device memory.
cudaError_t launch_tc(const ChunkArgs& a, cudaStream_t st);

// The partial results of every row added in order.
cudaError_t launch_join(const Args& g, int dtype, cudaStream_t st);

}  // namespace chunk
}  // namespace gbe
