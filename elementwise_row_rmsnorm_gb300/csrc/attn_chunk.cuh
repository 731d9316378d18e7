// attn_chunk.cuh -- what the kernels of new rows behind a cached prefix share:
// which keys a tile of rows sees, how its walk over them is cut, and how pieces
// of work are found.
//
// Sequence s holds n new rows and `len` keys, the rows' own keys last: row i is
// at place p = len - n + i and sees the keys
//
//   j <= p,  and under a window  j > p - window  or  j < sinks.
//
// Query heads that share a kv head share its keys, so a tile of rows is made of
// tokens and heads: row r is token r / heads, head r % heads.
//
// With few rows and many keys a tile's walk is cut into splits whose partial
// sums are joined afterwards.  How many is a function of the sequence and the
// call's head counts alone, so that a row's bits do not depend on the batch: a
// sequence is taken to have the GPU for itself, and gets the number at which
// kWave CTAs -- one to four rounds of them -- would be done soonest, an item
// costing its blocks of keys and kEnds more (its first copies, its join).
#pragma once

#include <stdint.h>

#include "attn_common.cuh"
#include "launch.h"

namespace gbe {
namespace chunk {

constexpr int kBlock = 128;        // keys that a split counts in
constexpr int kPairRows = 256;     // rows that it takes an item to have
constexpr int kWave = 152, kRounds = 4, kEnds = 3;
constexpr int kLeast = 8;          // blocks of a split at least
constexpr int kMostSplits = 128;

struct Args {
    ChunkArgs a;
    int group;             // query heads of a kv head
    int heads, parts;      // of a tile, and tiles that a group is cut into
    int tokens;            // of a tile
    int tiles_per_item;
    float* part_o;         // [entries, D]
    float2* part_ml;       // [entries]: running maximum (base 2), running sum
    int64_t per_seq;
    int most;
};

// The geometry of tiles of `rows` rows.
inline Args make_args(const ChunkArgs& a, int rows, int tiles_per_item) {
    Args g = {};
    g.a = a;
    g.group = (int)(a.Hq / a.Hkv);
    g.heads = g.group < rows ? g.group : rows;
    g.parts = (g.group + g.heads - 1) / g.heads;
    g.tokens = rows / g.heads;
    g.tiles_per_item = tiles_per_item;
    const int64_t keys = a.table == nullptr ? 0 : a.max_pages * a.c.page_size;
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
__device__ __forceinline__ Seq sequence(const ChunkArgs& a, int64_t b) {
    Seq s = {0, 0, 0};
    if (b >= a.n_seqs) return s;
    s.begin = (int)min(max((int64_t)a.starts[b], (int64_t)0), a.T);
    s.n = (int)max(min(max((int64_t)a.starts[b + 1], (int64_t)0), a.T) - s.begin, (int64_t)0);
    s.len = a.table == nullptr ? s.n
                               : (int)min(max((int64_t)a.lens[b], (int64_t)0), a.max_pages * a.c.page_size);
    return s;
}

__device__ __forceinline__ int splits_of(const Args& g, const Seq& s) {
    if (g.most == 1) return 1;
    const ChunkArgs& a = g.a;
    int64_t keys = s.len;
    if (a.window > 0) keys = min(keys, a.window + a.sinks + s.n);
    const int blocks = (int)((keys + kBlock - 1) / kBlock);
    const int64_t items = ((int64_t)s.n * g.group + kPairRows - 1) / kPairRows * a.Hkv;
    const int cap = min(g.most, blocks / kLeast);
    if (cap < 2 || items < 1 || items >= kWave * kRounds) return 1;
    const float u = (float)items;
    int best = 1, cost = ((int)items + kWave - 1) / kWave * (blocks + kEnds);
#pragma unroll
    for (int w = 1; w <= kRounds; ++w) {
        const int n = min(cap, (int)__fdividef((float)(w * kWave) + 0.5f, u));
        if (n < 2) continue;
        const int rounds = ((int)items * n + kWave - 1) / kWave;
        const int c = rounds * ((int)__fdividef((float)(blocks + n - 1) + 0.5f, (float)n) + kEnds);
        if (c < cost) cost = c, best = n;
    }
    return best;
}

// An item of work: tiles tile, tile + 1, ... (tiles_per_item of them, as far as
// there are) of a sequence, and one of the splits of their walk.
struct Item {
    Seq s;
    int seq, tile, tiles, split, splits;  // splits 0: no such item
};

// Finds items by their number, asked for in ascending order, by one whole warp:
// four sequences a lane, the next 128 when the number is past these.
class Finder {
  public:
    __device__ __forceinline__ explicit Finder(const Args& g) : g_(g) { load(); }

    __device__ __forceinline__ Item find(uint64_t index) {
        Item it = {};
        while (index >= base_ + total_) {
            first_ += 128;
            base_ += total_;
            if (first_ >= g_.a.n_seqs) {
                total_ = 0;
                first_ -= 128;
                return it;
            }
            load();
        }
        uint32_t left = (uint32_t)(index - base_);
        const int lane = threadIdx.x & 31;
        bool found = false;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (found) continue;
            if (left >= sum_[x]) {
                left -= sum_[x];
                continue;
            }
            uint32_t upto = count_[x];  // items of this lane's sequence and those before it
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, d);
                if (lane >= d) upto += y;
            }
            const int who = __ffs((int)__ballot_sync(0xFFFFFFFFu, upto > left)) - 1;
            it.s.begin = __shfl_sync(0xFFFFFFFFu, s_[x].begin, who);
            it.s.n = __shfl_sync(0xFFFFFFFFu, s_[x].n, who);
            it.s.len = __shfl_sync(0xFFFFFFFFu, s_[x].len, who);
            it.splits = __shfl_sync(0xFFFFFFFFu, splits_[x], who);
            left -= __shfl_sync(0xFFFFFFFFu, upto - count_[x], who);
            it.seq = (int)first_ + x * 32 + who;
            found = true;
        }
        const int tiles = tiles_of(it.s.n), items = (tiles + g_.tiles_per_item - 1) / g_.tiles_per_item;
        const int k = (int)(left / (uint32_t)it.splits);
        it.split = (int)(left - (uint32_t)k * (uint32_t)it.splits);
        it.tile = (items - 1 - k) * g_.tiles_per_item;  // the last rows, which see the most, first
        it.tiles = min(g_.tiles_per_item, tiles - it.tile);
        return it;
    }

  private:
    __device__ __forceinline__ int tiles_of(int n) const { return (n + g_.tokens - 1) / g_.tokens * g_.parts; }
    __device__ __forceinline__ void load() {
        total_ = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            count_[x] = 0, sum_[x] = 0, splits_[x] = 1;
            s_[x] = {0, 0, 0};
            if (first_ + x * 32 >= g_.a.n_seqs) continue;
            s_[x] = sequence(g_.a, first_ + x * 32 + (threadIdx.x & 31));
            if (s_[x].n > 0) {
                splits_[x] = splits_of(g_, s_[x]);
                count_[x] = (uint32_t)((tiles_of(s_[x].n) + g_.tiles_per_item - 1) / g_.tiles_per_item) *
                            (uint32_t)splits_[x];
            }
            sum_[x] = __reduce_add_sync(0xFFFFFFFFu, count_[x]);
            total_ += sum_[x];
        }
    }
    const Args& g_;
    int64_t first_ = 0;
    uint64_t base_ = 0;
    uint32_t total_ = 0, sum_[4], count_[4];
    Seq s_[4];
    int splits_[4];
};

// The blocks of `width` keys that some row of an item's tiles sees, as a list:
// those that hold a sink, then from the first under the window to the last row's
// place; and the part of it that is the item's split.
struct Walk {
    int first_place, last_place;  // of the item's rows
    int sinks;                    // blocks of sinks ahead of the window
    int window;                   // the window's first block
    int from, to;                 // the split's part of the list
    __device__ __forceinline__ int block(int i) const { return i < sinks ? i : window + (i - sinks); }
};
__device__ __forceinline__ Walk walk(const Args& g, const Item& it, int width) {
    Walk w;
    const int last_tile = it.tile + it.tiles - 1;
    w.first_place = it.s.len - it.s.n + it.tile / g.parts * g.tokens;
    w.last_place = it.s.len - it.s.n + min(it.s.n, (last_tile / g.parts + 1) * g.tokens) - 1;
    const int end = w.last_place < 0 ? 0 : w.last_place / width + 1;
    const int64_t low = g.a.window > 0 ? max((int64_t)w.first_place - g.a.window + 1, (int64_t)0) : 0;
    w.window = (int)min(low / width, (int64_t)end);
    w.sinks = (int)min((min(g.a.sinks, (int64_t)w.last_place + 1) + width - 1) / width, (int64_t)w.window);
    if (w.sinks < 0) w.sinks = 0;
    const int64_t n = w.sinks + end - w.window;
    w.from = (int)(n * it.split / it.splits);
    w.to = (int)(n * (it.split + 1) / it.splits);
    return w;
}

// Where a row's partial result of an item lies.
__device__ __forceinline__ int64_t part_at(const Args& g, const Item& it, int token, int head) {
    if (g.per_seq > 0)
        return it.seq * g.per_seq + ((int64_t)token * g.a.Hq + head) * it.splits + it.split;
    return ((int64_t)(it.s.begin + token) * g.a.Hq + head) * g.most + it.split;
}

// The tensor-core form: bf16 rows and, where there is a cache, one of a page at
// least; D <= 128, rows on the 16-byte grid, all in device memory.
cudaError_t launch_tc(const ChunkArgs& a, cudaStream_t st);

// The splits of every row added in order.
cudaError_t launch_join(const Args& g, int dtype, cudaStream_t st);

}  // namespace chunk
}  // namespace gbe
