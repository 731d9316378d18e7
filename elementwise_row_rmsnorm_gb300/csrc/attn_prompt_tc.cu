// attn_prompt_tc.cu -- causal attention over packed prompts on the tensor
// cores: bf16, D up to 128, rows on the 16-byte grid.
//
//   S = q k^T (f32, in tensor memory), p = 2^(c S - c m), c = |scale| log2(e),
//   O = sum p v, out = O / sum p
//
// A CTA works on two tiles of 128 query rows that share one kv head -- two
// heads of its group at the same rows, or neighbouring row tiles -- and walks
// the keys in blocks of 128 that a ring of shared-memory stages holds; then on
// the next pair, its copies and first products already under way while the last
// rows are written.  Three warpgroups: one of softmax for each tile (a thread
// owns a row), and one of which a warp hands out the pairs, another issues the
// tensor copies and two the products, each of a tile (one thread for both spent
// more on its waits than the products took).
//
// Tensor memory (512 columns): one S for both tiles, O of each, and the
// weights of each, rounded to bf16, which are the A operand of the second
// product.  A block of 128 keys costs a tile 512 clocks of either product and
// its warpgroup some 1400 clocks of softmax, so the products of a tile must not
// wait for its softmax: they follow one another as
//
//   S0 = q0 k(j+1)^T, O0 += p0 v(j), S1 = q1 k(j+1)^T, O1 += p1 v(j)
//
// S is handed over as soon as a warpgroup has it in registers, and each
// softmax then has 1500 clocks until its weights are due.  (With an S
// for each tile, overwritten by its weights, the next S had to wait for the
// product with v, and a round of both tiles took 3300 clocks, not 2048.)
//
// Weights of one bf16, 8 bits, are what the second product takes beside a v of
// bf16; the results are 1.2 to 1.3 times as far from the definition as their own
// rounding leaves them (0.0019 and 0.0021 of their norm, 0.0016).  A second bf16
// a weight, as decode keeps, would want 128 more columns than the 512 there are,
// and half as many clocks a round again.
//
// O is rescaled only when a row's maximum has grown by more than 2^8 over the
// one in use; until then weights go up to 2^8, which costs nothing in bf16 or
// f32 (both floats) and keeps sums far from overflow.
//
// Measured on a GB300: one sequence of 8192 tokens, 32 heads of 128 over 8 kv
// heads, 355 us (1.55 PFLOP/s, 0.79 of cuBLAS's bf16 rate), bound by the shared
// memory that the first product reads and by the softmax between; 12 sequences
// of up to 500 tokens 27 us, bound by the latency of one to four blocks a tile.
// (Of the softmax's 208 registers a thread five words spill.)
//
// Masked weights are exact zeros, but zero times an infinity or a NaN in a
// later row of v would reach the sum.  Rows of v behind the sequence's end are
// left out: of the block that crosses it, copies of 32, 8 and 1 rows bring those
// before the end, and zeros (from behind the tensor's end) in place of the others.
// That costs 0 to 3 % of a call of short prompts (100 of up to 50 tokens 45.9 ->
// 47.1 us, 12 of up to 500 27.0 -> 27.4 us); the rows written over with zeros by
// the softmax warps 3 to 9 %, by the issuing thread 1 to 5 %, copies of 8 and 1
// rows 1 to 7 %, of every power of two 1 to 11 %.  Within the sequence, rows that
// come out not finite are looked at once more (repair_row).  So a row's bits
// depend on its own sequence alone.
#include "attn_tiles.cuh"
#include "gbe_elementwise.h"
#include "launch.h"
#include "tensor_core.cuh"

namespace gbe {
namespace {

constexpr int kM = 128, kN = 128;
constexpr int kThreads = 384;  // three warpgroups: softmax of each tile, and the issuing warps
constexpr int kLoadWarp = 8, kItemWarp = 9, kMmaWarp = 10;  // products: a warp for each tile
constexpr float kGrowth = 8.0f;  // a maximum may lag this many powers of two

// Pair `index` of the tiles that share a kv head, the ones with the most keys
// first: a sequence of r row tiles has r * group tiles, tile u being head
// u % group of the group at rows (u / group) * kM.
struct Pair {
    int begin, len, unit, units;  // units 0: no such pair
};

// What the scheduling warp hands out; units < 0: nothing more.
struct Item {
    Pair p;
    int kvh;
};
constexpr int kItems = 4, kReaders = 11;  // items in hand; warps that read one: softmax, loads, products

struct Control {
    uint64_t q_full[2], q_empty, kv_full[8], kv_empty[8], s_full[2], s_free[2], p_ready[2], o_done[2], o_free[2];
    uint64_t drained[2];
    uint64_t item_full[kItems], item_empty[kItems];
    Item item[kItems];
    uint32_t tmem;
    int abort;
};

template <int DP>
struct Shape {
    static constexpr int kPanel = 128 * 128;              // 128 rows of 64 bf16
    static constexpr int kTile = kPanel * (DP / 64);      // 128 rows of DP
    static constexpr int kStages = DP == 128 ? 4 : 8;
    static constexpr int kOut = 8 * 32 * 128;             // 32 rows of 64 entries for each softmax warp
    static constexpr int kBytes = kTile * (2 + kStages) + kOut + 1024 + (int)sizeof(Control);
};

__device__ __forceinline__ Pair find_pair(const int32_t* starts, int n_seqs, int T, int group, uint32_t index) {
    auto tiles = [&](int n) { return (uint32_t)((n + kM - 1) / kM) * (uint32_t)group; };
    const SeqPiece p = find_piece(
        starts, n_seqs, T, index, [&](int n) { return (tiles(n) + 1) / 2; },
        [&](uint32_t rows, uint32_t seqs) {  // a sequence of an odd number of tiles leaves half a pair
            return ((rows / kM + seqs) * (uint32_t)group + (group & 1 ? seqs : 0u)) / 2;
        });
    if (p.index < 0) return {0, 0, 0, 0};
    return {p.begin, p.len, 2 * p.index, min(2, (int)tiles(p.len) - 2 * p.index)};
}

// Four consecutive values, widened.
__device__ __forceinline__ float4 load4(const void* base, int64_t i) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}

// One row in f32 from its own keys alone, by a whole warp: 32 keys at a time, a
// lane a key for the logits, a lane four entries for the output.
__device__ __noinline__ void exact_row(const PromptArgs& a, int begin, int row, int head) {
    const int lane = threadIdx.x & 31, D = (int)a.D, kvh = head / (int)(a.Hq / a.Hkv);
    const float c = a.scale * kLog2e;
    float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f), o = q;
    if (lane * 4 < D) q = load4(a.q, (begin + (int64_t)row) * a.q_stride + (int64_t)head * D + lane * 4);
    float m = -INFINITY, l = 0.0f;
    for (int k0 = 0; k0 <= row; k0 += 32) {
        const int j = k0 + lane;
        const bool seen = j <= row;
        const int64_t k_at = (begin + (int64_t)(seen ? j : row)) * a.k_stride + (int64_t)kvh * D;
        float s = 0.0f;
        for (int d = 0; d < D; d += 4) {
            const float4 k = load4(a.k, k_at + d);
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
                    load4(a.v, (begin + (int64_t)k0 + t) * a.v_stride + (int64_t)kvh * D + lane * 4);
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
        for (int e = 0; e < 4; ++e) Store<kBF16>::store1(a.out, at + e, m == -INFINITY ? 0.0f : y[e] / l);
    }
}

// Which of four consecutive values are infinite or NaN, a bit each.
__device__ __forceinline__ uint32_t not_finite4(const void* base, int64_t i) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
    return ((w.x & 0x7F80u) == 0x7F80u ? 1u : 0u) | ((w.x >> 16 & 0x7F80u) == 0x7F80u ? 2u : 0u) |
           ((w.y & 0x7F80u) == 0x7F80u ? 4u : 0u) | ((w.y >> 16 & 0x7F80u) == 0x7F80u ? 8u : 0u);
}

// A row that came out not finite: right as it is where the keys that it attends
// to made it so, but a weight of zero may also have met an infinity or a NaN of
// v behind the mask, in rows row + 1 .. end - 1, the sequence's in the tile.
// Computed again only if an entry is not finite, has such a value behind the
// mask, and has none before it.  By a whole warp; the row has been written.
__device__ __noinline__ void repair_row(const PromptArgs& a, int begin, int row, int end, int head) {
    const int lane = threadIdx.x & 31, D = (int)a.D, kvh = head / (int)(a.Hq / a.Hkv);
    const bool mine = lane * 4 < D;
    const int64_t v0 = (int64_t)begin * a.v_stride + (int64_t)kvh * D + lane * 4;
    const int64_t out0 = (begin + (int64_t)row) * a.out_stride + (int64_t)head * D + lane * 4;
    uint32_t open = mine ? not_finite4(a.out, out0) : 0u;  // entries that may have to be computed again
    uint32_t behind = 0;
    for (int j = row + 1; j < end && __any_sync(0xFFFFFFFFu, open & ~behind); j += 8)
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (mine && j + x < end) behind |= not_finite4(a.v, v0 + (int64_t)(j + x) * a.v_stride);
    open &= behind;
    for (int j = row; j >= 0; j -= 8) {
        if (!__any_sync(0xFFFFFFFFu, open)) return;
        uint32_t before = 0;
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if (mine && j - x >= 0) before |= not_finite4(a.v, v0 + (int64_t)(j - x) * a.v_stride);
        open &= ~before;
    }
    if (__any_sync(0xFFFFFFFFu, open)) exact_row(a, begin, row, head);
}

// Work item `round` of this CTA: rounds go back and forth over the CTAs, so that
// no CTA always gets the larger one.
__device__ __forceinline__ uint32_t item_of(int round) {
    return (uint32_t)round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
              const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mv32,
              const __grid_constant__ CUtensorMap mv8, const __grid_constant__ CUtensorMap mv1, PromptArgs a,
              uint32_t n_items) {
    using S = Shape<DP>;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    Control& ctl = *reinterpret_cast<Control*>(raw + (base - smem_addr(raw)) + S::kTile * (2 + S::kStages) + S::kOut);
    const uint32_t q_smem = base, kv_smem = base + 2 * S::kTile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = (int)(a.Hq / a.Hkv);
    volatile int* const abort = &ctl.abort;

    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&ctl.q_full[0]), 1);
        mbar_init(smem_addr(&ctl.q_full[1]), 1);
        mbar_init(smem_addr(&ctl.q_empty), 2);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(smem_addr(&ctl.kv_full[i]), 1);
            mbar_init(smem_addr(&ctl.kv_empty[i]), 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_addr(&ctl.s_full[t]), 1);
            mbar_init(smem_addr(&ctl.p_ready[t]), 4);
            mbar_init(smem_addr(&ctl.s_free[t]), 4);
            mbar_init(smem_addr(&ctl.o_done[t]), 1);
            mbar_init(smem_addr(&ctl.o_free[t]), 4);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(smem_addr(&ctl.item_full[i]), 1);
            mbar_init(smem_addr(&ctl.item_empty[i]), kReaders);
        }
        mbar_init(smem_addr(&ctl.drained[0]), 1);
        mbar_init(smem_addr(&ctl.drained[1]), 1);
        ctl.abort = 0;
        mbar_init_fence();
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
        tma_prefetch(&mv32);
        tma_prefetch(&mv8);
        tma_prefetch(&mv1);
    }
    pdl_begin();
    // (not ahead of it: a kernel before this one may have yet to take its share)
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&ctl.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;

    // Item i as its readers see it: tile t's head, first row and blocks of
    // keys up to its diagonal.
    struct Work {
        int begin, len, kvh, units, most;
        int head[2], row0[2], blocks[2];
    };
    auto as_work = [&](const Item& it) {
        Work w;
        w.begin = it.p.begin, w.len = it.p.len, w.kvh = it.kvh, w.units = it.p.units;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int u = it.p.unit + t;
            w.head[t] = it.kvh * group + u % group;
            w.row0[t] = u / group * kM;
            w.blocks[t] = t < w.units ? u / group + 1 : 0;
        }
        w.most = max(w.blocks[0], w.blocks[1]);
        return w;
    };
    // false: a wait gave up
    auto item_ready = [&](int i) { return mbar_wait(smem_addr(&ctl.item_full[i % kItems]), i / kItems & 1, abort); };
    auto item_read = [&](int i) { mbar_arrive(smem_addr(&ctl.item_empty[i % kItems])); };

    // Registers: 384 threads were launched with 168 each (64512); the softmax
    // warpgroups take 208, the issuing one keeps 80 (63488 in all).
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == kItemWarp) {
            bool ok = true;
            int i = 0;
            for (int round = 0; ok; ++round) {
                const uint32_t id = item_of(round);
                const bool end = (uint64_t)round * gridDim.x >= n_items;
                Item it = {{0, 0, 0, -1}, 0};
                if (!end) {
                    if (id >= n_items) continue;
                    it.kvh = (int)(id % (uint32_t)a.Hkv);
                    it.p = find_pair(a.starts, (int)a.n_seqs, (int)a.T, group, id / (uint32_t)a.Hkv);
                    if (it.p.units == 0) continue;
                }
                ok = __all_sync(0xFFFFFFFFu,
                                mbar_wait(smem_addr(&ctl.item_empty[i % kItems]), (i / kItems & 1) ^ 1, abort));
                if (!ok) break;
                if (lane == 0) {
                    ctl.item[i % kItems] = it;
                    mbar_arrive(smem_addr(&ctl.item_full[i % kItems]));
                }
                ++i;
                if (end) break;
            }
        } else if (warp == kLoadWarp) {
            if (elect_one()) {
                int g = 0, tiles[2] = {0, 0};  // loads of the ring and tiles of q so far
                bool ok = true;
                for (int i = 0; ok; ++i) {
                    if (!(ok = item_ready(i))) break;
                    const Work w = as_work(ctl.item[i % kItems]);
                    item_read(i);
                    if (w.units < 0) break;
                    for (int x = 0; ok && x < 2 * w.most; ++x) {  // k and v of each block in turn
                        const int stage = g % S::kStages;
                        ok = mbar_wait(smem_addr(&ctl.kv_empty[stage]), (g / S::kStages & 1) ^ 1, abort);
                        if (!ok) break;
                        const uint32_t full = smem_addr(&ctl.kv_full[stage]);
                        mbar_arrive_tx(full, S::kTile);
                        const uint32_t to = kv_smem + stage * S::kTile;
                        const int row = w.begin + (x >> 1) * kN, have = w.len - (x >> 1) * kN;
                        if (!(x & 1) || have >= kN) {
#pragma unroll
                            for (int p = 0; p < DP / 64; ++p)
                                tma_load_3d(to + p * S::kPanel, (x & 1) ? &mv : &mk, full, p * 64, w.kvh, row);
                        } else {  // v where the sequence ends within the block; from row T on there are zeros
                            auto part = [&](const CUtensorMap* m, int r) {
#pragma unroll
                                for (int p = 0; p < DP / 64; ++p)
                                    tma_load_3d(to + p * S::kPanel + r * 128, m, full, p * 64, w.kvh,
                                                r < have ? row + r : (int)a.T);
                            };
#pragma unroll 1
                            for (int r = 0; r < kN;) {
                                const int left = have - r;
                                if (r % 32 == 0 && (left >= 32 || left <= 0))
                                    part(&mv32, r), r += 32;
                                else if (r % 8 == 0 && (left >= 8 || left <= 0))
                                    part(&mv8, r), r += 8;
                                else
                                    part(&mv1, r), ++r;
                            }
                        }
                        ++g;
                        if (x == 0) {  // q, once the last item's is done with
                            ok = mbar_wait(smem_addr(&ctl.q_empty), (i & 1) ^ 1, abort);
                            if (!ok) break;
                            for (int t = 0; t < w.units; ++t) {
                                const uint32_t qb = smem_addr(&ctl.q_full[t]);
                                mbar_arrive_tx(qb, S::kTile);
#pragma unroll
                                for (int p = 0; p < DP / 64; ++p)
                                    tma_load_3d(q_smem + t * S::kTile + p * S::kPanel, &mq, qb, p * 64, w.head[t],
                                                w.begin + w.row0[t]);
                                ++tiles[t];
                            }
                        }
                    }
                }
                if (*abort) {  // nothing may still be on its way when the CTA ends
                    int none = 0;
                    for (int t = 0; t < 2; ++t)
                        if (tiles[t] > 0) mbar_wait(smem_addr(&ctl.q_full[t]), (tiles[t] - 1) & 1, &none);
                    for (int x = max(0, g - S::kStages); x < g; ++x)
                        mbar_wait(smem_addr(&ctl.kv_full[x % S::kStages]), x / S::kStages & 1, &none);
                }
            }
        } else if (elect_one()) {
            const int t = warp - kMmaWarp;
            const uint32_t idesc_s = bf16_idesc(kM, kN, false) | (a.scale < 0.0f ? 1u << 13 : 0u);
            constexpr uint32_t idesc_o = bf16_idesc(kM, DP, true), hi = smem_desc_hi(1024);
            const uint32_t q_lo = smem_desc_lo(q_smem + t * S::kTile, 16), k_lo = smem_desc_lo(kv_smem, 16);
            const uint32_t v_lo = smem_desc_lo(kv_smem, S::kPanel);
            const uint32_t o = tmem + 256 + t * 128, pw = tmem + 128 + t * 64;
            bool ok = true;
            int g = 0;              // the ring's loads before this item: k of block j is load g + 2 j
            int done[2] = {0, 0};   // blocks of each tile before this item
            int items = 0;          // items with a tile t
            int last_t = -1;        // the tile that S was last written for in the item before
            for (int i = 0; ok; ++i) {
                if (!(ok = item_ready(i))) break;
                const Work w = as_work(ctl.item[i % kItems]);
                item_read(i);
                if (w.units < 0) break;
                const int mine = w.blocks[t], theirs = w.blocks[t ^ 1];
                auto loaded = [&](int x) {
                    ok = ok && mbar_wait(smem_addr(&ctl.kv_full[x % S::kStages]), x / S::kStages & 1, abort);
                };
                // S is free once the block before in the order (0, j), (1, j), (0, j + 1), ... has been read
                auto s_free = [&](int j) {
                    int pt, pj;
                    if (t == 1) {
                        pt = j < theirs ? 0 : 1, pj = j < theirs ? j : j - 1;
                    } else {
                        pt = j - 1 < theirs ? 1 : 0, pj = j - 1;
                    }
                    if (pj < 0) pt = last_t;
                    // A wait by parity holds only where the phase before has completed.  The second tile's thread has
                    // passed over the first one's blocks of an item before that has no second tile: S of this item's
                    // first block, once it is there, says that those have been read.
                    if (t == 1 && j == 0 && last_t == 0)
                        ok = ok && mbar_wait(smem_addr(&ctl.s_full[0]), done[0] & 1, abort);
                    if (pt >= 0)
                        ok = ok && mbar_wait(smem_addr(&ctl.s_free[pt]), (done[pt] + pj) & 1, abort);
                };
                auto scores = [&](int j) {
                    loaded(g + 2 * j);
                    s_free(j);
                    if (!ok) return;
                    tc_fence_after();
                    const int stage = (g + 2 * j) % S::kStages;
                    const uint32_t k0 = k_lo + stage * (S::kTile >> 4);
#pragma unroll
                    for (int x = 0; x < DP / 16; ++x) {
                        const uint32_t off = ((x / 4) * S::kPanel + (x % 4) * 32) >> 4;
                        mma_ss(tmem, q_lo + off, hi, k0 + off, hi, idesc_s, x > 0);
                    }
                    mma_commit(smem_addr(&ctl.s_full[t]));
                    mma_commit(smem_addr(&ctl.kv_empty[stage]));
                    if (j + 1 == mine) mma_commit(smem_addr(&ctl.q_empty));
                };
                // (an item has a first tile always, a second one not)
                ok = mine > 0 ? mbar_wait(smem_addr(&ctl.q_full[t]), items & 1, abort)
                              : mbar_wait(smem_addr(&ctl.q_full[0]), i & 1, abort);
                if (mine > 0)
                    scores(0);
                else if (ok)
                    mbar_arrive(smem_addr(&ctl.q_empty));
                for (int j = 0; ok && j < mine; ++j) {
                    if (j + 1 < mine) scores(j + 1);
                    loaded(g + 2 * j + 1);
                    ok = ok && mbar_wait(smem_addr(&ctl.p_ready[t]), (done[t] + j) & 1, abort);
                    // O has been read for the last item
                    if (j == 0 && items > 0)
                        ok = ok && mbar_wait(smem_addr(&ctl.o_free[t]), (items - 1) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const int stage = (g + 2 * j + 1) % S::kStages;
                    const uint32_t v0 = v_lo + stage * (S::kTile >> 4);
#pragma unroll
                    for (int x = 0; x < kN / 16; ++x)
                        mma_ts(o, pw + x * 8, v0 + x * (2048 >> 4), hi, idesc_o, j > 0 || x > 0);
                    mma_commit(smem_addr(&ctl.o_done[t]));
                    mma_commit(smem_addr(&ctl.kv_empty[stage]));
                }
                // blocks that only the other tile works on
                for (int x = 2 * mine; ok && x < 2 * w.most; ++x) {
                    loaded(g + x);
                    if (ok) mbar_arrive(smem_addr(&ctl.kv_empty[(g + x) % S::kStages]));
                }
                g += 2 * w.most;
                done[0] += w.blocks[0], done[1] += w.blocks[1];
                items += mine > 0;
                last_t = w.blocks[1] > 0 ? 1 : 0;
            }
            // every product is done before tensor memory is given back
            mma_commit(smem_addr(&ctl.drained[t]));
            int none = 0;
            mbar_wait(smem_addr(&ctl.drained[t]), 0, &none);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
        const uint32_t ts = tmem + lanes, tp = tmem + 128 + t * 64 + lanes, to = tmem + 256 + t * 128 + lanes;
        // (never 0, so that c times the -inf of a masked place stays -inf)
        const float c = fmaxf(fabsf(a.scale) * kLog2e, __uint_as_float(1u));
        uint8_t* const stage = raw + (base - smem_addr(raw)) + S::kTile * (2 + S::kStages) + warp * (S::kOut / 8);
        bool ok = true;
        int done = 0;  // blocks of this tile before this item
        for (int i = 0; ok; ++i) {
            ok = __all_sync(0xFFFFFFFFu, item_ready(i));
            if (!ok) break;
            const Item it = ctl.item[i % kItems];
            __syncwarp();
            if (lane == 0) item_read(i);
            if (it.p.units < 0) break;
            if (t >= it.p.units) continue;
            const int u = it.p.unit + t, n = u / group + 1;
            const int row = u / group * kM + (threadIdx.x & 127);
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < n; ++j) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&ctl.s_full[t]), (done + j) & 1, abort));
                if (!ok) break;
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_ld32(ts + x * 32, s + x * 32);
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_wait_ld32(s + x * 32);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl.s_free[t]));
                if (j == n - 1) {  // the diagonal
                    const int seen = row - j * kN;
#pragma unroll
                    for (int x = 0; x < 128; ++x) s[x] = x <= seen ? s[x] : 0xFF800000u;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int x = 0; x < 128; x += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[x + e]), __uint_as_float(s[x + 4 + e])));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const bool grow = m == -INFINITY ? top > m : (top - m) * c > kGrowth;
                auto last_done = [&] {  // the product with the last weights is done
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&ctl.o_done[t]), (done + j - 1) & 1, abort));
                    tc_fence_after();
                };
                if (__any_sync(0xFFFFFFFFu, grow)) {
                    const float m2 = grow ? top : m;
                    if (j > 0) {
                        last_done();
                        if (!ok) break;
                        const float r = m == -INFINITY ? 0.0f : ex2((m - m2) * c);
                        l *= r;
#pragma unroll
                        for (int x = 0; x < DP / 32; ++x) {
                            uint32_t o[32];
                            tmem_ld32(to + x * 32, o);
                            tmem_wait_ld32(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * r);
                            tmem_st32(to + x * 32, o);
                        }
                    }
                    m = m2;
                }
                const float shift = m == -INFINITY ? 0.0f : -m * c;
                const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
                float2 sum[4] = {};
                uint32_t w[64];
#pragma unroll
                for (int e = 0; e < 64; ++e) {
                    float2 x = fma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2,
                                       shift2);
                    x.x = ex2(x.x), x.y = ex2(x.y);
                    sum[e & 3] = add2_rn(sum[e & 3], x);
                    w[e] = f32x2_to_bf16x2_bits(x.x, x.y);
                }
                const float2 add = add2_rn(add2_rn(sum[0], sum[1]), add2_rn(sum[2], sum[3]));
                l += add.x + add.y;
                if (j > 0) {
                    last_done();
                    if (!ok) break;
                }
                tmem_st32(tp, w);
                tmem_st32(tp + 32, w + 32);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl.p_ready[t]));
            }
            done += n;
            ok = ok && mbar_wait(smem_addr(&ctl.o_done[t]), (done - 1) & 1, abort);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
            const int head = it.kvh * group + u % group;
            const bool live = row < it.p.len;
            const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
            const int row0 = u / group * kM + (warp & 3) * 32;
            uint16_t* const out = static_cast<uint16_t*>(a.out) + (it.p.begin + (int64_t)row0) * a.out_stride +
                                  (int64_t)head * a.D;
            float2 bad = make_float2(0.0f, 0.0f);
            // 64 entries of the warp's rows at a time by way of shared memory, so
            // that a store covers 128 bytes of each of four rows (a thread storing
            // its own row took 5200 clocks a tile)
#pragma unroll
            for (int x = 0; x < DP / 64; ++x) {
                uint32_t o[64] = {};
                if (ok) {
                    tmem_ld32(to + x * 64, o);
                    tmem_ld32(to + x * 64 + 32, o + 32);
                    tmem_wait_ld32(o);
                    tmem_wait_ld32(o + 32);
                    if (x == DP / 64 - 1) {  // the next item may have O
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&ctl.o_free[t]));
                    }
                }
                __syncwarp();
                // a wait that gave up leaves NaN
                const float by = ok ? inv : __uint_as_float(0x7FC00000u);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    Vec16 v;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float2 f = mul2_rn(make_float2(__uint_as_float(o[e * 8 + 2 * y]),
                                                             __uint_as_float(o[e * 8 + 2 * y + 1])),
                                                 make_float2(by, by));
                        bad = fma2_rn(f, make_float2(0.0f, 0.0f), bad);  // 0, or NaN
                        v.w[y] = f32x2_to_bf16x2_bits(f.x, f.y);
                    }
                    *reinterpret_cast<Vec16*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = v;
                }
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = e * 4 + (lane >> 3), piece = lane & 7, d = x * 64 + piece * 8;
                    const Vec16 v = *reinterpret_cast<const Vec16*>(stage + r * 128 + ((piece ^ (r & 7)) << 4));
                    if (row0 + r < it.p.len && d < a.D) *reinterpret_cast<Vec16*>(out + r * a.out_stride + d) = v;
                }
            }
            uint32_t again = __ballot_sync(0xFFFFFFFFu, ok && live && bad.x + bad.y != 0.0f);
            __syncwarp();
            while (again) {
                const int r = __ffs((int)again) - 1;
                again &= again - 1;
                repair_row(a, it.p.begin, row0 + r, min(u / group * kM + kM, it.p.len), head);
            }
        }
        // a wait that gave up: NaN in every row of this CTA's tiles, done or not
        for (int round = 0; !ok && (uint64_t)round * gridDim.x < n_items; ++round) {
            const uint32_t id = item_of(round);
            if (id >= n_items) continue;
            const Pair p = find_pair(a.starts, (int)a.n_seqs, (int)a.T, group, id / (uint32_t)a.Hkv);
            const int u = p.unit + t, row = u / group * kM + (threadIdx.x & 127);
            if (t >= p.units || row >= p.len) continue;
            uint16_t* const out = static_cast<uint16_t*>(a.out) + (p.begin + (int64_t)row) * a.out_stride +
                                  ((int64_t)(id % (uint32_t)a.Hkv) * group + u % group) * a.D;
            for (int d = 0; d < a.D; ++d) out[d] = 0x7FC0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, 512);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeFn>(p);
        cudaGetLastError();
        return static_cast<EncodeFn>(nullptr);
    }();
    return fn;
}

// [T, H, D] bf16 with a token stride, copied in boxes of `rows` tokens of one
// head and 64 entries (128 bytes, swizzled by the place in shared memory, so
// that a box may begin at any row of a tile); zeros outside.
bool encode(CUtensorMap* m, const void* p, int64_t T, int64_t H, int64_t D, int64_t stride, cuuint32_t rows) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, rows}, step[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP>
cudaError_t go(const PromptArgs& a, cudaStream_t st) {
    CUtensorMap mq, mk, mv, mv32, mv8, mv1;
    if (!encode(&mq, a.q, a.T, a.Hq, a.D, a.q_stride, kM) || !encode(&mk, a.k, a.T, a.Hkv, a.D, a.k_stride, kN) ||
        !encode(&mv, a.v, a.T, a.Hkv, a.D, a.v_stride, kN) || !encode(&mv32, a.v, a.T, a.Hkv, a.D, a.v_stride, 32) ||
        !encode(&mv8, a.v, a.T, a.Hkv, a.D, a.v_stride, 8) || !encode(&mv1, a.v, a.T, a.Hkv, a.D, a.v_stride, 1))
        return cudaErrorNotSupported;
    constexpr int smem = Shape<DP>::kBytes;
    static FunctionLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(prompt_tc<DP>), smem);
    if (e != cudaSuccess) return e;
    const int64_t group = a.Hq / a.Hkv, seqs = a.n_seqs < a.T ? a.n_seqs : a.T;
    const int64_t pairs = ((a.T / kM + seqs) * group + (group & 1 ? seqs : 0)) / 2;
    const int64_t items = pairs * a.Hkv, sms = sm_count();
    return launch(prompt_tc<DP>, dim3((unsigned)(items < sms ? items : sms)), dim3(kThreads), smem, st, mq, mk, mv, mv32,
                  mv8, mv1, a, (uint32_t)items);
}

}  // namespace

cudaError_t launch_attn_prompt_tc(const PromptArgs& a, cudaStream_t st) {
    return a.D <= 64 ? go<64>(a, st) : go<128>(a, st);
}

}  // namespace gbe
