// attn_chunk_tc.cu -- attention of new rows behind a cached prefix, and of packed
// prompts under a sliding window, on the tensor cores: bf16 rows, D up to 128,
// on the 16-byte grid.
//
//   S = q k^T (f32, in tensor memory), p = 2^(c S - c m), c = |scale| log2(e),
//   O = sum p v, out = O / sum p
//
// over the keys that a row sees (attn_chunk.cuh).  A CTA goes from item to item:
// one or two tiles of 128 rows -- tokens and the query heads of a kv head, so
// that a few new tokens fill a tile and their keys are read once for all heads --
// and a split of the blocks of 128 keys that they see.  Three warpgroups, as
// attn_prompt_tc.cu has them: one of softmax for each tile (a thread owns a
// row), and one of which a warp finds the items, another issues the tensor
// copies, and two the products, each of a tile.  Tensor memory (512 columns)
// holds one S for both tiles, the weights of each, rounded to bf16, and O of
// each; the products follow one another as
//
//   S0 = q0 k(j+1)^T, O0 += p0 v(j), S1 = q1 k(j+1)^T, O1 += p1 v(j)
//
// Over an 8-bit cache two more warpgroups widen codes and scales to bf16, exactly.
// What their registers leave to the softmax warps does not hold a row of S, so S is
// not free early; each tile has one of its own, the weights take its place, and
// S(j+1) follows O += p v(j).
//
// Both tiles of an item walk the same blocks, so the one with the earlier rows
// may meet a block that none of them sees: its weights are zeros.
//
// Pages come by tensor copies too, of as many rows as divide a page and a block;
// each lane of the copying warp looks up the pages of its boxes a block ahead.
// Rows of v that no row of the sequence may look at -- behind its end, on pages
// that are not in the cache -- are zeros (from behind the tensor's end), since
// a weight of zero times an infinity or a NaN would reach the sum; keys among
// them are masked.  Within the sequence, a row that comes out not finite is
// looked at once more (repair_row).
//
// O is rescaled only when a row's maximum has grown by more than 2^8 over the
// one in use, as in attn_prompt_tc.cu.
//
// Weights are one bf16, 8 bits, as there and for the same reason: it is what a
// product with bf16 keys takes, and tensor memory is full (S, two tiles' weights, two
// O).  Results are 1.25 to 1.4 times as far from the definition as their own rounding
// leaves them (0.0021 to 0.0023 of their norm, 0.0016 to 0.0017); a single token's
// decode, which adds the rest of each weight as a second bf16, 1.0 times.  Sums of
// weights and of products are f32.
//
// Measured, with 32 heads over 8 of D 128 and pages of 64: 2048 tokens behind 30720
// 720 to 780 us, 1.37 to 1.46 PFLOP/s (softmax and products take turns on what the SM
// issues; the longer a GPU is kept at it, the slower); 24 sequences of up to 200 behind
// up to 8000 228 us; 64 of 5 behind 8000 412 us, 5.1 TB/s of keys; a prompt of 8192
// under a window of 1024 131 to 136 us.  Over an 8-bit cache the widening bounds it:
// 2048 behind 30720 1.17 ms, 64 of 5 behind 8000 530 to 545 us
// (eight warps take 1.2 to 1.5 thousand clocks for a block's k, as many for its v;
// with four 650 us, and one warp that waited for each block's pages and then for its
// scales 620).  Not kept: slots that share one tile's blocks, every other one each (545
// us), four warps for k alone and four for v (580), and pages asked into L2 a block
// ahead (bf16, 64 of 5: 426 us for 411).
#include "attn_chunk.cuh"
#include "attn_chunk_row.cuh"
#include "gbe_elementwise.h"
#include "kv_cache.cuh"
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace gbe {
namespace chunk {
namespace {

constexpr int kM = 128, kN = 128;
constexpr int kLoadWarp = 8, kItemWarp = 9, kMmaWarp = 10;  // products: a warp for each tile
constexpr int kWidenWarp = 12, kWidenWarps = 8;  // over an 8-bit cache
constexpr float kGrowth = 8.0f;  // a maximum may lag this many powers of two

// What the item warp hands out.  Of two tiles, tile t goes to slot t -- its
// softmax warpgroup, its thread of products and their tensor memory --; one alone
// goes to the other slot than the one before, so that its first products and
// weights are under way while the last one's rows are written.
struct Todo {
    Item item;
    Walk walk;
    int kvh, slot;  // slot -1: nothing more
    __device__ __forceinline__ int blocks() const { return walk.to - walk.from; }
    __device__ __forceinline__ bool two() const { return item.tiles == 2; }
    __device__ __forceinline__ bool has(int t) const { return two() || slot == t; }
    // the number of slot t's tile
    __device__ __forceinline__ int tile(int t) const { return item.tile + (two() ? t : 0); }
};
constexpr int kTodos = 4;  // in hand

struct Control {
    uint64_t q_full[2], q_empty[2], kv_full[8], kv_empty[8], s_full[2], s_free[2], s_last[2];
    uint64_t p_ready[2], o_done[2], o_free[2], drained[2], raw_full[3], raw_empty[3];
    uint64_t todo_full[kTodos], todo_empty[kTodos], todo_checked[kTodos];
    Todo todo[kTodos];
    int gone[kTodos];  // (once checked) whether a page of the item's walk is not in the cache
    uint32_t tmem;
    int state;  // of the CTA (patience.h)
};

template <int KV, int DP>
struct Shape {
    static constexpr bool kE4 = KV == GBE_KV_E4M3;
    static constexpr int kThreads = kE4 ? 640 : 384;
    // Registers of a thread: 384 threads were launched with 168 each (64512), the
    // softmax warpgroups take 208 and the issuing one keeps 80 (63488); of 640 with
    // 96 (61440), 144, 64 and the widening ones 64 (61440).
    static constexpr int kSoftmaxRegs = kE4 ? 144 : 208, kIssueRegs = kE4 ? 64 : 80, kWidenRegs = 64;
    static constexpr int kReaders = kE4 ? 19 : 11;        // warps that read an item: all but the one that finds it
    static constexpr int kPanel = 128 * 128;              // 128 rows of 64 bf16
    static constexpr int kTile = kPanel * (DP / 64);      // 128 rows of DP
    static constexpr int kStages = (kE4 ? 3 : 4) * (128 / DP);
    static constexpr int kOutRow = kE4 ? 32 : 64;         // bytes of a row on their way out
    static constexpr int kOut = 8 * 32 * kOutRow;         // 32 rows for each softmax warp
    // 8-bit rows on their way in, 64 bytes of each in a panel, and the scales and the pages of kAhead blocks
    static constexpr int kAhead = 8;
    static constexpr int kRaw = kE4 ? kN * DP : 0, kRaws = 3, kRawPanel = kN * 64;
    static constexpr int kRawAt = kTile * (2 + kStages) + kOut, kScaleAt = kRawAt + kRaws * kRaw;
    static constexpr int kPageAt = kScaleAt + (kE4 ? kAhead * 2 * kN : 0);
    static constexpr int kControlAt = kPageAt + (kE4 ? kAhead * 32 * 4 : 0);
    static constexpr int kBytes = kControlAt + 1024 + (int)sizeof(Control);
    // Tensor memory of slot t: O behind 256.  One S for both and weights of each; over an
    // 8-bit cache an S for each, of which the weights take the place.
    __host__ __device__ static constexpr int s_at(int t) { return kE4 ? 128 * t : 0; }
    __host__ __device__ static constexpr int p_at(int t) { return kE4 ? 128 * t : 128 + 64 * t; }
    // where piece c (16 bytes) of row r of a warp's rows lies on its way out
    __device__ static __forceinline__ int out_at(int r, int c) {
        constexpr int kPieces = kOutRow / 16, kSide = 8 / kPieces;  // rows side by side
        return r / kSide * 128 + ((((r % kSide) * kPieces + c) ^ (r / kSide & 7)) << 4);
    }
};

// The copies of a call: q; k and v in boxes of `rows` keys, and v in smaller ones
// (of 32, 8 and 1) where a sequence ends.
struct Maps {
    CUtensorMap q, k, v, v32, v8, v1;
};

// Row r of tile u: its token and head, and whether there is such a row.
struct Row {
    int token, head;
    bool there;
};
__device__ __forceinline__ Row row_of(const Args& g, const Item& it, int u, int r) {
    Row x;
    const int token0 = u / g.parts * g.tokens, head0 = u % g.parts * g.heads;
    x.token = token0 + r / g.heads;
    x.head = head0 + r % g.heads;
    x.there = r < g.tokens * g.heads && x.token < it.s.n && x.head < g.group;
    return x;
}

// After a wait that gave up: NaN in every row of this CTA's items, done or not.
// By one warp.
__device__ __noinline__ void give_up(const Args& g) {
    const ChunkArgs& a = g.a;
    Source items(g, true);
    Item it;
    int kvh;
    while (items.next(it, kvh))
        for (int r = threadIdx.x & 31; r < it.tiles * kM; r += 32) {
            const Row x = row_of(g, it, it.tile + r / kM, r % kM);
            if (!x.there) continue;
            const int head = kvh * g.group + x.head;
            if (it.splits > 1) g.part_ml[part_at(g, it, x.token, head)] = make_float2(0.0f, __uint_as_float(0x7FC00000u));
            uint16_t* const out =
                static_cast<uint16_t*>(a.out) + (it.s.begin + (int64_t)x.token) * a.out_stride + (int64_t)head * a.D;
            for (int d = 0; d < a.D; ++d) out[d] = 0x7FC0;
        }
}

// ---- an 8-bit cache's rows -----------------------------------------------------------

// Sixteen codes times 2^(byte - 127), exact in bf16 from 2^-126 on; byte 0:
// zeros.  A code's bits, its exponent and mantissa moved to where bf16 has them,
// are 2^-120 of its value; one product brings that and the scale.  False for what
// has to go through f32: rows of byte 135 and above (2^(byte - 7) is past bf16's
// range), and NaN codes, which that way come out as 480.
__device__ __forceinline__ bool widen16(const Vec16& codes, uint32_t byte, Vec16& lo, Vec16& hi) {
    uint32_t nan = 0, w[8];
    const uint32_t field = byte == 0 ? 0u : (byte + 120u) << 7, scale = field | field << 16;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        nan |= (codes.w[x] & 0x7F7F7F7Fu) + 0x01010101u;
        // the upper and the lower bytes of four results
        const uint32_t up = (codes.w[x] >> 4 & 0x07070707u) | (codes.w[x] & 0x80808080u);
        const uint32_t low = codes.w[x] << 4 & 0xF0F0F0F0u;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(w[2 * x]) : "r"(__byte_perm(low, up, 0x5140)), "r"(scale));
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(w[2 * x + 1]) : "r"(__byte_perm(low, up, 0x7362)), "r"(scale));
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) lo.w[x] = w[x], hi.w[x] = w[4 + x];
    return byte == 0 || (!(nan & 0x80808080u) && byte <= 134u);
}
__device__ __forceinline__ void widen16_f32(const Vec16& codes, uint32_t byte, Vec16& lo, Vec16& hi) {
    const float s = __uint_as_float(byte << 23);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        float f[4];
        e4m3x4_to_f32(codes.w[x], f);
        uint32_t* const w = x < 2 ? lo.w + 2 * x : hi.w + 2 * (x - 2);
        w[0] = f32x2_to_bf16x2_bits(f[0] * s, f[1] * s);
        w[1] = f32x2_to_bf16x2_bits(f[2] * s, f[3] * s);
    }
}

// The warps that widen an 8-bit cache's rows, as the copying warp brings them,
// into the ring.  Loads are counted over all items: k of block b is 2 b, v 2 b + 1.
template <int DP>
__device__ __forceinline__ void widen_rows(Control& ctl, uint8_t* const smem, const Args& g) {
    using S = Shape<GBE_KV_E4M3, DP>;
    constexpr int kPieces = DP / 16, kRows = kWidenWarps * 32 / kPieces, kTurns = kN / kRows;
    const int tid = threadIdx.x - kWidenWarp * 32, lane = threadIdx.x & 31;
    volatile int* const state = &ctl.state;
    auto until = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, state); };
    auto until_item = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, state, g.patience); };
    // Eight lanes have four pieces of 16 codes of two rows: what they read, and what
    // they write, a piece's halves one after the other, meets eight bank groups.
    const int panel = DP == 128 ? tid >> 3 & 1 : 0, piece = tid & 3;
    const int r0 = DP == 128 ? (tid >> 2 & 1) | tid >> 4 << 1 : tid >> 2;
    const uint8_t* const from = smem + S::kRawAt + panel * S::kRawPanel + r0 * 64 + piece * 16;
    uint8_t* const to = smem + 2 * S::kTile + panel * S::kPanel + r0 * 128;
    int load = 0;
    for (int i = 0;; ++i) {
        if (!__all_sync(0xFFFFFFFFu, until_item(smem_addr(&ctl.todo_full[i % kTodos]), i / kTodos & 1))) return;
        const int n = ctl.todo[i % kTodos].blocks(), slot = ctl.todo[i % kTodos].slot;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ctl.todo_empty[i % kTodos]));
        if (slot < 0) return;
        for (const int end = load + 2 * n; load < end; ++load) {
            const int raw = load % S::kRaws, stage = load % S::kStages;
            bool ok = until(smem_addr(&ctl.raw_full[raw]), load / S::kRaws & 1);
            ok = ok && until(smem_addr(&ctl.kv_empty[stage]), (load / S::kStages & 1) ^ 1);
            if (!__all_sync(0xFFFFFFFFu, ok)) return;
            const uint8_t* const scale = smem + S::kScaleAt + load % (2 * S::kAhead) * kN + r0;
            auto codes = [&](int x) { return *reinterpret_cast<const Vec16*>(from + raw * S::kRaw + x * (kRows * 64)); };
            auto write = [&](int x, const Vec16& lo, const Vec16& hi) {
                const int r = r0 + x * kRows, c = piece * 2;
                uint8_t* const line = to + stage * S::kTile + x * (kRows * 128);
                *reinterpret_cast<Vec16*>(line + ((c ^ (r & 7)) << 4)) = lo;
                *reinterpret_cast<Vec16*>(line + (((c + 1) ^ (r & 7)) << 4)) = hi;
            };
            uint32_t again = 0;
#pragma unroll
            for (int x = 0; x < kTurns; ++x) {
                Vec16 lo, hi;
                if (!widen16(codes(x), scale[x * kRows], lo, hi)) again |= 1u << x;
                write(x, lo, hi);
            }
#pragma unroll 1
            for (; again; again &= again - 1) {
                const int x = __ffs((int)again) - 1;
                Vec16 lo, hi;
                widen16_f32(codes(x), scale[x * kRows], lo, hi);
                write(x, lo, hi);
            }
            async_proxy_fence();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_addr(&ctl.kv_full[stage]));
                mbar_arrive(smem_addr(&ctl.raw_empty[raw]));
            }
        }
    }
}

// An item's rows and their scales on their way in, by the copying warp: pages that
// hold four rows of which the scales lie on the 4-byte grid.  A lane has rows
// 4 lane .. 4 lane + 3 of each block.  What one needs of another is asked for
// blocks ahead, into shared memory: a block's pages four, its scales, of which the
// pages have come by then, two.
template <int DP>
__device__ __forceinline__ bool load_codes(Control& ctl, uint8_t* const smem, const Maps& maps, const Args& g,
                                           const Walk& w, int len, int seq, int kvh, int box, int& loads) {
    using S = Shape<GBE_KV_E4M3, DP>;
    const KvCacheArgs& c = g.a.c;
    const int lane = threadIdx.x & 31, size = c.page_size, boxes = kN / box;
    const int32_t* const table = g.a.table + seq * g.a.max_pages;
    volatile int* const state = &ctl.state;
    auto until = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, state); };
    const uint32_t pages = smem_addr(smem) + S::kPageAt, scales = smem_addr(smem) + S::kScaleAt;
    const int base = loads / 2 - w.from;  // block x of the walk is block base + x of all
    auto ask_page = [&](int x) {
        const int j = w.block(x) * kN + 4 * lane;
        const bool here = x < w.to && j < len;
        cp_async4(pages + ((base + x) % S::kAhead * 32 + lane) * 4, table + (here ? j / size : 0), here ? 4 : 0);
    };
    auto page_of = [&](int x, int l) {
        return *reinterpret_cast<const volatile int32_t*>(smem + S::kPageAt + ((base + x) % S::kAhead * 32 + l) * 4);
    };
    // 0, which makes zeros of a row whatever its codes, behind the sequence's end and where there is no page
    auto ask_scales = [&](int x) {
        const int j = w.block(x) * kN + 4 * lane, page = page_of(x, lane);
        const bool here = x < w.to && j < len && page >= 0 && page < c.n_pages;
        const int64_t at = here ? ((int64_t)page * c.Hkv + kvh) * size + j % size : 0;
        const uint32_t to = scales + (base + x) % S::kAhead * (2 * kN) + 4 * lane;
        cp_async4(to, c.k_scale + at, here ? min(4, len - j) : 0);
        cp_async4(to + kN, c.v_scale + at, here ? min(4, len - j) : 0);
    };
    __syncwarp();
    for (int x = 0; x < 4; ++x) ask_page(w.from + x);
    cp_async_commit();
    cp_async_wait<0>();
    __syncwarp();
    for (int x = 0; x < 2; ++x) {
        ask_scales(w.from + x);
        cp_async_commit();
    }
    bool ok = true;
    for (int x = w.from; x < w.to; ++x) {
        const int j = w.block(x) * kN + lane * box;
        int page = (int)c.n_pages, row = 0;  // (from n_pages on: zeros)
        if (lane < boxes && j < len) {
            const int32_t p = page_of(x, lane * box / 4);
            if (p >= 0 && p < c.n_pages) page = p, row = j % size;
        }
        for (int kv = 0; kv < 2; ++kv, ++loads) {
            const int stage = loads % S::kRaws;
            ok = __all_sync(0xFFFFFFFFu,
                            until(smem_addr(&ctl.raw_empty[stage]), (loads / S::kRaws & 1) ^ 1));
            if (!ok) return false;
            const uint32_t full = smem_addr(&ctl.raw_full[stage]);
            const uint32_t to = smem_addr(smem) + S::kRawAt + stage * S::kRaw + lane * box * 64;
            if (lane < boxes) {
#pragma unroll
                for (int p = 0; p < DP / 64; ++p)
                    tma_load_4d(to + p * S::kRawPanel, kv == 0 ? &maps.k : &maps.v, full, p * 64, row, kvh, page);
            }
            if (kv == 0) {
                cp_async_wait<1>();  // this block's scales, the pages of the block after the next
                __syncwarp();
                ask_page(x + 4);
                ask_scales(x + 2);
                cp_async_commit();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_tx(full, S::kRaw);
        }
    }
    cp_async_wait<0>();
    return true;
}

template <int KV, int DP>
__global__ void __launch_bounds__(Shape<KV, DP>::kThreads, 1)
    chunk_tc(const __grid_constant__ Maps maps, const __grid_constant__ Args g, int box) {
    using S = Shape<KV, DP>;
    extern __shared__ uint8_t raw[];
    const ChunkArgs& a = g.a;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t* const smem = raw + (base - smem_addr(raw));
    Control& ctl = *reinterpret_cast<Control*>(smem + S::kControlAt);
    const uint32_t q_smem = base, kv_smem = base + 2 * S::kTile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* const state = &ctl.state;
    // for what a block's copies, products and weights take, and for an item (of which each slot may have another: the
    // first S of one comes behind the last keys of the other)
    auto until = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, state); };
    auto until_item = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, state, g.patience); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(smem_addr(&ctl.kv_full[i]), S::kE4 ? kWidenWarps : 1);
            mbar_init(smem_addr(&ctl.kv_empty[i]), 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_addr(&ctl.q_full[t]), 1);
            mbar_init(smem_addr(&ctl.q_empty[t]), 1);
            mbar_init(smem_addr(&ctl.s_last[t]), 4);
            mbar_init(smem_addr(&ctl.s_full[t]), 1);
            mbar_init(smem_addr(&ctl.p_ready[t]), 4);
            mbar_init(smem_addr(&ctl.s_free[t]), 4);
            mbar_init(smem_addr(&ctl.o_done[t]), 1);
            mbar_init(smem_addr(&ctl.o_free[t]), 4);
            mbar_init(smem_addr(&ctl.drained[t]), 1);
        }
        for (int i = 0; i < S::kRaws; ++i) {
            mbar_init(smem_addr(&ctl.raw_full[i]), 1);
            mbar_init(smem_addr(&ctl.raw_empty[i]), kWidenWarps);
        }
        for (int i = 0; i < kTodos; ++i) {
            mbar_init(smem_addr(&ctl.todo_full[i]), 1);
            mbar_init(smem_addr(&ctl.todo_checked[i]), 1);
            mbar_init(smem_addr(&ctl.todo_empty[i]), S::kReaders);
        }
        ctl.state = 0;
        mbar_init_fence();
        tma_prefetch(&maps.q);
        tma_prefetch(&maps.k);
        tma_prefetch(&maps.v);
    }
    pdl_begin();
    // (not ahead of it: a kernel before this one may have yet to take its share)
    if (warp == kMmaWarp) tmem_alloc(smem_addr(&ctl.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;

    // false: a wait gave up
    auto todo_ready = [&](int i) { return until_item(smem_addr(&ctl.todo_full[i % kTodos]), i / kTodos & 1); };
    auto todo_read = [&](int i) { mbar_arrive(smem_addr(&ctl.todo_empty[i % kTodos])); };

    if (S::kE4 && warp >= kWidenWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kWidenRegs));
        if constexpr (S::kE4) widen_rows<DP>(ctl, smem, g);
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kIssueRegs));
        if (warp == kItemWarp) {
            Source items(g, true);
            bool ok = true, more = true;
            int tiles[2] = {0, 0};  // of q so far
            int last = 1;           // the slot that S was last for
            Item q_item = {};       // whose q is to be fetched, once its slots' last one is done with
            int q_kvh = 0, q_slot = -1;
            auto load_q = [&](bool wait) {
                if (q_slot < 0) return;
                for (int t = 0; t < 2; ++t)
                    if (q_item.tiles == 2 || t == q_slot) {
                        const uint32_t bar = smem_addr(&ctl.q_empty[t]);
                        if (!wait && !__all_sync(0xFFFFFFFFu, mbar_try(bar, (tiles[t] & 1) ^ 1))) return;
                        ok = ok && __all_sync(0xFFFFFFFFu, until_item(bar, (tiles[t] & 1) ^ 1));
                        if (!ok) return;
                    }
                for (int t = 0; t < 2; ++t)
                    if (q_item.tiles == 2 || t == q_slot) {
                        const int u = q_item.tile + (q_item.tiles == 2 ? t : 0);
                        if (lane == 0) {
                            const uint32_t qb = smem_addr(&ctl.q_full[t]);
                            mbar_arrive_tx(qb, (DP / 64) * 128 * g.heads * g.tokens);
#pragma unroll
                            for (int p = 0; p < DP / 64; ++p)
                                tma_load_3d(q_smem + t * S::kTile + p * S::kPanel, &maps.q, qb, p * 64,
                                            q_kvh * g.group + u % g.parts * g.heads,
                                            q_item.s.begin + u / g.parts * g.tokens);
                        }
                        ++tiles[t];
                    }
                q_slot = -1;
            };
            for (int i = 0; ok && more; ++i) {
                Todo todo;
                more = items.next(todo.item, todo.kvh);
                todo.slot = -1;
                if (more) {
                    todo.walk = walk(g, todo.item);
                    todo.slot = todo.two() || todo.blocks() == 0 ? 0 : last ^ 1;
                    if (todo.blocks() > 0) last = todo.two() ? 1 : todo.slot;
                }
                ok = __all_sync(0xFFFFFFFFu,
                                until_item(smem_addr(&ctl.todo_empty[i % kTodos]), (i / kTodos & 1) ^ 1));
                if (!ok) break;
                if (lane == 0) {
                    ctl.todo[i % kTodos] = todo;
                    mbar_arrive(smem_addr(&ctl.todo_full[i % kTodos]));
                }
                load_q(true);  // the item's before
                if (!more || !ok) break;
                if (todo.blocks() > 0) q_item = todo.item, q_kvh = todo.kvh, q_slot = todo.slot;
                load_q(false);
                if constexpr (KV != kPacked) {
                    const Walk& w = todo.walk;
                    bool gone = false;
                    auto check = [&](int from, int to) {  // pages that hold keys from .. to - 1
                        to = min(to, todo.item.s.len);
                        const int32_t* const pages = a.table + todo.item.seq * a.max_pages;
                        for (int p = from / a.c.page_size + lane; p * (int64_t)a.c.page_size < to; p += 32)
                            gone = gone || pages[p] < 0 || pages[p] >= a.c.n_pages;
                    };
                    if (w.from < w.sinks) check(w.from * kN, min(w.to, w.sinks) * kN);
                    if (w.to > w.sinks) check(w.block(max(w.from, w.sinks)) * kN, w.block(w.to) * kN);
                    gone = __any_sync(0xFFFFFFFFu, gone);
                    if (lane == 0) {
                        ctl.gone[i % kTodos] = gone;
                        mbar_arrive(smem_addr(&ctl.todo_checked[i % kTodos]));
                    }
                }
            }
            if (*state > 0 && lane == 0) {  // nothing may still be on its way when the CTA ends
                int none = 0;
                for (int t = 0; t < 2; ++t)
                    if (tiles[t] > 0) mbar_wait(smem_addr(&ctl.q_full[t]), (tiles[t] - 1) & 1, &none);
            }
        } else if (warp == kLoadWarp) {
            int loads = 0;               // of the ring so far; of an 8-bit cache, of the one ahead of it
            bool ok = true;
            const int boxes = kN / box;  // of a block; a power of two
            // four rows' scales lie together, on the 4-byte grid
            const bool fours = S::kE4 && box >= 4 && ((uintptr_t)a.c.k_scale | (uintptr_t)a.c.v_scale) % 4 == 0;
            for (int i = 0; ok; ++i) {
                if (!(ok = __all_sync(0xFFFFFFFFu, todo_ready(i)))) break;
                const Todo& todo = ctl.todo[i % kTodos];
                const Walk w = todo.walk;
                const int kvh = todo.kvh, slot = todo.slot;
                const struct {
                    Seq s;
                    int seq;
                } it = {todo.item.s, todo.item.seq};
                __syncwarp();
                if (lane == 0) todo_read(i);
                if (slot < 0) break;
                if (w.from == w.to) continue;
                if constexpr (S::kE4) {
                    if (fours) {
                        ok = load_codes<DP>(ctl, smem, maps, g, w, it.s.len, it.seq, kvh, box, loads);
                        continue;
                    }
                }
                // box b of the walk's block x: the page (from n_pages on: zeros) and the row in it
                auto look_up = [&](int x, int b, int& page, int& row) {
                    const int j = w.block(x) * kN + b * box;
                    if constexpr (KV == kPacked) {
                        page = 0, row = it.s.begin + j;
                    } else {
                        page = (int)a.c.n_pages, row = 0;
                        if (x < w.to && b < boxes && j < it.s.len) {
                            const int page_i = j / a.c.page_size;
                            const int32_t p = a.table[it.seq * a.max_pages + page_i];
                            if (p >= 0 && p < a.c.n_pages) page = p, row = j - page_i * a.c.page_size;
                        }
                    }
                };
                constexpr int kPanel = S::kE4 ? S::kRawPanel : S::kPanel, kLine = S::kE4 ? 64 : 128;
                auto copy = [&](uint32_t to, const CUtensorMap* m, uint32_t full, int page, int row) {
#pragma unroll
                    for (int p = 0; p < DP / 64; ++p) {
                        if constexpr (KV == kPacked)
                            tma_load_3d(to + p * kPanel, m, full, p * 64, kvh, row);
                        else
                            tma_load_4d(to + p * kPanel, m, full, p * 64, row, kvh, page);
                    }
                };
                // An 8-bit cache's scales of rows 4 lane .. 4 lane + 3 of the walk's block x, a byte each; 0, which
                // makes zeros of a row whatever its codes, behind the sequence's end and where there is no page.
                uint32_t k_bytes = 0, v_bytes = 0;
                auto ask = [&](int x) {
                    k_bytes = v_bytes = 0;
                    const int j = w.block(x) * kN + 4 * lane;
                    int page = -1, row = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (x >= w.to || j + e >= it.s.len) break;
                        if (e == 0 || ++row == a.c.page_size) {
                            const int page_i = (j + e) / a.c.page_size;
                            row = j + e - page_i * a.c.page_size;
                            page = a.table[it.seq * a.max_pages + page_i];
                        }
                        if (page < 0 || page >= a.c.n_pages) continue;
                        const int64_t at = ((int64_t)page * a.c.Hkv + kvh) * a.c.page_size + row;
                        k_bytes |= (uint32_t)a.c.k_scale[at] << 8 * e;
                        v_bytes |= (uint32_t)a.c.v_scale[at] << 8 * e;
                    }
                };
                if constexpr (S::kE4) ask(w.from);
                int page, row;
                look_up(w.from, lane, page, row);
                for (int x = w.from; ok && x < w.to; ++x) {
                    const int have0 = it.s.len - w.block(x) * kN;  // of the block's rows
                    for (int kv = 0; kv < 2; ++kv) {
                        constexpr int kRing = S::kE4 ? S::kRaws : S::kStages, kBytes = S::kE4 ? S::kRaw : S::kTile;
                        const int stage = loads % kRing;
                        ok = __all_sync(0xFFFFFFFFu,
                                        until(smem_addr(S::kE4 ? &ctl.raw_empty[stage] : &ctl.kv_empty[stage]),
                                              (loads / kRing & 1) ^ 1));
                        if (!ok) break;
                        const uint32_t full = smem_addr(S::kE4 ? &ctl.raw_full[stage] : &ctl.kv_full[stage]);
                        const uint32_t to = S::kE4 ? smem_addr(smem) + S::kRawAt + stage * kBytes : kv_smem + stage * kBytes;
                        if constexpr (S::kE4) {
                            *reinterpret_cast<uint32_t*>(smem + S::kScaleAt + loads % (2 * S::kAhead) * kN + 4 * lane) =
                                kv == 0 ? k_bytes : v_bytes;
                            if (kv == 1) ask(x + 1);
                            __syncwarp();
                        }
                        if (lane == 0) mbar_arrive_tx(full, kBytes);
                        __syncwarp();
                        for (int b = lane; b < boxes; b += 32) {
                            if (b >= 32) look_up(x, b, page, row);
                            const int have = have0 - b * box;
                            const uint32_t at = to + b * box * kLine;
                            // (widening makes zeros of what is behind the end)
                            if (S::kE4 || kv == 0 || have >= box || (KV != kPacked && (have <= 0 || page == a.c.n_pages))) {
                                copy(at, kv == 0 ? &maps.k : &maps.v, full, page, row);
                                continue;
                            }
                            if constexpr (!S::kE4) {  // v where the sequence ends within the box: zeros from there on
                                for (int r = 0; r < box;) {
                                    const int left = have - r;
                                    auto part = [&](const CUtensorMap* m, int rows) {
                                        const bool zeros = left <= 0;
                                        copy(at + r * 128, m, full, zeros ? (int)a.c.n_pages : page,
                                             zeros && KV == kPacked ? (int)a.T : row + r);
                                        r += rows;
                                    };
                                    if (r % 32 == 0 && box >= 32 && (left >= 32 || left <= 0))
                                        part(&maps.v32, 32);
                                    else if (r % 8 == 0 && box >= 8 && (left >= 8 || left <= 0))
                                        part(&maps.v8, 8);
                                    else
                                        part(&maps.v1, 1);
                                }
                            }
                        }
                        if (boxes > 32) look_up(x, lane, page, row);  // (the last one of these was looked up last)
                        ++loads;
                    }
                    look_up(x + 1, lane, page, row);
                }
            }
            if constexpr (S::kE4) cp_async_wait<0>();  // as above
            __syncwarp();
            if (*state > 0 && lane == 0) {
                int none = 0;
                constexpr int kRing = S::kE4 ? S::kRaws : S::kStages;
                for (int x = max(0, loads - kRing); x < loads; ++x)
                    mbar_wait(smem_addr(S::kE4 ? &ctl.raw_full[x % kRing] : &ctl.kv_full[x % kRing]), x / kRing & 1,
                              &none);
            }
        } else if (elect_one()) {
            const int t = warp - kMmaWarp;
            const uint32_t idesc_s = bf16_idesc(kM, kN, false) | (a.scale < 0.0f ? 1u << 13 : 0u);
            constexpr uint32_t idesc_o = bf16_idesc(kM, DP, true), hi = smem_desc_hi(1024);
            const uint32_t q_lo = smem_desc_lo(q_smem + t * S::kTile, 16), k_lo = smem_desc_lo(kv_smem, 16);
            const uint32_t v_lo = smem_desc_lo(kv_smem, S::kPanel);
            const uint32_t o = tmem + 256 + t * 128;
            bool ok = true;
            int loads = 0;          // the ring's before this item: k of block j is load loads + 2 j
            int done[2] = {0, 0};   // blocks of each slot before this item
            int items = 0;          // items with blocks, of this slot
            int every = 0;          // and of either
            for (int i = 0; ok; ++i) {
                if (!(ok = todo_ready(i))) break;
                const Todo& todo = ctl.todo[i % kTodos];
                const int n = todo.blocks(), slot = todo.slot;
                const bool two = todo.two(), mine = todo.has(t);
                todo_read(i);
                if (slot < 0) break;
                if (n == 0) continue;
                auto loaded = [&](int x) {
                    ok = ok && until(smem_addr(&ctl.kv_full[x % S::kStages]), x / S::kStages & 1);
                };
                // S is free for an item once the last block of the item before has been read.  Both threads wait for
                // that at every item, so that neither passes over a phase (a wait by parity holds only where the phase
                // before has completed); two barriers in turn, for a thread may be as far behind as the other's item.
                if (!S::kE4 && every > 0)
                    ok = until(smem_addr(&ctl.s_last[(every - 1) & 1]), (every - 1) / 2 & 1);
                // And within it once the block before in the order (0, j), (1, j), (0, j + 1), ... has been.  (Over an
                // 8-bit cache it is free once the weights that took its place have met v.)
                auto s_free = [&](int j) {
                    if constexpr (S::kE4) {
                        if (done[t] + j > 0)
                            ok = ok && until(smem_addr(&ctl.o_done[t]), (done[t] + j - 1) & 1);
                    } else {
                        const int pt = !two ? t : t ^ 1, pj = two && t == 1 ? j : j - 1;
                        if (pj >= 0) ok = ok && until(smem_addr(&ctl.s_free[pt]), (done[pt] + pj) & 1);
                    }
                };
                auto scores = [&](int j) {
                    const int x = loads + 2 * j, stage = x % S::kStages;
                    loaded(x);
                    s_free(j);
                    if (!ok) return;
                    tc_fence_after();
                    const uint32_t k0 = k_lo + stage * (S::kTile >> 4);
#pragma unroll
                    for (int y = 0; y < DP / 16; ++y) {
                        const uint32_t off = ((y / 4) * S::kPanel + (y % 4) * 32) >> 4;
                        mma_ss(tmem + S::s_at(t), q_lo + off, hi, k0 + off, hi, idesc_s, y > 0);
                    }
                    mma_commit(smem_addr(&ctl.s_full[t]));
                    mma_commit(smem_addr(&ctl.kv_empty[stage]));
                    if (j + 1 == n) mma_commit(smem_addr(&ctl.q_empty[t]));
                };
                if (mine) {
                    ok = ok && until(smem_addr(&ctl.q_full[t]), items & 1);
                    if (!S::kE4) scores(0);
                }
                for (int j = 0; ok && mine && j < n; ++j) {
                    if (S::kE4)
                        scores(j);
                    else if (j + 1 < n)
                        scores(j + 1);
                    const int x = loads + 2 * j + 1, stage = x % S::kStages;
                    loaded(x);
                    ok = ok && until(smem_addr(&ctl.p_ready[t]), (done[t] + j) & 1);
                    // O has been read for the last item
                    if (j == 0 && items > 0) ok = ok && until(smem_addr(&ctl.o_free[t]), (items - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t v0 = v_lo + stage * (S::kTile >> 4);
#pragma unroll
                    for (int y = 0; y < kN / 16; ++y)
                        mma_ts(o, tmem + S::p_at(t) + y * 8, v0 + y * (2048 >> 4), hi, idesc_o, j > 0 || y > 0);
                    mma_commit(smem_addr(&ctl.o_done[t]));
                    mma_commit(smem_addr(&ctl.kv_empty[stage]));
                }
                // blocks that only the other slot works on
                for (int x = loads; ok && !mine && x < loads + 2 * n; ++x) {
                    loaded(x);
                    if (ok) mbar_arrive(smem_addr(&ctl.kv_empty[x % S::kStages]));
                }
                loads += 2 * n;
                if (two || slot == 0) done[0] += n;
                if (two || slot == 1) done[1] += n;
                items += mine;
                ++every;
            }
            // every product is done before tensor memory is given back
            mma_commit(smem_addr(&ctl.drained[t]));
            int none = 0;
            mbar_wait(smem_addr(&ctl.drained[t]), 0, &none);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kSoftmaxRegs));
        const int t = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
        const uint32_t ts = tmem + S::s_at(t) + lanes, tp = tmem + S::p_at(t) + lanes, to = tmem + 256 + t * 128 + lanes;
        // (never 0, so that c times the -inf of a masked place stays -inf)
        const float c = fmaxf(fabsf(a.scale) * kLog2e, __uint_as_float(1u));
        uint8_t* const stage = smem + S::kTile * (2 + S::kStages) + warp * (S::kOut / 8);
        bool ok = true;
        int done = 0;   // blocks of this slot before this item
        int every = 0;  // items with blocks, of either
        for (int i = 0; ok; ++i) {
            ok = __all_sync(0xFFFFFFFFu, todo_ready(i));
            if (!ok) break;
            // (what an item is stays where it is until its rows are written: registers are for S)
            const Todo& todo = ctl.todo[i % kTodos];
            const int n = todo.blocks();
            const bool end = todo.slot < 0;
            if (end || !todo.has(t)) {
                __syncwarp();
                if (lane == 0) todo_read(i);
                if (end) break;
                every += n > 0;
                continue;
            }
            bool gone = false;  // whether pages of the walk are not in the cache
            if constexpr (KV != kPacked) {
                ok = __all_sync(0xFFFFFFFFu,
                                until_item(smem_addr(&ctl.todo_checked[i % kTodos]), i / kTodos & 1));
                if (!ok) break;
                gone = ctl.gone[i % kTodos];
            }
            // S has been read; for the item's last time?
            auto s_read = [&](int j) {
                if (lane != 0) return;
                mbar_arrive(smem_addr(&ctl.s_free[t]));
                if (j == n - 1 && (t == 1 || !todo.two())) mbar_arrive(smem_addr(&ctl.s_last[every & 1]));
            };
            int place;
            bool idle;
            {
                const Row mine = row_of(g, todo.item, todo.tile(t), threadIdx.x & 127);
                place = todo.item.s.len - todo.item.s.n + mine.token;
                // a warp without a row that is there leaves its weights as they are: its rows of O are not looked at
                idle = !__any_sync(0xFFFFFFFFu, mine.there);
            }
            // every row of the warp sees the keys of a block that are before `sure`, and under a window behind `low`
            const int sure = __shfl_sync(0xFFFFFFFFu, place, 0) + 1;
            const int low = g.window > 0 ? __shfl_sync(0xFFFFFFFFu, place, 31) - g.window : -1;
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; idle && j < n; ++j) {
                ok = until_item(smem_addr(&ctl.s_full[t]), (done + j) & 1);
                if (!S::kE4) s_read(j);
                // (no sooner than the others: it would be counted for the weights before)
                if (j > 0) ok = ok && until(smem_addr(&ctl.o_done[t]), (done + j - 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                if (lane == 0) mbar_arrive(smem_addr(&ctl.p_ready[t]));
            }
            for (int j = 0; !idle && j < n; ++j) {
                const int k0 = todo.walk.block(todo.walk.from + j) * kN;
                const bool whole = !gone && k0 + kN <= sure && (k0 > low || k0 + kN <= g.sinks);
                if (KV != kPacked && gone) {  // (left where rows are written from: registers are for S)
#pragma unroll 1
                    for (int y = 0; y < 4; ++y) {
                        const int key = k0 + 32 * y + lane;
                        const bool here = key < todo.item.s.len && key_at<KV>(a, todo.item, todo.kvh, key) >= 0;
                        const uint32_t word = __ballot_sync(0xFFFFFFFFu, here);
                        if (lane == 0) reinterpret_cast<uint32_t*>(stage)[y] = word;
                    }
                    __syncwarp();
                }
                ok = __all_sync(0xFFFFFFFFu, until_item(smem_addr(&ctl.s_full[t]), (done + j) & 1));
                if (!ok) break;
                tc_fence_after();
                // a word's bits: which of 32 keys of the block are seen; the maximum of some logits, what is in use moved up
                auto seen = [&](int y) {
                    uint32_t word = seen_word(g, place, k0, y);
                    if (KV != kPacked && gone) word &= reinterpret_cast<const uint32_t*>(stage)[y];
                    return word;
                };
                auto last_done = [&] {  // the product with the last weights is done
                    ok = __all_sync(0xFFFFFFFFu, until(smem_addr(&ctl.o_done[t]), (done + j - 1) & 1));
                    tc_fence_after();
                };
                auto move_up = [&](float top) {
                    const bool grow = m == -INFINITY ? top > m : (top - m) * c > kGrowth;
                    if (!__any_sync(0xFFFFFFFFu, grow)) return;
                    const float m2 = grow ? top : m;
                    if (j > 0) {
                        if (!S::kE4) last_done();
                        if (!ok) return;
                        const float r = m == -INFINITY ? 0.0f : ex2((m - m2) * c);
                        l *= r;
#pragma unroll
                        for (int y = 0; y < DP; y += S::kE4 ? 16 : 32) {
                            uint32_t o[S::kE4 ? 16 : 32];
                            if constexpr (S::kE4)
                                tmem_ld16(to + y, o), tmem_wait_ld16(o);
                            else
                                tmem_ld32(to + y, o), tmem_wait_ld32(o);
#pragma unroll
                            for (uint32_t& e : o) e = __float_as_uint(__uint_as_float(e) * r);
                            if constexpr (S::kE4)
                                tmem_st16(to + y, o);
                            else
                                tmem_st32(to + y, o);
                        }
                    }
                    m = m2;
                };
                if constexpr (!S::kE4) {
                    // all of a row's logits in registers, and S given up at once
                    uint32_t s[128];
#pragma unroll
                    for (int y = 0; y < 4; ++y) tmem_ld32(ts + y * 32, s + y * 32);
#pragma unroll
                    for (int y = 0; y < 4; ++y) tmem_wait_ld32(s + y * 32);
                    tc_fence_before();
                    __syncwarp();
                    s_read(j);
                    if (!whole) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const uint32_t word = seen(y);
#pragma unroll
                            for (int e = 0; e < 32; ++e) s[32 * y + e] = word >> e & 1u ? s[32 * y + e] : 0xFF800000u;
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int y = 0; y < 128; y += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[y + e]), __uint_as_float(s[y + 4 + e])));
                    move_up(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                    if (!ok) break;
                    const float shift = m == -INFINITY ? 0.0f : -m * c;
                    const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
                    float2 sum[4] = {};
                    uint32_t p[64];
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        float2 y = fma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2,
                                           shift2);
                        y.x = ex2(y.x), y.y = ex2(y.y);
                        sum[e & 3] = add2_rn(sum[e & 3], y);
                        p[e] = f32x2_to_bf16x2_bits(y.x, y.y);
                    }
                    const float2 add = add2_rn(add2_rn(sum[0], sum[1]), add2_rn(sum[2], sum[3]));
                    l += add.x + add.y;
                    if (j > 0) {
                        last_done();
                        if (!ok) break;
                    }
                    tmem_st32(tp, p);
                    tmem_st32(tp + 32, p + 32);
                } else {
                    // The registers are the widening warps' too: keys 64 .. 95 are read once more.  (The product before
                    // this one was done with the weights before S took their place.)
                    uint32_t s[64], b[32];
                    auto read = [&](int y, uint32_t* to) { tmem_ld32(ts + 32 * y, to); };
                    auto there = [&](int y, uint32_t* to) {
                        tmem_wait_ld32(to);
                        if (whole) return;
                        const uint32_t word = seen(y);
#pragma unroll
                        for (int e = 0; e < 32; ++e) to[e] = word >> e & 1u ? to[e] : 0xFF800000u;
                    };
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    auto top = [&](const uint32_t* of) {
#pragma unroll
                        for (int y = 0; y < 32; y += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(of[y + e]), __uint_as_float(of[y + 4 + e])));
                    };
                    read(2, b), read(0, s), read(1, s + 32);
                    there(2, b);
                    top(b);
                    there(0, s), there(1, s + 32);
                    read(3, b);
                    top(s), top(s + 32);
                    there(3, b);
                    top(b);
                    move_up(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                    if (!ok) break;
                    const float shift = m == -INFINITY ? 0.0f : -m * c;
                    const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
                    float2 sum[2] = {};
                    auto weigh = [&](int y, const uint32_t* of) {
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 z = fma2_rn(make_float2(__uint_as_float(of[2 * e]), __uint_as_float(of[2 * e + 1])),
                                               c2, shift2);
                            z.x = ex2(z.x), z.y = ex2(z.y);
                            sum[e & 1] = add2_rn(sum[e & 1], z);
                            p[e] = f32x2_to_bf16x2_bits(z.x, z.y);
                        }
                        tmem_st16(tp + 16 * y, p);
                    };
                    weigh(3, b);
                    read(2, b);
                    weigh(0, s), weigh(1, s + 32);
                    there(2, b);
                    weigh(2, b);
                    const float2 add = add2_rn(sum[0], sum[1]);
                    l += add.x + add.y;
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl.p_ready[t]));
            }
            every += n > 0;
            done += n;
            if (n > 0) ok = ok && until(smem_addr(&ctl.o_done[t]), (done - 1) & 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            // nothing but NaN: a finite maximum, so that it reaches the join
            if (m == -INFINITY && l != l) m = -3.0e38f;
            const Item it = todo.item;
            const int kvh = todo.kvh;
            const Row mine = row_of(g, it, todo.tile(t), threadIdx.x & 127);
            const bool is_part = it.splits > 1;
            // where the row lies, of the partial results or of out; -1: there is none
            const int head = kvh * g.group + mine.head;
            const int64_t part = mine.there && is_part ? part_at(g, it, mine.token, head) : -1;
            const int64_t row = !mine.there ? -1
                                : is_part   ? part * a.D
                                            : (it.s.begin + (int64_t)mine.token) * a.out_stride + (int64_t)head * a.D;
            float2 bad = make_float2(0.0f, 0.0f);
            // Some bytes of the warp's rows at a time by way of shared memory, so that
            // a store covers all of them in several rows; 16 bytes a piece, which `piece`
            // makes of the row's entries at d
            constexpr int kPieces = S::kOutRow / 16, kSide = 32 / kPieces;  // rows that a store covers
            auto write = [&](char* base, int es, int d0, auto piece) {
                __syncwarp();
#pragma unroll
                for (int e = 0; e < kPieces; ++e)
                    *reinterpret_cast<Vec16*>(stage + S::out_at(lane, e)) = piece(e);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < kPieces; ++e) {
                    const int r = e * kSide + lane / kPieces, d = d0 + lane % kPieces * (16 / es);
                    const int64_t at = __shfl_sync(0xFFFFFFFFu, row, r);
                    const Vec16 v = *reinterpret_cast<const Vec16*>(stage + S::out_at(r, lane % kPieces));
                    if (at >= 0 && d < a.D) *reinterpret_cast<Vec16*>(base + (at + d) * es) = v;
                }
            };
            if (part >= 0) g.part_ml[part] = make_float2(m == -INFINITY || m == -3.0e38f ? m : m * c, l);
            const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
            // (rolled: code that runs once an item is fetched again each time)
#pragma unroll 1
            for (int x = 0; x < DP; x += 32) {
                uint32_t o[32] = {};
                if (n > 0) {
                    tmem_ld32(to + x, o);
                    tmem_wait_ld32(o);
                    if (x == DP - 32) {  // the next item may have O
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&ctl.o_free[t]));
                    }
                }
                const float by = is_part ? 1.0f : inv;
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 f = mul2_rn(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])),
                                             make_float2(by, by));
                    bad = fma2_rn(f, make_float2(0.0f, 0.0f), bad);  // 0, or NaN
                    o[e] = __float_as_uint(f.x), o[e + 1] = __float_as_uint(f.y);
                }
                if (is_part) {
                    constexpr int kEntries = S::kOutRow / 4;
#pragma unroll
                    for (int y = 0; y < 32; y += kEntries)
                        write(reinterpret_cast<char*>(g.part_o), 4, x + y, [&](int e) {
                            const uint32_t* const z = o + y + 4 * e;
                            return Vec16{{z[0], z[1], z[2], z[3]}};
                        });
                } else {
                    constexpr int kEntries = S::kOutRow / 2;
#pragma unroll
                    for (int y = 0; y < 32; y += kEntries)
                        write(static_cast<char*>(a.out), 2, x + y, [&](int e) {
                            Vec16 v;
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                v.w[z] = f32x2_to_bf16x2_bits(__uint_as_float(o[y + 8 * e + 2 * z]),
                                                              __uint_as_float(o[y + 8 * e + 2 * z + 1]));
                            return v;
                        });
                }
            }
            uint32_t again = __ballot_sync(0xFFFFFFFFu, mine.there && bad.x + bad.y != 0.0f);
            __syncwarp();
            if (again) {
                if (lane == 0) long_work_begins(state);
                for (; again; again &= again - 1) {
                    const int r = __ffs((int)again) - 1;
                    repair_row<KV>(g, it, kvh, __shfl_sync(0xFFFFFFFFu, mine.token, r),
                                   __shfl_sync(0xFFFFFFFFu, mine.head, r));
                }
                if (lane == 0) long_work_ends(state);
            }
            if (lane == 0) todo_read(i);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, 512);
    if (*state > 0 && warp == 0) give_up(g);
}

// k or v: pages of a cache, or packed rows; in boxes of `rows` keys of one head.
bool encode_kv(CUtensorMap* m, const ChunkArgs& a, bool second, cuuint32_t rows) {
    if (a.packed) {
        const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hkv, (cuuint64_t)a.T};
        const cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)(second ? a.v_stride : a.k_stride) * 2};
        const cuuint32_t box[3] = {64, 1, rows};
        return encode_bf16(m, second ? a.v : a.k, 3, dims, strides, box);
    }
    const KvCacheArgs& c = a.c;
    const cuuint64_t es = c.dtype == GBE_KV_E4M3 ? 1 : 2, page = (cuuint64_t)c.page_size * c.D * es;
    const cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.page_size, (cuuint64_t)c.Hkv, (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.D * es, page,
                                   c.n_pages > 1 ? (cuuint64_t)c.page_stride * es : page * c.Hkv};
    const cuuint32_t box[4] = {64, rows, 1, 1};
    if (es == 1) return encode_bytes(m, second ? c.v : c.k, 4, dims, strides, box);
    return encode_bf16(m, second ? c.v : c.k, 4, dims, strides, box);
}

template <int KV, int DP>
cudaError_t go(const ChunkArgs& a, cudaStream_t st) {
    using S = Shape<KV, DP>;
    const Args g = make_args(a, kM, 2, kN);
    cuuint32_t box = kN;  // keys of a copy: the largest power of two that divides a page, and at most a block
    if (KV != kPacked)
        while (a.c.page_size % box) box /= 2;
    Maps maps;
    const cuuint64_t dims[3] = {(cuuint64_t)a.D, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
    const cuuint64_t strides[2] = {(cuuint64_t)a.D * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t q_box[3] = {64, (cuuint32_t)g.heads, (cuuint32_t)g.tokens};
    if (!encode_bf16(&maps.q, a.q, 3, dims, strides, q_box)) return cudaErrorNotSupported;
    if (!encode_kv(&maps.k, a, false, box) || !encode_kv(&maps.v, a, true, box) ||
        !encode_kv(&maps.v32, a, true, box < 32 ? box : 32) || !encode_kv(&maps.v8, a, true, box < 8 ? box : 8) ||
        !encode_kv(&maps.v1, a, true, 1))
        return cudaErrorNotSupported;
    constexpr int smem = S::kBytes;
    static_assert(smem <= 227 * 1024);
    static FunctionLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(chunk_tc<KV, DP>), smem);
    if (e != cudaSuccess) return e;
    const int64_t seqs = a.n_seqs < a.T ? a.n_seqs : a.T, sms = sm_count();
    const int64_t pieces = (a.T / g.tokens + seqs) * g.parts * a.Hkv * g.most;
    return launch(chunk_tc<KV, DP>, dim3((unsigned)(pieces < sms ? pieces : sms)), dim3(S::kThreads), smem, st, maps, g,
                  (int)box);
}

}  // namespace

cudaError_t launch_tc(const ChunkArgs& a, cudaStream_t st) {
    if (a.packed) return a.D <= 64 ? go<kPacked, 64>(a, st) : go<kPacked, 128>(a, st);
    if (a.c.dtype == GBE_KV_E4M3) return a.D <= 64 ? go<GBE_KV_E4M3, 64>(a, st) : go<GBE_KV_E4M3, 128>(a, st);
    return a.D <= 64 ? go<GBE_KV_BF16, 64>(a, st) : go<GBE_KV_BF16, 128>(a, st);
}

}  // namespace chunk
}  // namespace gbe
