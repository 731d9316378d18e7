// attn_chunk.cu -- attention of new rows behind a cached prefix, and of packed
// prompts under a sliding window: f32, and what attn_chunk_tc.cu does not take;
// and the join of partial results, of both.
//
//   out[i, h] = sum_j p_ij v_j,  p_i = softmax_j(scale * q[i, h] . k_j)
//
// over the keys that row i sees (attn_chunk.cuh).  On the CUDA cores, f32
// throughout.  A CTA goes from item to item: 32 rows -- tokens and the query
// heads of a kv head -- and their keys, or a part of these, in tiles of 64 with the
// running maximum and sum of the softmax (base 2: scale * log2(e) is folded into q).
// Eight by sixteen threads, a thread holding 4 x 4 logits and 4 x D/16 of the
// output, two multiply-adds an instruction; up to D = 128 two groups of threads
// take every other tile and join their sums.  f32 rows come by asynchronous
// copies, v while the logits are formed and the next k while the output is; where
// a row lies is looked up a tile ahead.  The multiply-adds and their operands'
// loads from shared memory bound it: five sequences of up to 100 rows behind up to
// 900, 14 heads over 2 of D 64, window 500: 50 us; three prompts of up to 1000, 8
// heads of D 64, window 129: 50 us.
#include <new>
#include <type_traits>

#include "attn_chunk.cuh"
#include "gbe_elementwise.h"
#include "kv_cache.cuh"

namespace gbe {
namespace chunk {
namespace {

constexpr int kThreads = 128;  // of a group
constexpr int kN = 64, kM = 32, R = kM / 8;

template <int DP>
constexpr int kGroups = DP <= 128 ? 2 : 1;
template <int DP>
constexpr int kGroupFloats = 2 * kN * (DP + 4) + kM * (kN + 4);  // k, v and weights

// Where the rows of a tile's keys lie, looked up by 64 threads.
struct Places {
    int64_t at[kN];      // the first entry; -1: there is none, or nothing may be looked at
    int64_t scale[kN];   // of an 8-bit cache
    uint32_t live[2];
};

// 64 rows into shared memory as f32; zeros where there is none and behind D.
// SRC: the type that memory holds.
template <int SRC, int DP>
__device__ __forceinline__ void stage(float* dst, const void* src, const uint8_t* scales, const Places& pl, int D) {
    constexpr int W = DP + 4;
    for (int i = threadIdx.x & (kThreads - 1); i < kN * (DP / 8); i += kThreads) {
        const int r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
        float f[8] = {};
        const int64_t at = pl.at[r];
        if (at >= 0 && d < D) {
            if constexpr (SRC == GBE_KV_E4M3) {
                const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(src) + at + d);
                const float s = __uint_as_float((uint32_t)scales[pl.scale[r]] << 23);
                if (s != 0.0f) {  // zeros, whatever the codes
                    e4m3x4_to_f32(w.x, f);
                    e4m3x4_to_f32(w.y, f + 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] *= s;
                }
            } else {
                constexpr int V = Store<SRC>::V;
#pragma unroll
                for (int p = 0; p < 8 / V; ++p) {
                    float g[V];
                    Store<SRC>::unpack(ld_reuse(static_cast<const char*>(src) +
                                                (at + d + p * V) * (int64_t)sizeof(typename Store<SRC>::T)), g);
#pragma unroll
                    for (int e = 0; e < V; ++e) f[p * V + e] = g[e];
                }
            }
        }
        float4* o = reinterpret_cast<float4*>(dst + r * W + d);
        o[0] = make_float4(f[0], f[1], f[2], f[3]);
        o[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

template <int DP>
__device__ __forceinline__ void stage_async(float* dst, const float* src, const Places& pl, int D) {
    constexpr int W = DP + 4;
#pragma unroll 4
    for (int i = threadIdx.x & (kThreads - 1); i < kN * (DP / 4); i += kThreads) {
        const int r = i / (DP / 4), d = (i - r * (DP / 4)) * 4;
        const int64_t at = pl.at[r];
        const bool there = at >= 0 && d < D;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(dst + r * W + d)),
                     "l"(src + (there ? at + d : 0)), "r"(there ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// DT: of q and out.  KV: what the cache holds, or kPacked.  VEC: packed rows on
// the 16-byte grid (a cache's always are).
template <int DT, int KV, int DP, bool VEC>
__global__ void __launch_bounds__(kThreads* kGroups<DP>, 1) chunk_rows(const __grid_constant__ Args g) {
    constexpr int W = DP + 4, WP = kN + 4, Q4 = DP / 64;
    constexpr int SRC = KV == kPacked ? DT : KV;
    constexpr bool ASYNC = SRC == kF32 && VEC;
    extern __shared__ float sm[];
    const ChunkArgs& a = g.a;
    const int group = threadIdx.x / kThreads, tid = threadIdx.x & (kThreads - 1);
    float* const qs = sm;
    float* const ps = qs + kM * W + group * kGroupFloats<DP>;
    float* const ks = ps + kM * WP;
    float* const vs = ks + kN * W;
    __shared__ Places all_places[kGroups<DP>][2];
    Places(&places)[2] = all_places[group];
    auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kThreads) : "memory"); };
    __shared__ struct {
        Item item;
        int kvh;  // -1: nothing more
    } todo;
    pdl_begin();
    int kvh = 0;
    const int D = (int)a.D, ty = tid >> 4, tx = tid & 15;
    const int kv_heads = (int)a.Hkv;
    __shared__ alignas(8) unsigned char source_at[32][sizeof(Source)];  // the first warp's, out of its registers
    Source& source = *reinterpret_cast<Source*>(source_at[threadIdx.x & 31]);
    if (threadIdx.x < 32) new (&source) Source(g, false);

    for (;;) {
        __syncthreads();  // the last item is done with
        if (threadIdx.x < 32) {
            Item it;
            if (!source.next(it, kvh)) kvh = -1;
            if (threadIdx.x == 0) todo.item = it, todo.kvh = kvh;
        }
        __syncthreads();
        const Item it = todo.item;
        kvh = todo.kvh;
        if (kvh < 0) break;
        const Walk w = walk(g, it);
        const int token0 = it.tile / g.parts * g.tokens, head0 = it.tile % g.parts * g.heads;
        const int rows = g.tokens * g.heads;
        // row r of the tile: token and head of the group; false: the tile has no such row
        auto row_of = [&](int r, int& token, int& head) {
            token = token0 + r / g.heads;
            head = head0 + r % g.heads;
            return r < rows && token < it.s.n && head < g.group;
        };
        for (int i = threadIdx.x; i < kM * (DP / 4); i += kThreads * kGroups<DP>) {
            const int r = i / (DP / 4), d = (i - r * (DP / 4)) * 4;
            int token, head;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (row_of(r, token, head) && d < D) {
                const int64_t at = (it.s.begin + (int64_t)token) * a.q_stride + ((int64_t)kvh * g.group + head) * D + d;
                const float c = a.scale * kLog2e;
                x.x = Store<DT>::load1(a.q, at) * c;
                x.y = Store<DT>::load1(a.q, at + 1) * c;
                x.z = Store<DT>::load1(a.q, at + 2) * c;
                x.w = Store<DT>::load1(a.q, at + 3) * c;
            }
            *reinterpret_cast<float4*>(qs + r * W + d) = x;
        }
        // the thread's rows: the last key that each sees, and the first one under the window
        int last[R], low[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            last[i] = it.s.len - it.s.n + token0 + (ty * R + i) / g.heads;
            low[i] = a.window > 0 ? (int)max((int64_t)last[i] - a.window + 1, (int64_t)0) : 0;
        }
        const int sinks = (int)min(a.sinks, (int64_t)INT32_MAX);

        // where the keys of list entry x lie
        auto look_up = [&](int x, Places& pl) {
            if (tid >= kN) return;
            int64_t at = -1, scale = 0;
            const int j = w.block(x) * kN + tid;
            if (j < it.s.len) {
                if constexpr (KV == kPacked) {
                    at = it.s.begin + (int64_t)j;
                } else {
                    const int page_i = j / a.c.page_size, row = j - page_i * a.c.page_size;
                    const int32_t page = a.table[it.seq * a.max_pages + page_i];
                    if (page >= 0 && page < a.c.n_pages) {
                        at = page * a.c.page_stride + ((int64_t)kvh * a.c.page_size + row) * D;
                        scale = ((int64_t)page * kv_heads + kvh) * a.c.page_size + row;
                    }
                }
            }
            pl.at[tid] = at;
            pl.scale[tid] = scale;
            const uint32_t live = __ballot_sync(0xFFFFFFFFu, at >= 0);
            if ((tid & 31) == 0) pl.live[tid >> 5] = live;
        };
        const void* const k_src = KV == kPacked ? a.k : a.c.k;
        const void* const v_src = KV == kPacked ? a.v : a.c.v;
        // packed rows: places are of rows, and k and v have strides of their own
        auto fetch = [&](float* dst, const void* src, const uint8_t* scales, int64_t stride, Places& pl) {
            if constexpr (KV == kPacked) {
                constexpr int es = DT == kF32 ? 4 : 2;
                const char* const base = static_cast<const char*>(src) + (int64_t)kvh * D * es;
                // (the rows of a block follow one another)
                for (int i = tid; i < kN * (DP / 8); i += kThreads) {
                    const int r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
                    const bool there = pl.at[r] >= 0 && d < D;
                    const int64_t at = there ? pl.at[r] * stride + d : 0;
                    float* const to = dst + r * W + d;
                    if constexpr (ASYNC) {
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                             (uint32_t)__cvta_generic_to_shared(to + 4 * x)),
                                         "l"(base + (there ? (at + 4 * x) * es : 0)), "r"(there ? 16 : 0)
                                         : "memory");
                    } else {
                        float f[8] = {};
                        if (there) {
                            if constexpr (VEC) {
                                constexpr int V = Store<DT>::V;
#pragma unroll
                                for (int p = 0; p < 8 / V; ++p) {
                                    float y[V];
                                    Store<DT>::unpack(ld_reuse(base + (at + p * V) * es), y);
#pragma unroll
                                    for (int e = 0; e < V; ++e) f[p * V + e] = y[e];
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e) f[e] = Store<DT>::load1(base, at + e);
                            }
                        }
                        *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<float4*>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            } else if constexpr (ASYNC) {
                stage_async<DP>(dst, static_cast<const float*>(src), pl, D);
            } else {
                stage<SRC, DP>(dst, src, scales, pl, D);
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
        };

        float2 o[R][2 * Q4];
        float m[R], l[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2 * Q4; ++e) o[i][e] = make_float2(0.0f, 0.0f);
        }
        if (w.from + group < w.to) look_up(w.from + group, places[0]);
        __syncthreads();  // q and the first places are there
        if (w.from + group < w.to) fetch(ks, k_src, a.c.k_scale, a.k_stride, places[0]);
        int buf = 0;
        for (int x = w.from + group; x < w.to; x += kGroups<DP>, buf ^= 1) {
            const int k0 = w.block(x) * kN;
            sync();  // v of the tile before is done with
            fetch(vs, v_src, a.c.v_scale, a.v_stride, places[buf]);
            const bool more = x + kGroups<DP> < w.to;
            if (more) look_up(x + kGroups<DP>, places[buf ^ 1]);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            sync();  // k is there
            float2 s2[R][4] = {};  // sums over even and odd entries: two multiply-adds an instruction
#pragma unroll 4
            for (int d = 0; d < DP; d += 4) {
                float4 y[R], z[4];
#pragma unroll
                for (int i = 0; i < R; ++i) y[i] = *reinterpret_cast<const float4*>(qs + (ty * R + i) * W + d);
#pragma unroll
                for (int j = 0; j < 4; ++j) z[j] = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * W + d);
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s2[i][j] = fma2_rn(make_float2(y[i].x, y[i].y), make_float2(z[j].x, z[j].y), s2[i][j]);
                        s2[i][j] = fma2_rn(make_float2(y[i].z, y[i].w), make_float2(z[j].z, z[j].w), s2[i][j]);
                    }
            }
            float s[R][4];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
            uint32_t live[2] = {places[buf].live[0], places[buf].live[1]};
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            sync();  // k is done with, v and the next places are there
            if (more) fetch(ks, k_src, a.c.k_scale, a.k_stride, places[buf ^ 1]);
            // whether every row sees every key of the tile
            const bool clean = (live[0] & live[1]) == 0xFFFFFFFFu && k0 + kN - 1 <= w.first_place &&
                               (a.window == 0 || k0 > w.last_place - a.window || k0 + kN <= sinks);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float mx = m[i];
                bool seen[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = k0 + tx + 16 * j;
                    seen[j] = clean || ((live[j >> 1] >> (tx + 16 * (j & 1)) & 1u) && key <= last[i] &&
                                        (key >= low[i] || key < sinks));
                    // a NaN logit leaves a finite maximum, so that its NaN weight reaches the result
                    if (seen[j]) mx = fmaxf(mx, s[i][j] == s[i][j] ? s[i][j] : -3.0e38f);
                }
#pragma unroll
                for (int y = 8; y >= 1; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, y));
                const float r = m[i] == -INFINITY ? 0.0f : ex2(m[i] - mx);
                m[i] = mx;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = seen[j] ? (s[i][j] == -INFINITY ? 0.0f : ex2(s[i][j] - mx)) : 0.0f;
                    sum += p;
                    ps[(ty * R + i) * WP + tx + 16 * j] = p;
                }
#pragma unroll
                for (int y = 8; y >= 1; y >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, y);
                l[i] = fmaf(l[i], r, sum);
#pragma unroll
                for (int e = 0; e < 2 * Q4; ++e) o[i][e] = mul2_rn(o[i][e], make_float2(r, r));
            }
            __syncwarp();  // a row's weights come from its own half warp
            auto weigh = [&](auto masked) {
#pragma unroll 2
                for (int j = 0; j < kN; j += 4) {
                    float4 p[R];
#pragma unroll
                    for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(ps + (ty * R + i) * WP + j);
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                        for (int c = 0; c < Q4; ++c) {
                            const float4 v = *reinterpret_cast<const float4*>(vs + (j + jj) * W + tx * 4 + 64 * c);
#pragma unroll
                            for (int i = 0; i < R; ++i) {
                                const float w1 = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
                                if constexpr (decltype(masked)::value) {
                                    const int key = k0 + j + jj;
                                    if (!(live[j >> 5] >> ((j + jj) & 31) & 1u) || key > last[i] ||
                                        (key < low[i] && key >= sinks))
                                        continue;
                                }
                                const float2 w2 = make_float2(w1, w1);
                                o[i][2 * c] = fma2_rn(w2, make_float2(v.x, v.y), o[i][2 * c]);
                                o[i][2 * c + 1] = fma2_rn(w2, make_float2(v.z, v.w), o[i][2 * c + 1]);
                            }
                        }
                }
            };
            // What a row does not see has weight 0, which adds nothing but where v is not finite: then once more, without
            // such keys.  (Looked at one by one from the start: 542 us in place of 511 for three prompts of up to 4000
            // rows, 8 heads of 64, window 1000.)
            float2 before[R][2 * Q4];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int e = 0; e < 2 * Q4; ++e) before[i][e] = o[i][e];
            weigh(std::false_type{});
            float2 bad = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int e = 0; e < 2 * Q4; ++e) bad = fma2_rn(o[i][e], make_float2(0.0f, 0.0f), bad);  // 0, or NaN
            if (!clean && bad.x + bad.y != 0.0f) {
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int e = 0; e < 2 * Q4; ++e) o[i][e] = before[i][e];
                weigh(std::true_type{});
            }
        }
        if constexpr (kGroups<DP> == 2) {
            // the second group's sums by way of its own k
            float* const other = qs + kM * W + kGroupFloats<DP> + kM * WP;
            if (group == 1) {
                sync();
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    float* const to = other + (ty * R + i) * W;
#pragma unroll
                    for (int c = 0; c < Q4; ++c)
                        *reinterpret_cast<float4*>(to + tx * 4 + 64 * c) =
                            make_float4(o[i][2 * c].x, o[i][2 * c].y, o[i][2 * c + 1].x, o[i][2 * c + 1].y);
                    if (tx == 0) to[DP] = m[i], to[DP + 1] = l[i];
                }
            }
            __syncthreads();
            if (group == 1) continue;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float* const from = other + (ty * R + i) * W;
                const float m1 = from[DP], m2 = fmaxf(m[i], m1);
                const float r0 = m[i] == -INFINITY ? 0.0f : ex2(m[i] - m2), r1 = m1 == -INFINITY ? 0.0f : ex2(m1 - m2);
                m[i] = m2;
                l[i] = fmaf(l[i], r0, __fmul_rn(from[DP + 1], r1));
#pragma unroll
                for (int c = 0; c < Q4; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(from + tx * 4 + 64 * c);
                    o[i][2 * c].x = fmaf(o[i][2 * c].x, r0, __fmul_rn(v.x, r1));
                    o[i][2 * c].y = fmaf(o[i][2 * c].y, r0, __fmul_rn(v.y, r1));
                    o[i][2 * c + 1].x = fmaf(o[i][2 * c + 1].x, r0, __fmul_rn(v.z, r1));
                    o[i][2 * c + 1].y = fmaf(o[i][2 * c + 1].y, r0, __fmul_rn(v.w, r1));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            int token, head;
            if (!row_of(ty * R + i, token, head)) continue;
            head += kvh * g.group;
            const int64_t out = (it.s.begin + (int64_t)token) * a.out_stride + (int64_t)head * D;
            const bool is_part = it.splits > 1;
            const int64_t part = is_part ? part_at(g, it, token, head) : 0;
            const float inv = m[i] == -INFINITY ? 0.0f : 1.0f / l[i];
            if (is_part && tx == 0) g.part_ml[part] = make_float2(m[i], l[i]);
#pragma unroll
            for (int c = 0; c < Q4; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = tx * 4 + 64 * c + e;
                    const float y = e & 1 ? o[i][2 * c + e / 2].y : o[i][2 * c + e / 2].x;
                    if (d >= D) continue;
                    if (is_part)
                        g.part_o[part * D + d] = y;
                    else
                        Store<DT>::store1(a.out, out + d, m[i] == -INFINITY ? 0.0f : y * inv);
                }
        }
    }
}

// A warp two rows at a time, their partial results in order, four of each on
// their way, four entries a lane: a row has few of them, so that the latency of one
// behind the other is what it would cost.  0 where nothing was seen; a weight of 0
// still carries NaN on.
constexpr int kJoinWarps = 8, kJoinRows = 2, kJoinDepth = 4;
template <int DT, int DP>
__global__ void __launch_bounds__(kJoinWarps * 32) chunk_join(const __grid_constant__ Args g) {
    constexpr int kPieces = DP / 128;  // of four entries, of a lane
    pdl_begin();
    const ChunkArgs& a = g.a;
    const int lane = threadIdx.x & 31, D = (int)a.D;
    constexpr int kFour = DT == kF32 ? 16 : 8;  // bytes; where rows lie on their grid
    const bool fours = reinterpret_cast<uintptr_t>(a.out) % kFour == 0 && a.out_stride % 4 == 0;
    for (int64_t b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
        Item it = {};
        it.s = sequence(a, b);
        it.seq = (int)b;
        it.splits = cut_of(g, it.s).splits;
        if (it.splits == 1) continue;
        const int Hq = (int)a.Hq, rows = it.s.n * Hq, n = it.splits;  // (of fewer than kWave kRounds units)
        const int step = gridDim.y * kJoinWarps;
        for (int r0 = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); r0 < rows; r0 += kJoinRows * step) {
            int64_t at[kJoinRows];
            float m[kJoinRows], l[kJoinRows];
            float4 o[kJoinRows][kPieces] = {};
#pragma unroll
            for (int i = 0; i < kJoinRows; ++i) {
                const int r = min(r0 + i * step, rows - 1), token = r / Hq;
                at[i] = parts_at(g, it, token, r - token * Hq);
                m[i] = -INFINITY, l[i] = 0.0f;
            }
            for (int s0 = 0; s0 < n; s0 += kJoinDepth) {
                float2 ml[kJoinRows][kJoinDepth];
                float4 y[kJoinRows][kJoinDepth][kPieces];
#pragma unroll
                for (int i = 0; i < kJoinRows; ++i)
#pragma unroll
                    for (int s = 0; s < kJoinDepth; ++s) {
                        const bool there = s0 + s < n;
                        ml[i][s] = there ? g.part_ml[at[i] + s0 + s] : make_float2(-INFINITY, 0.0f);
#pragma unroll
                        for (int x = 0; x < kPieces; ++x) {
                            const int d = lane * 4 + x * 128;
                            y[i][s][x] = there && d < D
                                             ? *reinterpret_cast<const float4*>(g.part_o + (at[i] + s0 + s) * D + d)
                                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        }
                    }
#pragma unroll
                for (int i = 0; i < kJoinRows; ++i) {
                    float top = m[i];
#pragma unroll
                    for (int s = 0; s < kJoinDepth; ++s) top = fmaxf(top, ml[i][s].x);
                    const float back = m[i] == -INFINITY ? 0.0f : ex2(m[i] - top);
                    m[i] = top;
                    l[i] *= back;
#pragma unroll
                    for (int x = 0; x < kPieces; ++x)
                        o[i][x].x *= back, o[i][x].y *= back, o[i][x].z *= back, o[i][x].w *= back;
#pragma unroll
                    for (int s = 0; s < kJoinDepth; ++s) {
                        if (ml[i][s].x == -INFINITY) continue;
                        const float w = ex2(ml[i][s].x - top);
                        l[i] = fmaf(ml[i][s].y, w, l[i]);
#pragma unroll
                        for (int x = 0; x < kPieces; ++x) {
                            const float4 z = y[i][s][x];
                            o[i][x].x = fmaf(z.x, w, o[i][x].x);
                            o[i][x].y = fmaf(z.y, w, o[i][x].y);
                            o[i][x].z = fmaf(z.z, w, o[i][x].z);
                            o[i][x].w = fmaf(z.w, w, o[i][x].w);
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kJoinRows; ++i) {
                const int r = r0 + i * step, token = r / Hq;
                if (r >= rows) continue;
                const int64_t out = (it.s.begin + (int64_t)token) * a.out_stride + (int64_t)(r - token * Hq) * D + lane * 4;
#pragma unroll
                for (int x = 0; x < kPieces; ++x) {
                    if (lane * 4 + x * 128 >= D) continue;
                    float z[4] = {o[i][x].x, o[i][x].y, o[i][x].z, o[i][x].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = m[i] == -INFINITY ? 0.0f : z[e] / l[i];
                    const int64_t to = out + x * 128;
                    if (!fours) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) Store<DT>::store1(a.out, to + e, z[e]);
                    } else if constexpr (DT == kF32) {
                        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = make_float4(z[0], z[1], z[2], z[3]);
                    } else {
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) =
                            make_uint2(f32x2_to_bf16x2_bits(z[0], z[1]), f32x2_to_bf16x2_bits(z[2], z[3]));
                    }
                }
            }
        }
    }
}

template <int DT, int KV, int DP, bool VEC>
cudaError_t go(const ChunkArgs& a, cudaStream_t st) {
    const Args g = make_args(a, kM, 1, kN);
    constexpr int smem = (kM * (DP + 4) + kGroups<DP> * kGroupFloats<DP>) * 4;
    static FunctionLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(chunk_rows<DT, KV, DP, VEC>), smem);
    if (e != cudaSuccess) return e;
    const int64_t seqs = a.n_seqs < a.T ? a.n_seqs : a.T;
    const int64_t pieces = (a.T / g.tokens + seqs) * g.parts * a.Hkv * g.most;
    const int64_t most = 2 * (int64_t)sm_count();
    return launch(chunk_rows<DT, KV, DP, VEC>, dim3((unsigned)(pieces < most ? pieces : most)),
                  dim3(kThreads * kGroups<DP>), smem, st, g);
}

template <int DT, int KV, bool VEC>
cudaError_t pick(const ChunkArgs& a, cudaStream_t st) {
    if (a.D <= 64) return go<DT, KV, 64, VEC>(a, st);
    if (a.D <= 128) return go<DT, KV, 128, VEC>(a, st);
    return go<DT, KV, 256, VEC>(a, st);
}

}  // namespace

template <int DT>
static cudaError_t join(const Args& g, cudaStream_t st) {
    const int64_t ctas = 6 * (int64_t)sm_count(), x = g.a.n_seqs < ctas ? g.a.n_seqs : ctas;
    const int64_t rows = (g.a.T * g.a.Hq + kJoinWarps - 1) / kJoinWarps, share = (ctas + x - 1) / x;
    const dim3 grid((unsigned)x, (unsigned)(rows < share ? rows : share)), threads(kJoinWarps * 32);
    return g.a.D <= 128 ? launch(chunk_join<DT, 128>, grid, threads, 0, st, g)
                        : launch(chunk_join<DT, 256>, grid, threads, 0, st, g);
}

cudaError_t launch_join(const Args& g, int dtype, cudaStream_t st) {
    if (g.most == 1) return cudaSuccess;
    return dtype == GBE_F32 ? join<kF32>(g, st) : join<kBF16>(g, st);
}

}  // namespace chunk

ChunkRoom chunk_room(int64_t n_seqs, int64_t T, int64_t Hq, int64_t Hkv, int64_t keys, int64_t window, int64_t sinks) {
    using namespace chunk;
    ChunkRoom r = {1, 0, 0};
    if (window > 0 && window + sinks + kUnitRows < keys) keys = window + sinks + kUnitRows;
    int64_t most = (keys + 127) / 128 / (kLeast / 128);
    if (most > kWave * kRounds / Hkv) most = kWave * kRounds / Hkv;
    if (most < 2) return r;
    r.most = (int)most;
    // cut_of gives a sequence at most kWave kRounds items, of kUnitRows rows each
    const int64_t by_row = T * Hq * most, of_seq = (int64_t)kUnitRows * kWave * kRounds;
    const int64_t per_seq = of_seq < by_row ? of_seq : by_row;
    if (n_seqs * per_seq < by_row) r.per_seq = per_seq;
    r.entries = r.per_seq > 0 ? n_seqs * per_seq : by_row;
    return r;
}

cudaError_t launch_attn_chunk(const ChunkArgs& a, int dtype, bool vec, bool tensor, cudaStream_t st) {
    using namespace chunk;
    const bool paged = !a.packed, e4m3 = paged && a.c.dtype == GBE_KV_E4M3, bf16 = dtype == GBE_BF16;
    // Tensor copies start on 16 bytes in memory and on 128 in shared memory: over an 8-bit cache rows of a multiple of 16,
    // and pages of an even number of them, for a copy of one row would be of 64 bytes.
    const bool tc = bf16 && vec && tensor && a.D <= 128 &&
                    (!paged || (a.c.n_pages > 0 &&
                                (!e4m3 || (a.D % 16 == 0 && a.c.page_stride % 16 == 0 && a.c.page_size % 2 == 0))));
    cudaError_t e = cudaSuccess;
    if (tc)
        e = launch_tc(a, st);
    else if (!paged && bf16)
        e = vec ? pick<kBF16, kPacked, true>(a, st) : pick<kBF16, kPacked, false>(a, st);
    else if (!paged)
        e = vec ? pick<kF32, kPacked, true>(a, st) : pick<kF32, kPacked, false>(a, st);
    else if (bf16)
        e = e4m3 ? pick<kBF16, GBE_KV_E4M3, true>(a, st) : pick<kBF16, GBE_KV_BF16, true>(a, st);
    else
        e = e4m3 ? pick<kF32, GBE_KV_E4M3, true>(a, st) : pick<kF32, GBE_KV_F32, true>(a, st);
    return e != cudaSuccess ? e : launch_join(tc ? make_args(a, 128, 2, 128) : make_args(a, kM, 1, kN), dtype, st);
}

}  // namespace gbe
