// attn_chunk_row.cuh -- one row of a chunk, or a split of its keys, from the keys
// that it sees alone: for what the tensor cores' products cannot leave out, an
// infinity or a NaN of v behind a mask.  bf16 rows, D up to 128.
#pragma once

#include "attn_chunk.cuh"
#include "kv_cache.cuh"

namespace gbe {
namespace chunk {

constexpr int kKeys = 128;   // of a block of the walk

// The row of key j in k and v; -1: it lies on no page of the cache.
template <int KV>
__device__ __forceinline__ int64_t key_at(const ChunkArgs& a, const Item& it, int kvh, int j) {
    if constexpr (KV == kPacked) return it.s.begin + (int64_t)j;
    const int page_i = j / a.c.page_size, row = j - page_i * a.c.page_size;
    const int32_t page = a.table[it.seq * a.max_pages + page_i];
    if (page < 0 || page >= a.c.n_pages) return -1;
    return page * a.c.page_stride + ((int64_t)kvh * a.c.page_size + row) * a.D;
}

// Four consecutive values of a bf16 row, widened; on the 8-byte grid.
__device__ __forceinline__ float4 load4(const void* base, int64_t i) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + i);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}
template <int KV, bool V>
__device__ __forceinline__ float4 load_kv(const ChunkArgs& a, int kvh, int64_t at, int d) {
    if constexpr (KV == kPacked) {
        return load4(V ? a.v : a.k, at * (V ? a.v_stride : a.k_stride) + (int64_t)kvh * a.D + d);
    } else if constexpr (KV == GBE_KV_E4M3) {
        const int64_t page = at / a.c.page_stride, row = (at - page * a.c.page_stride) / a.D;
        const uint8_t byte = (V ? a.c.v_scale : a.c.k_scale)[page * a.c.Hkv * a.c.page_size + row];
        float f[4] = {};
        if (byte != 0) {  // (0: zeros, whatever the codes)
            e4m3x4_to_f32(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(V ? a.c.v : a.c.k) + at + d), f);
            const float scale = __uint_as_float((uint32_t)byte << 23);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] *= scale;
        }
        return make_float4(f[0], f[1], f[2], f[3]);
    } else {
        return load4(V ? a.c.v : a.c.k, at + d);
    }
}

// Which keys of a block, as bits, a row at `place` sees: word x is of keys
// k0 + 32 x and on.  (Places, windows and sinks are 2^30 at most.)
__device__ __forceinline__ uint32_t first_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t seen_word(const Args& g, int place, int k0, int x) {
    const int at = k0 + 32 * x;
    uint32_t m = first_bits(place + 1 - at);
    if (g.window > 0) m &= ~first_bits(place + 1 - g.window - at) | first_bits(g.sinks - at);
    return m;
}

// One row of an item in f32 from the keys that it sees alone, by a whole warp: 32
// keys at a time, a lane a key for the logits, a lane four entries for the output.
template <int KV>
static __device__ __noinline__ void exact_row(const Args& g, const Item& it, int kvh, int token, int head) {
    const ChunkArgs& a = g.a;
    const int lane = threadIdx.x & 31, D = (int)a.D, place = it.s.len - it.s.n + token;
    const float c = a.scale * kLog2e;
    const Walk w = walk(g, it);
    const int64_t row = (it.s.begin + (int64_t)token) * a.q_stride + ((int64_t)kvh * g.group + head) * D;
    float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f), o = q;
    if (lane * 4 < D) q = load4(a.q, row + lane * 4);
    float m = -INFINITY, l = 0.0f;
    for (int i = w.from * 4; i < w.to * 4; ++i) {
        const int k0 = w.block(i >> 2) * kKeys + (i & 3) * 32, j = k0 + lane;
        bool seen = seen_word(g, place, w.block(i >> 2) * kKeys, i & 3) >> lane & 1u;
        const int64_t at = seen ? key_at<KV>(a, it, kvh, j) : -1;
        seen = at >= 0;
        if (!__any_sync(0xFFFFFFFFu, seen)) continue;
        float s = 0.0f;
        for (int d = 0; d < D; d += 4) {
            const float4 k = seen ? load_kv<KV, false>(a, kvh, at, d) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
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
        for (uint32_t left = __ballot_sync(0xFFFFFFFFu, seen); left; left &= left - 1) {
            const int t = __ffs((int)left) - 1;
            const float weight = __shfl_sync(0xFFFFFFFFu, p, t);
            const int64_t from = __shfl_sync(0xFFFFFFFFu, at, t);
            if (lane * 4 < D) {
                const float4 v = load_kv<KV, true>(a, kvh, from, lane * 4);
                o.x = fmaf(weight, v.x, o.x);
                o.y = fmaf(weight, v.y, o.y);
                o.z = fmaf(weight, v.z, o.z);
                o.w = fmaf(weight, v.w, o.w);
            }
        }
    }
    const float y[4] = {o.x, o.y, o.z, o.w};
    if (it.splits > 1) {
        const int64_t part = part_at(g, it, token, kvh * g.group + head);
        if (lane * 4 < D) *reinterpret_cast<float4*>(g.part_o + part * D + lane * 4) = o;
        if (lane == 0) g.part_ml[part] = make_float2(m, l);
    } else if (lane * 4 < D) {
        const int64_t at = (it.s.begin + (int64_t)token) * a.out_stride + ((int64_t)kvh * g.group + head) * D + lane * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) Store<kBF16>::store1(a.out, at + e, m == -INFINITY ? 0.0f : y[e] / l);
    }
}

// A row that came out not finite: right as it is where the keys that it sees
// made it so, but a weight of zero may also have met an infinity or a NaN of v
// in a key of its blocks that it does not see, which makes NaN of the entry.
// Computed again only if an entry is NaN, has such a value there, and the values
// that it sees do not make NaN of it by themselves: a NaN among them or
// infinities of both signs.  (Of one sign they do not: the entry is that
// infinity.)  By a whole warp; the row has been written.
template <int KV>
static __device__ __noinline__ void repair_row(const Args& g, const Item& it, int kvh, int token, int head) {
    const ChunkArgs& a = g.a;
    const int lane = threadIdx.x & 31, D = (int)a.D, place = it.s.len - it.s.n + token;
    const bool mine = lane * 4 < D;
    const Walk w = walk(g, it);
    Odd now;
    if (mine) {
        if (it.splits > 1)
            now.meet(*reinterpret_cast<const float4*>(
                g.part_o + part_at(g, it, token, kvh * g.group + head) * D + lane * 4));
        else
            now.meet(load4(a.out, (it.s.begin + (int64_t)token) * a.out_stride +
                                      ((int64_t)kvh * g.group + head) * D + lane * 4));
    }
    uint32_t open = now.nan;  // entries that may have to be computed again
    // what they meet in the keys of the blocks, seen or not: an odd value, or of those seen ones that make NaN
    auto among = [&](bool seen) {
        Odd bad;
        auto found = [&] { return seen ? bad.lost() : bad.any(); };
        for (int i = (w.to - w.from) * 4 - 1; i >= 0; --i) {
            if (!__any_sync(0xFFFFFFFFu, open & ~found())) break;
            const int k0 = w.block(w.from + (i >> 2)) * kKeys;
            uint32_t keys = seen_word(g, place, k0, i & 3);
            if (!seen) keys = ~keys & first_bits(it.s.len - k0 - 32 * (i & 3));
            for (; keys; keys &= keys - 1) {
                const int64_t at = key_at<KV>(a, it, kvh, k0 + 32 * (i & 3) + __ffs((int)keys) - 1);
                if (at >= 0 && mine) bad.meet(load_kv<KV, true>(a, kvh, at, lane * 4));
            }
        }
        return found();
    };
    open &= among(false);
    open &= ~among(true);
    if (__any_sync(0xFFFFFFFFu, open)) exact_row<KV>(g, it, kvh, token, head);
}

}  // namespace chunk
}  // namespace gbe
