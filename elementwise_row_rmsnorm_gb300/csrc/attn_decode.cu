// attn_decode.cu -- attention of one new token per sequence over the paged
// key-value cache, split over the cache's length and joined.
//
//   out[b, h] = sum_j p_j v_j,  p = softmax_j(scale * q[b, h] . k_j),  j < lens[b]
//
// with k_j, v_j the cached rows of kv head h / (Hq / Hkv).  One CTA takes one
// chunk of one sequence's tokens for one kv head and up to H of its query
// heads; the chunk's length is a function of the sequence's length alone
// (chunk_tokens below), so a sequence's result has the same bits in a batch
// of any size.  Each CTA leaves the unnormalised sum, the running maximum and
// the running sum of its chunk in the workspace, and attn_join adds the
// chunks of a row in order.  A sequence of one chunk is written at once.
#include "attn_decode.cuh"
#include "gbe_elementwise.h"
#include "kv_cache.cuh"

namespace gbe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
using namespace decode;

// One 8-value piece of a cached row, widened to f32.
template <int KV>
struct Piece;
template <>
struct Piece<GBE_KV_F32> {
    Vec16 a, b;
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        const float* p = static_cast<const float*>(base) + i;
        a = ld_stream(p), b = ld_stream(p + 4);
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(a.w[e]), f[4 + e] = __uint_as_float(b.w[e]);
    }
};
template <>
struct Piece<GBE_KV_E4M3> {
    uint2 a;
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        a = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + i);
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        e4m3x4_to_f32(a.x, f);
        e4m3x4_to_f32(a.y, f + 4);
    }
};

// The CUDA-core form, for f32 queries: G lanes (the power of two at or above
// D / 8) hold one token's row, eight values each, so a warp walks 32 / G
// streams of tokens and each lane keeps the query heads' pieces and the
// output's in registers.  A stream takes four tokens at a time: their loads are
// on their way together (64 KB for a CTA's f32 rows, enough to cover HBM's
// latency from one CTA an SM), and the running maximum moves once for the four.
template <int KV, int H>
__global__ void __launch_bounds__(kThreads, 1) decode_rows(Args a, int lanes_log2) {
    constexpr int U = 4;
    extern __shared__ float sm[];  // [kWarps][H][D + 2]
    pdl_begin();
    const KvCacheArgs& c = a.c;
    const int G = 1 << lanes_log2, D = c.D;
    const Part p = find_part(a, blockIdx.x);
    if (p.t0 >= p.t1 && p.chunk > 0) return;
    const int b = p.b, kvh = p.kvh, t0 = p.t0, t1 = p.t1;
    const int h0 = kvh * a.group + p.part * H;            // first query head
    const int heads = min(H, a.group - p.part * H);

    const int sub = threadIdx.x & (G - 1), d0 = sub * 8;
    const bool mine = d0 < D;
    const int stream = threadIdx.x >> lanes_log2, streams = kThreads >> lanes_log2;

    float q[H][8], acc[H][8], m[H], l[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[h][e] = 0.0f;
            q[h][e] = 0.0f;
            if (mine && h < heads)
                q[h][e] = Store<kF32>::load1(a.q, b * a.q_stride + (int64_t)(h0 + h) * D + d0 + e) * a.scale;
        }
    }
    const int32_t* pages = a.table + (int64_t)b * a.max_pages;
    // all streams of a warp take the same number of steps, so that its
    // shuffles meet
    for (int base = t0; base < t1; base += U * streams) {
        Piece<KV> kp[U], vp[U];
        float ks[U], vs[U];
        bool good[U];
        int64_t at[U], si[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = base + u * streams + stream;
            const bool live = t < t1;
            const int page_i = live ? t / c.page_size : 0;
            const int32_t page = live ? pages[page_i] : -1;
            const int row = t - page_i * c.page_size;
            good[u] = page >= 0 && page < c.n_pages;
            at[u] = page * c.page_stride + ((int64_t)kvh * c.page_size + row) * D + d0;
            si[u] = ((int64_t)page * c.Hkv + kvh) * c.page_size + row;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            kp[u] = {}, vp[u] = {};
            ks[u] = vs[u] = 1.0f;
            if (good[u] && mine) kp[u].load(c.k, at[u]), vp[u].load(c.v, at[u]);
            if (KV == GBE_KV_E4M3 && good[u]) {
                ks[u] = __uint_as_float((uint32_t)c.k_scale[si[u]] << 23);
                vs[u] = __uint_as_float((uint32_t)c.v_scale[si[u]] << 23);
            }
        }
        float s[U][H];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float k[8];
            kp[u].widen(k);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                float x = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) x = fmaf(q[h][e], k[e], x);
                for (int y = G >> 1; y >= 1; y >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, y);
                s[u][h] = good[u] ? (KV == GBE_KV_E4M3 ? x * ks[u] : x) : -INFINITY;
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float m2 = m[h];
            // a NaN logit leaves a finite maximum, so that its NaN weight reaches the result
#pragma unroll
            for (int u = 0; u < U; ++u) m2 = fmaxf(m2, s[u][h] == s[u][h] ? s[u][h] : -3.0e38f);
            const float r = rescale(m[h], m2);
            m[h] = m2;
            l[h] *= r;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[h][e] *= r;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u][h] = s[u][h] == -INFINITY ? 0.0f : ex2(s[u][h] - m2);
                l[h] += s[u][h];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            vp[u].widen(v);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float w = KV == GBE_KV_E4M3 ? s[u][h] * vs[u] : s[u][h];
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[h][e] = fmaf(w, v[e], acc[h][e]);
            }
        }
    }
    // the warp's streams joined, pair by pair: both sides compute the same sums
    for (int x = G; x < 32; x <<= 1) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const float mo = __shfl_xor_sync(0xFFFFFFFFu, m[h], x), lo = __shfl_xor_sync(0xFFFFFFFFu, l[h], x);
            const float m2 = fmaxf(m[h], mo), r = rescale(m[h], m2), ro = rescale(mo, m2);
            l[h] = l[h] * r + lo * ro;
            m[h] = m2;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float o = __shfl_xor_sync(0xFFFFFFFFu, acc[h][e], x);
                acc[h][e] = __fadd_rn(__fmul_rn(acc[h][e], r), __fmul_rn(o, ro));
            }
        }
    }
    // and the warps in order, in shared memory
    const int W = D + 2, warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) < G) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float* o = sm + (warp * H + h) * W;
            if (mine)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[d0 + e] = acc[h][e];
            if (sub == 0) o[D] = m[h], o[D + 1] = l[h];
        }
    }
    __syncthreads();
    const bool whole = p.C >= p.n;
    for (int i = threadIdx.x; i < heads * D; i += kThreads) {
        const int h = i / D, d = i - h * D;
        float mx = -INFINITY;
#pragma unroll
        for (int s = 0; s < kWarps; ++s) mx = fmaxf(mx, sm[(s * H + h) * W + D]);
        float sum = 0.0f, o = 0.0f;
#pragma unroll
        for (int s = 0; s < kWarps; ++s) {
            const float* x = sm + (s * H + h) * W;
            if (x[D] == -INFINITY) continue;  // nothing seen; a weight of 0 still carries NaN on
            const float r = ex2(x[D] - mx);
            sum = fmaf(x[D + 1], r, sum), o = fmaf(x[d], r, o);
        }
        if (whole) {
            Store<kF32>::store1(a.out, b * a.out_stride + (int64_t)(h0 + h) * D + d,
                              mx == -INFINITY ? 0.0f : o / sum);
        } else {
            const int64_t row = ((int64_t)b * a.Hq + h0 + h) * a.split + p.chunk;
            a.part_o[row * D + d] = o;
            if (d == 0) a.part_ml[row] = make_float2(mx, sum);
        }
    }
}

// The chunks of one row added: one CTA a (sequence, query head).  Warp w adds
// chunks w, w + 8, ... in order, four entries a lane, and the warps' sums are
// added in order.  The loads of a warp's chunks do not wait on one another: one
// warp walking all 128 chunks of a long row took over 100 us.
constexpr int kJoinWarps = 8, kMostChunks = 128;
template <int DT>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_join(Args a) {
    __shared__ float weight[kMostChunks], sums[kJoinWarps];
    __shared__ float4 part[kJoinWarps][64];
    pdl_begin();
    const int64_t r = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.c.D;
    const int64_t b = r / a.Hq, h = r - b * a.Hq;
    const int64_t capacity = (int64_t)a.max_pages * a.c.page_size;
    const int32_t len = a.lens[b];
    const int n = len < 0 ? 0 : (int)(len < capacity ? len : capacity);
    const int C = chunk_tokens(n, a.split, a.least);
    if (C >= n) return;  // one chunk: already written
    const int chunks = (n + C - 1) / C;
    // every warp finds the maximum for itself
    const float2* ml = a.part_ml + r * a.split;
    float mx = -INFINITY;
    for (int s = lane; s < chunks; s += 32) mx = fmaxf(mx, ml[s].x);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
    // -1 marks a chunk in which nothing was seen; a weight of 0 still carries NaN on
    float l = 0.0f;
    for (int s = threadIdx.x; s < chunks; s += kJoinWarps * 32) {
        const float2 v = ml[s];
        const float w = v.x == -INFINITY ? -1.0f : ex2(v.x - mx);
        weight[s] = w;
        if (w >= 0.0f) l = fmaf(v.y, w, l);
    }
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
    if (lane == 0) sums[warp] = l;
    __syncthreads();
    float4 o[2] = {};
    const float* from = a.part_o + r * a.split * D + lane * 4;
#pragma unroll 4
    for (int s = warp; s < chunks; s += kJoinWarps) {
        const float w = weight[s];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (lane * 4 + x * 128 >= D) continue;
            const float4 v = *reinterpret_cast<const float4*>(from + (int64_t)s * D + x * 128);
            if (w >= 0.0f) {
                o[x].x = fmaf(v.x, w, o[x].x);
                o[x].y = fmaf(v.y, w, o[x].y);
                o[x].z = fmaf(v.z, w, o[x].z);
                o[x].w = fmaf(v.w, w, o[x].w);
            }
        }
    }
    part[warp][lane] = o[0];
    part[warp][32 + lane] = o[1];
    __syncthreads();
    float sum = 0.0f;
#pragma unroll
    for (int x = 0; x < kJoinWarps; ++x) sum += sums[x];
    if (threadIdx.x < D) {
        float y = 0.0f;
#pragma unroll
        for (int x = 0; x < kJoinWarps; ++x) y += reinterpret_cast<const float*>(part[x])[threadIdx.x];
        Store<DT>::store1(a.out, b * a.out_stride + h * D + threadIdx.x, mx == -INFINITY ? 0.0f : y / sum);
    }
}

template <int KV, int H>
cudaError_t go(Args a, int64_t B, cudaStream_t st) {
    int lg = 0;
    while ((8 << lg) < a.c.D) ++lg;
    a.parts = (a.group + H - 1) / H;
    const size_t smem = (size_t)kWarps * H * (a.c.D + 2) * 4;
    static FunctionLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(decode_rows<KV, H>), kWarps * H * 258 * 4);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(B * a.split * a.c.Hkv * a.parts));
    return launch(decode_rows<KV, H>, grid, dim3(kThreads), smem, st, a, lg);
}

template <int KV>
cudaError_t pick(const Args& a, int64_t B, cudaStream_t st) {
    if (a.group == 1) return go<KV, 1>(a, B, st);
    if (a.group == 2) return go<KV, 2>(a, B, st);
    if (a.group <= 4) return go<KV, 4>(a, B, st);
    return go<KV, 8>(a, B, st);
}

}  // namespace

// Chunks of 512 tokens and more: shorter ones cost more in fixed work and in
// partial results (4 * Hq / Hkv bytes written and read for every token and kv
// head) than the SMs they bring in are worth.  128 chunks at most, so that two
// sequences of 131072 tokens make 2048 CTAs.
DecodeSplit decode_split(int64_t page_size, int64_t max_pages) {
    DecodeSplit s;
    s.least = 512;
    const int64_t most = (page_size * max_pages + s.least - 1) / s.least;
    s.split = (int)(most < 1 ? 1 : most > kMostChunks ? kMostChunks : most);
    return s;
}

cudaError_t launch_attn_decode(const DecodeArgs& d, int dtype, cudaStream_t st) {
    Args a = {};
    const DecodeSplit s = decode_split(d.c.page_size, d.max_pages);
    a.q = d.q, a.out = d.out, a.q_stride = d.q_stride, a.out_stride = d.out_stride;
    a.c = d.c, a.table = d.table, a.lens = d.lens;
    a.Hq = (int)d.Hq, a.group = (int)(d.Hq / d.c.Hkv), a.max_pages = (int)d.max_pages;
    a.split = s.split, a.least = s.least, a.run = 1;
    a.scale = d.scale * kLog2e;
    a.part_o = static_cast<float*>(d.workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + d.B * d.Hq * s.split * d.c.D);
    cudaError_t e;
    if (dtype == GBE_BF16)
        e = decode::launch_mma(a, d.B, st);
    else
        e = d.c.dtype == GBE_KV_E4M3 ? pick<GBE_KV_E4M3>(a, d.B, st) : pick<GBE_KV_F32>(a, d.B, st);
    if (e != cudaSuccess || s.split == 1) return e;
    const dim3 rows((unsigned)(d.B * d.Hq)), threads(kJoinWarps * 32);
    return dtype == GBE_F32 ? launch(attn_join<kF32>, rows, threads, 0, st, a)
                            : launch(attn_join<kBF16>, rows, threads, 0, st, a);
}

}  // namespace gbe
