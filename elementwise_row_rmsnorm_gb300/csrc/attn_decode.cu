// attn_decode.cu -- attention of one new token per sequence over the paged
// key-value cache, split over the cache's length and joined.
//
//   out[b, h] = sum_j p_j v_j,  p = softmax_j(scale * q[b, h] . k_j),  j < lens[b],
//
// under a window j >= lens[b] - window or j < sinks (attn_decode.cuh says how the
// tokens between are passed over); with k_j, v_j the cached rows of kv head h / (Hq / Hkv).  One CTA takes one
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

// Threads of a CTA.  f32 rows: eight warps, for the small batches, where a chunk
// walked by four takes long enough to show (17 sequences of up to 2000 tokens, 7
// heads a kv head: 32 us with four, 29 with six, 22 with eight); a large batch
// with 8 heads a kv head pays for it, an SM holding one CTA of eight warps (64 x
// 4096: 606, 619 and 702 us).  8-bit rows: four, for with eight a chunk spends
// more on its ends (64 x 4096, 4 heads a kv head: 374 us, 320 us with four).
template <int KV>
constexpr int kThreadsOf = KV == GBE_KV_E4M3 ? 128 : 256;
template <int KV, int H>
constexpr int kResident = KV == GBE_KV_E4M3 ? (H == 8 ? 3 : 4) : H == 8 ? 1 : 2;  // CTAs an SM; of three 12 words spill
constexpr float kGrowth = 8.0f;  // powers of two that the maximum in use may lag
using namespace decode;

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* p, bool there) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p), "r"(there ? 16 : 0)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(p), "r"(there ? 8 : 0)
                     : "memory");
}

// The f32 form, on the CUDA cores: G lanes hold one token's row, eight values
// each, so a warp walks 32 / G streams of tokens, and a lane keeps the query
// heads' pieces and the output's in registers.  A lane's pieces of k and v come
// by asynchronous copies into a ring that is the lane's alone, kDepth tokens
// ahead, so that no wait but its own stands between a copy and its use; 16-byte
// pieces of the 32 lanes lie side by side.  Logits are summed over the G lanes
// by halves -- a lane passes on half of its heads at every step, and ends up
// with one -- so H heads take log2(H) + log2(G) - 1 + (H / 2 - 1) shuffles in
// place of H log2(G), and one exponential; the weights are passed back.
// Measured on a GB300: 64 x 4096 tokens, 32 heads of 128 over 8 kv heads, 523 us
// (4.1 TB/s, bound by instructions, shuffles foremost; over e4m3 320 us); 17 x
// up to 2000 tokens, 7 heads a kv head, 19 us (latency of a chunk and the join).
template <int KV, int H, int LG, bool WINDOW>
__global__ void __launch_bounds__(kThreadsOf<KV>, kResident<KV, H>) decode_rows(Args a) {
    constexpr bool E4 = KV == GBE_KV_E4M3;
    constexpr int kThreads = kThreadsOf<KV>, kWarps = kThreads / 32;
    constexpr int G = 1 << LG, LH = H == 1 ? 0 : H == 2 ? 1 : H == 4 ? 2 : 3;
    constexpr int kPieces = E4 ? 1 : 2, kBytes = E4 ? 8 : 16;         // of k, and as many of v, for a lane and token
    constexpr int kDepth = E4 ? 8 : 4, kSlot = 2 * kPieces * kBytes * 32;  // of a warp
    constexpr int streams = kThreads / G;
    extern __shared__ __align__(128) uint8_t raw[];  // the rings; then [kWarps][heads][D + 2]
    pdl_begin();
    const KvCacheArgs& c = a.c;
    const int D = c.D;
    const Part p = find_part(a, blockIdx.x);
    if (p.t0 >= p.t1 && p.chunk > 0) return;
    const int h0 = p.kvh * a.group + p.part * H;  // first query head
    const int heads = min(H, a.group - p.part * H);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & (G - 1), d0 = sub * 8;
    const bool mine = d0 < D;

    // the stream's token that is fetched next, and its page
    int tok = p.t0 + threadIdx.x / G, page_i, row;
    auto place = [&] {
        const int t = WINDOW ? p.seen.token(tok) : tok;
        page_i = t / c.page_size, row = t - page_i * c.page_size;
    };
    place();
    const int hop_pages = streams / c.page_size, hop_rows = streams - hop_pages * c.page_size;
    const int32_t* pages = a.table + (int64_t)p.b * a.max_pages;
    auto page_of = [&] { return tok < p.t1 ? pages[page_i] : -1; };
    int32_t page = page_of();
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(raw) + warp * kDepth * kSlot + lane * kBytes;
    uint32_t live = 0;  // bit i: the stream's token i steps ahead is there
    float scales[kDepth][2];
    auto fetch = [&](int slot, float (&sc)[2]) {
        const bool good = page >= 0 && page < c.n_pages && (!WINDOW || p.seen.sees(p.seen.token(tok), a.sinks));
        int64_t at = 0;
        if (good) {
            at = page * c.page_stride + ((int64_t)p.kvh * c.page_size + row) * D + d0;
            if constexpr (E4) {
                const int64_t si = ((int64_t)page * c.Hkv + p.kvh) * c.page_size + row;
                sc[0] = __uint_as_float((uint32_t)c.k_scale[si] << 23);
                sc[1] = __uint_as_float((uint32_t)c.v_scale[si] << 23);
            }
        }
        if (!mine) at = 0;
        if (good) {  // (lanes past D fill their places with zeros)
            const uint32_t to = ring + slot * kSlot;
            const uint8_t* k = static_cast<const uint8_t*>(c.k) + at * (E4 ? 1 : 4);
            const uint8_t* v = static_cast<const uint8_t*>(c.v) + at * (E4 ? 1 : 4);
#pragma unroll
            for (int x = 0; x < kPieces; ++x) {
                copy_async<kBytes>(to + x * kBytes * 32, k + x * kBytes, mine);
                copy_async<kBytes>(to + (kPieces + x) * kBytes * 32, v + x * kBytes, mine);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        tok += streams;
        page_i += hop_pages;
        row += hop_rows;
        if (row >= c.page_size) row -= c.page_size, ++page_i;
        if (WINDOW && tok >= p.seen.from && tok - streams < p.seen.from) place();  // past the gap
        page = page_of();
        return good;
    };
#pragma unroll
    for (int x = 0; x < kDepth - 1; ++x) live |= (uint32_t)fetch(x, scales[x]) << x;

    float2 q[H][4], acc[H][4];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc[h][e] = q[h][e] = make_float2(0.0f, 0.0f);
            if (mine && h < heads) {
                const int64_t at = p.b * a.q_stride + (int64_t)(h0 + h) * D + d0 + 2 * e;
                const float* from = static_cast<const float*>(a.q) + at;
                q[h][e] = make_float2(from[0] * a.scale, from[1] * a.scale);
            }
        }
    float m = -INFINITY, l = 0.0f;  // of the lane's own head, number sub >> (LG - LH)
    auto to_all = [&](float own, int h) {
        return __shfl_sync(0xFFFFFFFFu, own, (lane & ~(G - 1)) | (h << (LG - LH)));
    };
    // all streams of a CTA take the same number of steps, so that its shuffles meet
    const int steps = (p.t1 - p.t0 + streams - 1) / streams;
    int slot = 0;
    for (int step = 0; step < steps; ++step) {
        live |= (uint32_t)fetch(slot == 0 ? kDepth - 1 : slot - 1, scales[kDepth - 1]) << (kDepth - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        const uint8_t* const from = raw + warp * kDepth * kSlot + slot * kSlot + lane * kBytes;
        const bool good = live & 1u;
        auto piece = [&](int first, float2 (&f)[4]) {
            float y[8];
            if constexpr (E4) {
                uint2 w = *reinterpret_cast<const uint2*>(from + first * kBytes * 32);
                if (scales[0][first] == 0.0f) w = make_uint2(0u, 0u);  // zeros, whatever the codes
                e4m3x4_to_f32(w.x, y);
                e4m3x4_to_f32(w.y, y + 4);
            } else {
                const uint8_t* const at = from + first * kBytes * 32;
                *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(at);
                *reinterpret_cast<float4*>(y + 4) = *reinterpret_cast<const float4*>(at + kBytes * 32);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = make_float2(y[2 * e], y[2 * e + 1]);
        };
        float2 k[4];
        piece(0, k);
        float s[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float2 x = mul2_rn(q[h][0], k[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) x = fma2_rn(q[h][e], k[e], x);
            s[h] = x.x + x.y;
        }
#pragma unroll
        for (int b = 0; b < LH; ++b) {
            const int mask = G >> (b + 1), n = H >> (b + 1);
            const bool up = lane & mask;
#pragma unroll
            for (int x = 0; x < n; ++x) {
                const float send = up ? s[x] : s[x + n];
                s[x] = (up ? s[x + n] : s[x]) + __shfl_xor_sync(0xFFFFFFFFu, send, mask);
            }
        }
        float t = s[0];
#pragma unroll
        for (int mask = G >> (LH + 1); mask >= 1; mask >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, mask);
        if (E4) t *= scales[0][0];
        t = good ? t : -INFINITY;
        if (__any_sync(0xFFFFFFFFu, t > m + kGrowth || (t != t && m == -INFINITY))) {
            // (a NaN logit leaves a finite maximum, so that its NaN weight reaches the result)
            const float top = t == t ? t : -3.0e38f;
            const float m2 = top > m + kGrowth ? top : m, r = rescale(m, m2);
            m = m2;
            l *= r;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float rh = to_all(r, h);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[h][e] = mul2_rn(acc[h][e], make_float2(rh, rh));
            }
        }
        const float w = ex2(t - (m == -INFINITY ? 0.0f : m));
        l += w;
        if (good) {
            float2 v[4];
            piece(kPieces, v);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                // (the streams of a warp may differ in `good`: a shuffle within one stream's lanes)
                float wh = __shfl_sync(G == 32 ? 0xFFFFFFFFu : ((1u << G) - 1u) << (lane & ~(G - 1)), w,
                                       (lane & ~(G - 1)) | (h << (LG - LH)));
                if (E4) wh *= scales[0][1];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[h][e] = fma2_rn(make_float2(wh, wh), v[e], acc[h][e]);
            }
        }
        live >>= 1;
#pragma unroll
        for (int x = 0; x + 1 < kDepth; ++x) scales[x][0] = scales[x + 1][0], scales[x][1] = scales[x + 1][1];
        if (++slot == kDepth) slot = 0;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // the warp's streams joined, pair by pair: both sides compute the same sums
#pragma unroll
    for (int x = G; x < 32; x <<= 1) {
        const float mo = __shfl_xor_sync(0xFFFFFFFFu, m, x), lo = __shfl_xor_sync(0xFFFFFFFFu, l, x);
        const float m2 = fmaxf(m, mo), r = rescale(m, m2), ro = rescale(mo, m2);
        l = __fadd_rn(__fmul_rn(l, r), __fmul_rn(lo, ro));
        m = m2;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const float rh = to_all(r, h), roh = to_all(ro, h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float ox = __shfl_xor_sync(0xFFFFFFFFu, acc[h][e].x, x);
                const float oy = __shfl_xor_sync(0xFFFFFFFFu, acc[h][e].y, x);
                acc[h][e].x = __fadd_rn(__fmul_rn(acc[h][e].x, rh), __fmul_rn(ox, roh));
                acc[h][e].y = __fadd_rn(__fmul_rn(acc[h][e].y, rh), __fmul_rn(oy, roh));
            }
        }
    }
    // and the warps in order, in shared memory
    float* const sm = reinterpret_cast<float*>(raw + kWarps * kDepth * kSlot);
    const int W = D + 2;
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const float mh = to_all(m, h), lh = to_all(l, h);
        if (lane >= G || h >= heads) continue;
        float* o = sm + (warp * heads + h) * W;
        if (mine)
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(o + d0 + 2 * e) = acc[h][e];
        if (sub == 0) o[D] = mh, o[D + 1] = lh;
    }
    __syncthreads();
    const bool whole = p.C >= p.n;
    for (int i = threadIdx.x; i < heads * D; i += kThreads) {
        const int h = i / D, d = i - h * D;
        float mx = -INFINITY;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) mx = fmaxf(mx, sm[(x * heads + h) * W + D]);
        float sum = 0.0f, o = 0.0f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float* y = sm + (x * heads + h) * W;
            if (y[D] == -INFINITY) continue;  // nothing seen; a weight of 0 still carries NaN on
            const float r = ex2(y[D] - mx);
            sum = fmaf(y[D + 1], r, sum), o = fmaf(y[d], r, o);
        }
        if (whole) {
            Store<kF32>::store1(a.out, p.b * a.out_stride + (int64_t)(h0 + h) * D + d,
                                mx == -INFINITY ? 0.0f : o / sum);
        } else {
            const int64_t at = ((int64_t)p.b * a.Hq + h0 + h) * a.split + p.chunk;
            a.part_o[at * D + d] = o;
            if (d == 0) a.part_ml[at] = make_float2(mx, sum);
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
    const int n = find_seen(a, (int)b).n;
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

template <int KV, int H, int LG, bool WINDOW>
cudaError_t run(Args a, int64_t B, cudaStream_t st) {
    constexpr int kThreads = kThreadsOf<KV>, kWarps = kThreads / 32;
    constexpr int rings = kWarps * (KV == GBE_KV_E4M3 ? 8 * 512 : 4 * 2048);
    static FunctionLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(decode_rows<KV, H, LG, WINDOW>),
                                      rings + kWarps * H * ((8 << LG) + 2) * 4);
    if (e != cudaSuccess) return e;
    a.parts = (a.group + H - 1) / H;
    const int smem = rings + kWarps * (a.group < H ? a.group : H) * (a.c.D + 2) * 4;
    return launch(decode_rows<KV, H, LG, WINDOW>, dim3((unsigned)(B * a.split * a.c.Hkv * a.parts)), dim3(kThreads), smem, st,
                  a);
}

template <int KV, int H, bool WINDOW>
cudaError_t go(const Args& a, int64_t B, cudaStream_t st) {
    if (a.c.D <= 64) return run<KV, H, 3, WINDOW>(a, B, st);
    if (a.c.D <= 128) return run<KV, H, 4, WINDOW>(a, B, st);
    return run<KV, H, 5, WINDOW>(a, B, st);
}

template <int KV, bool WINDOW>
cudaError_t pick_heads(const Args& a, int64_t B, cudaStream_t st) {
    if (a.group == 1) return go<KV, 1, WINDOW>(a, B, st);
    if (a.group == 2) return go<KV, 2, WINDOW>(a, B, st);
    if (a.group <= 4) return go<KV, 4, WINDOW>(a, B, st);
    return go<KV, 8, WINDOW>(a, B, st);
}

template <int KV>
cudaError_t pick(const Args& a, int64_t B, cudaStream_t st) {
    return a.window > 0 ? pick_heads<KV, true>(a, B, st) : pick_heads<KV, false>(a, B, st);
}

}  // namespace

// Chunks of 512 tokens and more: shorter ones cost more in fixed work and in
// partial results (4 * Hq / Hkv bytes written and read for every token and kv
// head) than the SMs they bring in are worth.  128 chunks at most, so that two
// sequences of 131072 tokens make 2048 CTAs.
DecodeSplit decode_split(int64_t page_size, int64_t max_pages, int64_t window, int64_t sinks) {
    DecodeSplit s;
    s.least = 512;
    int64_t tokens = page_size * max_pages;
    if (window > 0 && window + sinks + 30 < tokens) tokens = window + sinks + 30;  // (both ends on 16 tokens' grid)
    const int64_t most = (tokens + s.least - 1) / s.least;
    s.split = (int)(most < 1 ? 1 : most > kMostChunks ? kMostChunks : most);
    return s;
}

cudaError_t launch_attn_decode(const DecodeArgs& d, int dtype, cudaStream_t st) {
    Args a = {};
    const DecodeSplit s = decode_split(d.c.page_size, d.max_pages, d.window, d.sinks);
    a.q = d.q, a.out = d.out, a.q_stride = d.q_stride, a.out_stride = d.out_stride;
    a.c = d.c, a.table = d.table, a.lens = d.lens;
    a.Hq = (int)d.Hq, a.group = (int)(d.Hq / d.c.Hkv), a.max_pages = (int)d.max_pages;
    a.window = (int)d.window, a.sinks = (int)d.sinks;
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
