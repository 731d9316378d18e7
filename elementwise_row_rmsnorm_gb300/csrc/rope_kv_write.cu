// rope_kv_write.cu -- q and k turned by their positions, q written, k and v
// stored into the paged cache, in one pass.
//
//   q'[t, h] = rot(q[t, h], pos[t]),  slot[t] <- (rot(k[t, h], pos[t]), v[t, h])
//
// The rotation is gbe_rope_qk's and what reaches the cache is gbe_kv_write's,
// bit for bit: k' is rounded to the storage type and, over an 8-bit cache, that
// value is encoded.  (A rounding to bf16 ahead of e4m3's: 2^-9 beside 2^-4, and
// it makes the cache's bytes those of the two calls.)
//
// Bound by HBM at prefill sizes, by the launch at decode sizes.  Apart, the two
// calls write k' and read it again and cost a launch more.  A group of lanes,
// the power of two at or above a head's lanes, holds a head at a time, sixteen
// values a lane in two pieces of eight: both members of its pairs in the half
// layout, neighbours otherwise; so a pair is turned in registers and an 8-bit
// row's largest magnitude takes log2 shuffles.  A lane goes through HEADS heads
// of its token, all loads ahead of the first store.  Angles are formed once a CTA,
// into shared memory: formed by the lanes, each its own, they bounded the kernel.
//
// Measured: 8192 tokens of 32 + 8 + 8 heads of 128 into 8 bits and read back from
// there (which takes 10 us) 50 us, 4.7 TB/s; 64 tokens 2.6 us a call in a graph.  A
// CTA's positions, angles and rows come one behind the other, so what hides them is
// more CTAs: three an SM, where two took 60 us; two heads a lane in four of them 51.
#include "gbe_elementwise.h"
#include "kv_cache.cuh"
#include "launch.h"
#include "rope.cuh"

namespace gbe {
namespace {

constexpr int kThreads = 256;
constexpr int kAngles = 1152;  // of a CTA, at most (see below)

// The lanes of a group, and how a token's heads are dealt out to groups.
struct Shape {
    int lanes_log2, pair_lanes;  // pair_lanes: of the half layout, the others hold what is not turned
    int q_chunks, k_chunks;
};

template <int DT>
__device__ __forceinline__ Values<DT, 8> narrow(const float (&f)[8]) {
    Values<DT, 8> v;
#pragma unroll
    for (int e = 0; e < Values<DT, 8>::W; ++e)
        v.w[e] = DT == kF32 ? __float_as_uint(f[e]) : f32x2_to_bf16x2_bits(f[2 * e], f[2 * e + 1]);
    return v;
}

// The largest of a row's finite magnitudes sets its scale; the row is spread
// over the lanes of `mask`, G of them.
__device__ __forceinline__ float row_max(float m, int G, uint32_t mask) {
    for (int s = G >> 1; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(mask, m, s));
    return m;
}

template <int DT, int KV, int LAYOUT, int HEADS>
__global__ void __launch_bounds__(kThreads, 3) rope_kv_rows(RopeKvArgs a, Shape sh, Divisor by_token, Divisor by_page,
                                                         Divisor by_half) {
    __shared__ float2 angles[kAngles];
    pdl_begin();
    constexpr bool E4 = KV == GBE_KV_E4M3;
    const KvCacheArgs& c = a.c;
    const int64_t lane_id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int G = 1 << sh.lanes_log2, sub = (int)lane_id & (G - 1);
    const uint32_t group = (uint32_t)(lane_id >> sh.lanes_log2);
    const uint32_t per = (uint32_t)(sh.q_chunks + 2 * sh.k_chunks), t = by_token.div(group);
    const bool there = t < a.T;  // (of whole groups)
    const uint32_t mask = (G == 32 ? 0xFFFFFFFFu : ((1u << G) - 1u)) << (threadIdx.x & 31 & ~(G - 1));
    int chunk = (int)(group - t * per);
    const bool is_q = chunk < sh.q_chunks;
    if (!is_q) chunk -= sh.q_chunks;
    const bool is_v = !is_q && chunk >= sh.k_chunks;
    if (is_v) chunk -= sh.k_chunks;
    const int h0 = chunk * HEADS, heads = min(HEADS, (is_q ? a.Hq : c.Hkv) - h0);

    // the lane's two pieces of a head, and which of their pairs it turns
    const int D = c.D, half = a.r >> 1;
    const bool pair_lane = LAYOUT == 0 && !is_v && sub < sh.pair_lanes;
    const int past = LAYOUT == 0 && !is_v ? sub - sh.pair_lanes : sub;
    const int d0 = pair_lane ? 8 * sub : 16 * past + (LAYOUT == 0 && !is_v ? a.r : 0);
    const int d1 = pair_lane ? half + 8 * sub : d0 + 8;
    const bool has0 = d0 < D, has1 = d1 < D;
    const bool turn0 = LAYOUT == 0 ? pair_lane : !is_v && d0 < a.r, turn1 = LAYOUT == 0 ? pair_lane : !is_v && d1 < a.r;

    const int64_t stride = is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride;
    const void* const from = is_q ? a.q : is_v ? a.v : a.k;
    const int64_t row0 = t * stride + (int64_t)h0 * D;
    const int32_t slot = is_q || !there ? -1 : a.slots[t];
    const bool good = !is_q && (uint32_t)slot < (uint32_t)(c.n_pages * c.page_size);
    if (!is_q && !good && slot != -1 && a.bad != nullptr && !is_v && chunk == 0 && sub == 0) atomicAdd(a.bad, 1);
    const bool work = there && (is_q || good);
    Values<DT, 8> x0[HEADS], x1[HEADS];
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
        x0[j] = {}, x1[j] = {};
        if (!work) continue;
        if (j < heads && has0) x0[j].template load<true>(from, row0 + (int64_t)j * D + d0);
        if (j < heads && has1) x1[j].template load<true>(from, row0 + (int64_t)j * D + d1);
    }
    int64_t ci = 0, si = 0;  // of head h0 in the cache, and of its scale
    if (!is_q) {
        const uint32_t page = by_page.div((uint32_t)slot), row = (uint32_t)slot - page * (uint32_t)c.page_size;
        ci = page * c.page_stride + ((int64_t)h0 * c.page_size + row) * D;
        si = ((int64_t)page * c.Hkv + h0) * c.page_size + row;
    }
    // The angles of the CTA's tokens, each formed once, while the rows are on their
    // way.  (A token has 2 G lanes at least and 8 G pairs at most, so these are at most
    // 8 G (254 / 2 G + 2): kAngles, at G = 16.)
    const uint32_t t0 = by_token.div((uint32_t)(((int64_t)blockIdx.x * kThreads) >> sh.lanes_log2));
    const uint32_t t1 = by_token.div((uint32_t)(((int64_t)blockIdx.x * kThreads + kThreads - 1) >> sh.lanes_log2));
    for (uint32_t x = threadIdx.x; x < (t1 - t0 + 1) * half; x += kThreads) {
        const uint32_t token = by_half.div(x);
        const int i = (int)(x - token * half);
        float2 y = make_float2(0.0f, 0.0f);
        if (t0 + token < a.T)
            angle<true>(a.pos[t0 + token], i, a.inv_freq, a.cos_sin, a.cache_len, half, y.x, y.y);
        angles[x] = y;
    }
    __syncthreads();
    if (!work) return;  // (whole groups)
    float cs[8], sn[8];
    if (turn0) {
        const float2* const from = angles + (t - t0) * half;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = LAYOUT == 0 ? d0 + e : (e < 4 ? d0 : d1) / 2 + (e & 3);
            if (i < half) cs[e] = from[i].x, sn[e] = from[i].y;
        }
    }
    void* const kv = is_v ? c.v : c.k;
    uint8_t* const scales = is_v ? c.v_scale : c.k_scale;
#pragma unroll
    for (int j = 0; j < HEADS; ++j) {
        if (j >= heads) break;
        if (turn0) {
            float f0[8], f1[8];
            x0[j].widen(f0);
            x1[j].widen(f1);
            if constexpr (LAYOUT == 0) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float2 u, w;
                    rotate2(make_float2(f0[e], f0[e + 1]), make_float2(f1[e], f1[e + 1]), make_float2(cs[e], cs[e + 1]),
                            make_float2(sn[e], sn[e + 1]), a.mu, u, w);
                    f0[e] = u.x, f0[e + 1] = u.y, f1[e] = w.x, f1[e + 1] = w.y;
                }
                x0[j] = narrow<DT>(f0), x1[j] = narrow<DT>(f1);
            } else {
                auto turn = [&](float (&f)[8], int e0) {
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        float2 u, w;
                        rotate2(make_float2(f[2 * e], f[2 * e + 2]), make_float2(f[2 * e + 1], f[2 * e + 3]),
                                make_float2(cs[e0 + e], cs[e0 + e + 1]), make_float2(sn[e0 + e], sn[e0 + e + 1]), a.mu, u,
                                w);
                        f[2 * e] = u.x, f[2 * e + 2] = u.y, f[2 * e + 1] = w.x, f[2 * e + 3] = w.y;
                    }
                };
                turn(f0, 0);
                x0[j] = narrow<DT>(f0);
                if (turn1) {
                    turn(f1, 4);
                    x1[j] = narrow<DT>(f1);
                }
            }
        }
        if (is_q) {
            const int64_t to = row0 + (int64_t)j * D;
            if (has0 && (turn0 || a.q != a.q_out)) x0[j].template store<true>(a.q_out, to + d0);
            if (has1 && (turn1 || a.q != a.q_out)) x1[j].template store<true>(a.q_out, to + d1);
            continue;
        }
        const int64_t to = ci + (int64_t)j * c.page_size * D;
        if constexpr (!E4) {
            if (has0) x0[j].template store<true>(kv, to + d0);
            if (has1) x1[j].template store<true>(kv, to + d1);
        } else {
            float f[16];
            {
                float f0[8], f1[8];
                x0[j].widen(f0);
                x1[j].widen(f1);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = f0[e], f[8 + e] = f1[e];
            }
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
            for (int s = G >> 1; s >= 1; s >>= 1) top = max(top, __shfl_xor_sync(mask, top, s));
            uint32_t byte = scale_byte(__uint_as_float(top));
            Values<GBE_KV_E4M3, 16> code;
            if (top >= 0x7F800000u || byte >= 247u) {  // (the same in all of the row's lanes)
                float m = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float y = fabsf(f[e]);
                    m = y <= 3.402823466e38f ? fmaxf(m, y) : m;  // infinities and NaN set no scale
                }
                byte = scale_byte(row_max(m, G, mask));
                code = encode<false>(f, byte);
            } else {
                code = encode<true>(f, byte);
            }
            if (sub == 0) scales[si + (int64_t)j * c.page_size] = (uint8_t)byte;
            uint8_t* const at = static_cast<uint8_t*>(kv) + to;
            if (has0) *reinterpret_cast<uint2*>(at + d0) = make_uint2(code.w[0], code.w[1]);
            if (has1) *reinterpret_cast<uint2*>(at + d1) = make_uint2(code.w[2], code.w[3]);
        }
    }
}

// Off the 16-byte grid, and widths that do not split into pieces of eight: a
// warp a head, turned into shared memory and stored from there.
template <int DT, int KV>
__global__ void __launch_bounds__(kThreads) rope_kv_scalar(RopeKvArgs a, int layout) {
    pdl_begin();
    using S = Store<DT>;
    constexpr bool E4 = KV == GBE_KV_E4M3;
    __shared__ float rows[kThreads / 32][256];
    const KvCacheArgs& c = a.c;
    const int lane = threadIdx.x & 31, per = a.Hq + 2 * c.Hkv;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = item / per;
    if (t >= a.T) return;
    int h = (int)(item - t * per);
    const bool is_q = h < a.Hq;
    if (!is_q) h -= a.Hq;
    const bool is_v = !is_q && h >= c.Hkv;
    if (is_v) h -= c.Hkv;
    const int32_t slot = is_q ? -1 : a.slots[t];
    if (!is_q && (uint32_t)slot >= (uint32_t)(c.n_pages * c.page_size)) {
        if (slot != -1 && a.bad != nullptr && !is_v && h == 0 && lane == 0) atomicAdd(a.bad, 1);
        return;
    }
    const int D = c.D, r = is_v ? 0 : a.r, half = r >> 1;
    const void* const from = is_q ? a.q : is_v ? a.v : a.k;
    const int64_t row = t * (is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride) + (int64_t)h * D;
    const int32_t p = is_v ? 0 : a.pos[t];
    float* const y = rows[threadIdx.x >> 5];
    for (int i = lane; i < half; i += 32) {
        float cs, sn, u, w;
        angle<true>(p, i, a.inv_freq, a.cos_sin, a.cache_len, half, cs, sn);
        const int ia = layout == 0 ? i : 2 * i, ib = layout == 0 ? i + half : 2 * i + 1;
        rotate(S::load1(from, row + ia), S::load1(from, row + ib), cs, sn, a.mu, u, w);
        y[ia] = S::round(u), y[ib] = S::round(w);
    }
    const bool in_place = is_q && a.q == a.q_out;  // then what is not turned is not touched
    for (int d = r + lane; d < D && !in_place; d += 32) y[d] = S::load1(from, row + d);
    __syncwarp();
    auto store = [&](void* dst, int64_t to, int n) {
        for (int d = lane; d < n; d += 32) {
            const uint32_t bits = __float_as_uint(y[d]);
            if (DT == kF32)
                static_cast<uint32_t*>(dst)[to + d] = bits;
            else
                static_cast<uint16_t*>(dst)[to + d] = (uint16_t)(bits >> 16);
        }
    };
    if (is_q) {
        store(a.q_out, row, in_place ? r : D);
        return;
    }
    const int64_t page = slot / c.page_size, at = slot - page * c.page_size;
    const int64_t to = page * c.page_stride + ((int64_t)h * c.page_size + at) * D;
    void* const kv = is_v ? c.v : c.k;
    if constexpr (!E4) {
        store(kv, to, D);
    } else {
        float m = 0.0f;
        for (int d = lane; d < D; d += 32) m = fmaxf(m, fabsf(y[d]) <= 3.402823466e38f ? fabsf(y[d]) : 0.0f);
        const uint32_t byte = scale_byte(row_max(m, 32, 0xFFFFFFFFu));
        if (lane == 0) (is_v ? c.v_scale : c.k_scale)[(page * c.Hkv + h) * c.page_size + at] = (uint8_t)byte;
        for (int d = lane * 8; d < D; d += 256) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = y[d + e];
            const Values<GBE_KV_E4M3, 8> code = encode<false>(f, byte);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(kv) + to + d) = make_uint2(code.w[0], code.w[1]);
        }
    }
}

template <int DT, int KV, int LAYOUT, int HEADS>
cudaError_t run(const RopeKvArgs& a, Shape sh, cudaStream_t st) {
    sh.q_chunks = ceil_div_i(a.Hq, HEADS);
    sh.k_chunks = ceil_div_i(a.c.Hkv, HEADS);
    const int per = sh.q_chunks + 2 * sh.k_chunks;
    const int64_t lanes = (a.T * per) << sh.lanes_log2;
    return launch(rope_kv_rows<DT, KV, LAYOUT, HEADS>, dim3((unsigned)((lanes + kThreads - 1) / kThreads)),
                  dim3(kThreads), 0, st, a, sh, Divisor((uint32_t)per), Divisor((uint32_t)a.c.page_size),
                  Divisor((uint32_t)(a.r > 0 ? a.r / 2 : 1)));
}

template <int DT, int KV, int LAYOUT>
cudaError_t pick(const RopeKvArgs& a, cudaStream_t st) {
    Shape sh = {0, LAYOUT == 0 ? a.r / 16 : 0, 0, 0};
    const int lanes = LAYOUT == 0 ? sh.pair_lanes + (a.c.D - a.r + 15) / 16 : 0, plain = (a.c.D + 15) / 16;
    while ((1 << sh.lanes_log2) < (lanes > plain ? lanes : plain)) ++sh.lanes_log2;
    constexpr int kHeads = DT == kF32 ? 2 : 4;
    const int64_t many = (a.T * (ceil_div_i(a.Hq, kHeads) + 2 * ceil_div_i(a.c.Hkv, kHeads))) << sh.lanes_log2;
    return many >= 1024 * (int64_t)sm_count() ? run<DT, KV, LAYOUT, kHeads>(a, sh, st)
                                              : run<DT, KV, LAYOUT, 1>(a, sh, st);
}

template <int DT, int KV>
cudaError_t go(const RopeKvArgs& a, int layout, bool vec, cudaStream_t st) {
    if (vec && a.r % (layout == 0 ? 16 : 8) == 0)
        return layout == 0 ? pick<DT, KV, 0>(a, st) : pick<DT, KV, 1>(a, st);
    const int64_t warps = a.T * (a.Hq + 2 * a.c.Hkv);
    return launch(rope_kv_scalar<DT, KV>, dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32))),
                  dim3(kThreads), 0, st, a, layout);
}

}  // namespace

cudaError_t launch_rope_kv_write(const RopeKvArgs& a, int layout, int dtype, bool vec, cudaStream_t st) {
    const bool e4m3 = a.c.dtype == GBE_KV_E4M3;
    if (dtype == GBE_F32)
        return e4m3 ? go<kF32, GBE_KV_E4M3>(a, layout, vec, st) : go<kF32, GBE_KV_F32>(a, layout, vec, st);
    return e4m3 ? go<kBF16, GBE_KV_E4M3>(a, layout, vec, st) : go<kBF16, GBE_KV_BF16>(a, layout, vec, st);
}

}  // namespace gbe
