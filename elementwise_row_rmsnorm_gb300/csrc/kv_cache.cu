// kv_cache.cu -- storing k and v rows of new tokens into a paged cache, and
// gathering cached rows back.
//
// The cache holds k and v as [n_pages, Hkv, page_size, D]; a token's slot is
// page * page_size + row.  Stored as they are (f32, bf16), rows are copied
// bit for bit.  Stored as e4m3, a row of D values has one power-of-two scale
// 2^(byte - 127): the least one, no smaller than 2^-126, that brings the
// row's largest finite magnitude to 448 (e4m3's largest) or below.  A
// power of two costs nothing against a scale of full precision -- e4m3 is
// a float, its relative step is the same at every scale -- and makes both
// directions exact but for the one rounding to e4m3: x * 2^-e never rounds
// in f32, and code * 2^e fits bf16's significand.
//
// Bound by HBM at prefill sizes and by the launch at decode sizes.  A row
// (one token, one head, k or v) belongs to a group of G lanes, G the power
// of two at or above D / 8, eight values a lane: 16 bytes of bf16 a load,
// and the row's largest magnitude by log2(G) shuffles within the group.  A
// lane keeps its place within a token (k or v, head, piece) and takes
// kUnroll tokens, all loads before the first store, so that what is left to
// compute for a token is where its slot lies: arithmetic on addresses was what
// bounded a form that divided for every row (write of 8192 tokens as e4m3
// 18.6 us, ALU at 79 %).  The largest magnitude is taken of the bits, two
// bf16 a word; a row that holds an infinity or a NaN goes through a slower
// branch.
#include "common.cuh"
#include "gbe_elementwise.h"
#include "kv_cache.cuh"
#include "launch.h"

namespace gbe {
namespace {

constexpr int kMostThreads = 512;
constexpr int kUnroll = 2;  // measured below

struct RowArgs {
    void* k;  // [T, Hkv, D], tokens `stride` apart: read by a write, written by a read
    void* v;
    int64_t k_stride, v_stride;
};

// A token has `items` = 2 Hkv G places for lanes; a CTA holds `slots_x` tokens
// side by side (or, of a token with many heads, the places from blockIdx.y on)
// and takes kUnroll of these one behind the other.
struct Shape {
    int lanes_log2, items, slots_x;
};

template <int DT, int KV, int N, bool VEC, bool WRITE>
__global__ void __launch_bounds__(kMostThreads) kv_rows(RowArgs a, KvCacheArgs c, const int32_t* slots, int64_t T,
                                                        Shape sh, Divisor by_page, int32_t* bad) {
    pdl_begin();
    const int G = 1 << sh.lanes_log2;
    const int side = threadIdx.x / sh.items;  // which of the tokens side by side
    const int item = threadIdx.x - side * sh.items + blockIdx.y * kMostThreads;
    const int sub = item & (G - 1), d0 = sub * N, hw = item >> sh.lanes_log2;
    const bool second = hw >= c.Hkv;
    const int head = second ? hw - c.Hkv : hw;
    // lanes past the CTA's last place take part in the shuffles alone
    const bool placed = side < sh.slots_x && head < c.Hkv;
    const bool mine = placed && d0 < c.D;
    const int64_t stride = second ? a.v_stride : a.k_stride;
    char* const rows = static_cast<char*>(second ? a.v : a.k);
    void* const kv = second ? c.v : c.k;
    uint8_t* const scales = second ? c.v_scale : c.k_scale;
    const int64_t x0 = (int64_t)head * c.D + d0, c0 = (int64_t)head * c.page_size * c.D + d0;
    const uint32_t capacity = (uint32_t)(c.n_pages * c.page_size);  // below 2^31

    const int64_t t0 = ((int64_t)blockIdx.x * kUnroll) * sh.slots_x + side;
    bool there[kUnroll], good[kUnroll];
    int64_t ci[kUnroll], si[kUnroll];
    Values<WRITE ? DT : KV, N> in[kUnroll];
    float scale[kUnroll];
    int32_t slot[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t t = t0 + u * sh.slots_x;
        there[u] = placed && t < T;
        slot[u] = there[u] ? slots[t] : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        good[u] = (uint32_t)slot[u] < capacity;
        if (slot[u] != -1 && !good[u] && bad != nullptr && item == 0) atomicAdd(bad, 1);
        const uint32_t at = good[u] ? (uint32_t)slot[u] : 0u;
        const uint32_t page = by_page.div(at), row = at - page * (uint32_t)c.page_size;
        ci[u] = page * c.page_stride + (c0 + (int64_t)row * c.D);
        si[u] = ((int64_t)page * c.Hkv + head) * c.page_size + row;
        in[u] = {};
        if (good[u] && mine) {
            if constexpr (WRITE)
                in[u].template load<VEC>(rows, (t0 + u * sh.slots_x) * stride + x0);
            else
                in[u].template load<true>(kv, ci[u]);
        }
        if constexpr (!WRITE && KV == GBE_KV_E4M3)
            scale[u] = good[u] ? __uint_as_float((uint32_t)scales[si[u]] << 23) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t xi = (t0 + u * sh.slots_x) * stride + x0;
        if constexpr (DT == KV) {
            if constexpr (WRITE) {
                if (good[u] && mine) in[u].template store<true>(kv, ci[u]);
            } else {
                if (there[u] && mine) in[u].template store<VEC>(rows, xi);  // zeros from a slot that is not there
            }
        } else if constexpr (WRITE) {
            float f[N];
            in[u].widen(f);
            uint32_t top = 0;  // the largest magnitude's bits; the lanes of a group share the row
            if constexpr (DT == kBF16) {
#pragma unroll
                for (int e = 0; e < N / 2; ++e) top = max_u16x2(top, in[u].w[e] & 0x7FFF7FFFu);
                for (int s = G >> 1; s >= 1; s >>= 1) top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
                top = max(top << 16, top & 0xFFFF0000u);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) top = max(top, in[u].w[e] & 0x7FFFFFFFu);
                for (int s = G >> 1; s >= 1; s >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
            }
            uint32_t byte = scale_byte(__uint_as_float(top));
            Values<GBE_KV_E4M3, N> out;
            if (__any_sync(0xFFFFFFFFu, top >= 0x7F800000u || byte >= 247u)) {
                float m = 0.0f;
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float v = fabsf(f[e]);
                    m = v <= 3.402823466e38f ? fmaxf(m, v) : m;  // infinities and NaN set no scale
                }
                for (int s = G >> 1; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
                byte = scale_byte(m);
                out = encode<false>(f, byte);
            } else {
                out = encode<true>(f, byte);
            }
            if (good[u] && sub == 0) scales[si[u]] = (uint8_t)byte;
            if (good[u] && mine) out.template store<true>(kv, ci[u]);
        } else {
            float f[N];
            if (scale[u] == 0.0f) {  // zeros, whatever the codes
                // (a branch: chosen word by word, 65536 tokens of f32 take 126 us, so 118 as without it)
                asm volatile("");
#pragma unroll
                for (int e = 0; e < N / 4; ++e) in[u].w[e] = 0u;
            }
            in[u].widen(f);
            Values<DT, N> out;
#pragma unroll
            for (int e = 0; e < N; ++e) f[e] = __fmul_rn(f[e], scale[u]);
            if constexpr (DT == kF32) {
#pragma unroll
                for (int e = 0; e < N; ++e) out.w[e] = __float_as_uint(f[e]);
            } else {
#pragma unroll
                for (int e = 0; e < N / 2; ++e) out.w[e] = f32x2_to_bf16x2_bits(f[2 * e], f[2 * e + 1]);
            }
            if (there[u] && mine) out.template store<VEC>(rows, xi);
        }
    }
}

template <int DT, int KV, int N, bool VEC, bool WRITE>
cudaError_t run(const RowArgs& a, const KvCacheArgs& c, const int32_t* slots, int64_t T, int32_t* bad,
                cudaStream_t st) {
    Shape sh = {0, 0, 1};
    while ((N << sh.lanes_log2) < c.D) ++sh.lanes_log2;
    sh.items = (2 * c.Hkv) << sh.lanes_log2;
    if (sh.items < kMostThreads / 2) sh.slots_x = kMostThreads / 2 / sh.items;
    const int threads = sh.items > kMostThreads ? kMostThreads : (sh.items * sh.slots_x + 31) / 32 * 32;
    const dim3 grid(ceil_div_i(T, (int64_t)sh.slots_x * kUnroll), ceil_div_i(sh.items, kMostThreads));
    if (sh.items > kMostThreads) sh.items = kMostThreads;  // of a CTA
    return launch(kv_rows<DT, KV, N, VEC, WRITE>, grid, dim3(threads), 0, st, a, c, slots, T, sh,
                  Divisor((uint32_t)c.page_size), bad);
}

// Sixteen values a lane between bf16 and e4m3 where both lie on the 16-byte
// grid, eight otherwise.  65536 tokens of 8 heads of 128 read back, 404 MB:
// 98 us with eight values and four tokens a lane, 71 us with sixteen and four,
// 61 us (6600 GB/s) with sixteen and two, 89 us with sixteen and eight; 8192
// tokens written: 13.0, 12.0, 10.9 and 11.9 us.
template <int DT, int KV, bool WRITE>
cudaError_t go(const RowArgs& a, const KvCacheArgs& c, const int32_t* slots, int64_t T, int32_t* bad, bool vec,
               cudaStream_t st) {
    if constexpr (DT == kBF16 && KV == GBE_KV_E4M3) {
        if (vec && c.D % 16 == 0 && c.page_stride % 16 == 0)
            return run<DT, KV, 16, true, WRITE>(a, c, slots, T, bad, st);
    }
    return vec ? run<DT, KV, 8, true, WRITE>(a, c, slots, T, bad, st)
               : run<DT, KV, 8, false, WRITE>(a, c, slots, T, bad, st);
}

template <bool WRITE>
cudaError_t pick(const RowArgs& a, const KvCacheArgs& c, const int32_t* slots, int64_t T, int32_t* bad, int dtype,
                 bool vec, cudaStream_t st) {
    const bool e4m3 = c.dtype == GBE_KV_E4M3;
    if (dtype == GBE_F32)
        return e4m3 ? go<kF32, GBE_KV_E4M3, WRITE>(a, c, slots, T, bad, vec, st)
                    : go<kF32, GBE_KV_F32, WRITE>(a, c, slots, T, bad, vec, st);
    return e4m3 ? go<kBF16, GBE_KV_E4M3, WRITE>(a, c, slots, T, bad, vec, st)
                : go<kBF16, GBE_KV_BF16, WRITE>(a, c, slots, T, bad, vec, st);
}

}  // namespace

cudaError_t launch_kv_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, const int32_t* slots,
                            int64_t T, const KvCacheArgs& c, int32_t* bad, int dtype, bool vec, cudaStream_t st) {
    const RowArgs a = {const_cast<void*>(k), const_cast<void*>(v), k_stride, v_stride};
    return pick<true>(a, c, slots, T, bad, dtype, vec, st);
}

cudaError_t launch_kv_read(void* k, int64_t k_stride, void* v, int64_t v_stride, const int32_t* slots, int64_t T,
                           const KvCacheArgs& c, int32_t* bad, int dtype, bool vec, cudaStream_t st) {
    const RowArgs a = {k, v, k_stride, v_stride};
    return pick<false>(a, c, slots, T, bad, dtype, vec, st);
}

}  // namespace gbe
