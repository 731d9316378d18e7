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
// and the row's largest magnitude by log2(G) shuffles within the group.
#include "common.cuh"
#include "gbe_elementwise.h"
#include "kv_cache.cuh"
#include "launch.h"

namespace gbe {
namespace {

constexpr int kThreads = 256;

// Eight values of a row starting at element i, widened to f32.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&f)[8]) {
    if constexpr (VEC && DT == kBF16) {
        Store<kBF16>::unpack(ld_stream(static_cast<const uint16_t*>(base) + i), f);
    } else if constexpr (VEC) {
        const float* p = static_cast<const float*>(base) + i;
        const Vec16 a = ld_stream(p), b = ld_stream(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(a.w[e]), f[4 + e] = __uint_as_float(b.w[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = Store<DT>::load1(base, i + e);
    }
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&f)[8]) {
    if constexpr (VEC && DT == kBF16) {
        st_stream(static_cast<uint16_t*>(base) + i, Store<kBF16>::pack(f));
    } else if constexpr (VEC) {
        Vec16 a, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) a.w[e] = __float_as_uint(f[e]), b.w[e] = __float_as_uint(f[4 + e]);
        st_stream(static_cast<float*>(base) + i, a);
        st_stream(static_cast<float*>(base) + i + 4, b);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) Store<DT>::store1(base, i + e, f[e]);
    }
}

// The scale byte of a row whose largest finite magnitude is m: 448 = 1.75 *
// 2^8, so with m = c * 2^x, 1 <= c < 2, the exponent is x - 8 when c <= 1.75
// and x - 7 above.
__device__ __forceinline__ uint32_t scale_byte(float m) {
    const uint32_t u = __float_as_uint(m);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // + 127
    return e < 1 ? 1u : (uint32_t)e;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

struct RowArgs {
    const void* x[2];  // k and v rows: [T, Hkv, D], tokens `stride` apart
    void* y[2];
    int64_t stride[2];
};

// rows of one launch: r = (token * 2 + which) * Hkv + head
template <int DT, int KV, bool VEC, bool WRITE>
__global__ void __launch_bounds__(kThreads) kv_rows(RowArgs a, KvCacheArgs c, const int32_t* slots, uint32_t n_rows,
                                                    int lanes_log2, int32_t* bad) {
    pdl_begin();
    const int G = 1 << lanes_log2;
    const int sub = threadIdx.x & (G - 1), d0 = sub * 8;
    const bool mine = d0 < c.D;
    const uint32_t r = (uint32_t)(((uint64_t)blockIdx.x * kThreads + threadIdx.x) >> lanes_log2);
    if (r >= n_rows) return;
    // a group's lanes are within one warp (G <= 32) and share their row, so
    // the shuffles below meet whole groups
    const uint32_t group = G == 32 ? 0xFFFFFFFFu : ((1u << G) - 1u) << ((threadIdx.x & 31) & ~(G - 1));
    const int head = (int)(r % (uint32_t)c.Hkv);
    const uint32_t tw = r / (uint32_t)c.Hkv;
    const int64_t t = tw >> 1;
    const int which = (int)(tw & 1);
    const int32_t slot = slots[t];
    const bool good = slot >= 0 && slot < c.n_pages * (int64_t)c.page_size;
    if (!good && slot != -1 && bad != nullptr && which == 0 && head == 0 && sub == 0) atomicAdd(bad, 1);
    const int64_t xi = t * a.stride[which] + (int64_t)head * c.D + d0;
    if (!good) {
        if (!WRITE && mine) {
            const float zero[8] = {};
            store8<DT, VEC>(a.y[which], xi, zero);
        }
        return;
    }
    const int64_t page = slot / c.page_size, row = slot % c.page_size;
    const int64_t ci = page * c.page_stride + ((int64_t)head * c.page_size + row) * c.D + d0;
    const int64_t si = (page * c.Hkv + head) * c.page_size + row;
    void* const kv = which ? c.v : c.k;
    uint8_t* const scales = which ? c.v_scale : c.k_scale;
    float f[8] = {};
    if constexpr (WRITE) {
        if (mine) load8<DT, VEC>(a.x[which], xi, f);
        if constexpr (KV == GBE_KV_E4M3) {
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = fabsf(f[e]);
                m = v <= 3.402823466e38f ? fmaxf(m, v) : m;  // infinities and NaN set no scale
            }
            for (int s = G >> 1; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(group, m, s));
            const uint32_t byte = scale_byte(m);
            if (sub == 0) scales[si] = (uint8_t)byte;
            if (mine) {
                const float inv = __uint_as_float((254u - byte) << 23);
                const float most = byte == 247u ? 240.0f : 448.0f;  // 256 * 2^120 would be past f32's range
                uint32_t w[2];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[e] = __fmul_rn(f[e], inv);
                    // infinities become NaN
                    f[e] = fabsf(f[e]) <= 448.0f ? copysignf(fminf(fabsf(f[e]), most), f[e])
                                                 : __uint_as_float(0x7FC00000u);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    w[e] = e4m3x2(f[4 * e], f[4 * e + 1]) | e4m3x2(f[4 * e + 2], f[4 * e + 3]) << 16;
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(kv) + ci) = make_uint2(w[0], w[1]);
            }
        } else {
            if (mine) store8<KV, true>(kv, ci, f);
        }
    } else if (mine) {
        if constexpr (KV == GBE_KV_E4M3) {
            const float scale = __uint_as_float((uint32_t)scales[si] << 23);
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(kv) + ci);
            e4m3x4_to_f32(w.x, f);
            e4m3x4_to_f32(w.y, f + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __fmul_rn(f[e], scale);
        } else {
            load8<KV, true>(kv, ci, f);
        }
        store8<DT, VEC>(a.y[which], xi, f);
    }
}

template <int DT, int KV, bool WRITE>
cudaError_t go(const RowArgs& a, const KvCacheArgs& c, const int32_t* slots, int64_t T, int32_t* bad, bool vec,
               cudaStream_t st) {
    int lg = 0;
    while ((8 << lg) < c.D) ++lg;
    const uint32_t n_rows = (uint32_t)(T * 2 * c.Hkv);  // at most 2^31, as the entry points check
    const dim3 grid(ceil_div_i((int64_t)n_rows << lg, kThreads));
    return vec ? launch(kv_rows<DT, KV, true, WRITE>, grid, dim3(kThreads), 0, st, a, c, slots, n_rows, lg, bad)
               : launch(kv_rows<DT, KV, false, WRITE>, grid, dim3(kThreads), 0, st, a, c, slots, n_rows, lg, bad);
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
    const RowArgs a = {{k, v}, {nullptr, nullptr}, {k_stride, v_stride}};
    return pick<true>(a, c, slots, T, bad, dtype, vec, st);
}

cudaError_t launch_kv_read(void* k, int64_t k_stride, void* v, int64_t v_stride, const int32_t* slots, int64_t T,
                           const KvCacheArgs& c, int32_t* bad, int dtype, bool vec, cudaStream_t st) {
    const RowArgs a = {{nullptr, nullptr}, {k, v}, {k_stride, v_stride}};
    return pick<false>(a, c, slots, T, bad, dtype, vec, st);
}

}  // namespace gbe
