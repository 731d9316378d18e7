// kv_cache.cuh -- device helpers shared by the kernels that read or write the paged cache.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "gbe_elementwise.h"

namespace gbe {

// Four e4m3 codes of a word, lowest byte first, widened exactly.
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* f) {
    uint32_t a, b;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(b) : "r"(w));
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f[0]), "=f"(f[1]) : "r"(a));
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f[2]), "=f"(f[3]) : "r"(b));
}

// n / d for n < 2^31: with 2^(s - 1) < d <= 2^s and m = ceil(2^(31 + s) / d),
// n m / 2^(31 + s) exceeds n / d by less than 2^-s <= 1 / d.
struct Divisor {
    uint32_t m;
    int s;
    explicit Divisor(uint32_t d) : s(0) {
        while ((1ull << s) < d) ++s;
        m = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> (31 + s)); }
};

// N values of type DT, as bits.
template <int DT, int N>
struct Values {
    static constexpr int kEs = DT == kF32 ? 4 : DT == kBF16 ? 2 : 1, W = N * kEs / 4;
    uint32_t w[W];
    template <bool VEC>
    __device__ __forceinline__ void load(const void* base, int64_t i) {
        const char* const p = static_cast<const char*>(base) + i * kEs;
        if constexpr (W == 2) {
            asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
        } else if constexpr (VEC) {
#pragma unroll
            for (int x = 0; x < W / 4; ++x) {
                const Vec16 v = ld_stream(p + 16 * x);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[4 * x + e] = v.w[e];
            }
        } else if constexpr (DT == kF32) {
#pragma unroll
            for (int e = 0; e < W; ++e) w[e] = reinterpret_cast<const uint32_t*>(p)[e];
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e)
                w[e] = (uint32_t)reinterpret_cast<const uint16_t*>(p)[2 * e] |
                       (uint32_t)reinterpret_cast<const uint16_t*>(p)[2 * e + 1] << 16;
        }
    }
    template <bool VEC>
    __device__ __forceinline__ void store(void* base, int64_t i) const {
        char* const p = static_cast<char*>(base) + i * kEs;
        if constexpr (W == 2) {
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (VEC) {
#pragma unroll
            for (int x = 0; x < W / 4; ++x) {
                Vec16 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v.w[e] = w[4 * x + e];
                st_stream(p + 16 * x, v);
            }
        } else if constexpr (DT == kF32) {
#pragma unroll
            for (int e = 0; e < W; ++e) reinterpret_cast<uint32_t*>(p)[e] = w[e];
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                reinterpret_cast<uint16_t*>(p)[2 * e] = (uint16_t)w[e];
                reinterpret_cast<uint16_t*>(p)[2 * e + 1] = (uint16_t)(w[e] >> 16);
            }
        }
    }
    __device__ __forceinline__ void widen(float (&f)[N]) const {
        if constexpr (DT == GBE_KV_E4M3) {
#pragma unroll
            for (int e = 0; e < W; ++e) e4m3x4_to_f32(w[e], f + 4 * e);
        } else if constexpr (DT == kF32) {
#pragma unroll
            for (int e = 0; e < W; ++e) f[e] = __uint_as_float(w[e]);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                f[2 * e] = __uint_as_float(w[e] << 16);
                f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            }
        }
    }
};

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

// The largest of the two 16-bit halves' maxima, half by half.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// The codes of a row's values at scale byte `byte`; PLAIN: all of them finite,
// and byte below 247.
template <bool PLAIN, int N>
__device__ __forceinline__ Values<GBE_KV_E4M3, N> encode(float (&f)[N], uint32_t byte) {
    const float inv = __uint_as_float((254u - byte) << 23);
    const float most = byte == 247u ? 240.0f : 448.0f;  // 256 * 2^120 would be past f32's range
#pragma unroll
    for (int e = 0; e < N; ++e) {
        f[e] = __fmul_rn(f[e], inv);
        if (!PLAIN)  // infinities become NaN
            f[e] = fabsf(f[e]) <= 448.0f ? fmaxf(fminf(f[e], most), -most) : __uint_as_float(0x7FC00000u);
    }
    Values<GBE_KV_E4M3, N> out;
#pragma unroll
    for (int e = 0; e < N / 4; ++e)
        out.w[e] = e4m3x2(f[4 * e], f[4 * e + 1]) | e4m3x2(f[4 * e + 2], f[4 * e + 3]) << 16;
    return out;
}

}  // namespace gbe
