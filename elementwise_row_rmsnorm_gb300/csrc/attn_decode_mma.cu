// attn_decode_mma.cu -- gbe_attn_decode for bf16 queries, over a bf16 or an
// e4m3 cache, with the products on the tensor cores.
//
// Bound by HBM: each cached row is read once, and four query heads to a kv
// head need only 4 (bf16) or 8 (e4m3) flops a byte, some 50 TFLOP/s.  So the
// small warp-wide products (mma.sync, 16 tokens by 8 heads) do, and rows go
// from global memory to registers in the very layout that they want, without
// shared memory:
//
//   S^T [16 tokens x 8 heads]  = K [16 x D] q^T       A: K, B: q
//   O^T [16 entries x 8 heads] += V^T [16 x 16] P^T   A: V, B: P
//
// A product may number its inner index as it likes as long as both operands
// agree, and its rows too.  With g = lane / 4 and t = lane % 4, lane (g, t)
// loads eight consecutive entries of K at 32 c + 8 t of tokens g and g + 8
// (four lanes: 64 bytes of a row), the inner index of the first product; and
// eight of V at 64 c + 8 g of tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9 (eight
// lanes: 128 bytes of a row), its rows in the second one, where pairs of
// tokens are put together by byte permutes.  P changes from the layout of a
// result to that of B by movmatrix.
//
// A CTA is four warps, each with steps of tokens of its own and its own
// running maximum, joined at the end in shared memory.  The maximum in use
// lags behind by up to 2^8 (as weights, floats all of them, may), so that a
// step costs one vote instead of a reduction.
//
// e4m3: codes widen to f16 exactly (one conversion for two), so the products
// are f16.  q is brought into f16's range by a power of two for each head; k's
// scale multiplies the logit, v's the weight, as 2^(byte - E) with a common E
// that lags like the maximum does (2^1; the maximum 2^2 here), times 2^12 so
// that the largest come near f16's end.  f16 then holds a weight to 2^-8 of
// itself, as bf16 would, down to 2^-29 of the row's largest, and to 2^-37 of
// that one below; a step with a scale more than 2^8 under E takes bf16 weights
// and values instead.
#include <type_traits>

#include "attn_decode.cuh"
#include "gbe_elementwise.h"
#include "kv_cache.cuh"

namespace gbe {
namespace decode {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kHeads = 8;           // query heads of a CTA
constexpr int kScaleGrowth = 1, kScaleDrop = 8;

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// The two e4m3 codes of the low (HI = 0) or high half of w, widened to f16.
template <int HI>
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
    uint32_t d;
    if (HI)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(w));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t f16x2_bf16x2(uint32_t x) {
    float lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi) : "r"(x));
    return f32x2_to_bf16x2_bits(lo, hi);
}

// Eight consecutive entries of a cached row.
template <int KV>
struct Eight {
    static constexpr int W = KV == GBE_KV_E4M3 ? 2 : 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const void* base, int64_t i, bool there) {
#pragma unroll
        for (int e = 0; e < W; ++e) w[e] = 0;
        if (!there) return;
        if constexpr (KV == GBE_KV_E4M3) {
            asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
                         : "=r"(w[0]), "=r"(w[1]) : "l"(static_cast<const uint8_t*>(base) + i));
        } else {
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "l"(static_cast<const uint16_t*>(base) + i));
        }
    }
};

template <int KV, int DP>
__global__ void __launch_bounds__(kThreads, DP <= 128 ? 4 : 2) decode_mma(Args a) {
    constexpr bool E4 = KV == GBE_KV_E4M3;
    constexpr float kGrowth = E4 ? 2.0f : 8.0f;  // powers of two that the maximum in use may lag
    constexpr int KC = DP / 32, VC = DP / 64;    // pieces of a K row, of a V row
    constexpr int SUB = E4 ? 2 : 1;              // groups of 16 tokens a step: as many bytes for either cache
    constexpr int kStep = 16 * SUB, kStride = kStep * kWarps;
    extern __shared__ float sm[];                // [kWarps][kHeads][DP + 2]
    pdl_begin();
    const KvCacheArgs& c = a.c;
    const Part p = find_part(a, blockIdx.x);
    if (p.t0 >= p.t1 && p.chunk > 0) return;
    const int D = c.D, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h0 = p.kvh * a.group + p.part * kHeads;
    const int heads = min(kHeads, a.group - p.part * kHeads);

    // where token base + lane % kStep lies: its page (-1: none) ...
    const int32_t* pages = a.table + (int64_t)p.b * a.max_pages;
    const int mine = lane & (kStep - 1);
    auto page_of = [&](int base) {
        const int tok = base + mine;
        return tok < p.t1 ? pages[tok / c.page_size] : -1;
    };
    // ... and its row's first element in k and v (-1: none) and scales
    struct Place {
        int64_t at;
        uint32_t scales;
    };
    auto place = [&](int base, int32_t page) {
        Place w = {-1, 0};
        if (page >= 0 && page < c.n_pages) {
            const int row = (base + mine) % c.page_size;
            w.at = page * c.page_stride + ((int64_t)p.kvh * c.page_size + row) * D;
            if constexpr (E4) {
                const int64_t si = ((int64_t)page * c.Hkv + p.kvh) * c.page_size + row;
                w.scales = (uint32_t)c.k_scale[si] | (uint32_t)c.v_scale[si] << 8;
            }
        }
        return w;
    };
    Eight<KV> k[SUB][2][KC], v[SUB][4][VC];
    auto load_k = [&](const Place& w) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t at = __shfl_sync(0xFFFFFFFFu, w.at, 16 * u + g + 8 * i);
#pragma unroll
                for (int x = 0; x < KC; ++x) {
                    const int d = x * 32 + t * 8;
                    k[u][i][x].load(c.k, at + d, at >= 0 && d < D);
                }
            }
    };
    auto load_v = [&](const Place& w) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t at = __shfl_sync(0xFFFFFFFFu, w.at, 16 * u + 2 * t + (i & 1) + 8 * (i >> 1));
#pragma unroll
                for (int x = 0; x < VC; ++x) {
                    const int d = x * 64 + g * 8;
                    v[u][i][x].load(c.v, at + d, at >= 0 && d < D);
                }
            }
    };

    int base = p.t0 + warp * kStep;
    Place now = place(base, page_of(base));
    load_k(now);
    load_v(now);
    int32_t page1 = page_of(base + kStride);

    // q of head g, the inner index of the first product as above
    uint32_t q[KC][4];
    float cs[2] = {a.scale, a.scale};  // what turns sums of heads 2 t, 2 t + 1 into logits of base 2
    {
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + p.b * a.q_stride + (int64_t)(h0 + g) * D;
#pragma unroll
        for (int x = 0; x < KC; ++x) {
            const int d = x * 32 + t * 8;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[x][e] = g < heads && d < D ? (uint32_t)src[d + 2 * e] | (uint32_t)src[d + 2 * e + 1] << 16 : 0u;
        }
        if constexpr (E4) {
            // the head's largest magnitude to 2^15: f16 then holds what is within 2^-29 of it whole
            uint32_t top = 0;
#pragma unroll
            for (int x = 0; x < KC; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, max(q[x][e] & 0x7FFFu, (q[x][e] >> 16) & 0x7FFFu));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            int e2 = (int)(top >> 7) - 127 - 14;  // infinities and NaN: taken as they are
            e2 = (top >> 7) == 255 ? 0 : max(-126, e2);
            const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
#pragma unroll
            for (int x = 0; x < KC; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    q[x][e] = f16x2(__uint_as_float(q[x][e] << 16) * down,
                                    __uint_as_float(q[x][e] & 0xFFFF0000u) * down);
            cs[0] *= __uint_as_float((uint32_t)(127 + __shfl_sync(0xFFFFFFFFu, e2, 8 * t)) << 23);
            cs[1] *= __uint_as_float((uint32_t)(127 + __shfl_sync(0xFFFFFFFFu, e2, 8 * t + 4)) << 23);
        }
    }

    float o[VC * 4][4];
#pragma unroll
    for (int x = 0; x < VC * 4; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int E = -1000;

    for (; base < p.t1; base += kStride) {
        float s[SUB][4];  // tokens g (heads 2 t, 2 t + 1) and g + 8 of each group
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.0f;
#pragma unroll
            for (int x = 0; x < KC; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    if constexpr (E4) {
                        const uint32_t f[4] = {e4m3x2_f16x2<0>(k[u][0][x].w[y]), e4m3x2_f16x2<0>(k[u][1][x].w[y]),
                                               e4m3x2_f16x2<1>(k[u][0][x].w[y]), e4m3x2_f16x2<1>(k[u][1][x].w[y])};
                        mma_f16(s[u], f, q[x][2 * y], q[x][2 * y + 1]);
                    } else {
                        const uint32_t f[4] = {k[u][0][x].w[2 * y], k[u][1][x].w[2 * y], k[u][0][x].w[2 * y + 1],
                                               k[u][1][x].w[2 * y + 1]};
                        mma_bf16(s[u], f, q[x][2 * y], q[x][2 * y + 1]);
                    }
                }
        }
        // the next step's K, and the page after it
        const Place next = place(base + kStride, page1);
        load_k(next);
        page1 = page_of(base + 2 * kStride);

        const uint32_t live = __ballot_sync(0xFFFFFFFFu, now.at >= 0);
        bool wide = false;
        if constexpr (E4) {
            const bool here = now.at >= 0;
            const int e = (int)(now.scales >> 8);
            if (__any_sync(0xFFFFFFFFu, here && e - E > kScaleGrowth)) {
                const int top = __reduce_max_sync(0xFFFFFFFFu, here ? e : 0);
                const int by = min(max(E, 0) - top, 0);
                const float r = by < -126 ? 0.0f : __uint_as_float((uint32_t)(127 + by) << 23);
                if (E >= 0) {
#pragma unroll
                    for (int x = 0; x < VC * 4; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[x][i] *= r;
                }
                E = max(E, top);
            }
            wide = __any_sync(0xFFFFFFFFu, here && e > 0 && E - e > kScaleDrop);
        }
        float vf[SUB][2];  // 2^(byte - E + 12) of v's scales
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool here = live >> (16 * u + g + 8 * i) & 1u;
                float ks = 1.0f;
                if constexpr (E4) {
                    const uint32_t w = __shfl_sync(0xFFFFFFFFu, now.scales, 16 * u + g + 8 * i);
                    ks = __uint_as_float((w & 255u) << 23);
                    const int by = (int)(w >> 8) - E + 12;
                    vf[u][i] = (w >> 8) == 0 || by < -126 ? 0.0f : __uint_as_float((uint32_t)(127 + by) << 23);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float& x = s[u][2 * i + h];
                    x = E4 ? x * cs[h] * ks : x * cs[h];
                    x = here ? x : -INFINITY;
                    // a NaN logit leaves a finite maximum, so that its NaN weight reaches the result
                    top[h] = fmaxf(top[h], x == x ? x : -3.0e38f);
                }
            }
        if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + kGrowth || top[1] > m[1] + kGrowth)) {
            float r[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], x));
                const float m2 = top[h] > m[h] + kGrowth ? top[h] : m[h];
                r[h] = rescale(m[h], m2);
                m[h] = m2;
                l[h] *= r[h];
            }
#pragma unroll
            for (int x = 0; x < VC * 4; ++x) {
                o[x][0] *= r[0];
                o[x][1] *= r[1];
                o[x][2] *= r[0];
                o[x][3] *= r[1];
            }
        }
        const float shift[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = ex2(s[u][i] - shift[i & 1]);
                l[i & 1] += w;
                s[u][i] = E4 ? w * vf[u][i >> 1] : w;
            }
        // o += V^T P^T; rows of the product: entries 64 x + 8 g + 2 y and + 2 y + 1
        auto weigh = [&](auto half) {
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t b0, b1;
                if constexpr (decltype(half)::value) {
                    b0 = transpose8(f16x2(s[u][0], s[u][1])), b1 = transpose8(f16x2(s[u][2], s[u][3]));
                } else {
                    b0 = transpose8(f32x2_to_bf16x2_bits(s[u][0], s[u][1]));
                    b1 = transpose8(f32x2_to_bf16x2_bits(s[u][2], s[u][3]));
                }
#pragma unroll
                for (int x = 0; x < VC; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t f[4];
                        if constexpr (E4) {
                            const uint32_t sel = y & 1 ? 0x7362u : 0x5140u;  // the two tokens' codes of both entries
                            const uint32_t w = __byte_perm(v[u][0][x].w[y >> 1], v[u][1][x].w[y >> 1], sel);
                            const uint32_t z = __byte_perm(v[u][2][x].w[y >> 1], v[u][3][x].w[y >> 1], sel);
                            f[0] = e4m3x2_f16x2<0>(w), f[1] = e4m3x2_f16x2<1>(w);
                            f[2] = e4m3x2_f16x2<0>(z), f[3] = e4m3x2_f16x2<1>(z);
                            if constexpr (decltype(half)::value) {
                                mma_f16(o[x * 4 + y], f, b0, b1);
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i) f[i] = f16x2_bf16x2(f[i]);
                                mma_bf16(o[x * 4 + y], f, b0, b1);
                            }
                        } else {
                            f[0] = __byte_perm(v[u][0][x].w[y], v[u][1][x].w[y], 0x5410);
                            f[1] = __byte_perm(v[u][0][x].w[y], v[u][1][x].w[y], 0x7632);
                            f[2] = __byte_perm(v[u][2][x].w[y], v[u][3][x].w[y], 0x5410);
                            f[3] = __byte_perm(v[u][2][x].w[y], v[u][3][x].w[y], 0x7632);
                            mma_bf16(o[x * 4 + y], f, b0, b1);
                        }
                    }
            }
        };
        if (E4 && !wide)
            weigh(std::bool_constant<E4>{});
        else
            weigh(std::false_type{});
        load_v(next);
        now = next;
    }

    // the warps' sums, joined in order
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], x);
    constexpr int W = DP + 2;
    if constexpr (E4) {
        const float back = __uint_as_float((uint32_t)max(E, 0) << 23);
#pragma unroll
        for (int x = 0; x < VC * 4; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[x][i] = o[x][i] * 0x1p-12f * back;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float* to = sm + (warp * kHeads + 2 * t + h) * W;
#pragma unroll
        for (int x = 0; x < VC * 4; ++x) {
            const int d = (x >> 2) * 64 + g * 8 + (x & 3) * 2;
            *reinterpret_cast<float2*>(to + d) = make_float2(o[x][h], o[x][2 + h]);
        }
        if (g == 0) to[DP] = m[h], to[DP + 1] = l[h];
    }
    __syncthreads();
    const bool whole = p.C >= p.n;
    for (int i = threadIdx.x; i < heads * DP; i += kThreads) {
        const int h = i / DP, d = i - h * DP;
        if (d >= D) continue;
        float mx = -INFINITY;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) mx = fmaxf(mx, sm[(x * kHeads + h) * W + DP]);
        float sum = 0.0f, y = 0.0f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float* z = sm + (x * kHeads + h) * W;
            if (z[DP] == -INFINITY) continue;  // nothing seen; a weight of 0 still carries NaN on
            const float r = ex2(z[DP] - mx);
            sum = fmaf(z[DP + 1], r, sum);
            y = fmaf(z[d], r, y);
        }
        if (whole) {
            Store<kBF16>::store1(a.out, p.b * a.out_stride + (int64_t)(h0 + h) * D + d, mx == -INFINITY ? 0.0f : y / sum);
        } else {
            const int64_t row = ((int64_t)p.b * a.Hq + h0 + h) * a.split + p.chunk;
            a.part_o[row * D + d] = y;
            if (d == 0) a.part_ml[row] = make_float2(mx, sum);
        }
    }
}

template <int KV, int DP>
cudaError_t go(Args a, int64_t B, cudaStream_t st) {
    constexpr int smem = kWarps * kHeads * (DP + 2) * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(decode_mma<KV, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e;
        }
    }
    a.parts = (a.group + kHeads - 1) / kHeads;
    return launch(decode_mma<KV, DP>, dim3((unsigned)(B * a.split * a.c.Hkv * a.parts)), dim3(kThreads), smem, st, a);
}

template <int KV>
cudaError_t pick(const Args& a, int64_t B, cudaStream_t st) {
    if (a.c.D <= 64) return go<KV, 64>(a, B, st);
    if (a.c.D <= 128) return go<KV, 128>(a, B, st);
    return go<KV, 256>(a, B, st);
}

}  // namespace

cudaError_t launch_mma(Args a, int64_t B, cudaStream_t st) {
    return a.c.dtype == GBE_KV_E4M3 ? pick<GBE_KV_E4M3>(a, B, st) : pick<GBE_KV_BF16>(a, B, st);
}

}  // namespace decode
}  // namespace gbe
