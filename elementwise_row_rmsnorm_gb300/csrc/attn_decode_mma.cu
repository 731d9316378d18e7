// attn_decode_mma.cu -- gbe_attn_decode for bf16 queries, over a bf16 or an
// e4m3 cache, with the products on the tensor cores.
//
// Bound by HBM: each cached row is read once, and four query heads to a kv
// head need only 4 (bf16) or 8 (e4m3) flops a byte, some 50 TFLOP/s.  So the
// small warp-wide products (mma.sync, 16 tokens by 8 heads) do:
//
//   S^T [16 tokens x 8 heads]  = K [16 x D] q^T       A: K, B: q
//   O^T [16 entries x 8 heads] += V^T [16 x 16] P^T   A: V, B: P
//
// A warp works on steps of 16 or 32 tokens of its own.  Asynchronous copies of
// 16 bytes a lane bring a step's rows of K and V (8 KB) into a ring of shared
// memory that is the warp's alone, so nothing waits on another warp and
// nothing but the step at hand is held in registers; three CTAs of four warps
// an SM keep about 96 KB on their way.  ldmatrix takes the rows out again
// (16-byte pieces are placed by the row's number modulo 8, so that eight rows
// meet eight different bank groups), transposing V; P changes from the layout
// of a result to that of B by movmatrix.
//
// The maximum in use lags behind by up to 2^8 (as weights, floats all of them,
// may), so that a step costs one vote instead of a reduction.  At the end of a
// chunk the warps' sums are joined in order; the ring is filling for the next
// chunk meanwhile, and a CTA takes several chunks one after another where there
// are enough of them.
//
// A bf16 cache takes weights as two bf16 each, 16 bits in all: the second product
// with v costs nothing that HBM would not have taken anyway, and the result is
// as good as its one rounding.
//
// Measured on a GB300, 32 heads of 128 over 8 kv heads: 64 sequences of up to
// 8192 tokens in bf16 165 us (6.5 TB/s, 0.97 of a plain copy's rate), 2 of 131072
// 164 us; 64 of 8192 in e4m3 190 us (5.7 TB/s, 0.85), bound by the instructions
// that widen codes and place pieces.
//
// e4m3: codes widen to f16 exactly (one conversion for two), so the products
// are f16; a product may number its inner index and its rows as it likes, so
// the order in which codes come out of ldmatrix is taken as it is.  q is
// brought into f16's range by a power of two for each head; k's scale
// multiplies the logit, v's the weight, as 2^(byte - E) with a common E that
// lags like the maximum does (2^1; the maximum 2^2 here), times 2^12 so that
// the largest come near f16's end.  f16 then holds a weight to 2^-8 of itself,
// as bf16 would, down to 2^-29 of the row's largest, and to 2^-37 of that one
// below; a step with a scale more than 2^8 under E takes bf16 weights and
// values instead.
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

// 16 bytes (SIZE 8: 8) into shared memory, the first `from` of them from memory and zeros behind them.
template <int SIZE>
__device__ __forceinline__ void copy_async(uint32_t to, const void* p, int from) {
    if (SIZE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p), "r"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(p), "r"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

template <int KV, int DP>
struct Shape {
    static constexpr int kEs = KV == GBE_KV_E4M3 ? 1 : 2;
    static constexpr int kRow = DP * kEs;                             // bytes of a row in shared memory
    static constexpr int kSub = kRow <= 128 ? 2 : 1;                  // groups of 16 tokens a step
    static constexpr int kStep = 16 * kSub, kStride = kStep * kWarps;
    static constexpr int kHalf = kStep * kRow, kStage = 2 * kHalf;    // K, then V
    static constexpr int kStages = kStage >= 8192 ? 2 : 4;
    static constexpr int kRing = kStages * kStage * kWarps;
    // where piece `c` (16 bytes) of row r lies
    __device__ static __forceinline__ uint32_t at(int r, int c) {
        if (kRow >= 128) return (uint32_t)(r * kRow + ((c ^ (r & 7)) << 4));
        return (uint32_t)((r >> 1) * 128 + (((((r & 1) << 2) + c) ^ (r >> 1 & 7)) << 4));
    }
};

template <int KV, int DP>
__global__ void __launch_bounds__(kThreads, DP <= 128 ? 3 : 1) decode_mma(Args a) {
    using S = Shape<KV, DP>;
    constexpr bool E4 = KV == GBE_KV_E4M3;
    constexpr float kGrowth = E4 ? 2.0f : 8.0f;  // powers of two that the maximum in use may lag
    constexpr int SUB = S::kSub, NST = S::kStages, es = S::kEs;
    constexpr int kPieces = S::kRow / 16, kTiles = DP / 16;
    extern __shared__ __align__(128) uint8_t raw[];
    float* const sm = reinterpret_cast<float*>(raw + S::kRing);  // [kWarps][heads][DP + 2]
    pdl_begin();
    const KvCacheArgs& c = a.c;
    const Part p = find_part(a, blockIdx.x);
    if (p.t0 >= p.t1 && p.chunk > 0) return;
    const int D = c.D, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h0 = p.kvh * a.group + p.part * kHeads;
    const int heads = min(kHeads, a.group - p.part * kHeads);

    // Lane i looks after token i of the step, first and kStride further at
    // every step: its page (-1: none) ...
    const int32_t* pages = a.table + (int64_t)p.b * a.max_pages;
    const int mine = lane & (S::kStep - 1);
    int tok = p.t0 + warp * S::kStep + mine, page_i = tok / c.page_size, row = tok - page_i * c.page_size;
    const int hop_pages = S::kStride / c.page_size, hop_rows = S::kStride - hop_pages * c.page_size;
    auto page_of = [&] { return tok < p.t1 ? pages[page_i] : -1; };
    int32_t page = page_of();
    // Rows of 16 tokens in a row lie in one page where pages hold a multiple
    // of 16 (chunks begin at multiples of 128): one address does for them.
    const bool runs = c.page_size % 16 == 0;
    const bool grid16 = !E4 || (D % 16 == 0 && c.page_stride % 16 == 0);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(raw) + warp * NST * S::kStage;
    uint32_t live[NST], scales[NST];  // of the steps in the ring, the one at hand first
    // ... and, a step later, its rows on their way into stage `into`, entry `q` of the above
    auto fetch = [&](int into, uint32_t& lives, uint32_t& sc) {
        int64_t at = 0;
        const bool here = page >= 0 && page < c.n_pages;
        sc = 0;
        if (here) {
            at = (page * c.page_stride + ((int64_t)p.kvh * c.page_size + row) * D) * es;
            if constexpr (E4) {
                const int64_t si = ((int64_t)page * c.Hkv + p.kvh) * c.page_size + row;
                sc = (uint32_t)c.k_scale[si] | (uint32_t)c.v_scale[si] << 8;
            }
        }
        lives = __ballot_sync(0xFFFFFFFFu, here);
        tok += S::kStride;
        page_i += hop_pages;
        row += hop_rows;
        if (row >= c.page_size) row -= c.page_size, ++page_i;
        page = page_of();
        if (lives == 0) {  // nothing to copy, and the step will be passed over
            copies_commit();
            return;
        }
        const uint32_t to = ring + into * S::kStage;
        constexpr int kCopies = S::kHalf / 512, kRows = 32 / kPieces;  // copies; rows that one of them covers
        const int r0 = lane / kPieces, piece = lane % kPieces;
        const int left = D * es - piece * 16, size = left < 0 ? 0 : left > 16 ? 16 : left;
        if (runs && grid16 && lives == 0xFFFFFFFFu) {
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                const int64_t x = __shfl_sync(0xFFFFFFFFu, at, 16 * u) + (size > 0 ? r0 * (D * es) + piece * 16 : 0);
                const uint8_t* ks = static_cast<const uint8_t*>(c.k) + x;
                const uint8_t* vs = static_cast<const uint8_t*>(c.v) + x;
#pragma unroll
                for (int i = 0; i < kCopies / SUB; ++i) {
                    const uint32_t at_smem = to + S::at(16 * u + i * kRows + r0, piece);
                    copy_async<16>(at_smem, ks, size);
                    copy_async<16>(at_smem + S::kHalf, vs, size);
                    ks += kRows * D * es, vs += kRows * D * es;
                }
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < kCopies; ++i) {
                const int r = i * kRows + r0;
                int64_t x = __shfl_sync(0xFFFFFFFFu, at, r);
                const int from = lives >> r & 1u ? size : 0;
                x = from > 0 ? x + piece * 16 : 0;
                const uint32_t at_smem = to + S::at(r, piece);
                const uint8_t* const ks = static_cast<const uint8_t*>(c.k) + x;
                const uint8_t* const vs = static_cast<const uint8_t*>(c.v) + x;
                if (grid16) {
                    copy_async<16>(at_smem, ks, from);
                    copy_async<16>(at_smem + S::kHalf, vs, from);
                } else {  // rows on the 8-byte grid
                    copy_async<8>(at_smem, ks, min(from, 8));
                    copy_async<8>(at_smem + 8, from > 8 ? ks + 8 : ks, max(from - 8, 0));
                    copy_async<8>(at_smem + S::kHalf, vs, min(from, 8));
                    copy_async<8>(at_smem + S::kHalf + 8, from > 8 ? vs + 8 : vs, max(from - 8, 0));
                }
            }
        }
        copies_commit();
    };
    const int steps = (p.t1 - p.t0 + S::kStride - 1) / S::kStride, chunk_steps = p.C / S::kStride;
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) fetch(i, live[i], scales[i]);

    // q of head g in the order of K's entries: of 16 at 16 x, two and two
    uint32_t q[kTiles][2];
    float cs[2] = {a.scale, a.scale};  // what turns sums of heads 2 t, 2 t + 1 into logits of base 2
    {
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + p.b * a.q_stride + (int64_t)(h0 + g) * D;
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = x * 16 + (E4 ? 4 * t + 2 * e : 8 * e + 2 * t);
                q[x][e] = g < heads && d < D ? (uint32_t)src[d] | (uint32_t)src[d + 1] << 16 : 0u;
            }
        if constexpr (E4) {
            // the head's largest magnitude to 2^15: f16 then holds what is within 2^-29 of it whole
            uint32_t top = 0;
#pragma unroll
            for (int x = 0; x < kTiles; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) top = max(top, max(q[x][e] & 0x7FFFu, (q[x][e] >> 16) & 0x7FFFu));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            int e2 = (int)(top >> 7) - 127 - 14;  // infinities and NaN: taken as they are
            e2 = (top >> 7) == 255 ? 0 : max(-126, e2);
            const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
#pragma unroll
            for (int x = 0; x < kTiles; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    q[x][e] = f16x2(__uint_as_float(q[x][e] << 16) * down,
                                    __uint_as_float(q[x][e] & 0xFFFF0000u) * down);
            cs[0] *= __uint_as_float((uint32_t)(127 + __shfl_sync(0xFFFFFFFFu, e2, 8 * t)) << 23);
            cs[1] *= __uint_as_float((uint32_t)(127 + __shfl_sync(0xFFFFFFFFu, e2, 8 * t + 4)) << 23);
        }
    }

    float o[kTiles][4], m[2], l[2];
    int E;
    auto restart = [&] {
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[x][e] = 0.0f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
        E = -1000;
    };
    restart();

    // The chunk's end: the warps' sums joined in order.
    auto finish = [&](int chunk) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 4; x <= 16; x <<= 1) l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], x);
        // nothing but NaN: a finite maximum, so that it reaches the result
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (m[h] == -INFINITY && l[h] != l[h]) m[h] = -3.0e38f;
        constexpr int W = DP + 2;
        if constexpr (E4) {
            const float back = __uint_as_float((uint32_t)max(E, 0) << 23);
#pragma unroll
            for (int x = 0; x < kTiles; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[x][i] = o[x][i] * 0x1p-12f * back;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (2 * t + h >= heads) continue;
            float* to = sm + (warp * heads + 2 * t + h) * W;
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
                const int d0 = E4 ? x * 16 + 2 * g : x * 16 + g, d1 = E4 ? d0 + 1 : d0 + 8;
                to[d0] = o[x][h];
                to[d1] = o[x][2 + h];
            }
            if (g == 0) to[DP] = m[h], to[DP + 1] = l[h];
        }
        __syncthreads();
        const bool alone = p.C >= p.n;
        for (int i = threadIdx.x; i < heads * DP; i += kThreads) {
            const int h = i / DP, d = i - h * DP;
            if (d >= D) continue;
            float mx = -INFINITY;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) mx = fmaxf(mx, sm[(x * heads + h) * W + DP]);
            float sum = 0.0f, y = 0.0f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float* z = sm + (x * heads + h) * W;
                if (z[DP] == -INFINITY) continue;  // nothing seen; a weight of 0 still carries NaN on
                const float r = ex2(z[DP] - mx);
                sum = fmaf(z[DP + 1], r, sum);
                y = fmaf(z[d], r, y);
            }
            if (alone) {
                Store<kBF16>::store1(a.out, p.b * a.out_stride + (int64_t)(h0 + h) * D + d,
                                     mx == -INFINITY ? 0.0f : y / sum);
            } else {
                const int64_t at = ((int64_t)p.b * a.Hq + h0 + h) * a.split + chunk;
                a.part_o[at * D + d] = y;
                if (d == 0) a.part_ml[at] = make_float2(mx, sum);
            }
        }
        __syncthreads();
    };
    if (steps == 0) finish(p.chunk);  // a sequence of no tokens

    int stage = 0, left_in_chunk = chunk_steps, chunk = p.chunk;
    for (int step = 0; step < steps; ++step) {
        __syncwarp();  // every lane is done with the stage that is filled next
        fetch(stage == 0 ? NST - 1 : stage - 1, live[NST - 1], scales[NST - 1]);
        copies_wait<NST - 1>();
        __syncwarp();
        if (live[0] != 0) {
            const uint32_t kb = ring + stage * S::kStage, vb = kb + S::kHalf;
            if constexpr (E4) {
                // a row whose scale byte is 0 stands for zeros, whatever its codes
                const uint32_t byte0 = (scales[0] & 0xFFu ? 0u : 1u) | (scales[0] >> 8 ? 0u : 2u);
                const bool here = lane < S::kStep && (live[0] >> lane & 1u);
                if (__any_sync(0xFFFFFFFFu, here && byte0)) {
                    if (here) {
                        uint8_t* const at = raw + (warp * NST + stage) * S::kStage;
                        for (int c0 = 0; c0 < kPieces; ++c0) {
                            uint4* const k = reinterpret_cast<uint4*>(at + S::at(lane, c0));
                            if (byte0 & 1u) *k = make_uint4(0u, 0u, 0u, 0u);
                            if (byte0 & 2u) *(k + S::kHalf / 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    __syncwarp();
                }
            }

            float s[SUB][4];  // tokens g (heads 2 t, 2 t + 1) and g + 8 of each group
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.0f;
                const int r = 16 * u + (lane & 15), c0 = lane >> 4;
#pragma unroll
                for (int x = 0; x < kPieces / 2; ++x) {
                    uint32_t f[4];
                    ldmatrix4(f, kb + S::at(r, 2 * x + c0));
                    if constexpr (E4) {
                        const uint32_t lo[4] = {e4m3x2_f16x2<0>(f[0]), e4m3x2_f16x2<0>(f[1]), e4m3x2_f16x2<1>(f[0]),
                                                e4m3x2_f16x2<1>(f[1])};
                        const uint32_t hi[4] = {e4m3x2_f16x2<0>(f[2]), e4m3x2_f16x2<0>(f[3]), e4m3x2_f16x2<1>(f[2]),
                                                e4m3x2_f16x2<1>(f[3])};
                        mma_f16(s[u], lo, q[2 * x][0], q[2 * x][1]);
                        mma_f16(s[u], hi, q[2 * x + 1][0], q[2 * x + 1][1]);
                    } else {
                        mma_bf16(s[u], f, q[x][0], q[x][1]);
                    }
                }
            }

            bool wide = false;
            if constexpr (E4) {
                const bool here = live[0] >> lane & 1u;
                const int e = (int)(scales[0] >> 8);
                if (__any_sync(0xFFFFFFFFu, here && e - E > kScaleGrowth)) {
                    const int top = __reduce_max_sync(0xFFFFFFFFu, here ? e : 0);
                    const int by = min(max(E, 0) - top, 0);
                    const float r = by < -126 ? 0.0f : __uint_as_float((uint32_t)(127 + by) << 23);
                    if (E >= 0) {
#pragma unroll
                        for (int x = 0; x < kTiles; ++x)
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
                    const bool here = live[0] >> (16 * u + g + 8 * i) & 1u;
                    float ks = 1.0f;
                    if constexpr (E4) {
                        const uint32_t w = __shfl_sync(0xFFFFFFFFu, scales[0], 16 * u + g + 8 * i);
                        ks = __uint_as_float((w & 255u) << 23);
                        const int by = (int)(w >> 8) - E + 12;
                        vf[u][i] = (w >> 8) == 0 || by < -126 ? 0.0f : __uint_as_float((uint32_t)(127 + by) << 23);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float& x = s[u][2 * i + h];
                        x = E4 ? x * cs[h] * ks : x * cs[h];
                        x = here ? x : -INFINITY;
                        top[h] = fmaxf(top[h], x);
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
                for (int x = 0; x < kTiles; ++x) {
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
            // o += V^T P^T
            auto weigh = [&](auto half) {
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    uint32_t b0, b1;
                    if constexpr (decltype(half)::value) {
                        b0 = transpose8(f16x2(s[u][0], s[u][1])), b1 = transpose8(f16x2(s[u][2], s[u][3]));
                    } else if constexpr (!E4) {  // cut off, not rounded
                        b0 = transpose8(__byte_perm(__float_as_uint(s[u][0]), __float_as_uint(s[u][1]), 0x7632));
                        b1 = transpose8(__byte_perm(__float_as_uint(s[u][2]), __float_as_uint(s[u][3]), 0x7632));
                    } else {
                        b0 = transpose8(f32x2_to_bf16x2_bits(s[u][0], s[u][1]));
                        b1 = transpose8(f32x2_to_bf16x2_bits(s[u][2], s[u][3]));
                    }
                    if constexpr (E4) {
                        const int r = 16 * u + (lane & 15), c0 = lane >> 4;
#pragma unroll
                        for (int x = 0; x < kPieces / 2; ++x) {
                            uint32_t w[4];
                            ldmatrix4_trans(w, vb + S::at(r, 2 * x + c0));
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                // two tokens' codes of both entries, side by side
                                const uint32_t w0 = __byte_perm(w[2 * y], 0, 0x3120);
                                const uint32_t w1 = __byte_perm(w[2 * y + 1], 0, 0x3120);
                                uint32_t f[4] = {e4m3x2_f16x2<0>(w0), e4m3x2_f16x2<1>(w0), e4m3x2_f16x2<0>(w1),
                                                 e4m3x2_f16x2<1>(w1)};
                                if constexpr (decltype(half)::value) {
                                    mma_f16(o[2 * x + y], f, b0, b1);
                                } else {
#pragma unroll
                                    for (int i = 0; i < 4; ++i) f[i] = f16x2_bf16x2(f[i]);
                                    mma_bf16(o[2 * x + y], f, b0, b1);
                                }
                            }
                        }
                    } else {
                        // the rest of each weight, cut off above, as a second bf16; never zero beside a weight that
                        // is not, so that an infinity of v is not met by a zero
                        float rest[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            rest[i] = fmaxf(s[u][i] - __uint_as_float(__float_as_uint(s[u][i]) & 0xFFFF0000u),
                                            s[u][i] * 0x1p-30f);
                        const uint32_t r0 = transpose8(f32x2_to_bf16x2_bits(rest[0], rest[1]));
                        const uint32_t r1 = transpose8(f32x2_to_bf16x2_bits(rest[2], rest[3]));
                        const int r = 16 * u + (lane & 7) + (lane >> 4) * 8, c0 = lane >> 3 & 1;
#pragma unroll
                        for (int x = 0; x < kTiles; ++x) {
                            uint32_t f[4];
                            ldmatrix4_trans(f, vb + S::at(r, 2 * x + c0));
                            mma_bf16(o[x], f, r0, r1);
                            mma_bf16(o[x], f, b0, b1);
                        }
                    }
                }
            };
            if (E4 && !wide)
                weigh(std::bool_constant<E4>{});
            else
                weigh(std::false_type{});
        }
#pragma unroll
        for (int i = 0; i + 1 < NST; ++i) live[i] = live[i + 1], scales[i] = scales[i + 1];
        if (++stage == NST) stage = 0;
        if (--left_in_chunk == 0 || step + 1 == steps) {
            finish(chunk++);
            restart();
            left_in_chunk = chunk_steps;
        }
    }
    copies_wait<0>();
}

template <int KV, int DP>
cudaError_t go(Args a, int64_t B, cudaStream_t st) {
    using S = Shape<KV, DP>;
    const int heads = a.group < kHeads ? a.group : kHeads;
    const int smem = S::kRing + kWarps * heads * (DP + 2) * 4;
    constexpr int most = S::kRing + kWarps * kHeads * (DP + 2) * 4;
    static FunctionLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(decode_mma<KV, DP>), most);
    if (e != cudaSuccess) return e;
    a.parts = (a.group + kHeads - 1) / kHeads;
    // Several chunks to a CTA while that leaves eight waves of CTAs, of e4m3 four
    // (64 x 0..8192 tokens: bf16 165 us, 170 with four; e4m3, 64 x 0..4000, 64 us
    // with eight, 62 with four).
    constexpr int kWaves = KV == GBE_KV_E4M3 ? 4 : 8;
    const int64_t rows = B * a.c.Hkv * a.parts, want = rows * a.split / (kWaves * 3 * (int64_t)sm_count());
    a.run = (int)(want < 1 ? 1 : want > a.split ? a.split : want);
    const int64_t runs = (a.split + a.run - 1) / a.run;
    return launch(decode_mma<KV, DP>, dim3((unsigned)(rows * runs)), dim3(kThreads), smem, st, a);
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
