// attn_prompt.cu -- causal attention over packed prompts with grouped heads:
// f32 storage, and what attn_prompt_tc.cu does not take.
//
//   out[i, h] = sum_j p_ij v_j,  p_i = softmax_j(scale * q[i, h] . k_j),
//   j <= i within i's sequence, k and v of kv head h / (Hq / Hkv)
//
// On the CUDA cores, in f32 throughout.  (Three tf32 products in place of one,
// on the tensor cores, came out 6 times as far from the definition as f32 sums
// and were not kept.)  One CTA takes 32 query rows of one head (64 where there
// are many) and walks the keys in tiles of 64 with the running maximum and sum
// of the softmax (base 2: scale * log2(e) is folded into q).  Eight by sixteen
// threads: a thread holds a 4 x 4 (8 x 4) piece of the logits and a 4 x D/16
// (8 x D/16) piece of the output in registers, two multiply-adds an
// instruction; q, k, v and the weights lie in shared memory as f32.  f32 rows on the 16-byte grid come by asynchronous copies, v while the
// logits are formed and the next k while the output is.  Bound by the rate of
// f32 multiply-adds (78 TFLOP/s) where there are tiles enough; 3 sequences of up
// to 1000 tokens, whose longest rows' CTAs are what is waited for, take 71 us.
#include <type_traits>

#include "attn_tiles.cuh"
#include "gbe_elementwise.h"
#include "launch.h"

namespace gbe {
namespace {

constexpr int kThreads = 128;  // of a group
constexpr int kN = 64;
// ROWS rows into shared memory as f32, times `scale`; zeros behind `rows` and D.
template <int DT, int DP, bool VEC, int ROWS>
__device__ __forceinline__ void stage(float* dst, const void* src, int64_t at, int64_t stride, int rows, int D,
                                      float scale) {
    constexpr int W = DP + 4;
    for (int i = threadIdx.x & (kThreads - 1); i < ROWS * (DP / 8); i += kThreads) {
        const int r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
        float f[8] = {};
        if (r < rows && d < D) {
            const int64_t x = at + r * stride + d;
            if constexpr (VEC) {
                constexpr int V = Store<DT>::V;
#pragma unroll
                for (int p = 0; p < 8 / V; ++p) {
                    float g[V];
                    const char* const from = static_cast<const char*>(src);
                    Store<DT>::unpack(ld_reuse(from + (x + p * V) * (int64_t)sizeof(typename Store<DT>::T)), g);
#pragma unroll
                    for (int e = 0; e < V; ++e) f[p * V + e] = g[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = Store<DT>::load1(src, x + e);
            }
        }
        float4* o = reinterpret_cast<float4*>(dst + r * W + d);
        o[0] = make_float4(f[0] * scale, f[1] * scale, f[2] * scale, f[3] * scale);
        o[1] = make_float4(f[4] * scale, f[5] * scale, f[6] * scale, f[7] * scale);
    }
}

// kN rows of f32 on their way into shared memory; zeros behind `rows` and D.
template <int DP>
__device__ __forceinline__ void stage_async(float* dst, const float* src, int64_t at, int64_t stride, int rows,
                                            int D) {
    constexpr int W = DP + 4;
#pragma unroll 4
    for (int i = threadIdx.x & (kThreads - 1); i < kN * (DP / 4); i += kThreads) {
        const int r = i / (DP / 4), d = (i - r * (DP / 4)) * 4;
        const bool there = r < rows && d < D;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(dst + r * W + d)),
                     "l"(src + (there ? at + r * stride + d : 0)), "r"(there ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Up to D = 128 two groups of threads take every other tile of keys each and
// join their sums at the end, which halves the walk of the longest rows.
template <int DP>
constexpr int kGroups = DP <= 128 ? 2 : 1;
template <int DP, int R>
constexpr int kGroupFloats = 2 * kN * (DP + 4) + 8 * R * (kN + 4);  // k, v and weights

// R: query rows of a thread, 8 R of a CTA.  A row's bits do not depend on it.
template <int DT, int DP, bool VEC, int R>
__global__ void __launch_bounds__(kThreads* kGroups<DP>, DP == 64 ? 2 : 1) prompt_rows(PromptArgs a) {
    constexpr int M = 8 * R, W = DP + 4, WP = kN + 4, Q4 = DP / 64;
    constexpr bool ASYNC = DT == kF32 && VEC;
    extern __shared__ float sm[];
    float* qs = sm;
    const int group = threadIdx.x / kThreads;
    float* const ps = qs + M * W + group * kGroupFloats<DP, R>;
    float* const ks = ps + M * WP;
    float* const vs = ks + kN * W;
    auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kThreads) : "memory"); };
    __shared__ SeqPiece where;
    pdl_begin();
    const int head = (int)(blockIdx.x % (unsigned)a.Hq);
    const unsigned index = blockIdx.x / (unsigned)a.Hq;
    if (threadIdx.x < 32) {
        const SeqPiece t = find_piece(a.starts, (int)a.n_seqs, (int)a.T, index,
                                      [](int n) { return (uint32_t)((n + M - 1) / M); },
                                      [](uint32_t rows, uint32_t seqs) { return rows / M + seqs; });
        if (threadIdx.x == 0) where = t;
    }
    __syncthreads();
    if (where.index < 0) return;
    const struct {
        int begin, len, row;
    } w = {where.begin, where.len, where.index * M};
    const int kvh = head / (int)(a.Hq / a.Hkv), D = (int)a.D;
    const int ty = threadIdx.x % kThreads >> 4, tx = threadIdx.x & 15;
    const int rows = min(M, w.len - w.row);
    if (group == 0)
        stage<DT, DP, VEC, M>(qs, a.q, (int64_t)(w.begin + w.row) * a.q_stride + (int64_t)head * D, a.q_stride, rows,
                               D, a.scale * kLog2e);
    float2 o[R][2 * Q4];
    float m[R], l[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < 2 * Q4; ++e) o[i][e] = make_float2(0.0f, 0.0f);
    }
    const int64_t k_at = (int64_t)w.begin * a.k_stride + (int64_t)kvh * D;
    const int64_t v_at = (int64_t)w.begin * a.v_stride + (int64_t)kvh * D;
    auto fetch_k = [&](int k0) {
        if constexpr (ASYNC)
            stage_async<DP>(ks, static_cast<const float*>(a.k), k_at + (int64_t)k0 * a.k_stride, a.k_stride,
                            min(kN, w.len - k0), D);
        else
            stage<DT, DP, VEC, kN>(ks, a.k, k_at + (int64_t)k0 * a.k_stride, a.k_stride, min(kN, w.len - k0), D,
                                   1.0f);
    };
    auto fetch_v = [&](int k0) {
        if constexpr (ASYNC)
            stage_async<DP>(vs, static_cast<const float*>(a.v), v_at + (int64_t)k0 * a.v_stride, a.v_stride,
                            min(kN, w.len - k0), D);
        else
            stage<DT, DP, VEC, kN>(vs, a.v, v_at + (int64_t)k0 * a.v_stride, a.v_stride, min(kN, w.len - k0), D,
                                   1.0f);
    };
    const int end = w.row + rows;
    constexpr int kHop = kGroups<DP> * kN;
    if (group * kN < end) fetch_k(group * kN);
    __syncthreads();  // q is there
    for (int k0 = group * kN; k0 < end; k0 += kHop) {
        const bool last = k0 + kN > w.row;  // the tile that holds the diagonal
        sync();  // v of the tile before is done with
        fetch_v(k0);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        sync();  // k is there
        float2 s2[R][4] = {};  // sums over even and odd entries: two multiply-adds an instruction
#pragma unroll 4
        for (int d = 0; d < DP; d += 4) {
            float4 x[R], y[4];
#pragma unroll
            for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float4*>(qs + (ty * R + i) * W + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * W + d);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s2[i][j] = fma2_rn(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), s2[i][j]);
                    s2[i][j] = fma2_rn(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), s2[i][j]);
                }
        }
        float s[R][4];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j].x + s2[i][j].y;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        sync();  // k is done with, and v is there
        if (k0 + kHop < end) fetch_k(k0 + kHop);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = w.row + ty * R + i;
            // a NaN logit leaves a finite maximum, so that its NaN weight reaches the result
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k0 + tx + 16 * j <= row) mx = fmaxf(mx, s[i][j] == s[i][j] ? s[i][j] : -3.0e38f);
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
            const float r = m[i] == -INFINITY ? 0.0f : ex2(m[i] - mx);
            m[i] = mx;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool seen = k0 + tx + 16 * j <= row;
                const float p = seen ? (s[i][j] == -INFINITY ? 0.0f : ex2(s[i][j] - mx)) : 0.0f;
                sum += p;
                ps[(ty * R + i) * WP + tx + 16 * j] = seen ? p : -1.0f;  // -1: no weight, and v is not looked at
            }
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
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
                            if (decltype(masked)::value && w1 < 0.0f) continue;
                            const float2 w2 = make_float2(w1, w1);
                            o[i][2 * c] = fma2_rn(w2, make_float2(v.x, v.y), o[i][2 * c]);
                            o[i][2 * c + 1] = fma2_rn(w2, make_float2(v.z, v.w), o[i][2 * c + 1]);
                        }
                    }
            }
        };
        if (last)
            weigh(std::true_type{});
        else
            weigh(std::false_type{});
    }
    if constexpr (kGroups<DP> == 2) {
        // the second group's sums by way of its own k
        float* const other = qs + M * W + kGroupFloats<DP, R> + M * WP;
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
        if (group == 1) return;
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
        if (ty * R + i >= rows) continue;
        const int64_t at = (int64_t)(w.begin + w.row + ty * R + i) * a.out_stride + (int64_t)head * D;
        const float inv = m[i] == -INFINITY ? 0.0f : 1.0f / l[i];
#pragma unroll
        for (int c = 0; c < Q4; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = tx * 4 + 64 * c + e;
                const float y = e & 1 ? o[i][2 * c + e / 2].y : o[i][2 * c + e / 2].x;
                if (d < D) Store<DT>::store1(a.out, at + d, m[i] == -INFINITY ? 0.0f : y * inv);
            }
    }
}

template <int DT, int DP, bool VEC, int R>
cudaError_t go(const PromptArgs& a, cudaStream_t st) {
    constexpr int smem = (8 * R * (DP + 4) + kGroups<DP> * kGroupFloats<DP, R>) * 4;
    static FunctionLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(prompt_rows<DT, DP, VEC, R>), smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = a.T / (8 * R) + (a.n_seqs < a.T ? a.n_seqs : a.T);
    const dim3 grid((unsigned)(tiles * a.Hq)), threads(kThreads * kGroups<DP>);
    return launch(prompt_rows<DT, DP, VEC, R>, grid, threads, smem, st, a);
}

// Eight rows a thread read a third less of shared memory for each multiply-add
// than four, but make half as many CTAs, each twice as long: for D in 65 .. 128
// and from four CTAs an SM on (1500 tokens, 32 heads of 128: 458 us, 537 us with
// four rows; with 4 heads 163 and 101 us).  Up to D = 64 four rows let two CTAs
// share an SM and are as fast (4096 tokens, 8 heads: 476 and 464 us); above 128
// eight would not fit registers.
template <int DT, bool VEC>
cudaError_t go128(const PromptArgs& a, cudaStream_t st) {
    return a.T / 64 * a.Hq >= 4 * (int64_t)sm_count() ? go<DT, 128, VEC, 8>(a, st) : go<DT, 128, VEC, 4>(a, st);
}

template <int DT, bool VEC>
cudaError_t pick(const PromptArgs& a, cudaStream_t st) {
    if constexpr (DT == kF32 || !VEC) {  // (bf16 on the grid up to D = 128 has a kernel of its own)
        if (a.D <= 64) return go<DT, 64, VEC, 4>(a, st);
        if (a.D <= 128) return go128<DT, VEC>(a, st);
    }
    return go<DT, 256, VEC, 4>(a, st);
}

}  // namespace

cudaError_t launch_attn_prompt(const PromptArgs& a, int dtype, bool vec, cudaStream_t st) {
    if (dtype == GBE_BF16 && vec && a.D <= 128) return launch_attn_prompt_tc(a, st);
    if (dtype == GBE_F32) return vec ? pick<kF32, true>(a, st) : pick<kF32, false>(a, st);
    return vec ? pick<kBF16, true>(a, st) : pick<kBF16, false>(a, st);
}

}  // namespace gbe
