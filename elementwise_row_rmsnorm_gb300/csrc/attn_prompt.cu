// attn_prompt.cu -- causal attention over packed prompts with grouped heads,
// on the CUDA cores: f32 storage, and any alignment.
//
//   out[i, h] = sum_j p_ij v_j,  p_i = softmax_j(scale * q[i, h] . k_j),
//   j <= i within i's sequence, k and v of kv head h / (Hq / Hkv)
//
// One CTA takes 64 query rows of one head and walks the keys in tiles of 64
// with the running maximum and sum of the softmax (base 2: scale * log2(e)
// is folded into q).  Sixteen by sixteen threads: a thread holds a 4 x 4
// piece of the logits and a 4 x D/16 piece of the output in registers; q, k,
// v and the weights are staged in shared memory as f32.
#include <type_traits>

#include "attn_tiles.cuh"
#include "common.cuh"
#include "gbe_elementwise.h"
#include "launch.h"

namespace gbe {
namespace {

constexpr int kThreads = 256;
constexpr int kM = 64, kN = 64;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 64 rows into shared memory as f32, times `scale`; zeros behind `rows` and D.
template <int DT, int DP, bool VEC>
__device__ __forceinline__ void stage(float* dst, const void* src, int64_t at, int64_t stride, int rows, int D,
                                      float scale) {
    constexpr int W = DP + 4;
    for (int i = threadIdx.x; i < kN * (DP / 8); i += kThreads) {
        const int r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
        float f[8] = {};
        if (r < rows && d < D) {
            const int64_t x = at + r * stride + d;
            if constexpr (VEC) {
                constexpr int V = Store<DT>::V;
#pragma unroll
                for (int p = 0; p < 8 / V; ++p) {
                    float g[V];
                    Store<DT>::unpack(
                        ld_reuse(static_cast<const char*>(src) + (x + p * V) * (int64_t)sizeof(typename Store<DT>::T)),
                        g);
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

template <int DT, int DP, bool VEC>
__global__ void __launch_bounds__(kThreads) prompt_rows(PromptArgs a) {
    constexpr int W = DP + 4, WP = kN + 4, Q4 = DP / 64;
    extern __shared__ float sm[];
    float* qs = sm;
    float* ks = qs + kM * W;
    float* vs = ks + kN * W;
    float* ps = vs + kN * W;
    __shared__ SeqTile where;
    pdl_begin();
    const int head = (int)(blockIdx.x % (unsigned)a.Hq);
    const unsigned index = blockIdx.x / (unsigned)a.Hq;
    if (threadIdx.x < 32) {
        const SeqTile t = find_tile(a.starts, (int)a.n_seqs, (int)a.T, kM, index);
        if (threadIdx.x == 0) where = t;
    }
    __syncthreads();
    const SeqTile w = where;
    if (w.row < 0) return;
    const int kvh = head / (int)(a.Hq / a.Hkv), D = (int)a.D;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    const int rows = min(kM, w.len - w.row);
    stage<DT, DP, VEC>(qs, a.q, (int64_t)(w.begin + w.row) * a.q_stride + (int64_t)head * D, a.q_stride, rows, D,
                       a.scale * kLog2e);
    float o[4][4 * Q4], m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4 * Q4; ++e) o[i][e] = 0.0f;
    }
    for (int k0 = 0; k0 < w.row + rows; k0 += kN) {
        const int keys = min(kN, w.len - k0);
        const bool last = k0 + kN > w.row;  // the tile that holds the diagonal
        __syncthreads();
        stage<DT, DP, VEC>(ks, a.k, (int64_t)(w.begin + k0) * a.k_stride + (int64_t)kvh * D, a.k_stride, keys, D,
                           1.0f);
        stage<DT, DP, VEC>(vs, a.v, (int64_t)(w.begin + k0) * a.v_stride + (int64_t)kvh * D, a.v_stride, keys, D,
                           1.0f);
        __syncthreads();
        float s[4][4] = {};
#pragma unroll 4
        for (int d = 0; d < DP; d += 4) {
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(qs + (ty * 4 + i) * W + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * W + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
                    s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                    s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
                    s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = w.row + ty * 4 + i;
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
                ps[(ty * 4 + i) * WP + tx + 16 * j] = seen ? p : -1.0f;  // -1: no weight, and v is not looked at
            }
#pragma unroll
            for (int x = 8; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
            l[i] = fmaf(l[i], r, sum);
#pragma unroll
            for (int e = 0; e < 4 * Q4; ++e) o[i][e] *= r;
        }
        __syncwarp();  // a row's weights come from its own half warp
        auto weigh = [&](auto masked) {
#pragma unroll 2
            for (int j = 0; j < kN; j += 4) {
                float4 p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(ps + (ty * 4 + i) * WP + j);
#pragma unroll
                for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                    for (int c = 0; c < Q4; ++c) {
                        const float4 v = *reinterpret_cast<const float4*>(vs + (j + jj) * W + tx * 4 + 64 * c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float w1 = jj == 0 ? p[i].x : jj == 1 ? p[i].y : jj == 2 ? p[i].z : p[i].w;
                            if (decltype(masked)::value && w1 < 0.0f) continue;
                            o[i][4 * c + 0] = fmaf(w1, v.x, o[i][4 * c + 0]);
                            o[i][4 * c + 1] = fmaf(w1, v.y, o[i][4 * c + 1]);
                            o[i][4 * c + 2] = fmaf(w1, v.z, o[i][4 * c + 2]);
                            o[i][4 * c + 3] = fmaf(w1, v.w, o[i][4 * c + 3]);
                        }
                    }
            }
        };
        if (last)
            weigh(std::true_type{});
        else
            weigh(std::false_type{});
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (ty * 4 + i >= rows) continue;
        const int64_t at = (int64_t)(w.begin + w.row + ty * 4 + i) * a.out_stride + (int64_t)head * D;
        const float inv = m[i] == -INFINITY ? 0.0f : 1.0f / l[i];
#pragma unroll
        for (int c = 0; c < Q4; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = tx * 4 + 64 * c + e;
                if (d < D) Store<DT>::store1(a.out, at + d, m[i] == -INFINITY ? 0.0f : o[i][4 * c + e] * inv);
            }
    }
}

template <int DT, int DP, bool VEC>
cudaError_t go(const PromptArgs& a, cudaStream_t st) {
    constexpr int smem = ((kM + 2 * kN) * (DP + 4) + kM * (kN + 4)) * 4;
    static FunctionLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(prompt_rows<DT, DP, VEC>), smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = a.T / kM + (a.n_seqs < a.T ? a.n_seqs : a.T);
    return launch(prompt_rows<DT, DP, VEC>, dim3((unsigned)(tiles * a.Hq)), dim3(kThreads), smem, st, a);
}

template <int DT, bool VEC>
cudaError_t pick(const PromptArgs& a, cudaStream_t st) {
    if (a.D <= 64) return go<DT, 64, VEC>(a, st);
    if (a.D <= 128) return go<DT, 128, VEC>(a, st);
    return go<DT, 256, VEC>(a, st);
}

}  // namespace

cudaError_t launch_attn_prompt(const PromptArgs& a, int dtype, bool vec, cudaStream_t st) {
    constexpr int64_t kFar = 1LL << 38;  // strides that a tensor copy can describe
    if (dtype == GBE_BF16 && vec && a.D <= 128 && a.q_stride < kFar && a.k_stride < kFar && a.v_stride < kFar)
        return launch_attn_prompt_tc(a, st);
    if (dtype == GBE_F32) return vec ? pick<kF32, true>(a, st) : pick<kF32, false>(a, st);
    return vec ? pick<kBF16, true>(a, st) : pick<kBF16, false>(a, st);
}

}  // namespace gbe
