// attn_prompt_tc.cu -- causal attention over packed prompts on the tensor
// cores: bf16, D up to 128, rows on the 16-byte grid.
//
//   S = q k^T (f32, in tensor memory), p = 2^(c S - c m), c = |scale| log2(e),
//   O = sum p v, out = O / sum p
//
// A CTA works on two tiles of 128 query rows that share one kv head -- two
// heads of its group at the same rows, or neighbouring row tiles -- and walks
// the keys in blocks of 128 that a ring of shared-memory stages holds.  Three
// warpgroups: one of softmax for each tile (a thread owns a row), and one of
// which a warp issues the tensor copies and another the products.
//
// Tensor memory (512 columns): one S for both tiles, O of each, and the
// weights of each, rounded to bf16, which are the A operand of the second
// product.  A block of 128 keys costs a tile 512 clocks of either product and
// its warpgroup some 1400 clocks of softmax, so the products of a tile must not
// wait for its softmax: they are issued in the order
//
//   S0 = q0 k(j+1)^T, O0 += p0 v(j), S1 = q1 k(j+1)^T, O1 += p1 v(j)
//
// S is handed over as soon as a warpgroup has it in registers, and each
// softmax then has 1500 clocks until its weights are asked for.  (With an S
// for each tile, overwritten by its weights, the next S had to wait for the
// product with v, and a round of both tiles took 3300 clocks, not 2048.)
//
// O is rescaled only when a row's maximum has grown by more than 2^8 over the
// one in use; until then weights go up to 2^8, which costs nothing in bf16 or
// f32 (both floats) and keeps sums far from overflow.
//
// Masked weights are exact zeros, but zero times an infinity or a NaN in a
// later row of v would reach the sum; a row that ends up not finite is
// therefore computed again by exact_row, which looks at its own keys alone.
#include "attn_tiles.cuh"
#include "common.cuh"
#include "gbe_elementwise.h"
#include "launch.h"
#include "tensor_core.cuh"

namespace gbe {
namespace {

constexpr int kM = 128, kN = 128;
constexpr int kThreads = 384;  // three warpgroups: softmax of each tile, and the issuing warps
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrowth = 8.0f;  // a maximum may lag this many powers of two

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int DP>
struct Shape {
    static constexpr int kPanel = 128 * 128;              // 128 rows of 64 bf16
    static constexpr int kTile = kPanel * (DP / 64);      // 128 rows of DP
    static constexpr int kStages = DP == 128 ? 5 : 9;
    static constexpr int kBytes = kTile * (2 + kStages) + 1024 + 512;
};

struct Control {
    uint64_t q_full, kv_full[9], kv_empty[9], s_full[2], s_free[2], p_ready[2], o_done[2], drained;
    uint32_t tmem;
    int abort;
    int begin, len, unit0, units;  // the sequence and its first tile here; how many tiles
};

// Pair `index` of the tiles that share a kv head, counted from the last
// sequence's last pair: a sequence of r row tiles has r * group tiles, tile u
// being head u % group of the group at rows (u / group) * kM.
struct Pair {
    int begin, len, unit, units;  // units 0: no such pair
};
__device__ __forceinline__ Pair find_pair(const int32_t* starts, int n_seqs, int T, int group, uint32_t index) {
    const int lane = threadIdx.x & 31;
    uint32_t before = 0;
    for (int top = n_seqs; top > 0; top -= 32) {
        const int b = top - 1 - lane;
        int s = 0, n = 0;
        if (b >= 0) {
            s = min(max(starts[b], 0), T);
            n = max(min(max(starts[b + 1], 0), T) - s, 0);
        }
        const uint32_t units = (uint32_t)((n + kM - 1) / kM) * (uint32_t)group;
        uint32_t sum = (units + 1) / 2;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, sum, x);
            if (lane >= x) sum += y;
        }
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, index < before + sum);
        if (hit) {
            const int who = __ffs((int)hit) - 1;
            const uint32_t upto = __shfl_sync(0xFFFFFFFFu, before + sum, who);
            const uint32_t own = __shfl_sync(0xFFFFFFFFu, units, who);
            Pair p;
            p.begin = __shfl_sync(0xFFFFFFFFu, s, who);
            p.len = __shfl_sync(0xFFFFFFFFu, n, who);
            p.unit = (int)(upto - 1 - index) * 2;
            p.units = min(2, (int)own - p.unit);
            return p;
        }
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    return {0, 0, 0, 0};
}

// One row in f32 from its own keys alone, by a whole warp: 32 keys at a time,
// a lane a key for the logits, a lane four entries for the output.
__device__ __noinline__ void exact_row(const PromptArgs& a, int begin, int row, int head) {
    const int lane = threadIdx.x & 31, D = (int)a.D, kvh = head / (int)(a.Hq / a.Hkv);
    const float c = a.scale * kLog2e;
    float q[4], o[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        q[e] = lane * 4 + e < D
                   ? Store<kBF16>::load1(a.q, (begin + (int64_t)row) * a.q_stride + (int64_t)head * D + lane * 4 + e)
                   : 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int k0 = 0; k0 <= row; k0 += 32) {
        const int j = k0 + lane;
        const bool seen = j <= row;
        float s = 0.0f;
        for (int d = 0; d < D; d += 4) {
            uint2 w = make_uint2(0, 0);
            if (seen)
                w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.k) + (begin + (int64_t)j) * a.k_stride +
                                                    (int64_t)kvh * D + d);
            s = fmaf(__shfl_sync(0xFFFFFFFFu, q[0], d >> 2), __uint_as_float(w.x << 16), s);
            s = fmaf(__shfl_sync(0xFFFFFFFFu, q[1], d >> 2), __uint_as_float(w.x & 0xFFFF0000u), s);
            s = fmaf(__shfl_sync(0xFFFFFFFFu, q[2], d >> 2), __uint_as_float(w.y << 16), s);
            s = fmaf(__shfl_sync(0xFFFFFFFFu, q[3], d >> 2), __uint_as_float(w.y & 0xFFFF0000u), s);
        }
        s *= c;
        // a NaN logit leaves a finite maximum, so that its NaN weight reaches the result
        float mx = seen ? fmaxf(m, s == s ? s : -3.0e38f) : m;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
        const float r = m == -INFINITY ? 0.0f : ex2(m - mx);
        const float p = !seen || s == -INFINITY ? 0.0f : ex2(s - mx);
        m = mx;
        float sum = p;
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        l = fmaf(l, r, sum);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= r;
        const int keys = min(32, row + 1 - k0);
        for (int t = 0; t < keys; ++t) {
            const float w = __shfl_sync(0xFFFFFFFFu, p, t);
            if (lane * 4 < D) {
                const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.v) +
                                                                (begin + (int64_t)k0 + t) * a.v_stride + (int64_t)kvh * D +
                                                                lane * 4);
                o[0] = fmaf(w, __uint_as_float(v.x << 16), o[0]);
                o[1] = fmaf(w, __uint_as_float(v.x & 0xFFFF0000u), o[1]);
                o[2] = fmaf(w, __uint_as_float(v.y << 16), o[2]);
                o[3] = fmaf(w, __uint_as_float(v.y & 0xFFFF0000u), o[3]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (lane * 4 + e < D)
            Store<kBF16>::store1(a.out, (begin + (int64_t)row) * a.out_stride + (int64_t)head * D + lane * 4 + e,
                                 m == -INFINITY ? 0.0f : o[e] / l);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
              const __grid_constant__ CUtensorMap mv, PromptArgs a) {
    using S = Shape<DP>;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    Control& ctl = *reinterpret_cast<Control*>(raw + (base - smem_addr(raw)) + S::kTile * (2 + S::kStages));
    const uint32_t q_smem = base, kv_smem = base + 2 * S::kTile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = (int)(a.Hq / a.Hkv);
    const int kvh = (int)(blockIdx.x % (unsigned)a.Hkv);
    volatile int* const abort = &ctl.abort;

    if (warp == kMmaWarp) tmem_alloc(smem_addr(&ctl.tmem), 512);
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&ctl.q_full), 1);
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(smem_addr(&ctl.kv_full[i]), 1);
            mbar_init(smem_addr(&ctl.kv_empty[i]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_addr(&ctl.s_full[t]), 1);
            mbar_init(smem_addr(&ctl.p_ready[t]), 4);
            mbar_init(smem_addr(&ctl.s_free[t]), 4);
            mbar_init(smem_addr(&ctl.o_done[t]), 1);
        }
        mbar_init(smem_addr(&ctl.drained), 1);
        ctl.abort = 0;
        mbar_init_fence();
        tma_prefetch(&mq);
        tma_prefetch(&mk);
        tma_prefetch(&mv);
    }
    pdl_begin();
    if (warp == 0) {
        const Pair p = find_pair(a.starts, (int)a.n_seqs, (int)a.T, group, blockIdx.x / (unsigned)a.Hkv);
        if (lane == 0) ctl.begin = p.begin, ctl.len = p.len, ctl.unit0 = p.unit, ctl.units = p.units;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    const int begin = ctl.begin, len = ctl.len, units = ctl.units;
    // tile t: head and first row, and the blocks of keys up to its diagonal
    int head[2], row0[2], blocks[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int u = ctl.unit0 + t;
        head[t] = kvh * group + u % group;
        row0[t] = u / group * kM;
        blocks[t] = t < units ? u / group + 1 : 0;
    }
    const int most = max(blocks[0], blocks[1]);

    // Registers: 384 threads were launched with 168 each (64512); the softmax
    // warpgroups take 208, the issuing one keeps 80 (63488 in all).
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == kLoadWarp) {
            if (units > 0 && elect_one()) {
                const uint32_t qb = smem_addr(&ctl.q_full);
                mbar_arrive_tx(qb, S::kTile * units);
                for (int t = 0; t < units; ++t)
#pragma unroll
                    for (int p = 0; p < DP / 64; ++p)
                        tma_load_3d(q_smem + t * S::kTile + p * S::kPanel, &mq, qb, p * 64, head[t], begin + row0[t]);
                int stage = 0, phase = 0, issued = 0;
                for (int i = 0; i < 2 * most; ++i) {  // k and v of each block in turn
                    if (!mbar_wait(smem_addr(&ctl.kv_empty[stage]), phase ^ 1, abort)) break;
                    const uint32_t full = smem_addr(&ctl.kv_full[stage]);
                    mbar_arrive_tx(full, S::kTile);
#pragma unroll
                    for (int p = 0; p < DP / 64; ++p)
                        tma_load_3d(kv_smem + stage * S::kTile + p * S::kPanel, (i & 1) ? &mv : &mk, full, p * 64, kvh,
                                    begin + (i >> 1) * kN);
                    ++issued;
                    if (++stage == S::kStages) stage = 0, phase ^= 1;
                }
                if (*abort) {  // nothing may still be on its way when the CTA ends
                    int none = 0;
                    mbar_wait(qb, 0, &none);
                    for (int i = max(0, issued - S::kStages); i < issued; ++i)
                        mbar_wait(smem_addr(&ctl.kv_full[i % S::kStages]), (i / S::kStages) & 1, &none);
                }
            }
        } else if (warp == kMmaWarp) {
            if (units > 0 && elect_one()) {
                const uint32_t idesc_s = bf16_idesc(kM, kN, false) | (a.scale < 0.0f ? 1u << 13 : 0u);
                constexpr uint32_t idesc_o = bf16_idesc(kM, DP, true);
                bool ok = mbar_wait(smem_addr(&ctl.q_full), 0, abort);
                // load i (k of block i / 2, or v) lies in stage i % kStages
                auto stage = [](int i) { return i % S::kStages; };
                auto loaded = [&](int i) {
                    return mbar_wait(smem_addr(&ctl.kv_full[stage(i)]), i / S::kStages & 1, abort);
                };
                auto release = [&](int i) { mma_commit(smem_addr(&ctl.kv_empty[stage(i)])); };
                int last_t = -1, last_j = 0;  // the tile and block that S was last written for
                auto scores = [&](int t, int j) {
                    if (last_t >= 0) ok = ok && mbar_wait(smem_addr(&ctl.s_free[last_t]), last_j & 1, abort);
                    if (!ok) return;
                    last_t = t, last_j = j;
                    tc_fence_after();
                    const uint32_t q0 = q_smem + t * S::kTile, k0 = kv_smem + stage(2 * j) * S::kTile;
#pragma unroll
                    for (int x = 0; x < DP / 16; ++x) {
                        const uint32_t off = (x / 4) * S::kPanel + (x % 4) * 32;
                        mma_ss(tmem, smem_desc(q0 + off, 16, 1024), smem_desc(k0 + off, 16, 1024), idesc_s, x > 0);
                    }
                    mma_commit(smem_addr(&ctl.s_full[t]));
                };
                auto weigh = [&](int t, int j) {
                    const uint32_t v0 = kv_smem + stage(2 * j + 1) * S::kTile;
                    ok = ok && mbar_wait(smem_addr(&ctl.p_ready[t]), j & 1, abort);
                    if (!ok) return;
                    tc_fence_after();
#pragma unroll
                    for (int x = 0; x < kN / 16; ++x)
                        mma_ts(tmem + 256 + t * 128, tmem + 128 + t * 64 + x * 8, smem_desc(v0 + x * 2048, S::kPanel, 1024),
                               idesc_o, j > 0 || x > 0);
                    mma_commit(smem_addr(&ctl.o_done[t]));
                };
                ok = ok && loaded(0);
                for (int t = 0; t < 2; ++t)
                    if (ok && blocks[t] > 0) scores(t, 0);
                if (ok) release(0);
                for (int j = 0; ok && j < most; ++j) {
                    if (j + 1 < most) ok = loaded(2 * j + 2);
                    for (int t = 0; t < 2; ++t) {
                        if (ok && j + 1 < blocks[t]) scores(t, j + 1);
                        if (t == 0) ok = ok && loaded(2 * j + 1);
                        if (t == 1 && ok && j + 1 < most) release(2 * j + 2);
                        if (ok && j < blocks[t]) weigh(t, j);
                    }
                    if (ok) release(2 * j + 1);
                }
                // every product is done before tensor memory is given back
                mma_commit(smem_addr(&ctl.drained));
                int none = 0;
                mbar_wait(smem_addr(&ctl.drained), 0, &none);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
        const uint32_t ts = tmem + lanes, tp = tmem + 128 + t * 64 + lanes, to = tmem + 256 + t * 128 + lanes;
        const int n = blocks[t], row = row0[t] + (threadIdx.x & 127);
        const float c = fabsf(a.scale) * kLog2e;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&ctl.s_full[t]), j & 1, abort));
            if (!ok) break;
            tc_fence_after();
            uint32_t s[128];
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_ld32(ts + x * 32, s + x * 32);
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_wait_ld32(s + x * 32);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl.s_free[t]));
            if (j == n - 1) {  // the diagonal
                const int seen = row - j * kN;
#pragma unroll
                for (int x = 0; x < 128; ++x) s[x] = x <= seen ? s[x] : 0xFF800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < 128; x += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[x + e]), __uint_as_float(s[x + 4 + e])));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const bool grow = m == -INFINITY ? top > m : (top - m) * c > kGrowth;
            auto last_done = [&] {  // the product with the last weights is done
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(smem_addr(&ctl.o_done[t]), (j - 1) & 1, abort));
                tc_fence_after();
            };
            if (__any_sync(0xFFFFFFFFu, grow)) {
                const float m2 = grow ? top : m;
                if (j > 0) {
                    last_done();
                    if (!ok) break;
                    const float r = m == -INFINITY ? 0.0f : ex2((m - m2) * c);
                    l *= r;
#pragma unroll
                    for (int x = 0; x < DP / 32; ++x) {
                        uint32_t o[32];
                        tmem_ld32(to + x * 32, o);
                        tmem_wait_ld32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * r);
                        tmem_st32(to + x * 32, o);
                    }
                }
                m = m2;
            }
            const float shift = m == -INFINITY ? 0.0f : -m * c;
            const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
            float2 sum[4] = {};
            uint32_t w[64];
#pragma unroll
            for (int e = 0; e < 64; ++e) {
                float2 x = fma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2, shift2);
                x.x = ex2(x.x), x.y = ex2(x.y);
                sum[e & 3] = add2_rn(sum[e & 3], x);
                w[e] = f32x2_to_bf16x2_bits(x.x, x.y);
            }
            const float2 add = add2_rn(add2_rn(sum[0], sum[1]), add2_rn(sum[2], sum[3]));
            l += add.x + add.y;
            if (j > 0) {
                last_done();
                if (!ok) break;
            }
            tmem_st32(tp, w);
            tmem_st32(tp + 32, w + 32);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl.p_ready[t]));
        }
        if (n > 0) {
            ok = ok && mbar_wait(smem_addr(&ctl.o_done[t]), (n - 1) & 1, abort);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
            const bool live = row < len;
            const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
            uint16_t* const out = static_cast<uint16_t*>(a.out) + (begin + (int64_t)row) * a.out_stride +
                                  (int64_t)head[t] * a.D;
            uint32_t bad = 0;
#pragma unroll
            for (int x = 0; x < DP / 32; ++x) {
                uint32_t o[32];
                if (ok) {
                    tmem_ld32(to + x * 32, o);
                    tmem_wait_ld32(o);
                }
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // a wait that gave up leaves NaN
                        f[i] = ok ? __uint_as_float(o[e + i]) * inv : __uint_as_float(0x7FC00000u);
                        if (!(fabsf(f[i]) <= 3.402823466e38f)) bad = 1;
                    }
                    if (live && x * 32 + e < a.D)
                        *reinterpret_cast<Vec16*>(out + x * 32 + e) = Store<kBF16>::pack(f);
                }
            }
            // rows that are not finite again, from their own keys alone
            uint32_t again = __ballot_sync(0xFFFFFFFFu, ok && live && bad);
            __syncwarp();
            while (again) {
                const int i = __ffs((int)again) - 1;
                again &= again - 1;
                exact_row(a, begin, row0[t] + (warp & 3) * 32 + i, head[t]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, 512);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeFn>(p);
        cudaGetLastError();
        return static_cast<EncodeFn>(nullptr);
    }();
    return fn;
}

// [T, H, D] bf16 with a token stride, copied in boxes of 128 tokens of one
// head and 64 entries (128 bytes, swizzled); zeros outside.
bool encode(CUtensorMap* m, const void* p, int64_t T, int64_t H, int64_t D, int64_t stride) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, 128}, step[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP>
cudaError_t go(const PromptArgs& a, cudaStream_t st) {
    CUtensorMap mq, mk, mv;
    if (!encode(&mq, a.q, a.T, a.Hq, a.D, a.q_stride) || !encode(&mk, a.k, a.T, a.Hkv, a.D, a.k_stride) ||
        !encode(&mv, a.v, a.T, a.Hkv, a.D, a.v_stride))
        return cudaErrorNotSupported;
    constexpr int smem = Shape<DP>::kBytes;
    static FunctionLimit limit;
    const cudaError_t e = limit.raise(reinterpret_cast<const void*>(prompt_tc<DP>), smem);
    if (e != cudaSuccess) return e;
    const int64_t group = a.Hq / a.Hkv, seqs = a.n_seqs < a.T ? a.n_seqs : a.T;
    const int64_t pairs = ((a.T / kM + seqs) * group + (group & 1 ? seqs : 0)) / 2;
    return launch(prompt_tc<DP>, dim3((unsigned)(pairs * a.Hkv)), dim3(kThreads), smem, st, mq, mk, mv, a);
}

}  // namespace

cudaError_t launch_attn_prompt_tc(const PromptArgs& a, cudaStream_t st) {
    return a.D <= 64 ? go<64>(a, st) : go<128>(a, st);
}

}  // namespace gbe
