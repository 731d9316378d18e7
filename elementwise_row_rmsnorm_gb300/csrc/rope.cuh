// rope.cuh -- the rotation's arithmetic, shared by every kernel that turns a
// head, so that their bits agree.
#pragma once

#include "common.cuh"

namespace gbe {

__device__ __forceinline__ void rotate(float a, float b, float c, float s, float mu, float& a2, float& b2) {
    a2 = __fmul_rn(mu, __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)));
    b2 = __fmul_rn(mu, __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c)));
}

// rotate() for two pairs at once, (a.x, b.x) by (c.x, s.x) and (a.y, b.y)
// by (c.y, s.y): the products and the scale two lanes at a time (packed
// f32x2 multiplies, each lane rounded as the scalar product), the sums
// scalar -- a packed multiply feeding a packed add may be fused into one
// rounding -- so the bits are rotate()'s.
__device__ __forceinline__ void rotate2(float2 a, float2 b, float2 c, float2 s, float mu, float2& a2, float2& b2) {
    const float2 ac = mul2_rn(a, c), bs = mul2_rn(b, s), as = mul2_rn(a, s), bc = mul2_rn(b, c);
    const float2 m = make_float2(mu, mu);
    a2 = mul2_rn(m, make_float2(__fsub_rn(ac.x, bs.x), __fsub_rn(ac.y, bs.y)));
    b2 = mul2_rn(m, make_float2(__fadd_rn(as.x, bc.x), __fadd_rn(as.y, bc.y)));
}

// cos / sin of the angle of pair i at position p: from the table when one is
// given and p lies inside it (it holds exactly these values), else formed.
template <bool CACHE>
__device__ __forceinline__ void angle(int32_t p, int i, const float* inv_freq, const float2* cache,
                                      int64_t cache_len, int half, float& c, float& s) {
    if (CACHE && p >= 0 && p < cache_len) {
        const float2 v = __ldg(cache + (int64_t)p * half + i);
        c = v.x;
        s = v.y;
    } else {
        rope_sincos(__fmul_rn((float)p, __ldg(inv_freq + i)), &s, &c);
    }
}

}  // namespace gbe
