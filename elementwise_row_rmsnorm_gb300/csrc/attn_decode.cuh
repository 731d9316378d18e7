// attn_decode.cuh -- what the kernels of gbe_attn_decode share.
#pragma once

#include <stdint.h>

#include "attn_common.cuh"
#include "launch.h"

namespace gbe {
namespace decode {

// A partial softmax's weight when its maximum m moves to m2: 0 while nothing
// has been seen (m = -inf).
__device__ __forceinline__ float rescale(float m, float m2) { return m == -INFINITY ? 0.0f : ex2(m - m2); }

// Tokens of a chunk for a sequence of n tokens: n / split of them in units
// of 128, at least `least`.
__device__ __forceinline__ int chunk_tokens(int n, int split, int least) {
    const int c = ((n + split - 1) / split + 127) & ~127;
    return c < least ? least : c;
}

struct Args {
    const void* q;
    void* out;
    int64_t q_stride, out_stride;
    KvCacheArgs c;
    const int32_t* table;
    const int32_t* lens;
    int Hq, group, max_pages;
    int split, least;     // chunks at most, tokens a chunk at least
    int parts;            // query-head parts of a kv head: ceil(group / H)
    int run;              // chunks that one CTA takes one after another
    float scale;          // times log2(e)
    int window, sinks;    // window 0: every token
    float* part_o;        // [B * Hq, split, D]
    float2* part_ml;      // [B * Hq, split]: running maximum (base 2), running sum
};

// What a sequence's token sees of it.  Under a window these are the first `sinks`
// tokens and those from `first` on; between the two there is a gap, and tokens
// are counted without it: from `from` on, token t is number t - gap.  Both ends
// of the gap are multiples of 16, so that tokens 16 i .. 16 i + 15 by number
// follow one another in memory where pages hold a multiple of 16; up to 15
// tokens behind the sinks and as many ahead of the window are counted, and not
// looked at.
struct Seen {
    int n;                  // tokens, counted without the gap
    int from, gap, first;   // (without a window: nothing is from `from` on, first is 0)
    __device__ __forceinline__ int token(int i) const { return i < from ? i : i + gap; }
    __device__ __forceinline__ bool sees(int token, int sinks) const { return token >= first || token < sinks; }
};
__device__ __forceinline__ Seen find_seen(const Args& a, int b) {
    const int64_t capacity = (int64_t)a.max_pages * a.c.page_size;
    const int32_t len = a.lens[b];
    Seen s = {len < 0 ? 0 : (int)(len < capacity ? len : capacity), INT32_MAX, 0, 0};
    if (a.window > 0 && s.n > a.window) {
        s.first = s.n - a.window;
        const int64_t from = ((int64_t)a.sinks + 15) & ~(int64_t)15, to = s.first & ~15;
        if (from < to) s.from = (int)from, s.gap = (int)(to - from), s.n -= s.gap;
    }
    return s;
}

// The CTA's part of the work, from its index: query-head part innermost, then
// kv head, then chunks.
struct Part {
    int b, kvh, chunk, part;  // chunk: the first of a.run
    Seen seen;
    int n, C, t0, t1;         // the sequence's tokens, tokens a chunk, and those of this CTA, without the gap
};
__device__ __forceinline__ Part find_part(const Args& a, uint32_t id) {
    Part p;
    p.part = (int)(id % (uint32_t)a.parts);
    id /= (uint32_t)a.parts;
    p.kvh = (int)(id % (uint32_t)a.c.Hkv);
    id /= (uint32_t)a.c.Hkv;
    const uint32_t runs = (uint32_t)((a.split + a.run - 1) / a.run);
    p.chunk = (int)(id % runs) * a.run;
    p.b = (int)(id / runs);
    p.seen = find_seen(a, p.b);
    p.n = p.seen.n;
    p.C = chunk_tokens(p.n, a.split, a.least);
    // (chunk, run at most 128 and C at most 2^30 / split + 127: no overflow)
    p.t0 = p.chunk * p.C;
    p.t1 = (int)min((int64_t)p.n, p.t0 + (int64_t)a.run * p.C);
    return p;
}

// The tensor-core form: bf16 queries.
cudaError_t launch_mma(Args a, int64_t B, cudaStream_t st);

}  // namespace decode
}  // namespace gbe
