// patience.h -- when a wait of a CTA gives up.
#pragma once

#include <stdint.h>

namespace gbe {

#ifdef __CUDACC__
#define GBE_BOTH __host__ __device__ __forceinline__
#else
#define GBE_BOTH inline
#endif

// Times are in ticks of 2^20 ns, 32 bits that wrap around: with 64 the chunk kernel
// over an 8-bit cache took 554 us where it takes 531.
constexpr uint32_t kPatience = 10000000000ull >> 20;  // ten seconds

// For waits until a warp is done with a list of up to `blocks` blocks of keys: as
// long again as that may take, at many times what a block takes (0.4 to 3 us); 178 s
// for 2^30 keys.
inline uint32_t patience_for(int64_t blocks) { return kPatience + (uint32_t)((blocks * 20000) >> 20); }

// What a CTA's waits look at, a word in shared memory: 0; less while as many warps
// are at work that has an end but may take long (a row computed again, key by key);
// kGaveUp and about once a wait has given up.
constexpr int kGaveUp = 1 << 20;

// A wait's time counts while nobody is at such work.  (Counted from its start
// alone, a row computed again over half a million keys ended the other warps'.)
struct Patience {
    uint32_t since = 0;  // 0: not begun
    GBE_BOTH bool over(uint32_t now, int state, uint32_t limit) {
        if (since == 0 || state < 0) since = now;
        return now - since > limit;
    }
};

#undef GBE_BOTH

}  // namespace gbe
