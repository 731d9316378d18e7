// kv_cache.cuh -- device helpers shared by the kernels that read the paged cache.
#pragma once

#include <stdint.h>

#include "common.cuh"

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

}  // namespace gbe
