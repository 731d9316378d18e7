// attn_common.cuh -- what the attention kernels share beyond common.cuh.
#pragma once

#include <atomic>

#include "common.cuh"

namespace gbe {

constexpr float kLog2e = 1.4426950408889634f;

// 2^x; 0 below 2^-126.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two multiply-adds in one instruction, each rounded once.
__device__ __forceinline__ float2 fma2_rn(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Dynamic shared memory past 48 KB is granted to a kernel once a device; one of
// these for each kernel remembers on which devices that has been done.
class FunctionLimit {
  public:
    cudaError_t raise(const void* kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) {
            const unsigned long long bit = 1ull << (dev & 63);
            if (dev < 64 && (done_.load(std::memory_order_acquire) & bit)) return cudaSuccess;
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e == cudaSuccess && dev < 64) done_.fetch_or(bit, std::memory_order_release);
        }
        if (e != cudaSuccess) cudaGetLastError();  // clear it; the caller reports e
        return e;
    }

  private:
    std::atomic<unsigned long long> done_{0};
};

}  // namespace gbe
