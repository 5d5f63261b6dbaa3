// f32x2.cuh - fp32 arithmetic two elements an instruction, each rounded as the
// scalar instruction rounds it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace amp {

// A pair in one 64-bit register (kept as such from the loads to the stores: as a
// pair of floats each operand would be moved into an aligned pair of registers
// first)
using f2 = uint64_t;
__device__ __forceinline__ f2 make_f2(float a, float b) {
    f2 c;
    asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(a), "f"(b));
    return c;
}
__device__ __forceinline__ float2 split(f2 a) {
    float2 c;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(c.x), "=f"(c.y) : "l"(a));
    return c;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 c;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(a), "l"(b));
    return c;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 c;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(a), "l"(b));
    return c;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 both(float v) { return make_f2(v, v); }
__device__ __forceinline__ float sum2(f2 a) {
    const float2 s = split(a);
    return s.x + s.y;
}

}  // namespace amp
