// Angles of rotary positions in fixed-point turns (rope.cu says why).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace csa {

// Turns per position of frequency f (radians), modulo 1, in units of 2^-64.
__device__ __forceinline__ uint64_t fixed_turns(double f) {
    double turns = f * 0.15915494309189533577;  // / 2 pi
    turns -= floor(turns);
    return __double2ull_rn(turns * 18446744073709551616.0);
}

__device__ __forceinline__ float2 cos_sin(int64_t p, uint64_t turns, float sign, float m) {
    const uint32_t frac = (uint32_t)(((uint64_t)p * turns) >> 32);  // of a turn, modulo 1
    const uint32_t upper = (frac + 128u) & ~255u;
    float s, c;
    sincospif((float)(int32_t)upper * 0x1p-31f, &s, &c);
    const float rest = (float)(int32_t)(frac - upper) * (0x1p-31f * 3.14159265f);  // radians
    return make_float2(m * fmaf(-rest, s, c), m * sign * fmaf(rest, c, s));
}

}  // namespace csa
