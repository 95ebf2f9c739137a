// Rows of 512 dims held in 384 bytes: the format and its arithmetic.
//
//   bytes   0-223  dims 0-447, 4 bits each: sign, two exponent bits, one bit
//                  of mantissa (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6)
//   bytes 224-251  an e4m3 scale for each group of 16 dims
//   byte  252      a power of two for the whole row, exponent + 127 (27 to 227)
//   bytes 253-255  zero
//   bytes 256-383  dims 448-511, the rotary ones, in bf16
//
// Eight dims make a 32-bit word: its low half holds dims 0, 2, 4, 6 from the
// lowest bits up, its high half dims 1, 3, 5, 7, so that one shift brings two
// neighbours to the same place of both halves, where bf16 has its bits.
//
// A held value is code x scale x 2^e: two, four and one significant bits, so
// it is exact in bf16 (and the products below are). The row's power of two puts
// its largest scale between 128 and 256 of e4m3's 448; groups down to 2^-17 of
// the largest keep a scale of their own. A code of 0 to 3 and a sign alone are
// a bf16 number 2^126 below the code's value, subnormal ones (0.5) included,
// and one multiplication brings it up.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace csa {
namespace q4 {

constexpr int kRow = 384;       // bytes
constexpr int kDims = 448;      // in 4 bits
constexpr int kGroup = 16;
constexpr int kScales = 224;    // first byte of the scales
constexpr int kExp = 252;
constexpr int kTail = 256;      // first byte of dims 448-511
constexpr int kMinExp = -100, kMaxExp = 100;

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Scale of a group as both halves of a bf16 pair; `unit` is the row's power of two.
__device__ __forceinline__ __nv_bfloat162 scale_pair(float scale, float unit) {
    return __float2bfloat162_rn(scale * unit);
}

// Two e4m3 scales (of neighbouring groups) as floats.
__device__ __forceinline__ float2 scales2(uint16_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Eight codes as four pairs of neighbouring dims, 2^126 below their values. A
// code's sign goes to bit 15 and the rest to bits 8-6 of its half: one product
// with two powers of two makes both shifts (a multiplication, of which the SM
// does as many as logical operations beside them; two shifts in its place made
// the pairs take a quarter longer).
__device__ __forceinline__ uint4 eight_small(uint32_t w) {
    const uint32_t v = w >> 8, place = 0x81c081c0u;
    return make_uint4(((w & 0x000f000fu) * 0x1040u) & place, ((w & 0x00f000f0u) * 0x104u) & place,
                      ((v & 0x000f000fu) * 0x1040u) & place, ((v & 0x00f000f0u) * 0x104u) & place);
}

__device__ __forceinline__ uint4 times(const uint4 &x, __nv_bfloat162 f) {
    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&in[i]), f);
        out[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// Eight codes times their group's scale.
__device__ __forceinline__ uint4 eight(uint32_t w, __nv_bfloat162 scale) {
    const uint32_t up = 0x7e807e80u;  // 2^126 twice
    return times(times(eight_small(w), *reinterpret_cast<const __nv_bfloat162 *>(&up)), scale);
}

// Dims 8 i .. 8 i + 7 of a row (i of 64), as they are held and as bf16 pairs.
struct Eight {
    uint4 v = {0, 0, 0, 0};
    uint32_t scale = 0, exp = 0;
    __device__ __forceinline__ void load(const uint8_t *row, int i) {  // nullptr: zeros
        if (!row) return;
        if (i < kDims / 8) {
            v.x = __ldg(reinterpret_cast<const uint32_t *>(row) + i);
            scale = __ldg(row + kScales + i / 2);
            exp = __ldg(row + kExp);
        } else {
            v = __ldg(reinterpret_cast<const uint4 *>(row + kTail) + (i - kDims / 8));
        }
    }
    __device__ __forceinline__ uint4 values(int i) const {
        return i < kDims / 8 ? eight(v.x, scale_pair(scales2((uint16_t)scale).x, pow2((int)exp - 127))) : v;
    }
};

}  // namespace q4
}  // namespace csa
