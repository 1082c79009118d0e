// The 8-bit floating point form of rows: e4m3 codes (1 sign, 4 exponent, 3
// mantissa bits, bias 7, no infinity, 0x7F NaN) and for each 128 of a row a
// scale 2^(b - 127) held as its biased exponent b (0xFF: NaN).
#pragma once

#include "tl_internal.h"

namespace tl {
namespace f8 {

typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));

constexpr uint32_t kInf = 0x7F800000u;

// biased exponent of the smallest power of two S with a <= 448 S; a by its bits, finite
__device__ __forceinline__ uint32_t scale_of(uint32_t a) {
    const int s = int(a >> 23) - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return uint32_t(s > 0 ? s : 0);
}

__device__ __forceinline__ float scale_value(uint32_t b) {
    return __builtin_bit_cast(float, b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
}

// the values of 8 codes, exact in fp32
__device__ __forceinline__ void values8(uint2 c, float s, float (&v)[8]) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], true);
        v[4 * h] = lo[0] * s;
        v[4 * h + 1] = lo[1] * s;
        v[4 * h + 2] = hi[0] * s;
        v[4 * h + 3] = hi[1] * s;
    }
}

// 8 codes times the scale of biased exponent b, as bfloat16: exact, a code having 4
// significant bits (within bfloat16's range).  The conversion reads only the
// exponent bits of its scale.
__device__ __forceinline__ bf8v widen(uint32_t lo, uint32_t hi, uint32_t b) {
    const float s = __builtin_bit_cast(float, b << 23);
    const bf2v p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
    const bf2v p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
    const bf2v p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
    const bf2v p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
    return bf8v{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// LDS byte address of a pointer into the workgroup's shared memory
__device__ __forceinline__ uint32_t lds_address(void* p) {
    return uint32_t(uintptr_t((__attribute__((address_space(3))) uint8_t*)(static_cast<uint8_t*>(p))));
}

}  // namespace f8
}  // namespace tl
