// Element types of the norm and the 4-bit calls: 8 consecutive elements to
// and from fp32, and the signed rotation of a 1024-block held by one wave.
#pragma once

#include "tl_internal.h"

namespace tl {
namespace elem {

struct F32 {
    static constexpr int kType = TL_F32, kBytes = 4;
};
struct F16 {
    static constexpr int kType = TL_F16, kBytes = 2;
};
struct BF16 {
    static constexpr int kType = TL_BF16, kBytes = 2;
};

__device__ __forceinline__ uint32_t f16_bits(float f) {
    return uint32_t(__builtin_bit_cast(uint16_t, _Float16(f)));
}

// fp32 -> bfloat16, nearest even; a NaN stays one (one instruction: in bit
// arithmetic a third of the norm's instructions were these roundings)
__device__ __forceinline__ uint32_t bf16_bits(float f) {
    return uint32_t(__builtin_bit_cast(uint16_t, __bf16(f)));
}

// the same of two, the first in the low half
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

template <typename T>
__device__ __forceinline__ float round_to(float f) {
    if (T::kType == TL_F16) return float(_Float16(f));
    if (T::kType == TL_BF16) return __builtin_bit_cast(float, bf16_bits(f) << 16);
    return f;
}

template <typename T>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
    if (T::kType == TL_F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (T::kType == TL_F16) {
                v[2 * j] = float(__builtin_bit_cast(_Float16, uint16_t(w[j])));
                v[2 * j + 1] = float(__builtin_bit_cast(_Float16, uint16_t(w[j] >> 16)));
            } else {
                v[2 * j] = __builtin_bit_cast(float, w[j] << 16);
                v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
            }
        }
    }
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// KEEP: the value is read again soon, by the same kernel.  What a kernel only
// writes is stored past the caches' replacement order, so that it does not push
// out what is still to be read
template <bool KEEP, typename V>
__device__ __forceinline__ void put(V* p, V v) {
    if (KEEP) *p = v;
    else __builtin_nontemporal_store(v, p);
}

template <typename T, bool KEEP = false>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
    uint32_t w[8];
    if (T::kType == TL_F32) {
        u32x4* q = reinterpret_cast<u32x4*>(static_cast<float*>(p) + i);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __builtin_bit_cast(uint32_t, v[j]);
        put<KEEP>(q, u32x4{w[0], w[1], w[2], w[3]});
        put<KEEP>(q + 1, u32x4{w[4], w[5], w[6], w[7]});
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = T::kType == TL_F16 ? f16_bits(v[2 * j]) | f16_bits(v[2 * j + 1]) << 16
                                      : bf16_pair(v[2 * j], v[2 * j + 1]);
        put<KEEP>(reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i), u32x4{w[0], w[1], w[2], w[3]});
    }
}

// v of lane l ^ m: DPP quad permutes for m = 1, 2, a lane permute through LDS's
// crossbar for m = 4, a rotation of a row of 16 for m = 8, swaps of rows and
// halves for m = 16, 32.  (Two DPP mirrors for m = 4 are slower in the rotation,
// which has no vector instructions to spare: 2048 x 5120 rows 21.1 us, 19.7 with
// the permute.)
__device__ __forceinline__ float lane_xor(float v, int m, int l) {
    const int b = __builtin_bit_cast(int, v);
    if (m == 1) return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(b, 0xB1, 0xF, 0xF, false));
    if (m == 2) return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(b, 0x4E, 0xF, 0xF, false));
    if (m == 4) return __shfl_xor(v, m, 64);
    if (m == 8) return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(b, 0x128, 0xF, 0xF, false));
    if (m == 16) {
        const auto sw = __builtin_amdgcn_permlane16_swap(uint32_t(b), uint32_t(b), false, false);
        return __builtin_bit_cast(float, (l & 16) ? sw[0] : sw[1]);
    }
    const auto sw = __builtin_amdgcn_permlane32_swap(uint32_t(b), uint32_t(b), false, false);
    return __builtin_bit_cast(float, l < 32 ? sw[1] : sw[0]);
}

// lane_xor's step m of a reduction, whose quads hold one value once m = 4 is
// reached: a mirrored half row does there
__device__ __forceinline__ float reduce_xor(float v, int m, int l) {
    if (m != 4) return lane_xor(v, m, l);
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x141, 0xF, 0xF, false));
}

// The unscaled transform H (s * v) of a 1024-block whose index bits lie in 4
// register and 6 lane bits, in any order (the matrix only asks which bits two
// indices share): the register bits are butterflied in registers, the lane
// bits with cross-lane exchanges; fp32 in a fixed order, 10 levels of sums.
// sg: the elements' sign bytes in register order.  The caller multiplies by
// 1/32 (exact).
__device__ __forceinline__ void rotate16(float (&v)[16], const uint4 sg, int l) {
    const uint32_t sw[4] = {sg.x, sg.y, sg.z, sg.w};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t neg = (sw[j >> 2] << (24 - 8 * (j & 3))) & 0x80000000u;
        v[j] = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, v[j]) ^ neg);
    }
#pragma unroll
    for (int h = 1; h < 16; h <<= 1)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (!(j & h)) {
                const float a = v[j], b = v[j + h];
                v[j] = a + b;
                v[j + h] = a - b;
            }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const float sgn = (l & m) ? -1.0f : 1.0f;
        float p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) p[j] = lane_xor(v[j], m, l);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __builtin_fmaf(v[j], sgn, p[j]);
    }
}

}  // namespace elem
}  // namespace tl
