// 4-bit weights with group scales: rounding of weight rows (after the signed
// rotation on demand, folded into the weights as for the ternary codes: page
// "OpenBonsai", section "How it works", steps 1 and 2) and their values.
//
//   a = max |w| of a group, S = binary16(a / 7), c = rint(w / S) in -8 .. 7,
//   w ~ c S
//
// Rounding a / 7 to binary16 from its 53-bit quotient cannot differ from
// rounding it once: a has 24 bits and a binary16 midpoint 12, so a quotient
// that is not a midpoint differs from one by more than 2^-28 of it.  Neither
// can c from a correctly rounded fp32 quotient: with S of 11 bits and k + 1/2
// of at most 4, w is a multiple of 2^-24 of itself away from S (k + 1/2), and
// that is more than half the quotient's last place for each k.
//
// Bound by memory: a lane reads 8 weights (32 or 16 bytes) and writes 4 bytes, a
// group's maximum is exchanged among 4 to 16 neighbouring lanes, nothing goes
// through LDS.  17408 x 5120 fp32 weights to 4 bits and back to binary16, 627
// MB, take 110 us in both launches together, 5.7 TB/s.  With the rotation a lane
// holds 16 neighbouring weights, so its loads lie 64 bytes from the next lane's:
// the way there takes 125 us instead of 71-82 (402 MB, 3.2 TB/s).
#include "elem.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;

constexpr int kThreads = 256;

// |v| as bits: NaN above infinity above numbers
__device__ __forceinline__ uint32_t abs_bits(float f) {
    return __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu;
}

__device__ __forceinline__ uint32_t group_max(uint32_t a, int lanes) {
    for (int m = 1; m < lanes; m <<= 1) {
        const uint32_t o = uint32_t(__shfl_xor(int(a), m, 64));
        a = o > a ? o : a;
    }
    return a;
}

// binary16 scale of a group whose largest |w| has these bits; NaN if it holds
// something that is not finite
__device__ __forceinline__ uint32_t q4_scale(uint32_t top) {
    if (top >= 0x7F800000u) return 0x7E00u;
    const double d = double(__builtin_bit_cast(float, top)) / 7.0;
    return d >= 65504.0 ? 0x7BFFu : uint32_t(__builtin_bit_cast(uint16_t, _Float16(d)));
}

// the word of 8 weights: even ones in the low half, odd ones in the high half
__device__ __forceinline__ uint32_t q4_word(const float* v, uint32_t scale) {
    const float s = float(__builtin_bit_cast(_Float16, uint16_t(scale)));
    const bool zero = !(s > 0.0f);   // 0 or NaN
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float r = __builtin_rintf(v[j] / s);
        const int c = zero ? 0 : int(__builtin_fminf(__builtin_fmaxf(r, -8.0f), 7.0f));
        w |= (uint32_t(c) & 15u) << (4 * (j >> 1) + 16 * (j & 1));
    }
    return w;
}

// One lane per 8 weights, a group being 4, 8 or 16 neighbouring lanes
template <typename T, int G>
__global__ __launch_bounds__(kThreads) void q4_quantize_kernel(const void* __restrict__ w,
                                                               int64_t words,
                                                               uint32_t* __restrict__ packed,
                                                               uint16_t* __restrict__ scales) {
    // words is a multiple of 16 (K % 128 == 0): a group's lanes leave together
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < words; i += stride) {
        float v[8];
        load8<T>(w, 8 * i, v);
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, abs_bits(v[j]));
        const uint32_t s = q4_scale(group_max(a, G / 8));
        packed[i] = q4_word(v, s);
        if (i % (G / 8) == 0) scales[i / (G / 8)] = uint16_t(s);
    }
}

// One wave per 1024-block of a row, 16 weights a lane
template <typename T, int G>
__global__ __launch_bounds__(kThreads) void q4_quantize_rotated_kernel(
    const void* __restrict__ w, const int8_t* __restrict__ signs, int64_t blocks, int64_t row_blocks,
    uint32_t* __restrict__ packed, uint16_t* __restrict__ scales) {
    const int l = threadIdx.x & 63;
    const int64_t stride = int64_t(gridDim.x) * (kThreads / 64);
    for (int64_t b = int64_t(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6); b < blocks; b += stride) {
        const int64_t i = b * kBlock + 16 * l;
        float v[16], h[8];
        load8<T>(w, i, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = h[j];
        load8<T>(w, i + 8, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 + j] = h[j];
        rotate16(v, *reinterpret_cast<const uint4*>(signs + (b % row_blocks) * kBlock + 16 * l), l);
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            v[j] *= 0.03125f;
            a = max(a, abs_bits(v[j]));
        }
        const uint32_t s = q4_scale(group_max(a, G / 16));
        *reinterpret_cast<uint2*>(packed + i / 8) = uint2{q4_word(v, s), q4_word(v + 8, s)};
        if (l % (G / 16) == 0) scales[i / G] = uint16_t(s);
    }
}

template <typename T, int G>
__global__ __launch_bounds__(kThreads) void q4_dequantize_kernel(const uint32_t* __restrict__ packed,
                                                                 const uint16_t* __restrict__ scales,
                                                                 int64_t words, void* __restrict__ w) {
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < words; i += stride) {
        const uint32_t q = packed[i];
        const float s = float(__builtin_bit_cast(_Float16, scales[i / (G / 8)]));
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = float(int32_t(q << (28 - 4 * (j >> 1) - 16 * (j & 1))) >> 28) * s;
        store8<T>(w, 8 * i, v);
    }
}

unsigned grid_for(int64_t work, int64_t per_wg) {
    const int64_t g = (work + per_wg - 1) / per_wg;
    return unsigned(g < (1 << 20) ? g : (1 << 20));
}

template <typename T, int G>
void quantize(const void* w, const int8_t* signs, int64_t n, int64_t k, uint8_t* packed,
              uint16_t* scales, hipStream_t stream) {
    uint32_t* out = reinterpret_cast<uint32_t*>(packed);
    if (signs) {
        const int64_t blocks = n * (k / kBlock);
        hipLaunchKernelGGL((q4_quantize_rotated_kernel<T, G>), dim3(grid_for(blocks, kThreads / 64)),
                           dim3(kThreads), 0, stream, w, signs, blocks, k / kBlock, out, scales);
    } else {
        const int64_t words = n * k / 8;
        hipLaunchKernelGGL((q4_quantize_kernel<T, G>), dim3(grid_for(words, kThreads)), dim3(kThreads), 0,
                           stream, w, words, out, scales);
    }
}

template <typename T, int G>
void dequantize(const uint8_t* packed, const uint16_t* scales, int64_t n, int64_t k, void* w,
                hipStream_t stream) {
    const int64_t words = n * k / 8;
    hipLaunchKernelGGL((q4_dequantize_kernel<T, G>), dim3(grid_for(words, kThreads)), dim3(kThreads), 0,
                       stream, reinterpret_cast<const uint32_t*>(packed), scales, words, w);
}

// f<T, G> for the type and group size
#define TL_Q4_DISPATCH(f, type, group)                                                              \
    (type == TL_F32    ? (group == 32 ? f<F32, 32> : group == 64 ? f<F32, 64> : f<F32, 128>)        \
     : type == TL_F16  ? (group == 32 ? f<F16, 32> : group == 64 ? f<F16, 64> : f<F16, 128>)        \
                       : (group == 32 ? f<BF16, 32> : group == 64 ? f<BF16, 64> : f<BF16, 128>))

}  // namespace

hipError_t launch_q4_quantize(const void* w, const int8_t* signs, int64_t n, int64_t k, int w_dtype,
                              int group, uint8_t* packed, uint16_t* scales, hipStream_t stream) {
    TL_Q4_DISPATCH(quantize, w_dtype, group)(w, signs, n, k, packed, scales, stream);
    return hipGetLastError();
}

hipError_t launch_q4_dequantize(const uint8_t* packed, const uint16_t* scales, int64_t n, int64_t k,
                                int group, void* w, int w_dtype, hipStream_t stream) {
    TL_Q4_DISPATCH(dequantize, w_dtype, group)(packed, scales, n, k, w, stream);
    return hipGetLastError();
}

}  // namespace tl
