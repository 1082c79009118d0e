// 8-bit floating point rows with block scales: rounding of rows (weights or
// activations) and their values.
//
//   a = max |x| over the finite of 128, S = 2^e, the smallest power of two from
//   2^-127 up with a <= 448 S;  c = e4m3(x / S), nearest even;  x ~ c S
//
// With a = f 2^p, 1 <= f < 2, and 448 = 1.75 * 2^8, e is p - 8 where f <= 1.75
// and p - 7 where it is not: taken from a's bits.  x / S is exact (a power of
// two; what leaves fp32's normal numbers on the way is far below half of e4m3's
// smallest, 2^-10, and rounds to 0), so codes follow exactly from x.
//
// Bound: memory.  A lane takes 8 values, so that a wave reads and writes whole cache
// lines and a block of 128 is 16 lanes, whose maximum takes four DPP steps and no LDS.
// us in a graph (traced): 17408 x 5120 float32 rounded 77 (446 MB, 5.8 TB/s), 4096 x
// 5120 bfloat16 11.8, a token 1.5; 17408 x 5120 back to binary16 41 (268 MB, 6.5 TB/s).
// (Two pieces a lane: 80; with stores past the caches' replacement order 76, but the
// product that reads the codes next takes 8 us longer, 4096 x 1024 x 5120 52 against 44
// with the rounding.)
#include "elem.h"
#include "f8.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;
using namespace f8;

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t abs_bits(float f) { return __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu; }

// largest of a row of 16 lanes
__device__ __forceinline__ uint32_t row16_max(uint32_t a) {
    const auto step = [&](int o) { a = uint32_t(o) > a ? uint32_t(o) : a; };
    step(__builtin_amdgcn_mov_dpp(int(a), 0xB1, 0xF, 0xF, false));    // lane ^ 1
    step(__builtin_amdgcn_mov_dpp(int(a), 0x4E, 0xF, 0xF, false));    // lane ^ 2
    step(__builtin_amdgcn_mov_dpp(int(a), 0x141, 0xF, 0xF, false));   // the other four of 8
    step(__builtin_amdgcn_mov_dpp(int(a), 0x140, 0xF, 0xF, false));   // the other 8
    return a;
}

// One lane per 8 values, a block being a row of 16 lanes
template <typename T>
__global__ __launch_bounds__(kThreads) void f8_quantize_kernel(const void* __restrict__ x, int64_t items,
                                                               uint2* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
    // items is a multiple of 16 (K % 128 == 0): a block's lanes leave together
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < items; i += stride) {
        float v[8];
        load8<T>(x, 8 * i, v);
        uint32_t a = 0, top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = abs_bits(v[j]);
            top = max(top, b);
            a = max(a, b < kInf ? b : 0u);
        }
        a = row16_max(a);
        const uint32_t s = scale_of(a);
        const float inv = __builtin_bit_cast(float, (254u - s) << 23);   // s <= 247
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w, true);
            c[h] = uint32_t(w);
        }
        if (top >= kInf) {      // e4m3 has no infinity: both become its NaN
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (abs_bits(v[j]) >= kInf) c[j >> 2] = (c[j >> 2] & ~(0xFFu << (8 * (j & 3)))) | 0x7Fu << (8 * (j & 3));
        }
        codes[i] = uint2{c[0], c[1]};
        if ((i & 15) == 0) scales[i >> 4] = uint8_t(s);
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void f8_dequantize_kernel(const uint2* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales,
                                                                 int64_t items, void* __restrict__ w) {
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < items; i += stride) {
        float v[8];
        values8(codes[i], scale_value(scales[i >> 4]), v);
        store8<T>(w, 8 * i, v);
    }
}

unsigned grid_for(int64_t items) {
    const int64_t g = (items + kThreads - 1) / kThreads;
    return unsigned(g < (1 << 20) ? g : (1 << 20));
}

}  // namespace

hipError_t launch_f8_quantize(const void* x, int64_t m, int64_t k, int x_dtype, uint8_t* codes, uint8_t* scales,
                              hipStream_t stream) {
    const int64_t items = m * k / 8;
    uint2* c = reinterpret_cast<uint2*>(codes);
    const dim3 grid(grid_for(items)), block(kThreads);
    if (x_dtype == TL_F32) hipLaunchKernelGGL(f8_quantize_kernel<F32>, grid, block, 0, stream, x, items, c, scales);
    else if (x_dtype == TL_F16) hipLaunchKernelGGL(f8_quantize_kernel<F16>, grid, block, 0, stream, x, items, c, scales);
    else hipLaunchKernelGGL(f8_quantize_kernel<BF16>, grid, block, 0, stream, x, items, c, scales);
    return hipGetLastError();
}

hipError_t launch_f8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n, int64_t k, void* w,
                                int w_dtype, hipStream_t stream) {
    const int64_t items = n * k / 8;
    const uint2* c = reinterpret_cast<const uint2*>(codes);
    const dim3 grid(grid_for(items)), block(kThreads);
    if (w_dtype == TL_F32) hipLaunchKernelGGL(f8_dequantize_kernel<F32>, grid, block, 0, stream, c, scales, items, w);
    else if (w_dtype == TL_F16) hipLaunchKernelGGL(f8_dequantize_kernel<F16>, grid, block, 0, stream, c, scales, items, w);
    else hipLaunchKernelGGL(f8_dequantize_kernel<BF16>, grid, block, 0, stream, c, scales, items, w);
    return hipGetLastError();
}

}  // namespace tl
