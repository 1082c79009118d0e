// Product of few tokens with 4-bit weights:
//
//   y[m, n] = sum_g S[n, g] * sum_{k in g} code[n, k] * x[m, k]
//
// One wave per weight row and up to four tokens; a lane takes every 64th word
// of 8 weights, whose products with the activations are summed in fp32 and
// multiplied by the word's scales; the lanes are added in a fixed order.
#include "elem.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;

constexpr int kThreads = 256;
constexpr int kTokens = 4;

template <int XT>
__device__ __forceinline__ void load_x(const void* x, const float* xs, int64_t m, int64_t k, int64_t i,
                                       float (&v)[8], float& scale) {
    scale = 1.0f;
    if (XT == TL_I8) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const int8_t*>(x) + m * k + i);
        for (int j = 0; j < 8; ++j)
            v[j] = float(int32_t((j < 4 ? u.x : u.y) << (24 - 8 * (j & 3))) >> 24);
        scale = xs[m * (k / 128) + i / 128];
    } else if (XT == TL_F16) {
        load8<F16>(x, m * k + i, v);
    } else {
        load8<BF16>(x, m * k + i, v);
    }
}

template <int XT>
__global__ __launch_bounds__(kThreads) void q4_gemv_kernel(const uint32_t* __restrict__ packed,
                                                           const uint16_t* __restrict__ scales,
                                                           int group, const void* __restrict__ x,
                                                           const float* __restrict__ xs, int64_t m,
                                                           int64_t n, int64_t k, void* __restrict__ y,
                                                           int y_dtype) {
    const int l = threadIdx.x & 63;
    const int64_t row = int64_t(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
    if (row >= n) return;
    const uint32_t* wr = packed + row * (k / 8);
    const uint16_t* sr = scales + row * (k / group);
    for (int64_t t0 = int64_t(blockIdx.y) * kTokens; t0 < m; t0 += int64_t(gridDim.y) * kTokens) {
        const int tokens = int(m - t0 < kTokens ? m - t0 : kTokens);
        float acc[kTokens] = {};
        for (int64_t i = l; i < k / 8; i += 64) {
            const uint32_t q = wr[i];
            const float s = float(__builtin_bit_cast(_Float16, sr[8 * i / group]));
            float c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                c[j] = float(int32_t(q << (28 - 4 * (j >> 1) - 16 * (j & 1))) >> 28);
            for (int t = 0; t < tokens; ++t) {
                float v[8], xsc, d = 0.0f;
                load_x<XT>(x, xs, t0 + t, k, 8 * i, v, xsc);
#pragma unroll
                for (int j = 0; j < 8; ++j) d = __builtin_fmaf(c[j], v[j], d);
                acc[t] = __builtin_fmaf(d, s * xsc, acc[t]);
            }
        }
        for (int t = 0; t < tokens; ++t) {
            float a = acc[t];
            for (int o = 32; o > 0; o >>= 1) a += __shfl_xor(a, o, 64);
            if (l == 0) {
                const int64_t at = (t0 + t) * n + row;
                if (y_dtype == TL_F32) static_cast<float*>(y)[at] = a;
                else static_cast<uint16_t*>(y)[at] = uint16_t(y_dtype == TL_F16 ? f16_bits(a) : bf16_bits(a));
            }
        }
    }
}

}  // namespace

int64_t q4_gemv_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_q4_gemv(const uint8_t* packed, const uint16_t* scales, int group, const void* x,
                          int x_dtype, const float* x_scales, int64_t m, int64_t n, int64_t k, void* y,
                          int y_dtype, void*, hipStream_t stream) {
    const int64_t tiles = (m + kTokens - 1) / kTokens;
    const dim3 grid(unsigned((n + kThreads / 64 - 1) / (kThreads / 64)), unsigned(tiles < 64 ? tiles : 64));
    const auto f = x_dtype == TL_I8    ? q4_gemv_kernel<TL_I8>
                   : x_dtype == TL_F16 ? q4_gemv_kernel<TL_F16>
                                       : q4_gemv_kernel<TL_BF16>;
    hipLaunchKernelGGL(f, grid, dim3(kThreads), 0, stream, reinterpret_cast<const uint32_t*>(packed), scales,
                       group, x, x_scales, m, n, k, y, y_dtype);
    return hipGetLastError();
}

}  // namespace tl
