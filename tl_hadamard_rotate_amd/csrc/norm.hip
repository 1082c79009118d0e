// Residual addition, root-mean-square norm and gain of activation rows, with
// the signed rotation of the ternary linear behind it (page "A 27-billion
// model that fits in 8.6 GB", paragraph 3) and 8-bit outputs on demand:
//
//   h = T(x + r),  y[k] = h[k] * gain[k] / sqrt(mean h^2 + eps),
//   out = y or R(y);  8 bits: a = max |value| of a group of 128, scale = a / 127,
//   code = rint(127 value / a)
//
// The row's factor 1 / sqrt(...) is common to all values, so it commutes with
// the rotation and cancels in the codes: both are taken of p = h * gain, and
// the factor is applied at the end.  Without the rotation p is exact in 64
// bits (24 by 24 bits), and the codes are decided there: a quotient of 16-bit
// types (22 bits by 22) lies on a tie only if the true one does.
//
// One workgroup per row, in two passes over it: the sum of squares (h goes to
// sum_out), then the values.  A lane handles the same elements in both, so the
// second pass may read h back from sum_out, which may be x or the residual.
#include <type_traits>

#include "elem.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxGrid = 1 << 20;   // workgroups of a launch; rows beyond it are looped over

struct I8 {
    static constexpr int kType = TL_I8, kBytes = 1;
};

// largest |p| of the lanes' group, NaN above infinity above numbers
template <typename P>
__device__ __forceinline__ P group_max(P a, int lanes) {
    for (int m = 1; m < lanes; m <<= 1) {
        const P o = __shfl_xor(a, m, 64);
        a = o > a || o != o ? o : a;
    }
    return a;
}

// E consecutive p of a lane (lanes l ^ 1 .. hold the rest of the group of 128)
// to codes and the group's scale
template <typename P, int E>
__device__ __forceinline__ void store_i8(const P (&p)[E], float inv, int64_t i, int64_t row_groups0, int64_t k0,
                                         bool on, int8_t* out, float* out_scales) {
    P a = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const P b = p[j] < 0 ? -p[j] : p[j];
        a = b > a || b != b ? b : a;
    }
    a = group_max(a, 128 / E);
    if (!on) return;
    const bool finite = a <= P(3.4028234663852886e38);
    uint32_t w[E / 4] = {};
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const int c = finite && a > 0 ? int(__builtin_rint(127.0 * double(p[j]) / double(a))) : 0;
        w[j >> 2] |= (uint32_t(c) & 0xFFu) << (8 * (j & 3));
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(out + i);
#pragma unroll
    for (int j = 0; j < E / 4; ++j) dst[j] = w[j];
    if (k0 % 128 == 0)
        out_scales[row_groups0 + k0 / 128] =
            finite ? float(a) * inv * (1.0f / 127.0f) : __builtin_nanf("");
}

template <typename T, typename O, bool ROT>
__global__ __launch_bounds__(kThreads) void rms_norm_kernel(const void* x, const void* residual,
                                                            const void* gain, const int8_t* signs,
                                                            int64_t m, int64_t k, float eps,
                                                            void* sum_out, void* out,
                                                            float* out_scales) {
    constexpr int E = ROT ? 16 : 8;   // consecutive elements of a lane
    __shared__ float part[kWaves];
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
        const int64_t base = row * k;
        float ss = 0.0f;
        for (int64_t i = int64_t(threadIdx.x) * E; i < k; i += kThreads * E)
#pragma unroll
            for (int e = 0; e < E; e += 8) {
                float v[8];
                load8<T>(x, base + i + e, v);
                if (residual) {
                    float r[8];
                    load8<T>(residual, base + i + e, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = round_to<T>(v[j] + r[j]);
                    if (sum_out) store8<T>(sum_out, base + i + e, v);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[j], v[j], ss);
            }
        for (int s = 1; s < 64; s <<= 1) ss += __shfl_xor(ss, s, 64);
        if (l == 0) part[wave] = ss;
        __syncthreads();
        ss = (part[0] + part[1]) + (part[2] + part[3]);
        __syncthreads();
        const float inv = 1.0f / sqrtf(ss / float(k) + eps);

        // whole waves take part in the exchanges, whether their elements exist or not
        const int64_t steps = (k + kThreads * E - 1) / (kThreads * E);
        for (int64_t st = 0; st < steps; ++st) {
            const int64_t i = (st * kThreads + threadIdx.x) * E;
            const bool on = i < k;
            using P = typename std::conditional<O::kType == TL_I8 && !ROT, double, float>::type;
            P p[E];
#pragma unroll
            for (int j = 0; j < E; ++j) p[j] = 0;
            if (on)
#pragma unroll
                for (int e = 0; e < E; e += 8) {
                    float v[8], g[8];
                    load8<T>(sum_out ? sum_out : x, base + i + e, v);
                    if (residual && !sum_out) {
                        float r[8];
                        load8<T>(residual, base + i + e, r);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = round_to<T>(v[j] + r[j]);
                    }
                    load8<T>(gain, i + e, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[e + j] = P(v[j]) * P(g[j]);
                }
            float scale = inv;
            if constexpr (ROT) {
                uint4 sg = uint4{0, 0, 0, 0};
                if (on) sg = *reinterpret_cast<const uint4*>(signs + i);
                rotate16(p, sg, l);
                scale *= 0.03125f;
            }
            if constexpr (O::kType == TL_I8) {
                store_i8<P, E>(p, scale, base + i, row * (k / 128), i, on, static_cast<int8_t*>(out),
                               out_scales);
            } else if (on) {
#pragma unroll
                for (int e = 0; e < E; e += 8) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = float(p[e + j]) * scale;
                    store8<O>(out, base + i + e, v);
                }
            }
        }
    }
}

template <typename T, typename O>
void launch(const void* x, const void* residual, const void* gain, const int8_t* signs, int64_t m,
            int64_t k, float eps, void* sum_out, void* out, float* out_scales, hipStream_t stream) {
    const dim3 grid(unsigned(m < kMaxGrid ? m : kMaxGrid));
    if (signs)
        hipLaunchKernelGGL((rms_norm_kernel<T, O, true>), grid, dim3(kThreads), 0, stream, x, residual,
                           gain, signs, m, k, eps, sum_out, out, out_scales);
    else
        hipLaunchKernelGGL((rms_norm_kernel<T, O, false>), grid, dim3(kThreads), 0, stream, x, residual,
                           gain, signs, m, k, eps, sum_out, out, out_scales);
}

template <typename T>
void launch_to(int out_dtype, const void* x, const void* residual, const void* gain,
               const int8_t* signs, int64_t m, int64_t k, float eps, void* sum_out, void* out,
               float* out_scales, hipStream_t stream) {
    switch (out_dtype) {
        case TL_F32: return launch<T, F32>(x, residual, gain, signs, m, k, eps, sum_out, out, out_scales, stream);
        case TL_F16: return launch<T, F16>(x, residual, gain, signs, m, k, eps, sum_out, out, out_scales, stream);
        case TL_BF16: return launch<T, BF16>(x, residual, gain, signs, m, k, eps, sum_out, out, out_scales, stream);
        default: return launch<T, I8>(x, residual, gain, signs, m, k, eps, sum_out, out, out_scales, stream);
    }
}

}  // namespace

hipError_t launch_rms_norm(const void* x, const void* residual, const void* gain, const int8_t* signs,
                           int64_t m, int64_t k, int x_dtype, float eps, void* sum_out, void* out,
                           int out_dtype, float* out_scales, hipStream_t stream) {
    const auto run = x_dtype == TL_F32 ? launch_to<F32> : x_dtype == TL_F16 ? launch_to<F16> : launch_to<BF16>;
    run(out_dtype, x, residual, gain, signs, m, k, eps, sum_out, out, out_scales, stream);
    return hipGetLastError();
}

}  // namespace tl
