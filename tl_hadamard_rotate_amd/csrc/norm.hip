// Residual addition, root-mean-square norm and gain of activation rows, with
// the signed rotation of the ternary linear behind it (page "A 27-billion
// model that fits in 8.6 GB", paragraph 3) and 8-bit outputs on demand:
//
//   h = T(x + r),  y[k] = h[k] * gain[k] / sqrt(mean h^2 + eps),
//   out = y or R(y);  8 bits: a = max |value| of a group of 128, scale = a / 127,
//   code = rint(127 value / a)
//
// The row's factor 1 / sqrt(...) is common to all values, so it commutes with
// the rotation and cancels in the codes: both are taken of p = h * gain, in
// fp32 like the rotation's sums, and the factor is applied at the end.  Without the rotation p is exact in 64
// bits (24 by 24 bits), and close codes are decided there: a quotient of 16-bit
// types (22 bits by 22) lies on a tie only if the true one does.
//
// One workgroup per row.  A wave holds one or two 1024-blocks in registers,
// lane l elements 8l .. 8l + 7 and 512 + 8l .. of each, so that every load is 1
// KB of memory (the rotation's index bits are then 4 register and 6 lane bits):
// each input is read once and each output written once, and the rotation runs
// while the waves' sums of squares are on their way through LDS.  Rows past
// kLongRow are gone through twice: the sum of squares (h goes to sum_out), then
// the values; a lane handles the same elements in both passes, so the second
// may read h back from sum_out, which may be x or the residual.
//
// Bound by memory for many rows, by the launch for few.  Outputs are stored
// past the caches' replacement order: 4096 x 5120 bfloat16 rows with a residual
// (168 MB) 27.8 us, 6.0 TB/s, against 39 with ordinary stores; as 8-bit codes
// (147 MB) 28.7 us with gains around 1, 38.6 with a gain of ones, whose quotients
// lie near ties more often.  2048 rotated binary16 rows (84 MB) 18.9 us, 4.5 TB/s:
// the rotation's 10 levels; 4096 of them as 8-bit codes 57 us, the rotation's and
// the codes' instructions.  One row of 5120 4.6-5.3 us, 16 to 8 bits 5.7.
#include <type_traits>

#include "elem.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kLongRow = 24576;     // elements; 12 waves of two blocks: longer rows do not fit in registers
constexpr int kMaxGrid = 1 << 20;   // workgroups of a launch; rows beyond it are looped over

struct I8 {
    static constexpr int kType = TL_I8, kBytes = 1;
};

// values of a lane as the output takes them: h * g, or h that was rotated
template <typename P, bool ROT>
__device__ __forceinline__ P value(float h, float g) {
    return ROT ? P(h) : P(h) * P(g);
}

// largest |value| of the 16 lanes that hold 128 elements, NaN above infinity
// above numbers: the order of their bits
template <typename P, bool ROT>
__device__ __forceinline__ P abs_max(const float (&h)[8], const float (&g)[8], int l) {
    using B = typename std::conditional<sizeof(P) == 4, uint32_t, uint64_t>::type;
    B a = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const B b = __builtin_bit_cast(B, value<P, ROT>(h[j], g[j])) & (~B(0) >> 1);
        a = b > a ? b : a;
    }
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) {
        B o;
        if constexpr (sizeof(P) == 4) o = __builtin_bit_cast(B, reduce_xor(__builtin_bit_cast(float, a), m, l));
        else o = __shfl_xor(a, m, 64);
        a = o > a ? o : a;
    }
    return __builtin_bit_cast(P, a);
}

// 8 consecutive elements of a lane (its row of 16 lanes holds the group of 128)
// to codes at out and, by the group's first lane, its scale.  All lanes of a
// wave come here.  The codes are taken in fp32, whose quotients are off by less
// than 127 * 4.1 * 2^-24 < 3.2e-5 (the roundings of value, a, 127 / a and the
// product); a wave with one nearer than 4e-5 to a tie (4 % of the waves), or
// whose 127 / a is no number, decides them in 64 bits: by the quotient, or,
// where the values are fp32, by the exact remainder (eight quotients at once
// beside the rotation's registers went to scratch: one row of 5120 took 5 us
// more).
template <bool ROT>
__device__ __forceinline__ void store_i8(const float (&h)[8], const float (&g)[8], float inv, bool on, int l,
                                         int8_t* out, float* out_scale) {
    const float a = abs_max<float, ROT>(h, g, l);   // the rounded largest value: rounding keeps the order
    const bool finite = a <= 3.4028234663852886e38f;
    const float up = ROT && a < 1e-30f ? 0x1p100f : 1.0f;
    bool slow = !ROT && !(a > 1e-30f);
    const float r = 127.0f / (a * up);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = value<float, ROT>(h[j], g[j]) * up * r;
        q[j] = __builtin_rintf(t);
        slow |= __builtin_fabsf(t - q[j]) > 0.5f - 4e-5f;
    }
    if (__ballot(slow && finite && on)) {
        if constexpr (ROT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const double e = __builtin_fma(127.0, double(h[j]), -double(q[j]) * double(a));
                const double gap = 2.0 * __builtin_fabs(e) - double(a);
                if (gap > 0 || (gap == 0 && (int(q[j]) & 1))) q[j] += e > 0 ? 1.0f : -1.0f;
            }
        } else {
            const double d = abs_max<double, ROT>(h, g, l);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                q[j] = d > 0 ? float(__builtin_rint(127.0 * value<double, ROT>(h[j], g[j]) / d)) : 0.0f;
        }
    }
    if (!on) return;
    // (inv is 0 or NaN where the row has an infinity, a NaN or squares past fp32:
    // all its values are 0 or NaN then)
    const bool none = !finite || !(inv > 0.0f) || (ROT && a == 0);
    uint32_t w[2] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = none ? 0 : int(q[j]);
        w[j >> 2] |= (uint32_t(c) & 0xFFu) << (8 * (j & 3));
    }
    put<false>(reinterpret_cast<u32x2*>(out), u32x2{w[0], w[1]});
    if ((l & 15) == 0) *out_scale = finite ? a * inv * (1.0f / 127.0f) : __builtin_nanf("");
}

// a lane's 8 consecutive elements written, `scale` the row's factor: taken before
// the gain, as h * scale stays within sqrt(K) where h * gain may pass fp32
template <typename O, bool ROT>
__device__ __forceinline__ void store_out(const float (&h)[8], const float (&g)[8], float scale, bool on, int l,
                                          int64_t at, int64_t group, void* out, float* out_scales) {
    if constexpr (O::kType == TL_I8) {
        store_i8<ROT>(h, g, scale, on, l, static_cast<int8_t*>(out) + at, out_scales + group);
    } else if (on) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ROT ? h[j] * scale : h[j] * scale * g[j];
        store8<O>(out, at, v);
    }
}

// sum over the wave, the same in every lane
__device__ __forceinline__ float wave_sum(float v, int l) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += reduce_xor(v, m, l);
    return v;
}

// NB 1024-blocks a wave, as many waves as the row needs
template <typename T, typename O, bool ROT, int NB>
__global__ __launch_bounds__(NB == 1 ? 1024 : 768) void rms_norm_kernel(const void* x, const void* residual,
                                                                         const void* gain, const int8_t* signs,
                                                                         int64_t m, int64_t k, float eps,
                                                                         void* sum_out, void* out,
                                                                         float* out_scales) {
    __shared__ float part[2][16];
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = int(blockDim.x >> 6);
    const float inv_k = 1.0f / float(k);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x, turn ^= 1) {
        const int64_t base = row * k;
        float h[NB][2][8], g[NB][2][8];
        uint4 sg[NB];
        float ss = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t i = 1024 * (wave + int64_t(b) * waves) + 512 * e + 8 * l;
                if (i < k) load8<T>(x, base + i, h[b][e]);
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[b][e][j] = 0.0f;
            }
        if (residual) {
            float r[NB][2][8];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int64_t i = 1024 * (wave + int64_t(b) * waves) + 512 * e + 8 * l;
                    if (i < k) load8<T>(residual, base + i, r[b][e]);
                    else
#pragma unroll
                        for (int j = 0; j < 8; ++j) r[b][e][j] = 0.0f;
                }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[b][e][j] = round_to<T>(h[b][e][j] + r[b][e][j]);
                }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t i = 1024 * (wave + int64_t(b) * waves) + 512 * e + 8 * l;
                if (i < k) load8<T>(gain, i, g[b][e]);
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[b][e][j] = 0.0f;
                if (ROT) {
                    const uint2 s = i < k ? *reinterpret_cast<const uint2*>(signs + i) : uint2{0, 0};
                    if (e == 0) sg[b].x = s.x, sg[b].y = s.y;
                    else sg[b].z = s.x, sg[b].w = s.y;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(h[b][e][j], h[b][e][j], ss);
            }
        ss = wave_sum(ss, l);
        if (l == 0) part[turn][wave] = ss;
        if (sum_out)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int64_t i = 1024 * (wave + int64_t(b) * waves) + 512 * e + 8 * l;
                    if (i < k) store8<T>(sum_out, base + i, h[b][e]);
                }
        if constexpr (ROT)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = h[b][j >> 3][j & 7] * g[b][j >> 3][j & 7];
                rotate16(v, sg[b], l);
#pragma unroll
                for (int j = 0; j < 16; ++j) h[b][j >> 3][j & 7] = v[j];
            }
        __syncthreads();   // (the other set of sums is written next)
        ss = 0.0f;
        for (int w = 0; w < waves; ++w) ss += part[turn][w];
        float scale = 1.0f / sqrtf(ss * inv_k + eps);
        if (ROT) scale *= 0.03125f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t i = 1024 * (wave + int64_t(b) * waves) + 512 * e + 8 * l;
                store_out<O, ROT>(h[b][e], g[b][e], scale, i < k, l, base + i, (base + i) / 128, out, out_scales);
            }
    }
}

template <typename T, typename O, bool ROT>
__global__ __launch_bounds__(kThreads) void rms_norm_long_kernel(const void* x, const void* residual,
                                                                 const void* gain, const int8_t* signs,
                                                                 int64_t m, int64_t k, float eps,
                                                                 void* sum_out, void* out,
                                                                 float* out_scales) {
    __shared__ float part[kWaves];
    const int l = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
        const int64_t base = row * k;
        const auto element = [&](int64_t b, int e) { return 1024 * (b + wave) + 512 * e + 8 * l; };
        const auto load_h = [&](int64_t i, const void* from, bool add, float (&v)[8]) {
            load8<T>(from, base + i, v);
            if (add) {
                float r[8];
                load8<T>(residual, base + i, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = round_to<T>(v[j] + r[j]);
            }
        };
        float ss = 0.0f;
        for (int64_t b = 0; 1024 * b < k; b += kWaves)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t i = element(b, e);
                if (i >= k) continue;
                float v[8];
                load_h(i, x, residual != nullptr, v);
                if (sum_out) store8<T, true>(sum_out, base + i, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(v[j], v[j], ss);
            }
        ss = wave_sum(ss, l);
        if (l == 0) part[wave] = ss;
        __syncthreads();
        ss = (part[0] + part[1]) + (part[2] + part[3]);
        __syncthreads();
        float scale = 1.0f / sqrtf(ss / float(k) + eps);
        if (ROT) scale *= 0.03125f;
        // whole waves take part in the exchanges, whether their elements exist or not
        for (int64_t b = 0; 1024 * b < k; b += kWaves) {
            float h[2][8] = {}, g[2][8] = {};
            uint2 sg[2] = {};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t i = element(b, e);
                if (i >= k) continue;
                load_h(i, sum_out ? sum_out : x, residual && !sum_out, h[e]);
                load8<T>(gain, i, g[e]);
                if (ROT) sg[e] = *reinterpret_cast<const uint2*>(signs + i);
            }
            if constexpr (ROT) {
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = h[j >> 3][j & 7] * g[j >> 3][j & 7];
                rotate16(v, uint4{sg[0].x, sg[0].y, sg[1].x, sg[1].y}, l);
#pragma unroll
                for (int j = 0; j < 16; ++j) h[j >> 3][j & 7] = v[j];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t i = element(b, e);
                store_out<O, ROT>(h[e], g[e], scale, i < k, l, base + i, (base + i) / 128, out, out_scales);
            }
        }
    }
}

template <typename T, typename O, bool ROT>
void launch_row(const void* x, const void* residual, const void* gain, const int8_t* signs, int64_t m,
                int64_t k, float eps, void* sum_out, void* out, float* out_scales, hipStream_t stream) {
    const dim3 grid(unsigned(m < kMaxGrid ? m : kMaxGrid));
    const int blocks = int((k + 1023) / 1024);
    if (blocks <= 16)
        hipLaunchKernelGGL((rms_norm_kernel<T, O, ROT, 1>), grid, dim3(64 * blocks), 0, stream, x, residual, gain,
                           signs, m, k, eps, sum_out, out, out_scales);
    else if (k <= kLongRow)
        hipLaunchKernelGGL((rms_norm_kernel<T, O, ROT, 2>), grid, dim3(64 * ((blocks + 1) / 2)), 0, stream, x,
                           residual, gain, signs, m, k, eps, sum_out, out, out_scales);
    else
        hipLaunchKernelGGL((rms_norm_long_kernel<T, O, ROT>), grid, dim3(kThreads), 0, stream, x, residual, gain,
                           signs, m, k, eps, sum_out, out, out_scales);
}

template <typename T, typename O>
void launch(const void* x, const void* residual, const void* gain, const int8_t* signs, int64_t m,
            int64_t k, float eps, void* sum_out, void* out, float* out_scales, hipStream_t stream) {
    if (signs) launch_row<T, O, true>(x, residual, gain, signs, m, k, eps, sum_out, out, out_scales, stream);
    else launch_row<T, O, false>(x, residual, gain, signs, m, k, eps, sum_out, out, out_scales, stream);
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
