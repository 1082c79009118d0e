// Embedding lookup: rows of a table of 4-bit or 8-bit floating point weights,
// times a factor,
//
//   out[m, k] = value(ids[m], k) * factor   (0 for an id outside the table)
//
// value is exact in fp32, the product is rounded there and once more to the
// output's type.  A lane takes 8 values; nothing is shared, so the bound is
// memory (a prompt) or the latency of two dependent loads, id then row (a token).
// us traced: 4096 rows of 5120 8-bit codes to bfloat16 12 (42 MB written), a row of 4-bit ones
// 1.7.  Outputs are stored to stay in the caches, for the norm that reads them next: past
// the replacement order the lookup is faster and the two together are not (us in a graph,
// alone and with the norm: 4096 x 5120 float32 24.4 45.2, past it 23.1 49.2; with eight
// buffers in turn 27.4 45.6, past it 23.1 47.8; bfloat16 14.6 33.5, past it 14.8 34.7).
#include "elem.h"
#include "f8.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;
using namespace f8;

constexpr int kThreads = 256;

// 8 values of table row `id` from its place j (in eights)
template <int G>   // 4-bit codes with a scale per G
struct Q4 {
    static __device__ __forceinline__ void load(const uint8_t* codes, const void* scales, int64_t id, uint32_t eights,
                                                uint32_t j, float (&v)[8]) {
        const uint32_t q = reinterpret_cast<const uint32_t*>(codes)[id * eights + j];
        const uint16_t h = static_cast<const uint16_t*>(scales)[id * (eights / (G / 8)) + j / (G / 8)];
        const float s = float(__builtin_bit_cast(_Float16, h));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = float(int32_t(q << (28 - 4 * (i >> 1) - 16 * (i & 1))) >> 28) * s;
    }
};

struct E4M3 {
    static __device__ __forceinline__ void load(const uint8_t* codes, const void* scales, int64_t id, uint32_t eights,
                                                uint32_t j, float (&v)[8]) {
        const uint2 c = reinterpret_cast<const uint2*>(codes)[id * eights + j];
        values8(c, scale_value(static_cast<const uint8_t*>(scales)[id * (eights / 16) + j / 16]), v);
    }
};

// U pieces of 8 values a lane, all asked for before the first is stored
template <typename W, typename T, int U>
__global__ __launch_bounds__(kThreads) void rows_kernel(const uint8_t* __restrict__ codes,
                                                        const void* __restrict__ scales,
                                                        const int32_t* __restrict__ ids, int64_t m, int64_t n,
                                                        uint32_t eights, float factor, void* __restrict__ out) {
    // the workgroup's first item by one division of scalars, a lane's by 32-bit ones
    const int64_t first = int64_t(blockIdx.x) * (kThreads * U), row0 = first / eights;
    const uint32_t off0 = uint32_t(first - row0 * eights) + threadIdx.x;
    int64_t row[U];
    uint32_t j[U];
    int32_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t off = off0 + u * kThreads;
        row[u] = row0 + off / eights;
        j[u] = off % eights;
        id[u] = row[u] < m ? ids[row[u]] : -1;
    }
    float v[U][8] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (id[u] < 0 || id[u] >= n) continue;
        W::load(codes, scales, id[u], eights, j[u], v[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] *= factor;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (row[u] < m) store8<T, true>(out, 8 * (row[u] * eights + j[u]), v[u]);
}

template <typename W, int U>
hipError_t rows(const uint8_t* codes, const void* scales, const int32_t* ids, int64_t m, int64_t n, int64_t k,
                float factor, void* out, int out_dtype, hipStream_t stream) {
    const auto kernel = out_dtype == TL_F32   ? rows_kernel<W, F32, 1>
                        : out_dtype == TL_F16 ? rows_kernel<W, F16, U>
                                              : rows_kernel<W, BF16, U>;
    const int per = kThreads * (out_dtype == TL_F32 ? 1 : U);
    const uint32_t eights = uint32_t(k / 8);
    const int64_t most = (int64_t(1) << 31) / eights;       // rows of a launch, whose lanes count in 32 bits
    for (int64_t at = 0; at < m; at += most) {
        const int64_t left = m - at < most ? m - at : most;
        hipLaunchKernelGGL(kernel, dim3(unsigned((left * eights + per - 1) / per)), dim3(kThreads), 0, stream,
                           codes, scales, ids + at, left, n, eights, factor,
                           static_cast<uint8_t*>(out) + at * k * (out_dtype == TL_F32 ? 4 : 2));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Two pieces a lane for outputs of 2 bytes where there are many.  us in a graph with one
// and two: 4096 rows of 5120 8-bit codes to bfloat16 12.9 12.3 (outputs beyond the cache
// 18.4 16.9), 16384 of 1024 11.1 10.8, 512 of 5120 4.2 4.4; to float32 4096 of 5120 26.6
// 27.7.
template <typename W>
hipError_t rows(const uint8_t* codes, const void* scales, const int32_t* ids, int64_t m, int64_t n, int64_t k,
                float factor, void* out, int out_dtype, hipStream_t stream) {
    return m * k >= int64_t(1) << 23 ? rows<W, 2>(codes, scales, ids, m, n, k, factor, out, out_dtype, stream)
                                     : rows<W, 1>(codes, scales, ids, m, n, k, factor, out, out_dtype, stream);
}

}  // namespace

hipError_t launch_q4_rows(const uint8_t* packed, const uint16_t* scales, int group, const int32_t* ids, int64_t m,
                          int64_t n, int64_t k, float factor, void* out, int out_dtype, hipStream_t stream) {
    return group == 32   ? rows<Q4<32>>(packed, scales, ids, m, n, k, factor, out, out_dtype, stream)
           : group == 64 ? rows<Q4<64>>(packed, scales, ids, m, n, k, factor, out, out_dtype, stream)
                         : rows<Q4<128>>(packed, scales, ids, m, n, k, factor, out, out_dtype, stream);
}

hipError_t launch_f8_rows(const uint8_t* codes, const uint8_t* scales, const int32_t* ids, int64_t m, int64_t n,
                          int64_t k, float factor, void* out, int out_dtype, hipStream_t stream) {
    return rows<E4M3>(codes, scales, ids, m, n, k, factor, out, out_dtype, stream);
}

}  // namespace tl
