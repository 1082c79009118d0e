// Logits made ready for drawing a token: penalties for tokens that occurred,
// biases, a grammar's mask.  For row m and token v, x in fp32:
//
//   seen   = v occurs among the row's history        x = x > 0 ? x / r : x * r   if seen
//   count  = its occurrences after the prompt        x = x - f * count - p (count > 0)
//   named  = the last bias of the row that names v   x = x + bias                if named
//   mask bit 0                                       x = -infinity
//
// A workgroup owns a slice of one row's tokens, 8 a lane.  It asks for its
// logits first; while they are on the way it goes through the row's whole
// history and biases and marks in LDS what falls into its slice (occurrences
// after the prompt counted in the low 31 bits of a word, the prompt's in the top
// one; the largest place of a bias that names the token): integer additions and
// maxima, whose order does not show.
#include <cmath>

#include "elem.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;

constexpr uint32_t kPrompt = 0x80000000u;

struct Args {
    const void* logits;
    const int32_t *history, *history_lens, *prompt_lens;
    const float *repetition, *presence, *frequency;
    const int32_t* bias_ids;
    const float* bias_values;
    const uint8_t* mask;
    void* out;
    int64_t v, h, b;
    uint32_t slices;
};

// 8 elements at any alignment of the type (rows of an odd vocabulary)
template <typename T>
struct Raw {
    uint32_t w[2 * T::kBytes];
};

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = T::kType == TL_F32   ? __builtin_bit_cast(float, r.w[j % (2 * T::kBytes)])
               : T::kType == TL_F16 ? float(__builtin_bit_cast(_Float16, uint16_t(r.w[j >> 1] >> (16 * (j & 1)))))
                                    : __builtin_bit_cast(float, j & 1 ? r.w[j >> 1] & 0xFFFF0000u : r.w[j >> 1] << 16);
}

template <typename T>
__device__ __forceinline__ void pack(const float (&x)[8], Raw<T>& r) {
    if constexpr (T::kType == TL_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j] = __builtin_bit_cast(uint32_t, x[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r.w[j] = T::kType == TL_F16 ? f16_bits(x[2 * j]) | f16_bits(x[2 * j + 1]) << 16
                                        : bf16_pair(x[2 * j], x[2 * j + 1]);
    }
}

template <typename T>
using Elem = std::conditional_t<T::kBytes == 4, uint32_t, uint16_t>;

template <typename T, typename U>
__global__ __launch_bounds__(1024) void adjust_logits_kernel(const Args a) {
    extern __shared__ uint32_t lds[];
    const uint32_t tid = threadIdx.x, threads = blockDim.x, width = 8 * threads;
    const int64_t row = blockIdx.x / a.slices;
    const int64_t first = int64_t(blockIdx.x - uint32_t(row) * a.slices) * width;   // of the slice
    const int64_t at = first + 8 * tid;                                             // of the lane
    const int64_t left = a.v - at;
    const Elem<T>* in = static_cast<const Elem<T>*>(a.logits) + row * a.v + at;
    Elem<U>* out = static_cast<Elem<U>*>(a.out) + row * a.v + at;

    Raw<T> raw = {};
    uint32_t allowed = 0xFFu;
    if (left >= 8) {
        __builtin_memcpy(&raw, in, sizeof(raw));
    } else {
        Elem<T> e[8] = {};
        for (int j = 0; j < 8; ++j)
            if (j < left) e[j] = in[j];
        __builtin_memcpy(&raw, e, sizeof(raw));
    }
    if (a.mask && left > 0) allowed = a.mask[row * ((a.v + 31) / 32 * 4) + (at >> 3)];

    uint32_t* const counts = lds;
    uint32_t* const named = lds + (a.history ? width : 0);
    if (a.history || a.bias_ids) {
        const uint32_t words = (a.history ? width : 0) + (a.bias_ids ? width : 0);
        for (uint32_t i = tid; i < words; i += threads) lds[i] = 0;
        __syncthreads();
        if (a.history) {
            int64_t len = a.history_lens ? a.history_lens[row] : a.h;
            len = len < 0 ? 0 : len > a.h ? a.h : len;
            const int64_t prompt = a.prompt_lens ? a.prompt_lens[row] : 0;
            const int32_t* ids = a.history + row * a.h;
            for (int64_t i = tid; i < len; i += threads) {
                const uint64_t d = uint64_t(int64_t(ids[i]) - first);
                if (d < width) {
                    if (i >= prompt) atomicAdd(&counts[d], 1u);
                    else atomicOr(&counts[d], kPrompt);
                }
            }
        }
        if (a.bias_ids) {
            const int32_t* ids = a.bias_ids + row * a.b;
            for (int64_t i = tid; i < a.b; i += threads) {
                const uint64_t d = uint64_t(int64_t(ids[i]) - first);
                if (d < width) atomicMax(&named[d], uint32_t(i + 1));
            }
        }
        __syncthreads();
    }
    if (left <= 0) return;

    float x[8];
    unpack<T>(raw, x);
    if (a.history) {
        const float r = a.repetition ? a.repetition[row] : 1.0f;
        const float p = a.presence ? a.presence[row] : 0.0f;
        const float f = a.frequency ? a.frequency[row] : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t c = counts[8 * tid + j];
            if (c) {
                const uint32_t n = c & ~kPrompt;
                if (a.repetition) x[j] = x[j] > 0.0f ? x[j] / r : x[j] * r;
                if (n) x[j] = x[j] - f * float(n) - p;
            }
        }
    }
    if (a.bias_ids) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t c = named[8 * tid + j];
            if (c) x[j] += a.bias_values[row * a.b + c - 1];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (!(allowed >> j & 1)) x[j] = -__builtin_inff();

    Raw<U> res;
    pack<U>(x, res);
    if (left >= 8) {
        __builtin_memcpy(out, &res, sizeof(res));
    } else {
        Elem<U> e[8];
        __builtin_memcpy(e, &res, sizeof(res));
        for (int j = 0; j < 8; ++j)
            if (j < left) out[j] = e[j];
    }
}

template <typename T, typename U>
hipError_t launch(Args a, int64_t m, hipStream_t stream) {
    const unsigned threads = 1024, width = 8 * threads;
    a.slices = unsigned((a.v + width - 1) / width);
    const unsigned lds = 4 * width * unsigned((a.history ? 1 : 0) + (a.bias_ids ? 1 : 0));
    hipLaunchKernelGGL((adjust_logits_kernel<T, U>), dim3(unsigned(m * a.slices)), dim3(threads), lds, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_out(const Args& a, int64_t m, int out_dtype, hipStream_t stream) {
    return out_dtype == TL_F32   ? launch<T, F32>(a, m, stream)
           : out_dtype == TL_F16 ? launch<T, F16>(a, m, stream)
                                 : launch<T, BF16>(a, m, stream);
}

}  // namespace

hipError_t launch_adjust_logits(const void* logits, int64_t m, int64_t v, int dtype, const int32_t* history,
                                int64_t h, const int32_t* history_lens, const int32_t* prompt_lens,
                                const float* repetition, const float* presence, const float* frequency,
                                const int32_t* bias_ids, const float* bias_values, int64_t b, const uint32_t* mask,
                                void* out, int out_dtype, hipStream_t stream) {
    // (a history of no tokens, or biases of none, are as good as absent)
    const Args a = {logits, h ? history : nullptr, history_lens, prompt_lens, repetition, presence, frequency,
                    b ? bias_ids : nullptr, bias_values, reinterpret_cast<const uint8_t*>(mask), out, v, h, b, 0};
    return dtype == TL_F32   ? launch_out<F32>(a, m, out_dtype, stream)
           : dtype == TL_F16 ? launch_out<F16>(a, m, out_dtype, stream)
                             : launch_out<BF16>(a, m, out_dtype, stream);
}

}  // namespace tl
