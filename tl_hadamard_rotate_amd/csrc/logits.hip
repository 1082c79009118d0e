// Logits made ready for drawing a token: penalties for tokens that occurred,
// biases, a grammar's mask.  For row m and token v, x in fp32:
//
//   seen   = v occurs among the row's history        x = x > 0 ? x / r : x * r   if seen
//   count  = its occurrences after the prompt        x = x - f * count - p (count > 0)
//   named  = the last bias of the row that names v   x = x + bias                if named
//   mask bit 0                                       x = -infinity
//
// A workgroup owns a slice of one row's tokens, 4 a lane and I times that.  It asks
// for its logits first; while they are on the way it goes through the row's whole
// history and biases and marks in LDS what falls into its slice: occurrences after
// the prompt counted, the prompt's in the top bit; the largest place of a bias that
// names the token.  Integer additions and maxima, whose order does not show.
#include <type_traits>

#include "elem.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;

struct Args {
    const void* logits;
    const int32_t *history, *history_lens, *prompt_lens;
    const float *repetition, *presence, *frequency;
    const int32_t* bias_ids;
    const float* bias_values;
    const uint8_t* mask;
    void* out;
    int64_t v, h, b, row0;       // row0: the launch's first row
    uint32_t slices;
    bool stream;                 // stores past the caches' replacement order
};

// 4 elements, at any alignment of the type (rows of an odd vocabulary)
template <typename T>
struct Raw {
    uint32_t w[T::kBytes];
};

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&x)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        x[j] = T::kType == TL_F32   ? __builtin_bit_cast(float, r.w[j % T::kBytes])
               : T::kType == TL_F16 ? float(__builtin_bit_cast(_Float16, uint16_t(r.w[j >> 1] >> (16 * (j & 1)))))
                                    : __builtin_bit_cast(float, j & 1 ? r.w[j >> 1] & 0xFFFF0000u : r.w[j >> 1] << 16);
}

template <typename T>
__device__ __forceinline__ void pack(const float (&x)[4], Raw<T>& r) {
    if constexpr (T::kType == TL_F32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r.w[j] = __builtin_bit_cast(uint32_t, x[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            r.w[j] = T::kType == TL_F16 ? f16_bits(x[2 * j]) | f16_bits(x[2 * j + 1]) << 16
                                        : bf16_pair(x[2 * j], x[2 * j + 1]);
    }
}

// ids [i, i + 4) of n, -1 past them
__device__ __forceinline__ int4 ids4(const int32_t* ids, uint32_t i, uint32_t n) {
    int4 v = {-1, -1, -1, -1};
    if (i + 4 <= n) {
        __builtin_memcpy(&v, ids + i, 16);
    } else if (i < n) {
        v.x = ids[i];
        if (i + 1 < n) v.y = ids[i + 1];
        if (i + 2 < n) v.z = ids[i + 2];
    }
    return v;
}

template <typename T>
using Elem = std::conditional_t<T::kBytes == 4, uint32_t, uint16_t>;

// What LDS holds of a token, 32 or 16 bits of it
template <bool WIDE>
struct Table {
    static constexpr uint32_t kBits = WIDE ? 32 : 16, kTop = 1u << (kBits - 1), kBytes = kBits / 8;
    uint32_t* words;

    __device__ __forceinline__ uint32_t shift(uint32_t d) const { return WIDE ? 0 : 16 * (d & 1); }
    __device__ __forceinline__ uint32_t* word(uint32_t d) const { return words + (WIDE ? d : d >> 1); }
    // one more after the prompt; in the prompt
    __device__ __forceinline__ void count(uint32_t d) const { atomicAdd(word(d), 1u << shift(d)); }
    __device__ __forceinline__ void note(uint32_t d) const { atomicOr(word(d), kTop << shift(d)); }
    __device__ __forceinline__ void raise(uint32_t d, uint32_t to) const {
        if (WIDE) {
            atomicMax(word(d), to);
        } else {    // half a word: tried again where the other half, or this one, was changed meanwhile
            uint32_t was = *word(d);
            while ((was >> shift(d) & 0xFFFFu) < to) {
                const uint32_t now = atomicCAS(word(d), was, (was & ~(0xFFFFu << shift(d))) | to << shift(d));
                if (now == was) break;
                was = now;
            }
        }
    }
    // of 4 tokens from d (a multiple of 4)
    __device__ __forceinline__ void get4(uint32_t d, uint32_t (&v)[4]) const {
        if (WIDE) {
            const uint4 w = *reinterpret_cast<const uint4*>(word(d));
            v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(word(d));
            v[0] = w.x & 0xFFFFu, v[1] = w.x >> 16, v[2] = w.y & 0xFFFFu, v[3] = w.y >> 16;
        }
    }
};

// 4 elements as one vector, aligned as an element is (of a copy of bytes the compiler
// makes stores of 12 and 4 bytes, one of them shared with the row's end)
template <typename U>
using Vector = uint32_t __attribute__((ext_vector_type(U::kBytes), aligned(U::kBytes)));

template <typename U>
__device__ __forceinline__ Vector<U> as_vector(const Raw<U>& r) {
    Vector<U> v;
#pragma unroll
    for (int j = 0; j < U::kBytes; ++j) v[j] = r.w[j];
    return v;
}

template <typename T, typename U, int I, bool WIDE>
__global__ __launch_bounds__(1024) void adjust_logits_kernel(const Args a) {
    extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
    const uint32_t tid = threadIdx.x, threads = blockDim.x, width = 4 * I * threads;
    const uint32_t at_row = blockIdx.x / a.slices;
    const int64_t row = a.row0 + at_row;
    const uint32_t first = (blockIdx.x - at_row * a.slices) * width;     // token of the slice
    const uint32_t v = uint32_t(a.v);
    const Elem<T>* in = static_cast<const Elem<T>*>(a.logits) + row * a.v;
    Elem<U>* out = static_cast<Elem<U>*>(a.out) + row * a.v;
    const uint8_t* mask = a.mask ? a.mask + row * ((a.v + 31) / 32 * 4) : nullptr;

    Raw<T> raw[I];
    uint32_t allowed[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const uint32_t at = first + 4 * (tid + i * threads);
        raw[i] = Raw<T>{};
        if (at + 4 <= v) {
            __builtin_memcpy(&raw[i], in + at, sizeof(raw[i]));
        } else if (at < v) {
            Elem<T> e[4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (at + j < v) e[j] = in[at + j];
            __builtin_memcpy(&raw[i], e, sizeof(raw[i]));
        }
        allowed[i] = mask && at < v ? mask[at >> 3] >> (at & 4) : 0xFu;
    }

    const Table<WIDE> counts{lds}, named{lds + (a.history ? width * Table<WIDE>::kBytes / 4 : 0)};
    if (a.history || a.bias_ids) {
        // the first ids are asked for before anything waits, whatever the row's length
        // (the buffer has them), and looked at once LDS is clear
        const int32_t* ids = a.history + row * a.h;
        const int32_t* bias_ids = a.bias_ids + row * a.b;
        int4 next[2];
        int32_t next_bias = -1;
        uint32_t len = uint32_t(a.h);
        int64_t prompt = 0;
        if (a.history) {
#pragma unroll
            for (int j = 0; j < 2; ++j) next[j] = ids4(ids, 4 * (tid + j * threads), len);
            if (a.history_lens) {
                const int32_t n = a.history_lens[row];
                len = n < 0 ? 0 : uint32_t(n) < len ? uint32_t(n) : len;
            }
            if (a.prompt_lens) prompt = a.prompt_lens[row];
        }
        if (a.bias_ids && tid < a.b) next_bias = bias_ids[tid];
        const uint32_t quads = (a.history && a.bias_ids ? 2 : 1) * (width * Table<WIDE>::kBytes / 16);
        for (uint32_t i = tid; i < quads; i += threads) reinterpret_cast<uint4*>(lds)[i] = uint4{0, 0, 0, 0};
        __syncthreads();
        // (an id outside the slice, a negative one too, is far from its first token)
        if (a.history) {
            const auto mark = [&](int32_t id, uint32_t at) {
                const uint32_t d = uint32_t(id) - first;
                if (d < width && at < len) {
                    if (at >= prompt) counts.count(d);
                    else counts.note(d);
                }
            };
            for (uint32_t i = 4 * tid; i < len; i += 8 * threads) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t at = i + 4 * j * threads;
                    mark(next[j].x, at);
                    mark(next[j].y, at + 1);
                    mark(next[j].z, at + 2);
                    mark(next[j].w, at + 3);
                    next[j] = ids4(ids, at + 8 * threads, len);
                }
            }
        }
        if (a.bias_ids) {
            for (uint32_t i = tid; i < a.b; i += threads) {
                const uint32_t d = uint32_t(next_bias) - first;
                if (d < width) named.raise(d, i + 1);
                if (i + threads < a.b) next_bias = bias_ids[i + threads];
            }
        }
        __syncthreads();
    }

    const float r = a.repetition ? a.repetition[row] : 1.0f;
    const float p = a.presence ? a.presence[row] : 0.0f;
    const float f = a.frequency ? a.frequency[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const uint32_t d = 4 * (tid + i * threads), at = first + d;
        if (at >= v) break;
        float x[4];
        unpack<T>(raw[i], x);
        if (a.history) {
            uint32_t c[4];
            counts.get4(d, c);
            if (c[0] | c[1] | c[2] | c[3]) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t n = c[j] & (Table<WIDE>::kTop - 1);
                    if (a.repetition && c[j]) x[j] = x[j] > 0.0f ? x[j] / r : x[j] * r;
                    if (n) x[j] = x[j] - f * float(n) - p;
                }
            }
        }
        if (a.bias_ids) {
            uint32_t c[4];
            named.get4(d, c);
            if (c[0] | c[1] | c[2] | c[3]) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c[j]) x[j] += a.bias_values[row * a.b + c[j] - 1];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (!(allowed[i] >> j & 1)) x[j] = -__builtin_inff();

        Raw<U> res;
        pack<U>(x, res);
        if (at + 4 <= v) {
            Vector<U>* const to = reinterpret_cast<Vector<U>*>(out + at);
            if (a.stream) {     // (the empty statements keep the compiler from making one plain store of both)
                asm volatile("");
                __builtin_nontemporal_store(as_vector(res), to);
                asm volatile("");
            } else {
                *to = as_vector(res);
            }
        } else {
            Elem<U> e[4];
            __builtin_memcpy(e, &res, sizeof(res));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (at + j < v) out[at + j] = e[j];
        }
    }
}

template <typename T, typename U, int I, bool WIDE>
hipError_t launch(Args a, int64_t m, unsigned threads, hipStream_t stream) {
    const auto kernel = adjust_logits_kernel<T, U, I, WIDE>;
    const unsigned width = 4 * I * threads;
    const unsigned lds = Table<WIDE>::kBytes * width * unsigned((a.history ? 1 : 0) + (a.bias_ids ? 1 : 0));
    static_assert(Table<WIDE>::kBytes * 4 * I * 1024 * 2 <= 64 * 1024, "LDS");
    a.slices = unsigned((a.v + width - 1) / width);
    const int64_t most = (int64_t(1) << 31) / threads / a.slices;   // rows of a launch, whose lanes count in 32 bits
    for (a.row0 = 0; a.row0 < m; a.row0 += most) {
        const int64_t left = m - a.row0 < most ? m - a.row0 : most;
        hipLaunchKernelGGL(kernel, dim3(unsigned(left * a.slices)), dim3(threads), lds, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// 16 bits hold a count below 32768 and a place below 65536.  Every workgroup goes
// through the whole history, so slices are long (16384 tokens) where that leaves two
// workgroups a compute unit, short where there are few rows and little history.  us in
// a graph, slices of 2048, 8192, 16384, 32768 tokens: 64 rows of 131072 bfloat16 to
// float32 logits, 8192 ids, 300 biases 22.7 18.3 16.8 17.9; one row of float32, 2048
// ids, 16 biases 4.6 5.3 7.2 10.7.  The first moves 52 MB: the reads overlap the ids
// of the history, the stores (33 MB, 6 us) begin when those are done.
// Outputs of half the 256 MB last-level cache and more are stored past the caches'
// replacement order, us alone and with a maximum over each row behind: 512 rows of
// 131072 float32 94 and 145 (99 and 153), 256 37 and 86 (49 and 93); 128 20 and 58 (22
// and 47), 64 14.8 and 53 (17 and 41).
template <typename T, typename U>
hipError_t launch_sized(const Args& a, int64_t m, hipStream_t stream) {
    const int64_t cus = cu_count(), slots = m * ((a.v + 8191) / 8192);
    if (a.h >= 32768 || a.b >= 65536) return launch<T, U, 2, true>(a, m, 1024, stream);
    if ((a.history || a.bias_ids) && slots >= 4 * cus) return launch<T, U, 4, false>(a, m, 1024, stream);
    return launch<T, U, 2, false>(a, m, slots < cus && a.h <= 4096 ? 256 : 1024, stream);
}

template <typename T>
hipError_t launch_out(const Args& a, int64_t m, int out_dtype, hipStream_t stream) {
    return out_dtype == TL_F32   ? launch_sized<T, F32>(a, m, stream)
           : out_dtype == TL_F16 ? launch_sized<T, F16>(a, m, stream)
                                 : launch_sized<T, BF16>(a, m, stream);
}

}  // namespace

hipError_t launch_adjust_logits(const void* logits, int64_t m, int64_t v, int dtype, const int32_t* history,
                                int64_t h, const int32_t* history_lens, const int32_t* prompt_lens,
                                const float* repetition, const float* presence, const float* frequency,
                                const int32_t* bias_ids, const float* bias_values, int64_t b, const uint32_t* mask,
                                void* out, int out_dtype, hipStream_t stream) {
    // (a history of no tokens, or biases of none, are as good as absent)
    const Args a = {logits, h ? history : nullptr, history_lens, prompt_lens, repetition, presence, frequency,
                    b ? bias_ids : nullptr, bias_values, reinterpret_cast<const uint8_t*>(mask), out, v, h, b, 0, 0,
                    m * v * (out_dtype == TL_F32 ? 4 : 2) >= int64_t(1) << 27};
    return dtype == TL_F32   ? launch_out<F32>(a, m, out_dtype, stream)
           : dtype == TL_F16 ? launch_out<F16>(a, m, out_dtype, stream)
                             : launch_out<BF16>(a, m, out_dtype, stream);
}

}  // namespace tl
