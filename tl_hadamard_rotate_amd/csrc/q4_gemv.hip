// Product of few tokens with 4-bit weights on the matrix cores:
//
//   y[m, n] = sum_g S[n, g] * sum_{k in g} code[n, k] * x[m, k]
//
// v_mfma_f32_16x16x32_f16 (8 bits: v_mfma_i32_16x16x64_i8, 16x16x32 for groups
// of 32) with 16 tokens as A rows and 16 weight rows as B columns.  Lane
// (q, c) = (lane / 16, lane % 16) loads the 16 bytes of row c that hold octets
// 4q .. 4q + 3 of a 128-weight chunk; two swaps across the quarters of the wave
// (v_permlane16_swap, v_permlane32_swap) hand it the octets q, q + 4, q + 8,
// q + 12 instead, so that each MFMA covers 32 (64) consecutive weights, which
// lie in one scale group, and reads the activations of 16 tokens in runs of 64
// bytes.  The sums of a group leave the matrix cores in fp32 (exact int32 for
// 8 bits) and are multiplied by the group's scale in fp32.
//
// Decode: a nibble n of two's complement is code + 8 = n ^ 8.  For binary16,
// (w & 0x000F000F) ^ 0x64086408 is the pair 1024 + (code + 8) and (w & 0x00F000F0)
// ^ 0x64806480 the pair 1024 + 16 (code + 8); one packed add or fma makes them
// the codes, exactly.  For 8 bits, w & 0xF0F0F0F0 and (w << 4) & 0xF0F0F0F0 are
// four signed bytes 16 * code each; the 1/16 goes into the scale.
//
// bfloat16 activations become binary16 under a power of two per token and
// chunk, chosen so that the largest of the chunk lies in [2^14, 2^15): 8
// significant bits fit exactly down to binary16's smallest normal number,
// 2^-28 of the largest; smaller ones are off by at most 2^-29 of it.  The
// power of two is applied to the sums, as the scales of 8-bit activations are.
//
// Work split: a workgroup owns 16 R weight rows and all of K; its waves split
// K into runs of chunks and add their partial sums through LDS in a fixed
// order.  A wave keeps D chunks of weights and activations on the way.
#include "elem.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef unsigned short ushort2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef int int4v __attribute__((ext_vector_type(4)));

constexpr int kMaxWaves = 8;

// a's upper half-wave exchanged with b's lower one; odd rows of 16 of a with
// even ones of b
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
    const auto s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = s[0];
    b = s[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto s = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = s[0];
    b = s[1];
}

// 8 codes of a word as binary16, in order
__device__ __forceinline__ half8v decode_f16(uint32_t w) {
    const half2v off = {_Float16(-1032.0f), _Float16(-1032.0f)};
    const half2v off16 = {_Float16(-72.0f), _Float16(-72.0f)};
    const half2v r16 = {_Float16(0.0625f), _Float16(0.0625f)};
    const uint32_t v = w >> 8;
    const half2v a = __builtin_bit_cast(half2v, (w & 0x000F000Fu) ^ 0x64086408u) + off;
    const half2v b = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (w & 0x00F000F0u) ^ 0x64806480u), r16, off16);
    const half2v c = __builtin_bit_cast(half2v, (v & 0x000F000Fu) ^ 0x64086408u) + off;
    const half2v d = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (v & 0x00F000F0u) ^ 0x64806480u), r16, off16);
    return half8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// What a lane holds of one 128-chunk of its token: 16-bit types, octet q + 4j
// in x[j]; 8 bits, the 16 bytes of octet pair q + 4j in x[j] (groups of 32:
// octet q + 4j in half of x[j / 2])
template <int XT>
struct Act {
    uint4 x[XT == TL_I8 ? 2 : 4];
    float scale;   // 8 bits only
};

template <int XT, int G>
__device__ __forceinline__ void load_act(const uint8_t* xp, const float* sp, int q, Act<XT>& a) {
    if constexpr (XT != TL_I8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) a.x[j] = *reinterpret_cast<const uint4*>(xp + 64 * j + 16 * q);
    } else if constexpr (G == 32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint2 u = *reinterpret_cast<const uint2*>(xp + 32 * j + 8 * q);
            if (j & 1) a.x[j >> 1].z = u.x, a.x[j >> 1].w = u.y;
            else a.x[j >> 1].x = u.x, a.x[j >> 1].y = u.y;
        }
        a.scale = *sp;
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) a.x[j] = *reinterpret_cast<const uint4*>(xp + 64 * j + 16 * q);
        a.scale = *sp;
    }
}

// bfloat16 -> binary16 times a power of two common to the token's chunk; the
// factor that undoes it
__device__ __forceinline__ float convert_bf16(uint4 (&x)[4]) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[4 * j] = x[j].x, w[4 * j + 1] = x[j].y, w[4 * j + 2] = x[j].z, w[4 * j + 3] = x[j].w;
    ushort2v top = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(ushort2v, w[i] & 0x7FFF7FFFu));
    uint32_t a = top[0] > top[1] ? top[0] : top[1], b = a;
    swap16(a, b);   // the other quarters' largest
    a = a > b ? a : b;
    b = a;
    swap32(a, b);
    a = a > b ? a : b;
    const int e = int(a >> 7);              // biased exponent of the largest
    const int d = e > 29 ? e - 29 : 0;      // it becomes 29 in binary16
    const unsigned short down = static_cast<unsigned short>(d << 7);
    const ushort2v dv = {down, down};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const ushort2v t = __builtin_bit_cast(ushort2v, w[i] & 0x7FFF7FFFu);
        const ushort2v u = __builtin_elementwise_sub_sat(t, dv) << static_cast<unsigned short>(3);
        w[i] = (w[i] & 0x80008000u) | __builtin_bit_cast(uint32_t, u);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = uint4{w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]};
    return e == 255 ? __builtin_nanf("") : __builtin_bit_cast(float, uint32_t(d + 15) << 23);
}

// 8-bit activations in the order of a decoded word: octets (0 4 1 5 2 6 3 7)
__device__ __forceinline__ void order_i8(uint4& v) {
    const uint32_t a = v.x, b = v.y, c = v.z, d = v.w;
    v.x = __builtin_amdgcn_perm(b, a, 0x05010400u);
    v.y = __builtin_amdgcn_perm(b, a, 0x07030602u);
    v.z = __builtin_amdgcn_perm(d, c, 0x05010400u);
    v.w = __builtin_amdgcn_perm(d, c, 0x07030602u);
}

template <int XT, int R, int MT>
struct Step {
    uint4 w[R];
    uint2 s[R];        // the chunk's 1, 2 or 4 binary16 scales of row c
    Act<XT> x[MT];
};

// y rows' sums of one chunk added to acc[r][t]: lane (q, c) holds weight row
// 16 r + c and tokens 16 t + 4 q .. + 3
template <int XT, int G, int R, int MT>
__device__ __forceinline__ void consume(Step<XT, R, MT>& st, int q, float4v (&acc)[R][MT]) {
    float f[MT][4];    // factors of the lane's four tokens (bfloat16, 8 bits)
    if constexpr (XT != TL_F16) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            float own;
            if constexpr (XT == TL_BF16) own = convert_bf16(st.x[t].x);
            else own = st.x[t].scale * 0.0625f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[t][i] = __builtin_bit_cast(
                    float, __builtin_amdgcn_ds_bpermute(4 * (4 * q + i), __builtin_bit_cast(int, own)));
            if constexpr (XT == TL_I8) {
                order_i8(st.x[t].x[0]);
                order_i8(st.x[t].x[1]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        uint32_t w[4] = {st.w[r].x, st.w[r].y, st.w[r].z, st.w[r].w};
        if constexpr (XT != TL_I8 || G == 32) {   // octets q, q + 4, q + 8, q + 12
            swap32(w[0], w[2]);
            swap32(w[1], w[3]);
            swap16(w[0], w[1]);
            swap16(w[2], w[3]);
        } else {                                  // octet pairs q, q + 4
            swap16(w[0], w[2]);
            swap16(w[1], w[3]);
            swap32(w[0], w[2]);
            swap32(w[1], w[3]);
        }
        constexpr int NS = 128 / G;               // scales of the chunk
        const uint32_t sb[2] = {st.s[r].x, st.s[r].y};
#pragma unroll
        for (int g = 0; g < NS; ++g) {
            const float s = float(__builtin_bit_cast(_Float16, uint16_t(sb[g >> 1] >> (16 * (g & 1)))));
            if constexpr (XT != TL_I8) {
                float4v d[MT] = {};
#pragma unroll
                for (int j = 4 / NS * g; j < 4 / NS * (g + 1); ++j) {
                    const half8v b = decode_f16(w[j]);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        d[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            __builtin_bit_cast(half8v, st.x[t].x[j]), b, d[t], 0, 0, 0);
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[r][t][i] = __builtin_fmaf(d[t][i], XT == TL_F16 ? s : s * f[t][i], acc[r][t][i]);
            } else {
                int4v d[MT] = {};
                if constexpr (G == 32) {
                    const uint32_t lo = (w[g] << 4) & 0xF0F0F0F0u, hi = w[g] & 0xF0F0F0F0u;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const uint4 xv = st.x[t].x[g >> 1];
                        const uint2 xo = (g & 1) ? uint2{xv.z, xv.w} : uint2{xv.x, xv.y};
                        d[t] = __builtin_amdgcn_mfma_i32_16x16x32_i8(
                            int64_t(uint64_t(xo.y) << 32 | xo.x), int64_t(uint64_t(hi) << 32 | lo), d[t], 0, 0, 0);
                    }
                } else {
#pragma unroll
                    for (int j = 2 / NS * g; j < 2 / NS * (g + 1); ++j) {
                        const int4v b = {int((w[2 * j] << 4) & 0xF0F0F0F0u), int(w[2 * j] & 0xF0F0F0F0u),
                                         int((w[2 * j + 1] << 4) & 0xF0F0F0F0u), int(w[2 * j + 1] & 0xF0F0F0F0u)};
#pragma unroll
                        for (int t = 0; t < MT; ++t)
                            d[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                                __builtin_bit_cast(int4v, st.x[t].x[j]), b, d[t], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[r][t][i] = __builtin_fmaf(float(d[t][i]), s * f[t][i], acc[r][t][i]);
            }
        }
    }
}

struct Args {
    const uint8_t* packed;
    const uint16_t* scales;
    const uint8_t* x;
    const float* xs;
    void* y;
    int64_t n, k;
    int m, y_dtype;
};

template <int XT, int G, int R, int MT, int D>
__global__ __launch_bounds__(64 * kMaxWaves) void q4_gemv_kernel(const Args p) {
    extern __shared__ __attribute__((aligned(16))) float red[];   // [wave][t][r][row][token]
    constexpr int kXB = XT == TL_I8 ? 1 : 2;
    constexpr int NS = 128 / G;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int waves = int(blockDim.x >> 6);
    const int q = lane >> 4, c = lane & 15;
    const int chunks = int(p.k / 128);
    const int row_bytes = int(p.k / 2);
    const int64_t n0 = int64_t(blockIdx.x) * (16 * R);
    const int rows = int(p.n - n0 < 16 * R ? p.n - n0 : 16 * R);
    const int64_t m0 = int64_t(blockIdx.y) * (16 * MT);
    const int tokens = int(p.m - m0 < 16 * MT ? p.m - m0 : 16 * MT);

    // rows and tokens that do not exist repeat the last one; their sums are
    // not stored
    const uint8_t* wt = p.packed + n0 * row_bytes;
    const uint16_t* st = p.scales + n0 * (int64_t(chunks) * NS);
    const uint8_t* xt = p.x + m0 * p.k * kXB;
    const float* xst = XT == TL_I8 ? p.xs + m0 * chunks : nullptr;
    uint32_t woff[R], soff[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = 16 * r + c < rows ? 16 * r + c : rows - 1;
        woff[r] = uint32_t(row) * uint32_t(row_bytes) + 16u * uint32_t(q);
        soff[r] = uint32_t(row) * uint32_t(chunks * NS);
    }
    uint32_t xoff[MT], xsoff[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int tok = 16 * t + c < tokens ? 16 * t + c : tokens - 1;
        xoff[t] = uint32_t(tok) * uint32_t(p.k) * kXB;
        xsoff[t] = uint32_t(tok) * uint32_t(chunks);
    }

    // this wave's chunks [beg, end)
    const int share = (chunks + waves - 1) / waves;
    const int beg = wave * share;
    const int end = beg + share < chunks ? beg + share : chunks;

    Step<XT, R, MT> ring[D];
    const auto load = [&](int g, Step<XT, R, MT>& s) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s.w[r] = *reinterpret_cast<const uint4*>(wt + int64_t(g) * 64 + woff[r]);
            const uint16_t* sp = st + int64_t(g) * NS + soff[r];
            if (NS == 1) s.s[r].x = *sp;
            else if (NS == 2) s.s[r].x = *reinterpret_cast<const uint32_t*>(sp);
            else s.s[r] = *reinterpret_cast<const uint2*>(sp);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
            load_act<XT, G>(xt + int64_t(g) * (128 * kXB) + xoff[t], XT == TL_I8 ? xst + g + xsoff[t] : nullptr, q,
                            s.x[t]);
    };
    float4v acc[R][MT] = {};
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (beg + d < end) load(beg + d, ring[d]);
    for (int g = beg; g < end; g += D)
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (g + d >= end) break;
            consume<XT, G, R, MT>(ring[d], q, acc);
            if (g + d + D < end) load(g + d + D, ring[d]);
        }

    // partial sums, then the waves added in order
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r)
            *reinterpret_cast<float4v*>(red + ((wave * MT + t) * R + r) * 256 + c * 16 + 4 * q) = acc[r][t];
    __syncthreads();
    for (int i = threadIdx.x; i < rows * tokens; i += int(blockDim.x)) {
        const int tok = i / rows, row = i - tok * rows;
        const float* src = red + ((tok >> 4) * R + (row >> 4)) * 256 + (row & 15) * 16 + (tok & 15);
        float v = 0.0f;
        for (int w = 0; w < waves; ++w) v += src[w * (MT * R * 256)];
        const int64_t at = (m0 + tok) * p.n + n0 + row;
        if (p.y_dtype == TL_F32) static_cast<float*>(p.y)[at] = v;
        else static_cast<uint16_t*>(p.y)[at] = uint16_t(p.y_dtype == TL_F16 ? f16_bits(v) : bf16_bits(v));
    }
}

struct Plan {
    int r, waves;
};

Plan q4_plan(int64_t, int64_t n, int64_t k) {
    const int64_t cus = cu_count();
    Plan p;
    p.r = n >= 64 * cus ? 4 : n >= 32 * cus ? 2 : 1;
    p.waves = k >= 8 * 128 ? 8 : int(k / 128);
    return p;
}

template <int XT, int G, int R, int MT>
hipError_t launch(const Args& a, int waves, hipStream_t stream) {
    constexpr int D = MT * R >= 8 ? 2 : MT * R >= 4 ? 3 : 4;
    const auto kernel = q4_gemv_kernel<XT, G, R, MT, D>;
    const int lds = waves * MT * R * 1024;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kMaxWaves * MT * R * 1024);
    if (e != hipSuccess) return e;
    const dim3 grid(unsigned((a.n + 16 * R - 1) / (16 * R)), unsigned((a.m + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), lds, stream, a);
    return hipGetLastError();
}

template <int XT, int G>
hipError_t launch_rows(const Args& a, const Plan& p, hipStream_t stream) {
    if (a.m <= 16) {
        if (p.r == 4) return launch<XT, G, 4, 1>(a, p.waves, stream);
        if (p.r == 2) return launch<XT, G, 2, 1>(a, p.waves, stream);
        return launch<XT, G, 1, 1>(a, p.waves, stream);
    }
    if (a.m <= 32) {
        if (p.r == 4) return launch<XT, G, 4, 2>(a, p.waves, stream);
        if (p.r == 2) return launch<XT, G, 2, 2>(a, p.waves, stream);
        return launch<XT, G, 1, 2>(a, p.waves, stream);
    }
    if (p.r >= 2) return launch<XT, G, 2, 4>(a, p.waves, stream);
    return launch<XT, G, 1, 4>(a, p.waves, stream);
}

}  // namespace

int64_t q4_gemv_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_q4_gemv(const uint8_t* packed, const uint16_t* scales, int group, const void* x,
                          int x_dtype, const float* x_scales, int64_t m, int64_t n, int64_t k, void* y,
                          int y_dtype, void*, hipStream_t stream) {
    // a grid's second dimension ends at 65535: at most 65535 * 16 tokens a launch
    constexpr int64_t kMaxTokens = 65535 * 16;
    const int64_t xb = x_dtype == TL_I8 ? 1 : 2, yb = y_dtype == TL_F32 ? 4 : 2;
    const Plan p = q4_plan(m, n, k);
    for (int64_t m0 = 0; m0 < m; m0 += kMaxTokens) {
        const int64_t mt = m - m0 < kMaxTokens ? m - m0 : kMaxTokens;
        const Args a = {packed, scales, static_cast<const uint8_t*>(x) + m0 * k * xb,
                        x_scales ? x_scales + m0 * (k / 128) : nullptr,
                        static_cast<uint8_t*>(y) + m0 * n * yb, n, k, int(mt), y_dtype};
#define TL_Q4_GROUP(XT)                                             \
    (group == 32   ? launch_rows<XT, 32>(a, p, stream)              \
     : group == 64 ? launch_rows<XT, 64>(a, p, stream)              \
                   : launch_rows<XT, 128>(a, p, stream))
        const hipError_t e = x_dtype == TL_I8    ? TL_Q4_GROUP(TL_I8)
                             : x_dtype == TL_F16 ? TL_Q4_GROUP(TL_F16)
                                                 : TL_Q4_GROUP(TL_BF16);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tl
