// Product of few tokens with 4-bit weights on the matrix cores:
//
//   y[m, n] = sum_g S[n, g] * sum_{k in g} code[n, k] * x[m, k]
//
// v_mfma_f32_16x16x32_f16 (8 bits: v_mfma_i32_16x16x64_i8, 16x16x32 for groups
// of 32) with 16 tokens as A rows and 16 weight rows as B columns.  Lane
// (q, c) = (lane / 16, lane % 16) loads the 16 bytes of row c that hold octets
// 4q .. 4q + 3 of a 128-weight chunk.  Which weights a matrix instruction sums
// is free as long as they share a scale and both operands agree: in groups of
// 128 the four octets go in as loaded, in groups of 64 (32) one (two) swaps
// across the quarters of the wave bring the octets of a group together.  The
// sums of a group leave the matrix cores in fp32 (exact int32 for 8 bits) and
// are multiplied by the group's scale in fp32.
//
// Decode.  A nibble n of two's complement is code + 8 = n ^ 8.  For 16-bit
// activations, (w & 0x000F000F) ^ 0x64086408 is the binary16 pair 1024 + (code
// + 8) and (w & 0x00F000F0) ^ 0x64806480 the pair 1024 + 16 (code + 8); one
// packed add or fma makes them the codes, exactly: the known way to widen
// interleaved 4-bit integers through the mantissa of 1024 + n.  (Feeding code + 8 as a
// subnormal pattern and taking the 8 off the sums saves those, but then rows
// of small codes carry the rounding errors of 8 * sum x.)  For 8 bits, w &
// 0xF0F0F0F0 and (w << 4) & 0xF0F0F0F0 are four signed bytes 16 * code each;
// the 1/16 goes into the scale.
//
// bfloat16 activations become binary16 under a power of two per token and
// chunk, chosen so that the largest of the chunk lies in [2^14, 2^15): 8
// significant bits fit exactly down to binary16's smallest normal number,
// 2^-28 of the largest; smaller ones are off by at most 2^-29 of it.  The
// power of two is applied to the sums, as the scales of 8-bit activations are.
//
// Work split.  K is cut into `parts` of L chunks such that the activations of
// a part fit in LDS; a workgroup stages one part once and each of its waves
// then goes through tiles of 16 weight rows on its own, without a barrier,
// its weights in a ring of D chunks that is refilled in pairs, 128 bytes of a row
// at a time (one chunk at a time: 131072 x 5120 of one token 66 us, 62.5 in
// pairs).  Where rows are few, KS waves share a tile,
// each a run of the part's chunks, and add their sums through LDS.  With
// several parts the sums go to the workspace and a second kernel adds them.
// All sums are taken in a fixed order.  A tile's scales, one run of memory or
// a piece of each row, go through the wave's own LDS, SEG chunks at a time:
// read as they are used, 2 bytes from each of 16 rows, they took longer than
// the weights.  Both come by loads that write LDS directly (through registers
// they waited for one another), in places of 16 (4) bytes a lane in order; the
// pieces of a token's activations are exchanged by 3 bits of its number, so
// that 8 tokens at one place lie on different banks.
//
// Bound.  One token: the weights' bytes from HBM (131072 x 5120 in groups of 128,
// 346 MB, 60.6 us, 5.7 TB/s; a plain read of as much 55 us).  Few tokens: besides
// that the staging of a part's activations, which every workgroup does before its
// first product, and the second kernel (5120 x 17408 by 8 bfloat16 tokens, 47 MB,
// 19.1 us; traced one by one, 21.5 and 4.1).  From some 40 tokens on the
// instructions: decoding, and one fma for each group, token and row (32003 x 5120
// in groups of 32 by 45 tokens, 42.7 us, traced 40.2 and 5.8: counters give 18.6
// us of vector and 6.3 of matrix instructions on each SIMD and 13.1 us of LDS
// reads on each compute unit, 6.5 of them bank conflicts, which two waves a SIMD
// overlap little).  Narrow matrices from 17 tokens on: the split leaves most
// compute units idle (1024 x 5120 by 20 8-bit tokens 12.4 us in 16 workgroups; by
// 16 tokens 7.5 us).
#include <cmath>

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
typedef unsigned int uint4v __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;    // of a workgroup

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

// value of lane ^ 1, lane ^ 2, the other four of 8, the other 8 of 16
template <int STEP>
__device__ __forceinline__ uint32_t row16(uint32_t a) {
    constexpr int kCtrl[4] = {0xB1, 0x4E, 0x141, 0x140};
    return uint32_t(__builtin_amdgcn_mov_dpp(int(a), kCtrl[STEP], 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t row16_max(uint32_t a) {
    const auto step = [&](uint32_t o) { a = o > a ? o : a; };
    step(row16<0>(a));
    step(row16<1>(a));
    step(row16<2>(a));
    step(row16<3>(a));
    return a;
}

// 8 bfloat16 values of a lane, 128 of its row of 16 lanes, to binary16 times a
// power of two common to the 128; returns the factor that undoes it
__device__ __forceinline__ float convert_bf16(uint4v& v) {
    uint32_t w[4] = {v[0], v[1], v[2], v[3]};
    ushort2v top = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(ushort2v, w[i] & 0x7FFF7FFFu));
    const int e = int(row16_max(top[0] > top[1] ? top[0] : top[1]) >> 7);   // biased exponent of the largest
    const int d = e > 29 ? e - 29 : 0;      // it becomes 29 in binary16
    const unsigned short down = static_cast<unsigned short>(d << 7);
    const ushort2v dv = {down, down};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ushort2v t = __builtin_bit_cast(ushort2v, w[i] & 0x7FFF7FFFu);
        const ushort2v u = __builtin_elementwise_sub_sat(t, dv) << static_cast<unsigned short>(3);
        w[i] = (w[i] & 0x80008000u) | __builtin_bit_cast(uint32_t, u);
    }
    v = uint4v{w[0], w[1], w[2], w[3]};
    return e == 255 ? __builtin_nanf("") : __builtin_bit_cast(float, uint32_t(d + 15) << 23);
}

// 8-bit activations in the order of a decoded word: octets (0 4 1 5 2 6 3 7)
__device__ __forceinline__ void order_i8(uint4v& v) {
    const uint32_t a = v[0], b = v[1], c = v[2], d = v[3];
    v = uint4v{__builtin_amdgcn_perm(b, a, 0x05010400u), __builtin_amdgcn_perm(b, a, 0x07030602u),
               __builtin_amdgcn_perm(d, c, 0x05010400u), __builtin_amdgcn_perm(d, c, 0x07030602u)};
}

// a load of B bytes a lane that writes LDS itself, lane i at l + max(B, 4) * i
template <int B>
__device__ __forceinline__ void load_lds(const void* g, void* l) {
    const auto from = (const __attribute__((address_space(1))) void*)g;
    const auto to = (__attribute__((address_space(3))) void*)l;
    if constexpr (B == 16) __builtin_amdgcn_global_load_lds(from, to, 16, 0, 0);
    else if constexpr (B == 4) __builtin_amdgcn_global_load_lds(from, to, 4, 0, 0);
    else __builtin_amdgcn_global_load_lds(from, to, 2, 0, 0);
}

// Wait until at most N loads are on the way.  By the builtin, which the compiler
// counts: behind a wait it cannot see, it takes the loads into LDS for pending
// and waits for every later load before it reads LDS.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | 15 << 8 | (N >> 4) << 14);
    asm volatile("" ::: "memory");
}

// Octets of the chunk that lane quarter q and (16 bits, or groups of 32) word
// j, (8 bits) pair of words j, meet in: first_octet(q) + octet_step(j)
template <int G>
__device__ __forceinline__ int first_octet(int q) {
    return G == 128 ? 4 * q : G == 64 ? 4 * (q & 1) + 2 * (q >> 1) : q;
}
template <int G>
constexpr int octet_step(int j, bool pair) {
    if (pair) return G == 128 ? 2 * j : 8 * j;
    return G == 128 ? j : G == 64 ? 8 * (j >> 1) + (j & 1) : 4 * j;
}

template <int XT>
constexpr int chunk_bytes() { return XT == TL_I8 ? 128 : 256; }
// fp32 factors a chunk has per token beside its activations (bfloat16, 8 bits)
template <int XT>
constexpr int chunk_floats() { return XT == TL_F16 ? 0 : 1; }

// One chunk's sums added to acc[t]: lane (q, c) holds weight row c and tokens
// 16 t + 4 q .. + V - 1.  In LDS: xa[t] the lane's token's activations (xsw[t]
// in the offset: where the lane starts, exchanged by the token's bits), fa[t]
// the chunk's factors of tokens 16 t + 4 q .. + 3, sc its scales of row c.
template <int XT, int G, int MT, int V>
__device__ __forceinline__ void consume(const uint4v& wr, const uint8_t* const (&xa)[MT], const int (&xsw)[MT],
                                        const uint8_t* sc, const float* const (&fa)[MT], float (&acc)[MT][V]) {
    constexpr int NS = 128 / G;               // scales of the chunk
    constexpr bool kPair = XT == TL_I8 && G != 32;
    constexpr int NX = kPair ? 2 : 4;         // matrix instructions along K
    uint32_t w[4] = {wr[0], wr[1], wr[2], wr[3]};
    if constexpr (G != 128) {
        swap32(w[0], w[2]);
        swap32(w[1], w[3]);
    }
    if constexpr (G == 32) {
        swap16(w[0], w[1]);
        swap16(w[2], w[3]);
    }
    float4v f[MT];
    if constexpr (XT != TL_F16)
#pragma unroll
        for (int t = 0; t < MT; ++t)
            f[t] = *reinterpret_cast<const float4v*>(fa[t]);
    uint32_t sb[2] = {};
    if constexpr (NS == 1) sb[0] = *reinterpret_cast<const uint16_t*>(sc);
    else if constexpr (NS == 2) sb[0] = *reinterpret_cast<const uint32_t*>(sc);
    else {
        const uint2 u = *reinterpret_cast<const uint2*>(sc);
        sb[0] = u.x, sb[1] = u.y;
    }
    float s[NS];
#pragma unroll
    for (int g = 0; g < NS; ++g)
        s[g] = float(__builtin_bit_cast(_Float16, uint16_t(sb[g >> 1] >> (16 * (g & 1))))) *
               (XT == TL_I8 ? 0.0625f : 1.0f);
    float4v d[MT];
    int4v di[MT];
#pragma unroll
    for (int j = 0; j < NX; ++j) {
        const bool first = j % (NX / NS) == 0, last = (j + 1) % (NX / NS) == 0;
        const int g = j / (NX / NS);
        constexpr int kOctet = XT == TL_I8 ? 8 : 16;   // bytes
        const int at = kOctet * octet_step<G>(j, kPair);
        if constexpr (XT != TL_I8) {
            half8v a[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) a[t] = *reinterpret_cast<const half8v*>(xa[t] + (at ^ xsw[t]));
            const half8v b = decode_f16(w[j]);
#pragma unroll
            for (int t = 0; t < MT; ++t)
                d[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[t], b, first ? float4v{} : d[t], 0, 0, 0);
        } else if constexpr (!kPair) {
            const uint32_t lo = (w[j] << 4) & 0xF0F0F0F0u, hi = w[j] & 0xF0F0F0F0u;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint2 v = *reinterpret_cast<const uint2*>(xa[t] + (at ^ xsw[t]));
                const uint32_t xl = __builtin_amdgcn_perm(v.y, v.x, 0x05010400u);
                const uint32_t xh = __builtin_amdgcn_perm(v.y, v.x, 0x07030602u);
                di[t] = __builtin_amdgcn_mfma_i32_16x16x32_i8(int64_t(uint64_t(xh) << 32 | xl),
                                                              int64_t(uint64_t(hi) << 32 | lo),
                                                              first ? int4v{} : di[t], 0, 0, 0);
            }
        } else {
            const uint32_t u = w[2 * j], v = w[2 * j + 1];
            const int4v b = {int((u << 4) & 0xF0F0F0F0u), int(u & 0xF0F0F0F0u), int((v << 4) & 0xF0F0F0F0u),
                             int(v & 0xF0F0F0F0u)};
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                uint4v x = *reinterpret_cast<const uint4v*>(xa[t] + (at ^ xsw[t]));
                order_i8(x);
                di[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(int4v, x), b,
                                                              first ? int4v{} : di[t], 0, 0, 0);
            }
        }
        if (last)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float v;
                    if constexpr (XT == TL_I8) v = float(di[t][i]);
                    else v = d[t][i];
                    acc[t][i] = __builtin_fmaf(v, XT == TL_F16 ? s[g] : s[g] * f[t][i], acc[t][i]);
                }
    }
}

struct Args {
    const uint8_t* packed;
    const uint16_t* scales;
    const uint8_t* x;
    const float* xs;
    void* y;
    float* sums;     // parts > 1: fp32 [part][m][n], parts sums_stride(m * n) apart
    int64_t n, k;
    int m, y_dtype;
    // parts of L chunks; KS waves share a tile, LW = ceil(L / KS) chunks each;
    // tiles of 16 rows, row groups (workgroups of a part); chunks whose
    // scales a wave has in LDS at a time, and their bytes
    int parts, l, ks, lw, tiles, groups, seg, s_bytes;
};

// floats from one part's sums to the next's, which start on 16 bytes
__host__ __device__ constexpr int64_t sums_stride(int64_t count) { return (count + 3) / 4 * 4; }

__device__ __forceinline__ void store_y(void* y, int64_t at, float v, int y_dtype) {
    if (y_dtype == TL_F32) static_cast<float*>(y)[at] = v;
    else static_cast<uint16_t*>(y)[at] = uint16_t(y_dtype == TL_F16 ? f16_bits(v) : bf16_bits(v));
}

template <int XT, int G, int MT, int D, int V>
__global__ __launch_bounds__(64 * kWaves, MT == 1 ? 4 : 2) void q4_gemv_kernel(const Args p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    constexpr int kCB = chunk_bytes<XT>();
    constexpr int kPieces = kCB / 16;         // 16-byte pieces of a token's chunk
    constexpr int kF = chunk_floats<XT>();
    constexpr int NS = 128 / G;
    const int tid = threadIdx.x, threads = int(blockDim.x);
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = threads >> 6;
    const int q = lane >> 4, c = lane & 15;
    const int chunks = int(p.k / 128);
    const int row_bytes = int(p.k / 2);
    const int part = int(blockIdx.x) % p.parts, group = int(blockIdx.x) / p.parts;
    const int ks = wave % p.ks, tw = wave / p.ks, tws = waves / p.ks;
    const int64_t m0 = int64_t(blockIdx.y) * (16 * MT);
    const int tokens = int(p.m - m0 < 16 * MT ? p.m - m0 : 16 * MT);
    // the part's chunks [c0, c0 + len), this wave's [w0, w0 + mine) of them
    const int c0 = part * p.l;
    const int len = chunks - c0 < p.l ? chunks - c0 : p.l;
    const int w0 = ks * p.lw;
    const int left = len - w0;
    const int mine = left < 0 ? 0 : left < p.lw ? left : p.lw;

    // LDS: activations [token][chunk], factors [chunk][TS], TS the tokens
    // rounded up to fours, the waves' scales [row][chunk]; at the end partial sums (KS > 1)
    const int xstride = len * kCB;
    const int ts = (tokens + 3) / 4 * 4;
    uint8_t* const lx = smem;
    float* const lf = reinterpret_cast<float*>(lx + tokens * p.l * kCB);
    uint8_t* const ls = reinterpret_cast<uint8_t*>(lf + p.l * (kF * ts)) + wave * p.s_bytes;
    float* const red = reinterpret_cast<float*>(smem);

    // this wave's tiles: tile, tile + stride, ...
    const int stride = p.groups * tws;
    int tile = group * tws + tw;

    // Weights on the way: D chunks of a tile.  voff: the lane's row of the tile
    // (rows that do not exist repeat the last one; their sums are not stored).
    uint4v buf[D];
    uint32_t voff = 0;
    const auto enter = [&](int t) {
        const int64_t n0 = int64_t(t) * 16;
        const int last = int(p.n - n0 < 16 ? p.n - n0 : 16) - 1;
        voff = uint32_t(c < last ? c : last) * uint32_t(row_bytes) + 16u * uint32_t(q);
        return p.packed + (n0 * row_bytes + int64_t(c0 + w0) * 64);
    };
    // chunk i into place d (past the end the last one again)
    const auto fetch = [&](const uint8_t* b, int i, int d) {
        buf[d] = *reinterpret_cast<const uint4v*>(b + 64 * (i < mine ? i : mine - 1) + voff);
    };
    const auto fetch_first = [&](const uint8_t* b) {
#pragma unroll
        for (int d = 0; d < D; ++d) fetch(b, d, d);
    };
    // Scales of chunks [i0, i0 + SEG) of this wave's of a tile into its LDS,
    // [row][chunk]: one run of memory when they are all of the rows, else
    // places of 4 bytes (a scale, or two)
    constexpr int kPlaces = NS > 2 ? NS / 2 : 1;
    const auto load_s = [&](int t, int i0) {
        const int64_t n0 = int64_t(t) * 16;
        const int rows = int(p.n - n0 < 16 ? p.n - n0 : 16);
        const int span = mine - i0 < p.seg ? mine - i0 : p.seg;
        const uint16_t* const src = p.scales + (n0 * chunks + c0 + w0 + i0) * NS;
        if (span == chunks) {
            const int count = rows * span * NS;
            for (int i = 0; i < count / 8; i += 64)
                if (i + lane < count / 8) load_lds<16>(src + 8 * (i + lane), ls + 16 * i);
            const int tail = count / 8 * 8 + lane;   // the end of the scales
            if (tail < count) reinterpret_cast<uint16_t*>(ls)[tail] = src[tail];
        } else {
            const int per_row = span * kPlaces, count = rows * per_row;
            const float inv = 1.0f / float(per_row);
            for (int i = 0; i < count; i += 64) {
                const int u = i + lane, row = int((float(u) + 0.5f) * inv);   // exact: u < 2^16
                if (u < count)
                    load_lds<NS == 1 ? 2 : 4>(src + int64_t(row) * (chunks * NS) + (u - row * per_row) * (NS == 1 ? 1 : 2),
                                              ls + 4 * i);
            }
        }
    };
    const bool work = tile < p.tiles && mine > 0;
    const uint8_t* base = p.packed;

    // the part's activations (and their scales) to LDS
    {
        const uint8_t* const xt = p.x + (m0 * p.k + int64_t(c0) * 128) * (kCB / 128);
        const int per_token = len * kPieces, count = tokens * per_token;
        const float inv = 1.0f / float(per_token);
        for (int i = 64 * wave; i < count; i += threads) {
            const int u = i + lane, t = int((float(u) + 0.5f) * inv);   // exact: u < 2^16
            if (u < count)
                load_lds<16>(xt + int64_t(t) * p.k * (kCB / 128) + 16 * ((u - t * per_token) ^ (t & 7)), lx + 16 * i);
        }
        if constexpr (XT == TL_I8)
            for (int i = 64 * wave; i < len * ts; i += threads) {
                const int u = i + lane, slot = u / ts, t = u - slot * ts;
                if (slot < len && t < tokens) load_lds<4>(p.xs + (m0 + t) * chunks + c0 + slot, lf + i);
            }
    }
    if (work) {
        load_s(tile, 0);
        base = enter(tile);
        fetch_first(base);
    }
    wait_loads<0>();
    __syncthreads();
    if constexpr (XT == TL_BF16) {
        const int count = tokens * len;   // (token, chunk), a row of 16 lanes each
        const float inv = 1.0f / float(len);
        for (int i = tid >> 4; i < count; i += threads >> 4) {
            uint4v* const at = reinterpret_cast<uint4v*>(lx) + 16 * i + c;
            uint4v v = *at;
            const float f = convert_bf16(v);
            *at = v;
            const int t = int((float(i) + 0.5f) * inv);   // exact: i < 2^16
            if (c == 0) lf[(i - t * len) * ts + t] = f;
        }
        __syncthreads();
    }

    const uint8_t* xa[MT];
    int xsw[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int tok = 16 * t + c < tokens ? 16 * t + c : tokens - 1;   // absent tokens repeat the last
        xa[t] = lx + tok * xstride + w0 * kCB;
        xsw[t] = (first_octet<G>(q) * (XT == TL_I8 ? 8 : 16)) ^ (16 * (tok & 7));
    }
    const float* fa[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t)   // (factors of absent tokens: any)
        fa[t] = lf + w0 * (kF * ts) + (16 * t + 4 * q < ts ? 16 * t + 4 * q : ts - 4);
    for (; tile < p.tiles; tile += stride) {
        float acc[MT][V] = {};
        const int64_t n0 = int64_t(tile) * 16;
        const int rows = int(p.n - n0 < 16 ? p.n - n0 : 16);
        const bool more = tile + stride < p.tiles;
        int seg0 = 0;
        for (int i0 = 0; i0 < mine;) {
            if (i0 == seg0 + p.seg) {
                seg0 = i0;
                load_s(tile, seg0);
                wait_loads<0>();
            }
            const int span = mine - seg0 < p.seg ? mine - seg0 : p.seg;
            const int s_step = span == chunks ? 2 * NS : 4 * kPlaces, row_step = span * s_step;   // bytes
            const uint8_t* const sc = ls + c * row_step - seg0 * s_step;
            const auto step = [&](int i, const uint4v& w) {
                const uint8_t* xc[MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) xc[t] = xa[t] + i * kCB;
                const float* fc[MT];
#pragma unroll
                for (int t = 0; t < MT; ++t) fc[t] = fa[t] + i * (kF * ts);
                consume<XT, G, MT, V>(w, xc, xsw, sc + i * s_step, fc, acc);
            };
            if (i0 + D < mine) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    step(i0 + d, buf[d]);
                    if (d & 1) fetch(base, i0 + D + d - 1, d - 1);
                    if ((d & 1) || d == D - 1) fetch(base, i0 + D + d, d);
                }
            } else {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    if (i0 + d >= mine) break;
                    step(i0 + d, buf[d]);
                }
            }
            i0 += D;
        }
        if (p.ks > 1) {
            // (one tile a wave then)
            __syncthreads();
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < V; ++i) red[(wave * MT + t) * 256 + (4 * q + i) * 16 + c] = acc[t][i];
            break;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int tok = 16 * t + 4 * q + i;
                if (c >= rows || tok >= tokens) continue;
                const int64_t at = (m0 + tok) * p.n + n0 + c;
                if (p.parts > 1) p.sums[part * sums_stride(int64_t(p.m) * p.n) + at] = acc[t][i];
                else store_y(p.y, at, acc[t][i], p.y_dtype);
            }
        if (more) {
            // the next tile's scales (the old ones have been read), then its
            // weights; all but the latter are awaited
            load_s(tile + stride, 0);
            asm volatile("" ::: "memory");
            base = enter(tile + stride);
            fetch_first(base);
            wait_loads<D>();
        }
    }
    if (p.ks > 1) {
        // waves without a tile meet the others at both barriers
        if (tile >= p.tiles) __syncthreads();
        __syncthreads();
        const int64_t n0 = int64_t(group) * tws * 16;
        const int rows = int(p.n - n0 < tws * 16 ? p.n - n0 : tws * 16);
        for (int o = tid; o < rows * tokens; o += threads) {
            const int tok = o / rows, row = o - tok * rows;
            const float* src = red + ((row / 16 * p.ks) * MT + (tok >> 4)) * 256 + (tok & 15) * 16 + row % 16;
            float v = 0.0f;
            for (int w = 0; w < p.ks; ++w) v += src[w * (MT * 256)];
            const int64_t at = (m0 + tok) * p.n + n0 + row;
            if (p.parts > 1) p.sums[part * sums_stride(int64_t(p.m) * p.n) + at] = v;
            else store_y(p.y, at, v, p.y_dtype);
        }
    }
}

// y = the parts' sums added in order
__global__ __launch_bounds__(256) void q4_join_kernel(const float* __restrict__ sums, int parts, int64_t count,
                                                      void* __restrict__ y, int y_dtype) {
    const int64_t stride = sums_stride(count);
    for (int64_t i = 4 * (int64_t(blockIdx.x) * 256 + threadIdx.x); i < count; i += int64_t(gridDim.x) * 1024) {
        float4v v = *reinterpret_cast<const float4v*>(sums + i);
#pragma unroll 4
        for (int s = 1; s < parts; ++s) v += *reinterpret_cast<const float4v*>(sums + s * stride + i);
        if (i + 4 > count) {
            for (int j = 0; j < count - i; ++j) store_y(y, i + j, v[j], y_dtype);
        } else if (y_dtype == TL_F32) {
            *reinterpret_cast<float4v*>(static_cast<float*>(y) + i) = v;
        } else {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = y_dtype == TL_F16 ? f16_bits(v[j]) : bf16_bits(v[j]);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + i) = uint2{h[0] | h[1] << 16, h[2] | h[3] << 16};
        }
    }
}

constexpr int64_t kLdsCu = 160 * 1024;
constexpr int64_t kOnePart = 16384;   // M * K that is never cut into parts: its activations fit in LDS
constexpr int64_t kMaxSums = int64_t(1) << 28;   // bytes of the parts' sums, if 64 tokens' fit in them
// Scales of a wave in LDS, 20 KB of a workgroup's 80.  Longer runs come in segments,
// each of which waits for the weights on the way; that shows nowhere (17408 rows in
// groups of 64, one token: K = 5120 3.47 TB/s, 5248 3.42, 5632 3.50, 6144 3.73)
constexpr int kScaleLds = 2560;

// How a call is split; the same for the workspace and the launch.
struct Plan {
    int mt, l, parts, ks, d, seg;
    int64_t s_bytes, lds;
};

// Chunks of weights a wave has on the way: 2 or 4.  64 tokens: 4 spill (17408 x
// 5120 by binary16 28.8 us with 2, 30.1 with 1; for bfloat16 in groups of 128 2 do
// as well, 20 bytes a lane).  Up to 16 tokens, 2 against 4, means over six shapes from
// 1024 x 5120 to 32003 x 5120 and 5120 x 17408 at 1, 4 and 16 tokens: binary16 in
// groups of 128 2 to 3 % shorter (131072 x 5120 of one token 62.0 us, 64.2 with 4),
// in groups of 64 and 32 0 to 2 % longer (the worst: 32003 x 5120 of one token 21.4
// us, 19.4 with 4; the best: 17408 x 5120 of 4 16.7 and 17.8); bfloat16 1 to 5 %
// shorter, but for one token in groups of 128 (1 % longer); 8 bits: one token 4 to
// 6 % shorter, several 1 to 5 % longer (10240 x 4096 of 4 9.5 us, 8.6 with 4), in
// groups of 32 1 to 3 % shorter.  The rule goes by the types' means.  32 and 48
// tokens: 32003 x 5120 of 20 binary16 27.7 us, 26.3 with 4.  (Two row tiles of a
// wave that share the activations' reads are slower from 8 to 64 tokens on most
// shapes: 5120 x 17408 by 20 tokens 22.8 us, 18.1 with one.)
template <int XT>
constexpr int ring_depth(int mt, bool one_token) {
    return mt == 4 || (mt == 1 && (one_token || XT != TL_I8)) ? 2 : 4;
}

// LDS bytes of a workgroup with parts of l chunks, and of a wave's scales
template <int XT, int G>
void size_lds(Plan& p, int64_t tokens) {
    const int lw = (p.l + p.ks - 1) / p.ks;
    int chunk = 16 * (G == 128 ? 4 : 256 / G);        // bytes of a chunk's scales
    if (p.parts == 1 && p.ks == 1 && lw * chunk / (G == 128 ? 2 : 1) <= kScaleLds) chunk = 16 * (256 / G);
    p.seg = lw;
    if (lw * chunk > kScaleLds) p.seg = kScaleLds / chunk / p.d * p.d;   // whole steps
    p.s_bytes = (p.seg * chunk + 15) / 16 * 16;
    p.lds = tokens * int64_t(p.l) * chunk_bytes<XT>() + int64_t(p.l) * chunk_floats<XT>() * ((tokens + 3) / 4 * 16) +
            kWaves * p.s_bytes;
    const int64_t red = p.ks > 1 ? int64_t(kWaves) * p.mt * 1024 : 0;
    if (p.lds < red) p.lds = red;
}

// The split with the least estimated time.  What it weighs was measured at N x
// K from 1024 x 5120 to 131072 x 5120: weights arrive at 5.3 bytes per ps
// once about 0.7 of the waves that fit are busy (0.4 of that with few), more
// waves than fit cost a tenth, tiles that do not divide among the waves half of
// what they leave idle (without that, 17408 x 5120 by 45 8-bit tokens took 27.3
// us, 22.8 with); staged activations at 12; a second kernel costs 2 us and its
// sums 6 bytes per ps.
template <int XT, int G>
Plan q4_plan(int64_t m, int64_t n, int64_t k) {
    const int64_t chunks = k / 128, cus = cu_count();
    Plan p, best = {};
    double least = 0;
    p.mt = m <= 16 ? 1 : m <= 32 ? 2 : m <= 48 ? 3 : 4;
    const int64_t tokens = m < 16 * p.mt ? m : 16 * p.mt, slices = (m + 16 * p.mt - 1) / (16 * p.mt);
    p.d = ring_depth<XT>(p.mt, m == 1);
    // one token tile: two workgroups on a compute unit; more: one
    const int64_t per_cu = p.mt == 1 ? 2 : 1, room = kLdsCu / per_cu;
    const int64_t tiles = (n + 15) / 16, slots = cus * per_cu * kWaves;
    const int64_t fewest = chunks * tokens * chunk_bytes<XT>() / room;   // fewer parts do not fit
    for (p.ks = kWaves; p.ks >= 1; p.ks /= 2) {
        int tried = 0;
        for (p.parts = fewest > 1 ? int(fewest) : 1; p.parts <= chunks && tried < 5; ++p.parts) {
            if (p.parts > 1 && m * k <= kOnePart) break;
            p.l = int((chunks + p.parts - 1) / p.parts);
            size_lds<XT, G>(p, tokens);
            if (p.lds > room || (chunks + p.l - 1) / p.l != p.parts) continue;
            ++tried;
            if (p.ks > 1 && p.l < p.ks) continue;
            const double waves = double(tiles) * p.parts * p.ks * slices;
            const double busy = waves < 0.7 * slots ? waves / (0.7 * slots) : 1.0;
            const double over = p.ks > 1 && waves > 1.125 * slots ? 1.1 : 1.0;
            double groups = double((tiles + kWaves / p.ks - 1) / (kWaves / p.ks)) * p.parts;
            if (p.ks == 1 && groups > double(cus * per_cu)) groups = double(cus * per_cu);
            // tiles a wave goes through, over their mean
            double uneven = 1.0;
            if (p.ks == 1) {
                const double each = double(tiles) / (double(kWaves) * groups / p.parts);
                uneven = 0.5 + 0.5 * std::ceil(each) / each;
            }
            double us = double(n) * k / 2 * slices / 5.3e6 * over * uneven / (0.4 + 0.6 * busy) +
                        groups * slices * double(tokens) * p.l * chunk_bytes<XT>() / 12e6;
            if (p.parts > 1) us += 2.0 + double(p.parts) * m * n * 8 / 6e6;
            if (least == 0 || us < least) {
                least = us;
                best = p;
            }
        }
    }
    return best;
}

// Tokens of one launch: whole slices, so many that the parts' sums stay within
// kMaxSums (one slice if it does not fit) and the grid's second dimension ends
// at 65535
int64_t launch_tokens(const Plan& p, int64_t n) {
    const int64_t most = 65535 * 16, fit = p.parts > 1 ? kMaxSums / (4 * p.parts * n) / 64 * 64 : most;
    return fit < 64 ? 64 : fit < most ? fit : most;
}

template <int XT, int G, int MT, int V>
hipError_t launch(Args a, const Plan& p, hipStream_t stream) {
    const auto kernel = q4_gemv_kernel<XT, G, MT, ring_depth<XT>(MT, V == 1), V>;
    a.parts = p.parts;
    a.l = p.l;
    a.ks = p.ks;
    a.lw = (p.l + p.ks - 1) / p.ks;
    a.tiles = int((a.n + 15) / 16);
    const int tws = kWaves / p.ks;
    a.groups = (a.tiles + tws - 1) / tws;
    const int per_cu = MT == 1 ? 2 : 1;
    const int most = per_cu * cu_count() / p.parts > 0 ? per_cu * cu_count() / p.parts : 1;
    if (p.ks == 1 && a.groups > most) a.groups = most;
    a.seg = p.seg;
    a.s_bytes = int(p.s_bytes);
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), 160 * 1024);
    if (e != hipSuccess) return e;
    const dim3 grid(unsigned(a.groups * a.parts), unsigned((a.m + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), unsigned(p.lds), stream, a);
    if (p.parts > 1) {
        const int64_t count = int64_t(a.m) * a.n, g = (count + 1023) / 1024;
        hipLaunchKernelGGL(q4_join_kernel, dim3(unsigned(g < 8192 ? g : 8192)), dim3(256), 0, stream, a.sums, a.parts,
                           count, a.y, a.y_dtype);
    }
    return hipGetLastError();
}

template <int XT, int G>
hipError_t launch_rows(const Args& all, int64_t m, hipStream_t stream) {
    const Plan p = q4_plan<XT, G>(m, all.n, all.k);
    const int64_t step = launch_tokens(p, all.n), yb = all.y_dtype == TL_F32 ? 4 : 2;
    // (the last launch of several may be of few tokens, or one: their plan)
    for (int64_t m0 = 0; m0 < m; m0 += step) {
        Args a = all;
        a.x += m0 * all.k * (chunk_bytes<XT>() / 128);
        if (XT == TL_I8) a.xs += m0 * (all.k / 128);
        a.y = static_cast<uint8_t*>(all.y) + m0 * all.n * yb;
        a.m = int(m - m0 < step ? m - m0 : step);
        const hipError_t e = m == 1        ? launch<XT, G, 1, 1>(a, p, stream)
                             : p.mt == 1 ? launch<XT, G, 1, 4>(a, p, stream)
                             : p.mt == 2 ? launch<XT, G, 2, 4>(a, p, stream)
                             : p.mt == 3 ? launch<XT, G, 3, 4>(a, p, stream)
                                         : launch<XT, G, 4, 4>(a, p, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int64_t q4_gemv_need(int64_t m, int64_t n, int64_t k, int x_dtype, int group) {
    if (m * k <= kOnePart) return 0;
    const auto bytes = [&](const Plan& p) {
        const int64_t step = launch_tokens(p, n);
        return p.parts > 1 ? p.parts * sums_stride((m < step ? m : step) * n) * 4 : int64_t(0);
    };
#define TL_Q4_NEED(XT)                                      \
    bytes(group == 32   ? q4_plan<XT, 32>(m, n, k)          \
          : group == 64 ? q4_plan<XT, 64>(m, n, k)          \
                        : q4_plan<XT, 128>(m, n, k))
    return x_dtype == TL_I8 ? TL_Q4_NEED(TL_I8) : x_dtype == TL_F16 ? TL_Q4_NEED(TL_F16) : TL_Q4_NEED(TL_BF16);
}

int64_t q4_gemv_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    int64_t most = 0;
    for (const int x_dtype : {TL_F16, TL_BF16, TL_I8})
        for (const int group : {32, 64, 128}) {
            const int64_t b = q4_gemv_need(m, n, k, x_dtype, group);
            most = b > most ? b : most;
        }
    return most;
}

hipError_t launch_q4_gemv(const uint8_t* packed, const uint16_t* scales, int group, const void* x,
                          int x_dtype, const float* x_scales, int64_t m, int64_t n, int64_t k, void* y,
                          int y_dtype, void* ws, hipStream_t stream) {
    const Args a = {packed, scales, static_cast<const uint8_t*>(x), x_scales, y, static_cast<float*>(ws),
                    n, k, 0, y_dtype, 0, 0, 0, 0, 0, 0, 0, 0};
#define TL_Q4_GROUP(XT)                                                \
    (group == 32   ? launch_rows<XT, 32>(a, m, stream)                 \
     : group == 64 ? launch_rows<XT, 64>(a, m, stream)                 \
                   : launch_rows<XT, 128>(a, m, stream))
    return x_dtype == TL_I8    ? TL_Q4_GROUP(TL_I8)
           : x_dtype == TL_F16 ? TL_Q4_GROUP(TL_F16)
                               : TL_Q4_GROUP(TL_BF16);
}

}  // namespace tl
