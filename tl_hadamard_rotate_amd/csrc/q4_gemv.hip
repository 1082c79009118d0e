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
// Work split: a workgroup owns a tile of 16 R TW weight rows; its TW KS waves
// are TW sets of 16 R rows, each split along K into KS runs of chunks whose
// partial sums are added through LDS in a fixed order.  A wave keeps D chunks
// of weights on the way.  Activations and scales go through LDS: read from
// memory as the matrix cores want them, the scales (2 bytes from each of 16
// rows) took longer than the weights, and the activations of 16 tokens (64
// bytes from each row, a power of two apart, so from few L2 channels) as long
// as the weights.  Activations that fit in LDS are loaded once and stay while
// the workgroup goes through its tiles; others (PH) come in phases, P chunks
// of each of the KS runs at a time.
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

constexpr int kThreads = 512;   // at most

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

// largest of the 16 lanes of a row (as bfloat16 magnitudes)
__device__ __forceinline__ uint32_t row16_max(uint32_t a) {
    const auto step = [&](uint32_t o) { a = o > a ? o : a; };
    step(uint32_t(__builtin_amdgcn_mov_dpp(int(a), 0xB1, 0xF, 0xF, false)));    // lane ^ 1
    step(uint32_t(__builtin_amdgcn_mov_dpp(int(a), 0x4E, 0xF, 0xF, false)));    // lane ^ 2
    step(uint32_t(__builtin_amdgcn_mov_dpp(int(a), 0x141, 0xF, 0xF, false)));   // the other four of 8
    step(uint32_t(__builtin_amdgcn_mov_dpp(int(a), 0x140, 0xF, 0xF, false)));   // the other 8 of 16
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

// One chunk's sums added to acc[r][t]: lane (q, c) holds weight row 16 r + c
// and tokens 16 t + 4 q .. + 3.  In LDS: xa[t] the lane's token's activations
// of the chunk, sc the chunk's scales of row c (row 16 r + c is r * row_step
// elements further), fa the factors of tokens 4 q .. of the chunk (bfloat16, 8
// bits).
template <int XT, int G, int R, int MT>
__device__ __forceinline__ void consume(const uint4 (&wr)[R], const uint8_t* const (&xa)[MT], const uint16_t* sc,
                                        int row_step, const float* fa, int q, float4v (&acc)[R][MT]) {
    constexpr int NS = 128 / G;               // scales of the chunk
    constexpr int NX = XT == TL_I8 && G != 32 ? 2 : 4;   // matrix instructions along K
    uint32_t w[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        w[r][0] = wr[r].x, w[r][1] = wr[r].y, w[r][2] = wr[r].z, w[r][3] = wr[r].w;
        if constexpr (NX == 4) {              // octets q, q + 4, q + 8, q + 12
            swap32(w[r][0], w[r][2]);
            swap32(w[r][1], w[r][3]);
            swap16(w[r][0], w[r][1]);
            swap16(w[r][2], w[r][3]);
        } else {                              // octet pairs q, q + 4
            swap16(w[r][0], w[r][2]);
            swap16(w[r][1], w[r][3]);
            swap32(w[r][0], w[r][2]);
            swap32(w[r][1], w[r][3]);
        }
    }
    float4v f[MT];
    if constexpr (XT != TL_F16)
#pragma unroll
        for (int t = 0; t < MT; ++t) f[t] = *reinterpret_cast<const float4v*>(fa + 16 * t);
    float s[R][NS];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        uint32_t sb[2];
        if constexpr (NS == 1) sb[0] = sc[r * row_step];
        else if constexpr (NS == 2) sb[0] = *reinterpret_cast<const uint32_t*>(sc + r * row_step);
        else {
            const uint2 u = *reinterpret_cast<const uint2*>(sc + r * row_step);
            sb[0] = u.x, sb[1] = u.y;
        }
#pragma unroll
        for (int g = 0; g < NS; ++g)
            s[r][g] = float(__builtin_bit_cast(_Float16, uint16_t(sb[g >> 1] >> (16 * (g & 1))))) *
                      (XT == TL_I8 ? 0.0625f : 1.0f);
    }
    float4v d[R][MT];
    int4v di[R][MT];
#pragma unroll
    for (int j = 0; j < NX; ++j) {
        const bool first = j % (NX / NS) == 0, last = (j + 1) % (NX / NS) == 0;
        const int g = j / (NX / NS);
        if constexpr (XT != TL_I8) {
            half8v a[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) a[t] = *reinterpret_cast<const half8v*>(xa[t] + 64 * j);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const half8v b = decode_f16(w[r][j]);
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    d[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[t], b, first ? float4v{} : d[r][t], 0, 0, 0);
            }
        } else if constexpr (G == 32) {
            int64_t a[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) a[t] = *reinterpret_cast<const int64_t*>(xa[t] + 32 * j);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t lo = (w[r][j] << 4) & 0xF0F0F0F0u, hi = w[r][j] & 0xF0F0F0F0u;
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    di[r][t] = __builtin_amdgcn_mfma_i32_16x16x32_i8(a[t], int64_t(uint64_t(hi) << 32 | lo),
                                                                     first ? int4v{} : di[r][t], 0, 0, 0);
            }
        } else {
            int4v a[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) a[t] = *reinterpret_cast<const int4v*>(xa[t] + 64 * j);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const uint32_t u = w[r][2 * j], v = w[r][2 * j + 1];
                const int4v b = {int((u << 4) & 0xF0F0F0F0u), int(u & 0xF0F0F0F0u), int((v << 4) & 0xF0F0F0F0u),
                                 int(v & 0xF0F0F0F0u)};
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    di[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[t], b, first ? int4v{} : di[r][t], 0, 0, 0);
            }
        }
        if (last)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v;
                        if constexpr (XT == TL_I8) v = float(di[r][t][i]);
                        else v = d[r][t][i];
                        acc[r][t][i] = __builtin_fmaf(v, XT == TL_F16 ? s[r][g] : s[r][g] * f[t][i], acc[r][t][i]);
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
    // the launch's split: KS runs of C chunks, P of each in a phase; tiles of
    // rows, how many a workgroup takes, of how many the scales are in LDS
    int ks, c, p, tiles, per_wg, s_tiles;
};

__device__ __forceinline__ void store_y(void* y, int64_t at, float v, int y_dtype) {
    if (y_dtype == TL_F32) static_cast<float*>(y)[at] = v;
    else static_cast<uint16_t*>(y)[at] = uint16_t(y_dtype == TL_F16 ? f16_bits(v) : bf16_bits(v));
}

template <int XT, int G, int R, int MT, int D, bool PH>
__global__ __launch_bounds__(kThreads, MT == 1 ? 4 : 2) void q4_gemv_kernel(const Args p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    constexpr int kXB = XT == TL_I8 ? 1 : 2;
    constexpr int kPieces = 8 * kXB;          // 16-byte pieces of a token's chunk
    constexpr int kLanePiece = XT == TL_I8 && G == 32 ? 8 : 16;   // bytes of x a lane reads at a time
    constexpr int NS = 128 / G;
    const int tid = threadIdx.x, threads = int(blockDim.x);
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int q = lane >> 4, c = lane & 15;
    const int chunks = int(p.k / 128);
    const int row_bytes = int(p.k / 2);
    const int ks = wave % p.ks, tw = wave / p.ks, tws = (threads >> 6) / p.ks;
    const int tile_rows = 16 * R * tws;
    const int64_t m0 = int64_t(blockIdx.y) * (16 * MT);
    const int tokens = int(p.m - m0 < 16 * MT ? p.m - m0 : 16 * MT);
    const int slots = PH ? p.ks * p.p : chunks;   // chunks of activations in LDS
    const int tile0 = int(blockIdx.x) * p.per_wg;
    const int tile1 = tile0 + p.per_wg < p.tiles ? tile0 + p.per_wg : p.tiles;

    // LDS: activations [token][slot], factors [slot][16 MT], two sets of
    // partial sums [ks][tw][t][r][row][token], scales [row][chunk]
    const int xstride = slots * (128 * kXB) + 16;   // 16: rows on different banks
    const int red_set = (threads >> 6) * (MT * R * 256);
    uint8_t* const lx = smem;
    float* const lf = reinterpret_cast<float*>(lx + tokens * xstride);
    float* const red = lf + (XT == TL_F16 ? 0 : slots * 16 * MT);
    uint16_t* const lsc = reinterpret_cast<uint16_t*>(red + (p.ks > 1 ? 2 * red_set : 0));

    // this wave's chunks are ks * C + [0, mine)
    const int left = chunks - ks * p.c;
    const int mine = left < 0 ? 0 : left < p.c ? left : p.c;

    // Weights on the way: chunk i of a tile in ring[i % D].  voff: the lane's
    // rows of a tile (rows that do not exist repeat the last one; their sums
    // are not stored).
    uint4 ring[D][R];
    uint32_t voff[R], vnext[R];
    const uint8_t *base, *nbase = nullptr;
    const auto tile_count = [&](int tile) {
        const int64_t rest = p.n - int64_t(tile) * tile_rows;
        return int(rest < tile_rows ? rest : tile_rows);
    };
    const auto enter = [&](int tile, uint32_t (&v)[R]) {
        const int last = tile_count(tile) - 1;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = 16 * (R * tw + r) + c;
            v[r] = uint32_t(row < last ? row : last) * uint32_t(row_bytes) + 16u * uint32_t(q);
        }
        return p.packed + (int64_t(tile) * tile_rows * row_bytes + int64_t(ks) * p.c * 64);
    };
    const auto fetch = [&](const uint8_t* b, const uint32_t (&v)[R], uint4 (&w)[R]) {
#pragma unroll
        for (int r = 0; r < R; ++r) w[r] = *reinterpret_cast<const uint4*>(b + v[r]);
    };
    base = enter(tile0, voff);
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < mine) fetch(base + 64 * d, voff, ring[d]);

    // activations of phase ph to LDS
    const auto stage_x = [&](int ph) {
        constexpr int U = 4;
        const uint8_t* const xt = p.x + m0 * p.k * kXB;
        const float* const xst = XT == TL_I8 ? p.xs + m0 * chunks : nullptr;
        const int per_token = slots * kPieces;
        int t = tid / per_token, e = tid - t * per_token;
        while (t < tokens) {
            uint4v v[U] = {};
            int dst[U];     // byte of the piece in LDS, -1: none
            int fd[U];      // its factor's place, -1: another lane's
            float f[U] = {};
#pragma unroll
            for (int u = 0; u < U; ++u) {
                dst[u] = fd[u] = -1;
                if (t < tokens) {
                    const int slot = e / kPieces;
                    int g = slot;
                    if (PH) {
                        const int run = slot / p.p, i = ph * p.p + (slot - run * p.p);
                        g = i < p.c ? run * p.c + i : chunks;
                    }
                    if (g < chunks) {
                        dst[u] = t * xstride + 16 * e;
                        v[u] = *reinterpret_cast<const uint4v*>(xt + (int64_t(t) * p.k + int64_t(g) * 128) * kXB +
                                                               16 * (e % kPieces));
                        if (XT != TL_F16 && e % kPieces == 0) {
                            fd[u] = slot * (16 * MT) + t;
                            if (XT == TL_I8) f[u] = xst[int64_t(t) * chunks + g];
                        }
                    }
                    e += threads;
                    while (e >= per_token) {
                        e -= per_token;
                        ++t;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // (a chunk's lanes are a row of 16 or half of one, present or
                // absent together)
                if (dst[u] >= 0) {
                    if constexpr (XT == TL_BF16) f[u] = convert_bf16(v[u]);
                    if constexpr (XT == TL_I8) order_i8(v[u]);
                    *reinterpret_cast<uint4v*>(lx + dst[u]) = v[u];
                    if (XT != TL_F16 && fd[u] >= 0) lf[fd[u]] = f[u];
                }
            }
        }
    };
    // scales: of s_tiles tiles from `tile` on, one run of memory; PH: of a tile's
    // chunks of phase ph
    const auto stage_s = [&](int tile, int ph) {
        const int64_t n0 = int64_t(tile) * tile_rows;
        const uint16_t* const src = p.scales + n0 * (chunks * NS);
        if constexpr (PH) {
            const int units = tile_count(tile) * slots;
            for (int u = tid; u < units; u += threads) {
                const int row = u / slots, slot = u - row * slots, run = slot / p.p;
                const int i = ph * p.p + (slot - run * p.p), g = run * p.c + i;
                if (i >= p.c || g >= chunks) continue;
                const uint16_t* const from = src + (int64_t(row) * chunks + g) * NS;
                uint16_t* const to = lsc + u * NS;
                if constexpr (NS == 1) *to = *from;
                else if constexpr (NS == 2) *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
                else *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from);
            }
        } else {
            const int64_t have = (p.n - n0) * (chunks * NS);
            const int want = p.s_tiles * tile_rows * chunks * NS;
            const int count = int(have < want ? have : want);
            for (int i = 8 * tid; i < count; i += 8 * threads) {
                if (i + 8 <= count) *reinterpret_cast<uint4*>(lsc + i) = *reinterpret_cast<const uint4*>(src + i);
                else
                    for (int j = i; j < count; ++j) lsc[j] = src[j];
            }
        }
    };
    stage_s(tile0, 0);
    stage_x(0);
    __syncthreads();

    const uint8_t* xa[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int tok = 16 * t + c < tokens ? 16 * t + c : tokens - 1;   // absent tokens repeat the last
        xa[t] = lx + tok * xstride + kLanePiece * q;
    }
    int s_tile = 0, set = 0;
    for (int tile = tile0; tile < tile1; ++tile) {
        float4v acc[R][MT] = {};
        const int64_t n0 = int64_t(tile) * tile_rows;
        const int rows = tile_count(tile);
        if (tile + 1 < tile1) nbase = enter(tile + 1, vnext);
        const int srow = slots * NS;    // elements of a row of scales in LDS
        const uint16_t* const sc = lsc + (s_tile * tile_rows + 16 * R * tw + c) * srow;
        int ph = 0;
        do {
            const int beg = PH ? ph * p.p : 0;
            const int end = PH && beg + p.p < mine ? beg + p.p : mine;
            for (int i0 = beg; i0 < end; i0 += D)
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    const int i = i0 + d;
                    if (i >= end) break;
                    const int slot = PH ? ks * p.p + (i - beg) : ks * p.c + i;
                    const uint8_t* xc[MT];
#pragma unroll
                    for (int t = 0; t < MT; ++t) xc[t] = xa[t] + slot * (128 * kXB);
                    consume<XT, G, R, MT>(ring[d], xc, sc + slot * NS, 16 * srow, lf + slot * (16 * MT) + 4 * q, q, acc);
                    // the chunk that uses this place next, of this tile or the next
                    if (i + D < mine) fetch(base + 64 * (i + D), voff, ring[d]);
                    else if (tile + 1 < tile1) fetch(nbase + 64 * d, vnext, ring[d]);
                }
            if constexpr (PH) {
                ++ph;
                const bool more = ph * p.p < p.c;
                if (more || tile + 1 < tile1) {
                    __syncthreads();
                    stage_s(more ? tile : tile + 1, more ? ph : 0);
                    stage_x(more ? ph : 0);
                    if (more) __syncthreads();   // else the one below
                }
            }
        } while (PH && ph * p.p < p.c);
        base = nbase;
#pragma unroll
        for (int r = 0; r < R; ++r) voff[r] = vnext[r];

        if (p.ks > 1) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int r = 0; r < R; ++r)
                    *reinterpret_cast<float4v*>(red + set * red_set + ((wave * MT + t) * R + r) * 256 + c * 16 + 4 * q) =
                        acc[r][t];
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = 16 * (R * tw + r) + c, tok = 16 * t + 4 * q + e;
                        if (row < rows && tok < tokens)
                            store_y(p.y, (m0 + tok) * p.n + n0 + row, acc[r][t][e], p.y_dtype);
                    }
        }
        if (!PH && ++s_tile == p.s_tiles && tile + 1 < tile1) {
            __syncthreads();
            stage_s(tile + 1, 0);
            s_tile = 0;
        }
        // (one barrier a tile: the other set of partial sums is written next,
        // and read by nobody once all have come here again)
        __syncthreads();
        if (p.ks > 1) {
            for (int o = tid; o < rows * tokens; o += threads) {
                const int tok = o / rows, row = o - tok * rows;
                const int w0 = row / (16 * R), rr = row - w0 * (16 * R);
                const float* src = red + set * red_set + (w0 * p.ks * MT * R + ((tok >> 4) * R + (rr >> 4))) * 256 +
                                   (rr & 15) * 16 + (tok & 15);
                float v = 0.0f;
                for (int w = 0; w < p.ks; ++w) v += src[w * (MT * R * 256)];
                store_y(p.y, (m0 + tok) * p.n + n0 + row, v, p.y_dtype);
            }
            set ^= 1;
        }
    }
}

constexpr int64_t kLdsCu = 160 * 1024;
constexpr int64_t kOneX = 84 * 1024;     // activations that stay in LDS
constexpr int64_t kScaleLds = 24 * 1024; // scales of several tiles

// Waves: KS runs of K (8, so that a workgroup reads long pieces of few rows),
// the rest sets of rows.  Activations in phases (PH) where they, or a tile's
// scales, do not fit in LDS.
template <int XT, int G, int R, int MT, int D, bool PH>
hipError_t launch(Args a, hipStream_t stream) {
    const auto kernel = q4_gemv_kernel<XT, G, R, MT, D, PH>;
    constexpr int kChunkX = XT == TL_I8 ? 128 : 256, NS = 128 / G;
    const int64_t chunks = a.k / 128;
    const int waves = PH || chunks >= 8 ? 8 : int(chunks);
    const int64_t tokens = a.m < 16 * MT ? a.m : 16 * MT;
    int64_t tile_rows = 0, fixed = 0, lds = 0;
    const auto size = [&](int64_t slots) {   // LDS without scales
        return tokens * (slots * kChunkX + 16) + (XT == TL_F16 ? 0 : slots * 64 * MT) +
               (a.ks > 1 ? 2 * waves * MT * R * 1024 : 0);
    };
    for (a.ks = waves;; a.ks /= 2) {
        tile_rows = 16 * R * (waves / a.ks);
        a.c = int((chunks + a.ks - 1) / a.ks);
        a.p = a.c;
        if (!PH) {
            fixed = size(chunks);
            break;
        }
        // the longest phase (a multiple of D, at most all) that lets two
        // workgroups run on a compute unit
        const auto phase = [&](int64_t pp) { return size(a.ks * pp) + tile_rows * a.ks * pp * NS * 2; };
        a.p = (a.c + D - 1) / D * D;
        while (a.p > D && phase(a.p) > kLdsCu / 2) a.p -= D;
        fixed = size(int64_t(a.ks) * a.p);
        if (phase(a.p) <= kLdsCu / 2 || a.ks == 1) break;
    }
    a.tiles = int((a.n + tile_rows - 1) / tile_rows);
    const int64_t s_tile = tile_rows * (PH ? int64_t(a.ks) * a.p : chunks) * NS * 2;
    // as many workgroups as run at once, each with a run of tiles
    const auto split = [&](int64_t per_cu) {
        const int64_t most = per_cu * cu_count();
        a.per_wg = int((a.tiles + most - 1) / most);
        const int64_t room = kLdsCu / per_cu - fixed;
        const int64_t fit = (room < kScaleLds ? room : kScaleLds) / s_tile;
        a.s_tiles = PH || fit < 1 ? 1 : fit < a.per_wg ? int(fit) : a.per_wg;
        lds = fixed + a.s_tiles * s_tile;
    };
    split(2);
    if (lds > kLdsCu / 2) split(1);
    if (lds > kLdsCu) return hipErrorInvalidValue;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), int(kLdsCu));
    if (e != hipSuccess) return e;
    const dim3 grid(unsigned((a.tiles + a.per_wg - 1) / a.per_wg), unsigned((a.m + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), unsigned(lds), stream, a);
    return hipGetLastError();
}

template <int XT, int G, int R>
hipError_t launch_mt(const Args& a, hipStream_t stream) {
    if (a.m > 48) return launch<XT, G, G == 32 ? 1 : R, 4, 2, true>(a, stream);   // (registers)
    if (a.m > 32) return launch<XT, G, R, 3, 2, true>(a, stream);
    if (a.m > 16) return launch<XT, G, R, 2, 2, true>(a, stream);
    const int64_t chunks = a.k / 128;
    if (a.m * chunks * (XT == TL_I8 ? 128 : 256) > kOneX || 16 * R * chunks * (256 / G) > kScaleLds)
        return launch<XT, G, R, 1, 2, true>(a, stream);
    return launch<XT, G, R, 1, 4, false>(a, stream);
}

template <int XT, int G>
hipError_t launch_rows(const Args& a, hipStream_t stream) {
    return a.n >= 32 * int64_t(cu_count()) ? launch_mt<XT, G, 2>(a, stream) : launch_mt<XT, G, 1>(a, stream);
}

}  // namespace

int64_t q4_gemv_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_q4_gemv(const uint8_t* packed, const uint16_t* scales, int group, const void* x,
                          int x_dtype, const float* x_scales, int64_t m, int64_t n, int64_t k, void* y,
                          int y_dtype, void*, hipStream_t stream) {
    // a grid's second dimension ends at 65535: at most 65535 * 16 tokens a launch
    constexpr int64_t kMaxTokens = 65535 * 16;
    const int64_t xb = x_dtype == TL_I8 ? 1 : 2, yb = y_dtype == TL_F32 ? 4 : 2;
    for (int64_t m0 = 0; m0 < m; m0 += kMaxTokens) {
        const int64_t mt = m - m0 < kMaxTokens ? m - m0 : kMaxTokens;
        const Args a = {packed, scales, static_cast<const uint8_t*>(x) + m0 * k * xb,
                        x_scales ? x_scales + m0 * (k / 128) : nullptr,
                        static_cast<uint8_t*>(y) + m0 * n * yb, n, k, int(mt), y_dtype, 0, 0, 0, 0, 0, 0};
#define TL_Q4_GROUP(XT)                                             \
    (group == 32   ? launch_rows<XT, 32>(a, stream)              \
     : group == 64 ? launch_rows<XT, 64>(a, stream)              \
                   : launch_rows<XT, 128>(a, stream))
        const hipError_t e = x_dtype == TL_I8    ? TL_Q4_GROUP(TL_I8)
                             : x_dtype == TL_F16 ? TL_Q4_GROUP(TL_F16)
                                                 : TL_Q4_GROUP(TL_BF16);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace tl
