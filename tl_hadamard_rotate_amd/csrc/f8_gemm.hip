// Product of rows and weights in 8-bit floating point on the matrix cores:
//
//   y[m, n] = sum_k X[m, k] * W[n, k],   X, W = e4m3 code * 2^(scale of its 128)
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes both operands' codes and scales as they
// are: weights are the A rows, tokens the B columns.
#include "elem.h"
#include "f8.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;

typedef int int8v __attribute__((ext_vector_type(8)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;
typedef __attribute__((address_space(3))) uint8_t lds_u8;

constexpr int kThreads = 512;    // 8 waves: 4 along the weight rows, 2 along the tokens
constexpr int kRows = 256;       // weight rows of a tile
constexpr int kStep = 64;        // K of a step

struct Args {
    const uint8_t *w, *ws, *x, *xs;
    void* y;
    float* sums;
    int64_t m, n, k;
    int y_dtype, groups;             // groups: K / 128
    int tiles_m, tiles_n, tiles, whole, splits, chunk_a, chunk_b;
};

// 16 (1) bytes a lane from base + offset to LDS, lane i at `to` + 16 (4) i.
// Written out, with the waits of the loop: the compiler would make every LDS
// read wait for every load on the way into LDS.
__device__ __forceinline__ void load_lds16(const uint8_t* base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(to), "v"(offset), "s"(base)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_lds1(const uint8_t* base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, %2"
                 :
                 : "s"(to), "v"(offset), "s"(base)
                 : "memory", "m0");
}

__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    return reinterpret_cast<const uint8_t*>(uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(u)))) |
                                            uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(u >> 32)))) << 32);
}

// One 32 x 32 tile of a lane's sums to y: register r of lane (q, c) is weight row
// 8 (r / 4) + 4 q + r % 4 and token c of the tile
__device__ __forceinline__ void store_tile(const float16v& acc, const Args& a, int64_t n0, int64_t token, int q) {
    if (a.y_dtype == TL_F32) {
        float* y = static_cast<float*>(a.y) + token * a.n;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int64_t n = n0 + 8 * g + 4 * q;
            const float v[4] = {acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
            if (token >= a.m) continue;
            if (n + 4 <= a.n) {
                __builtin_memcpy(y + n, v, 16);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (n + r < a.n) y[n + r] = v[r];
            }
        }
        return;
    }
    uint16_t* y = static_cast<uint16_t*>(a.y) + token * a.n;
    const auto pair = [&](float u, float v) {
        return a.y_dtype == TL_F16 ? f16_bits(u) | f16_bits(v) << 16 : bf16_pair(u, v);
    };
    // the halves of the wave exchange rows, so that each lane has 8 in a row
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
        const auto s0 = __builtin_amdgcn_permlane32_swap(pair(acc[4 * g], acc[4 * g + 1]),
                                                         pair(acc[4 * g + 4], acc[4 * g + 5]), false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(pair(acc[4 * g + 2], acc[4 * g + 3]),
                                                         pair(acc[4 * g + 6], acc[4 * g + 7]), false, false);
        const uint32_t v[4] = {s0[0], s1[0], s0[1], s1[1]};
        const int64_t n = n0 + 8 * (g + q);
        if (token >= a.m) continue;
        if (n + 8 <= a.n) {
            __builtin_memcpy(y + n, v, 16);
        } else {
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (n + r < a.n) y[n + r] = uint16_t(v[r >> 1] >> (16 * (r & 1)));
        }
    }
}

__device__ __forceinline__ void tile_origin(const Args& a, int tile, int tokens, int64_t& n0, int64_t& m0) {
    // four rows of tokens' tiles at a time, those fastest
    const int per = 4 * a.tiles_n, band = tile / per, in = tile - band * per;
    const int high = a.tiles_m - 4 * band < 4 ? a.tiles_m - 4 * band : 4;
    m0 = int64_t(4 * band + in % high) * tokens;
    n0 = int64_t(in / high) * kRows;
}

__device__ __forceinline__ bf8v widen(uint32_t a, uint32_t b, float s) {
    const bf2v p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, false);
    const bf2v p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, s, true);
    const bf2v p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, false);
    const bf2v p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, s, true);
    return bf8v{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

template <int IT, bool WIDE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void f8_gemm_kernel(const Args a) {
    constexpr int kTokens = 64 * IT;
    constexpr int kStage = (kRows + kTokens) * kStep, kScaleStage = (kRows + kTokens) * 4;
    constexpr int kTokenLoads = kTokens / 16, kPerWave = kTokenLoads < 8 ? 1 : kTokenLoads / 8;
    constexpr int kLoads = 2 + kPerWave;        // of a wave in a step, and one of scales every other step
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const uint32_t lds = uint32_t(uintptr_t((__attribute__((address_space(3))) uint8_t*)(smem)));
    constexpr uint32_t kXStages = 4 * kRows * kStep;
    const uint32_t scale_lds = lds + 4 * kStage;

    int tile, sp = 0, slot = 0;
    bool split = false;
    if (int(blockIdx.x) < 8 * a.chunk_a) {
        tile = int(blockIdx.x & 7) * a.chunk_a + int(blockIdx.x >> 3);
        if (tile >= a.whole) return;
    } else {
        const int u = int(blockIdx.x) - 8 * a.chunk_a;
        slot = (u & 7) * a.chunk_b + (u >> 3);
        if (slot >= (a.tiles - a.whole) * a.splits) return;
        tile = a.whole + slot / a.splits;
        sp = slot % a.splits;
        split = a.splits > 1;
    }
    int64_t m0, n0;
    tile_origin(a, tile, kTokens, n0, m0);
    const int g0 = split ? int(int64_t(sp) * a.groups / a.splits) : 0;
    const int g1 = split ? int(int64_t(sp + 1) * a.groups / a.splits) : a.groups;
    const int steps = 2 * (g1 - g0);

    const int tid = threadIdx.x, l = tid & 63, q = l >> 5, c = l & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = 64 * (wave & 3), wt = 32 * IT * (wave >> 2);

    // lane i of a load of 1 KB brings 16 bytes of row i / 4 to place i % 4, those
    // of chunk (i % 4) ^ ((row / 4) % 4): 16 rows read at one chunk meet all banks
    const uint8_t* const wb = a.w + n0 * a.k + int64_t(g0) * 128;
    const uint8_t* const xb = a.x + m0 * a.k + int64_t(g0) * 128;
    const uint8_t* const wsb = a.ws + n0 * a.groups + g0;
    const uint8_t* const xsb = a.xs + m0 * a.groups + g0;
    const uint32_t k32 = uint32_t(a.k);
    const int64_t left_n = a.n - n0, left_m = a.m - m0;
    const auto row_n = [&](int r) { return uint32_t(r < left_n ? r : left_n - 1); };   // rows past the end: the last
    const auto row_m = [&](int r) { return uint32_t(r < left_m ? r : left_m - 1); };
    const uint32_t chunk = 16u * uint32_t((l & 3) ^ ((l >> 4) & 3));
    uint32_t w_off[2], x_off[kPerWave];
    uint32_t w_to[2], x_to[kPerWave];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        w_off[u] = row_n(32 * wave + 16 * u + (l >> 2)) * k32 + chunk;
        w_to[u] = uint32_t(32 * wave + 16 * u) * kStep;
    }
#pragma unroll
    for (int u = 0; u < kPerWave; ++u) {
        const int first = 16 * ((kPerWave * wave + u) % kTokenLoads);
        x_off[u] = row_m(first + (l >> 2)) * k32 + chunk;
        x_to[u] = kXStages + uint32_t(first) * kStep;
    }
    const int sw = wave % (4 + IT);     // 64 rows' scales
    const bool s_w = sw < 4;
    const uint8_t* const sb = s_w ? wsb : xsb;
    const uint32_t s_off = (s_w ? row_n(64 * sw + l) : row_m(64 * (sw - 4) + l)) * uint32_t(a.groups);
    const uint32_t s_to = scale_lds + 256u * uint32_t(sw);

    // load u of step t (past the end: of the last one again)
    const auto load_w = [&](int t, int stage, int u) {
        const uint32_t at = uint32_t(t < steps ? t : steps - 1) * kStep;
        load_lds16(wb + at, w_off[u], lds + uint32_t(stage) * kRows * kStep + w_to[u]);
    };
    const auto load_x = [&](int t, int stage, int u) {
        const uint32_t at = uint32_t(t < steps ? t : steps - 1) * kStep;
        load_lds16(xb + at, x_off[u], lds + uint32_t(stage) * kTokens * kStep + x_to[u]);
    };
    const auto load_scales = [&](int t, int stage) {
        const uint32_t g = uint32_t(t < steps ? t : steps - 1) >> 1;
        load_lds1(sb + g, s_off, s_to + uint32_t(stage) * kScaleStage);
    };

    // a lane's fragment of a 32-row tile: 32 bytes of row c, at 32 q
    const uint32_t f0 = uint32_t(c) * kStep + 16u * uint32_t((2 * q) ^ ((c >> 2) & 3));
    const uint32_t w_at = lds + uint32_t(wn) * kStep + f0, x_at = lds + kXStages + uint32_t(wt) * kStep + f0;
    const uint32_t w_at1 = w_at ^ 16u, x_at1 = x_at ^ 16u;
    const uint32_t ws_at = scale_lds + 4u * uint32_t(wn + c), xs_at = scale_lds + 4u * uint32_t(kRows + wt + c);
    const auto fragment = [&](uint32_t lo_at, uint32_t hi_at) {
        const u32x4 lo = *reinterpret_cast<lds_u32x4*>(lo_at), hi = *reinterpret_cast<lds_u32x4*>(hi_at);
        return int8v{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]), int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
    };

    int8v wf[2][2], xf[IT];
    int wsc[2][2], xsc[IT];
    const auto read_w = [&](int buf, int stage, int i) {
        const uint32_t at = uint32_t(stage) * kRows * kStep + 32u * kStep * uint32_t(i);
        wf[buf][i] = fragment(w_at + at, w_at1 + at);
    };
    const auto read_x = [&](int stage, int j) {
        const uint32_t at = uint32_t(stage) * kTokens * kStep + 32u * kStep * uint32_t(j);
        xf[j] = fragment(x_at + at, x_at1 + at);
    };
    const auto read_ws = [&](int buf, int stage) {
        const uint32_t at = uint32_t(stage) * kScaleStage;
#pragma unroll
        for (int i = 0; i < 2; ++i) wsc[buf][i] = int(*reinterpret_cast<lds_u32*>(ws_at + at + 128u * uint32_t(i)));
    };
    const auto read_xs = [&](int stage, int j) {
        const uint32_t at = uint32_t(stage) * kScaleStage;
        xsc[j] = int(*reinterpret_cast<lds_u32*>(xs_at + at + 128u * uint32_t(j)));
    };

    float16v acc[2][IT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < IT; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    load_scales(0, 0);
#pragma unroll
    for (int t = 0; t < 3; ++t) {
#pragma unroll
        for (int u = 0; u < 2; ++u) load_w(t, t, u);
#pragma unroll
        for (int u = 0; u < kPerWave; ++u) load_x(t, t, u);
    }
    load_scales(2, 1);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    read_ws(0, 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) read_w(0, 0, i);
#pragma unroll
    for (int j = 0; j < IT; ++j) read_xs(0, j), read_x(0, j);

    const auto step = [&](int t, auto s_c) {
        constexpr int S = decltype(s_c)::value, cur = S & 1, nxt = cur ^ 1, group = S >> 1;
#pragma unroll
        for (int j = 0; j < IT; ++j) {
            if constexpr (WIDE) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const bf8v xv = widen(uint32_t(xf[j][2 * h]), uint32_t(xf[j][2 * h + 1]),
                                          __builtin_bit_cast(float, xsc[j] << 23));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                    const bf8v wv = widen(uint32_t(wf[cur][i][2 * h]), uint32_t(wf[cur][i][2 * h + 1]),
                                  __builtin_bit_cast(float, wsc[group][i] << 23));
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wv, xv, acc[i][j], 0, 0, 0);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        wf[cur][i], xf[j], acc[i][j], 0, 0, 0, wsc[group][i], 0, xsc[j]);
            }
            if (j == 0) {
                if (S & 1) read_ws(group ^ 1, group ^ 1);
                read_w(nxt, (S + 1) & 3, 0);
                read_w(nxt, (S + 1) & 3, 1);
            }
            if (S & 1) read_xs(group ^ 1, j);
            read_x((S + 1) & 3, j);
            constexpr int D = IT == 4 ? 0 : 0;
            if (j == D || IT == 1) load_w(t + 3, (S + 3) & 3, 0), load_w(t + 3, (S + 3) & 3, 1);
            if (IT == 1) load_x(t + 3, (S + 3) & 3, 0);
            if (IT > 1 && j == D + 1) {
#pragma unroll
                for (int u = 0; u < kPerWave; ++u) load_x(t + 3, (S + 3) & 3, u);
            }
            if (S & 1 && j == IT - 1) load_scales(t + 3, ((S + 3) >> 1) & 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_sched_barrier(0);
        // all but this step's own loads are there: what the next step reads
        if (S & 1) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads + 1) : "memory");
        else asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    using C0 = std::integral_constant<int, 0>;
    using C1 = std::integral_constant<int, 1>;
    using C2 = std::integral_constant<int, 2>;
    using C3 = std::integral_constant<int, 3>;
    int t = 0;
    for (; t + 4 <= steps; t += 4) {
        step(t, C0{});
        step(t + 1, C1{});
        step(t + 2, C2{});
        step(t + 3, C3{});
    }
    if (t < steps) {
        step(t, C0{});
        step(t + 1, C1{});
    }
    // loads into stages nobody reads may still be on the way: wait for them before
    // the workgroup's LDS goes to another
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    if (split) {
        float* mine = a.sums + size_t(slot) * (kRows * kTokens);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < IT; ++j)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    *reinterpret_cast<float4v*>(mine + (wt + 32 * j + c) * kRows + wn + 32 * i + 2 * r + 4 * q) =
                        float4v{acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < IT; ++j)
            store_tile(acc[i][j], a, n0 + wn + 32 * i, m0 + wt + 32 * j + c, q);
}

// ---- many tokens: 256 x 256 tiles, 8-bit matrix instructions ----

constexpr int kScalePitch = 52;      // LDS bytes of a row's scales: 48, and 4 so that rows meet different banks
constexpr int kSegment = 48;         // groups whose scales are in LDS at a time
constexpr int kBigLds = 2 * 32768 + 4 * 16384 + 512 * kScalePitch;
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void f8_gemm_big_kernel(const Args a) {
    constexpr int kTokens = 256;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const uint32_t lds = uint32_t(uintptr_t((__attribute__((address_space(3))) uint8_t*)(smem)));
    const uint32_t x_lds = lds + 65536, scale_lds = lds + 131072;

    int tile, sp = 0, slot = 0;
    bool split = false;
    if (int(blockIdx.x) < 8 * a.chunk_a) {
        tile = int(blockIdx.x & 7) * a.chunk_a + int(blockIdx.x >> 3);
        if (tile >= a.whole) return;
    } else {
        const int u = int(blockIdx.x) - 8 * a.chunk_a;
        slot = (u & 7) * a.chunk_b + (u >> 3);
        if (slot >= (a.tiles - a.whole) * a.splits) return;
        tile = a.whole + slot / a.splits;
        sp = slot % a.splits;
        split = a.splits > 1;
    }
    int64_t m0, n0;
    tile_origin(a, tile, kTokens, n0, m0);
    const int g0 = split ? int(int64_t(sp) * a.groups / a.splits) : 0;
    const int g1 = split ? int(int64_t(sp + 1) * a.groups / a.splits) : a.groups;
    const int blocks = g1 - g0;

    const int tid = threadIdx.x, l = tid & 63, q = l >> 5, c = l & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = 64 * (wave & 3), half = wave >> 2, wt = 128 * half;

    const uint8_t* const wb = uniform(a.w + n0 * a.k + int64_t(g0) * 128);
    const uint8_t* const xb = uniform(a.x + m0 * a.k + int64_t(g0) * 128);
    const uint32_t k32 = uint32_t(a.k);
    const int64_t left_n = a.n - n0, left_m = a.m - m0;
    const auto row_n = [&](int r) { return uint32_t(r < left_n ? r : left_n - 1); };   // rows past the end: the last
    const auto row_m = [&](int r) { return uint32_t(r < left_m ? r : left_m - 1); };
    uint32_t w_off[4], x_off[2][2];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        w_off[u] = row_n(8 * (4 * wave + u) + (l >> 3)) * k32 + 16u * uint32_t((l & 7) ^ (4 * (u & 1) + (l >> 4)));
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = 8 * (2 * wave + u) + (l >> 3);
            x_off[p][u] = row_m(128 * (r >> 6) + 64 * p + (r & 63)) * k32 + 16u * uint32_t((l & 7) ^ (4 * (u & 1) + (l >> 4)));
        }
    const auto load_w = [&](int b, uint32_t s, int u) {
        load_lds16(wb + 128u * uint32_t(b < blocks ? b : blocks - 1), w_off[u], lds + s * 32768u + uint32_t(4 * wave + u) * 1024u);
    };
    const auto load_x = [&](int b, int p, uint32_t s, int u) {
        load_lds16(xb + 128u * uint32_t(b < blocks ? b : blocks - 1), x_off[p][u], x_lds + s * 16384u + uint32_t(2 * wave + u) * 1024u);
    };
    // scales of groups [s0, s0 + 48) of the tile's rows, a row a lane
    const auto stage_scales = [&](int s0) {
        const uint8_t* from =
            (tid < 256 ? a.ws + (n0 + row_n(tid)) * a.groups : a.xs + (m0 + row_m(tid - 256)) * a.groups) + g0 + s0;
        const int left = blocks - s0;
        lds_u32* to = reinterpret_cast<lds_u32*>(scale_lds + uint32_t(tid) * kScalePitch);
        uint32_t v[kSegment / 4] = {};
#pragma unroll
        for (int j = 0; j < kSegment / 4; ++j)
            if (4 * j + 4 <= left) __builtin_memcpy(&v[j], from + 4 * j, 4);
#pragma unroll
        for (int j = 0; j < kSegment / 4; ++j) to[j] = v[j];
        if (left < kSegment)
            for (int e = left & ~3; e < left; ++e) reinterpret_cast<lds_u8*>(to)[e] = from[e];
    };

    const uint32_t f = uint32_t(c) * 128u + 16u * uint32_t((2 * q) ^ ((c >> 1) & 7));
    uint32_t w_at[2][2], x_at[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            w_at[h][e] = lds + uint32_t(wn) * 128u + (f ^ (64u * h) ^ (16u * e));
            x_at[h][e] = x_lds + uint32_t(half) * 8192u + (f ^ (64u * h) ^ (16u * e));
        }
    const auto fragment = [&](uint32_t lo_at, uint32_t hi_at) {
        const u32x4 lo = *reinterpret_cast<lds_u32x4*>(lo_at), hi = *reinterpret_cast<lds_u32x4*>(hi_at);
        return int8v{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]), int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
    };
    int8v wf[2][2], xf[2][2];     // [h][i], [h][jj]
    int wsc[2], wsn[2], xsc[2][2];
    // (flip: 32768 where the block after the current one's is meant, whose stages lie there)
    const auto read_w = [&](uint32_t flip, int h, int i) {
        const uint32_t at = uint32_t(i) * 4096u;
        return fragment((w_at[h][0] ^ flip) + at, (w_at[h][1] ^ flip) + at);
    };
    const auto read_x = [&](uint32_t flip, int p, int h, int jj) {
        const uint32_t at = uint32_t(p) * 16384u + uint32_t(jj) * 4096u;
        return fragment((x_at[h][0] ^ flip) + at, (x_at[h][1] ^ flip) + at);
    };
    uint32_t ws_at = scale_lds + uint32_t(wn + c) * kScalePitch, xs_at = scale_lds + uint32_t(256 + wt + c) * kScalePitch;
    const auto read_ws = [&](int (&v)[2], uint32_t g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = *reinterpret_cast<lds_u8*>(ws_at + g + 32u * kScalePitch * uint32_t(i));
    };
    const auto read_xs = [&](uint32_t g, int p) {
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) xsc[p][jj] = *reinterpret_cast<lds_u8*>(xs_at + g + 32u * kScalePitch * uint32_t(2 * p + jj));
    };

    float16v acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

#pragma unroll
    for (int u = 0; u < 4; ++u) load_w(0, 0, u);
#pragma unroll
    for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) load_x(t >> 1, t & 1, t, u);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_w(1, 1, u);
    stage_scales(0);
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 2; ++i) wf[0][i] = read_w(0, 0, i);
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) xf[0][jj] = read_x(0, 0, 0, jj);
    read_ws(wsc, 0);
    read_xs(0, 0);

    for (int s0 = 0;;) {
    const int end = blocks < s0 + kSegment ? blocks : s0 + kSegment;
#pragma unroll 1
    for (int b = s0; b < end; ++b) {
        const uint32_t par = uint32_t(b) & 1;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            // K half 0, then 1: what a half no longer needs is read for its next use
            constexpr int E = 4;        // matrix instructions of a half
#pragma unroll
            for (int e = 0; e < 2 * E; ++e) {
                const int h = e / E, i = (e % E) >> 1, jj = e & 1;
                acc[i][2 * p + jj] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    wf[h][i], xf[h][jj], acc[i][2 * p + jj], 0, 0, 0, wsc[i], 0, xsc[p][jj]);
                if (e < 2) xf[1][e] = read_x(0, p, 1, e);
                if (p == 0 && e < E) {
                    if (e == 1 || e == 2) wf[1][e - 1] = read_w(0, 1, e - 1);
                }
                if (p == 0 && e == E) read_xs(0, 1);
                if (e >= E && e < E + 2) xf[0][e - E] = read_x(p ? 32768u : 0u, p ^ 1, 0, e - E);
                if (p == 1 && (e == E + 1 || e == E + 2)) wf[0][e - E - 1] = read_w(32768u, 0, e - E - 1);
                if (p == 1 && e == E) read_ws(wsn, 1);
                if (p == 1 && e == E + 1) read_xs(1, 0);
                if (p == 0) {
                    if (e % 4 == 1) load_x(b + 1, 1, (2 * (par ^ 1)) + 1, e / 4);
                } else {
                    if (e % 4 == 1) load_x(b + 2, 0, 2 * par, e / 4);
                    else if (e % 4 != 3) load_w(b + 2, par, 2 * (e / 4) + (e % 4 == 2));
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            // all but this phase's own loads are there: what the next phase reads
            if (p) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(6) : "memory");
            else asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(2) : "memory");
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) w_at[h][e] ^= 32768u, x_at[h][e] ^= 32768u;
        ws_at += 1;
        xs_at += 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) wsc[i] = wsn[i];
    }
    s0 = end;
    if (s0 >= blocks) break;
    __syncthreads();    // (the last reads of scales)
    stage_scales(s0);
    __syncthreads();
    ws_at -= kSegment;
    xs_at -= kSegment;
    read_ws(wsc, 0);
    read_xs(0, 0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    if (split) {
        float* mine = a.sums + size_t(slot) * (kRows * kTokens);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    *reinterpret_cast<float4v*>(mine + (wt + 32 * j + c) * kRows + wn + 32 * i + 2 * r + 4 * q) =
                        float4v{acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
        return;
    }
    // through LDS, 128 tokens by 64 weight rows a wave, so that a store writes whole
    // cache lines: chunk e of 8 weight rows of a token in another place for each token
    asm volatile("s_barrier" ::: "memory");
        const auto place = [&](int token, int e) { return uint32_t(token) * 128u + 16u * uint32_t(e ^ ((token >> 1) & 7)); };
    const uint32_t mine = lds + 16384u * uint32_t(wave);
    const auto pair = [&](float u, float v) {
        return a.y_dtype == TL_F16 ? f16_bits(u) | f16_bits(v) << 16 : bf16_pair(u, v);
    };
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                const float16v& v = acc[i][j];
                const auto s0 = __builtin_amdgcn_permlane32_swap(pair(v[4 * g], v[4 * g + 1]), pair(v[4 * g + 4], v[4 * g + 5]), false, false);
                const auto s1 = __builtin_amdgcn_permlane32_swap(pair(v[4 * g + 2], v[4 * g + 3]), pair(v[4 * g + 6], v[4 * g + 7]), false, false);
                *reinterpret_cast<lds_u32x4*>(mine + place(32 * j + c, 4 * i + g + q)) = u32x4{s0[0], s1[0], s0[1], s1[1]};
            }
    const int64_t n = n0 + wn + 8 * ((l & 7));
    const bool whole_lines = a.n % 64 == 0;
#pragma unroll
    for (int z = 0; z < 16; ++z) {
        const int r = (8) * z + (l >> 3);
        const u32x4 v = *reinterpret_cast<lds_u32x4*>(mine + place(r, l & 7));
        const int64_t token = m0 + wt + r;
        if (token >= a.m) continue;
        uint16_t* y = static_cast<uint16_t*>(a.y) + token * a.n + n;
        if (n + 8 <= a.n) {
            if (whole_lines) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y));
            else __builtin_memcpy(y, &v, 16);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (n + k < a.n) y[k] = uint16_t(v[k >> 1] >> (16 * (k & 1)));
        }
    }
}

// The parts of a tile's sums added in their order
template <int IT>
__global__ __launch_bounds__(256) void f8_join_kernel(const Args a) {
    constexpr int kTokens = 64 * IT;
    // 8 weight rows of a token a lane
    const int t = int(blockIdx.x) / (kTokens / 8), e = 8 * (int(blockIdx.x) % (kTokens / 8)) + int(threadIdx.x >> 5);
    int64_t m0, n0;
    tile_origin(a, a.whole + t, kTokens, n0, m0);
    const int64_t token = m0 + e, n = n0 + 8 * (threadIdx.x & 31);
    if (token >= a.m) return;
    const float4v* parts = reinterpret_cast<const float4v*>(a.sums + size_t(t) * a.splits * (kRows * kTokens) + e * kRows) + 2 * (threadIdx.x & 31);
    float4v lo = parts[0], hi = parts[1];
    for (int p = 1; p < a.splits; ++p) {
        parts += kRows * kTokens / 4;
        lo += parts[0];
        hi += parts[1];
    }
    const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    if (a.y_dtype == TL_F32) {
        float* y = static_cast<float*>(a.y) + token * a.n + n;
        if (n + 8 <= a.n) __builtin_memcpy(y, v, 32);
        else
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (n + k < a.n) y[k] = v[k];
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = a.y_dtype == TL_F16 ? f16_bits(v[2 * k]) | f16_bits(v[2 * k + 1]) << 16 : bf16_pair(v[2 * k], v[2 * k + 1]);
    uint16_t* y = static_cast<uint16_t*>(a.y) + token * a.n + n;
    if (n + 8 <= a.n) __builtin_memcpy(y, w, 16);
    else
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (n + k < a.n) y[k] = uint16_t(w[k >> 1] >> (16 * (k & 1)));
}

struct Plan {
    int it, splits;
    int64_t tiles_m, tiles_n, tiles, whole;
};

constexpr int64_t kMaxParts = 512;

Plan make_plan(int64_t m, int64_t n, int64_t k) {
    Plan p;
    p.it = m <= 64 ? 1 : m <= 128 ? 2 : 4;
    p.tiles_m = (m + 64 * p.it - 1) / (64 * p.it);
    p.tiles_n = (n + kRows - 1) / kRows;
    p.tiles = p.tiles_m * p.tiles_n;
    const int64_t cus = cu_count(), rem = p.tiles % cus, groups = k / 128;
    p.whole = p.tiles;
    p.splits = 1;
    double best = double(groups);
    for (int s = 2; rem && s <= 32 && s <= groups / 2 && rem * s <= kMaxParts; ++s) {
        const double cost = double((rem * s + cus - 1) / cus) * (double((groups + s - 1) / s) + 1.0) + 0.02 * double(rem * s) + 2.0;
        if (cost < best - 1.0) {
            best = cost;
            p.whole = p.tiles - rem;
            p.splits = s;
        }
    }
    return p;
}

template <int IT, bool WIDE>
hipError_t launch(Args a, const Plan& p, hipStream_t stream) {
    constexpr bool kBig = IT == 4 && !WIDE;
    const auto kernel = kBig ? f8_gemm_big_kernel : f8_gemm_kernel<IT, kBig || WIDE>;
    constexpr int lds = kBig ? kBigLds : 4 * (kRows + 64 * IT) * kStep + 2 * (kRows + 64 * IT) * 4;
    hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), lds);
    if (e != hipSuccess) return e;
    const int64_t items = (p.tiles - p.whole) * p.splits;
    a.tiles_m = int(p.tiles_m);
    a.tiles_n = int(p.tiles_n);
    a.tiles = int(p.tiles);
    a.whole = int(p.whole);
    a.splits = p.splits;
    a.chunk_a = int((p.whole + 7) / 8);
    a.chunk_b = int((items + 7) / 8);
    hipLaunchKernelGGL(kernel, dim3(unsigned(8 * (a.chunk_a + a.chunk_b))), dim3(kThreads), lds, stream, a);
    if (p.splits > 1) {
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(f8_join_kernel<IT>, dim3(unsigned(8 * IT * (p.tiles - p.whole))), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

constexpr int64_t kFewTokens = 64;

}  // namespace

int64_t f8_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (m <= kFewTokens) return 0;
    const Plan p = make_plan(m, n, k);
    return p.splits > 1 ? (p.tiles - p.whole) * p.splits * kRows * 64 * p.it * 4 : 0;
}

hipError_t launch_f8_gemm(const uint8_t* codes, const uint8_t* scales, const uint8_t* x, const uint8_t* x_scales,
                          int64_t m, int64_t n, int64_t k, void* y, int y_dtype, void* ws, hipStream_t stream) {
    if (m <= kFewTokens) return launch_f8_gemv(codes, scales, x, x_scales, m, n, k, y, y_dtype, stream);
    const Plan p = make_plan(m, n, k);
    const Args a = {codes, scales, x, x_scales, y, static_cast<float*>(ws), m, n, k, y_dtype, int(k / 128), 0, 0, 0, 0, 0, 0, 0};
    if (y_dtype == TL_F32)
        return p.it == 1 ? launch<1, true>(a, p, stream) : p.it == 2 ? launch<2, true>(a, p, stream) : launch<4, true>(a, p, stream);
    return p.it == 1 ? launch<1, false>(a, p, stream) : p.it == 2 ? launch<2, false>(a, p, stream) : launch<4, false>(a, p, stream);
}

}  // namespace tl
