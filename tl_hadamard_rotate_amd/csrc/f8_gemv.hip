// Product of few tokens (or few weights) in 8-bit floating point, exact products:
//
//   y[m, n] = sum_k X[m, k] * W[n, k],   X, W = e4m3 code * 2^(scale of its 128)
//
// code * scale is a bfloat16 number: one instruction makes two of them, and
// v_mfma_f32_16x16x32_bf16 multiplies them exactly and sums in fp32.  (The 8-bit
// matrix instructions would gain nothing: few tokens are bound by the weights' bytes.)
//
// 16 weight rows are the A rows, 16 tokens (or twice 16) the B columns; absent tokens
// repeat the last.  Lane (q, c) = (lane / 16, lane % 16) takes 32 bytes of row c of a
// chunk of 128, at 32 q: which of the chunk's places a matrix instruction sums is free
// as long as both operands agree.
//
// Every wave works on its own: R tiles of 16 weight rows, a run of K's chunks, and
// a ring of D of them in its own LDS, filled by loads that write LDS directly and
// whose waits are counted by hand (through registers, with the compiler's waits, a
// wave had hardly more than one chunk on the way: 17408 x 5120 of one token 43 us,
// now 20).  A load takes whole cache lines, 128 bytes of each of 8 rows.  The
// activations of a chunk come through the same ring.  A workgroup is the `ks` waves
// that share a tile, each a run of the chunks; their sums meet in LDS in order.
// Scales, one byte of each row a chunk, come 32 chunks at a time.
//
// Bound: the weights' bytes from HBM.  In a graph, weights not in the caches: 131072
// x 5120 of one token 108 us (6.2 TB/s), 17408 x 5120 of one 20 us, of sixteen 24,
// 5120 x 17408 of one 21, 1024 x 5120 of one 6.0 (bound by one wave's loads, one
// after another).
#include "elem.h"
#include "f8.h"
#include "tl_internal.h"

namespace tl {
namespace {

using namespace elem;
using namespace f8;

typedef float float4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) float4v lds_float4;

constexpr int kDepth = 3;        // chunks of the ring
constexpr int kSegment = 32;     // chunks whose scales a wave holds at a time
constexpr int kScaleRow = 40;    // LDS bytes of a row of them: 8-byte aligned, 16 rows on different banks

struct Args {
    const uint8_t *codes, *scales, *x, *xs;
    void* y;
    int64_t m, n, k;
    int y_dtype, chunks, ks;
};

// 16 bytes a lane from its address to LDS, lane i at `to` + 16 i.  Written out: the
// compiler would make every read of LDS wait for every load on the way there.
template <bool NT>
__device__ __forceinline__ void load_lds16(const uint8_t* from, uint32_t to) {
    if (NT) asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(to), "v"(from) : "memory", "m0");
    else asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory", "m0");
}

// scales [s0, s0 + 32) of 16 rows to LDS: lane 4 r + p brings 8 of row r, `from`
// being that row's; where the row ends in a word, the row's last word is shifted
__device__ __forceinline__ void stage_scales(const uint8_t* from, int s0, int chunks, uint32_t lds, int l) {
    const int i = s0 + 8 * (l & 3);
    uint32_t w[2] = {};
    if (chunks >= 4) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int at = i + 4 * j, in = at < chunks - 4 ? at : chunks - 4, off = at - in < 3 ? at - in : 3;
            uint32_t v;
            __builtin_memcpy(&v, from + in, 4);
            w[j] = v >> (8 * off);
        }
    } else {
        for (int j = 0; j < 3; ++j)
            if (i + j < chunks) w[0] |= uint32_t(from[i + j]) << (8 * j);
    }
    *reinterpret_cast<lds_u32x2*>(lds + kScaleRow * uint32_t(l >> 2) + 8u * uint32_t(l & 3)) = u32x2{w[0], w[1]};
}

template <int R, int XI>
constexpr int wave_bytes() { return kDepth * (2 * R + XI) * 1024 + 16 * kScaleRow * (R + (XI + 1) / 2); }

// R tiles of 16 weight rows a wave, XI loads of 8 tokens, T tiles of 16 of them
template <int R, int XI>
__global__ __launch_bounds__(512) void f8_gemv_kernel(const Args a) {
    constexpr int T = (XI + 1) / 2, kLoads = 2 * R + XI, kSlot = kLoads * 1024, kWave = wave_bytes<R, XI>();
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int l = threadIdx.x & 63, q = l >> 4, c = l & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t ring = lds_address(smem) + uint32_t(wave) * kWave, scales = ring + kDepth * kSlot;
    const int64_t n0 = 16 * R * int64_t(blockIdx.x);
    const auto row = [&](int i) { return n0 + i < a.n ? n0 + i : a.n - 1; };
    const int64_t m0 = 16 * T * int64_t(blockIdx.y);
    const auto token = [&](int i) { return m0 + i < a.m ? m0 + i : a.m - 1; };

    // lane i of a load brings the piece of row i / 8 that belongs in place i % 8, piece
    // (i % 8) ^ (row / 2) % 8: 16 rows read at one piece meet all banks
    const int c0 = int(int64_t(wave) * a.chunks / a.ks), c1 = int(int64_t(wave + 1) * a.chunks / a.ks);
    const uint8_t* wp[2 * R];
    const uint8_t* xp[XI];
#pragma unroll
    for (int u = 0; u < 2 * R; ++u)
        wp[u] = a.codes + row(8 * u + (l >> 3)) * a.k + 16 * ((l & 7) ^ (4 * (u & 1) + (l >> 4))) + 128 * int64_t(c0);
#pragma unroll
    for (int u = 0; u < XI; ++u)
        xp[u] = a.x + token(8 * u + (l >> 3)) * a.k + 16 * ((l & 7) ^ (4 * (u & 1) + (l >> 4))) + 128 * int64_t(c0);
    const auto load = [&](int t, uint32_t slot) {       // chunk t of the wave's (past them: the last again)
        const int64_t at = 128 * int64_t(t < c1 - c0 ? t : c1 - c0 - 1);
#pragma unroll
        for (int u = 0; u < 2 * R; ++u) load_lds16<true>(wp[u] + at, slot + 1024u * u);
#pragma unroll
        for (int u = 0; u < XI; ++u) load_lds16<false>(xp[u] + at, slot + 1024u * (2 * R + u));
    };
    // (of 8 tokens the lanes from 8 on read the first again, and drop what they get)
    const int ct = XI == 1 ? c & 7 : c;
    const uint32_t fw = uint32_t(c) * 128u + 16u * uint32_t((2 * q) ^ ((c >> 1) & 7));
    const uint32_t fx = uint32_t(ct) * 128u + 16u * uint32_t((2 * q) ^ ((ct >> 1) & 7)) + 2048u * R;

    float4v acc[R][T] = {};
#pragma unroll
    for (int i = 0; i < kDepth; ++i) load(i, ring + uint32_t(i) * kSlot);
    uint32_t slot = ring;
    for (int s0 = c0; s0 < c1; s0 += kSegment) {
        const int s1 = s0 + kSegment < c1 ? s0 + kSegment : c1;
#pragma unroll
        for (int r = 0; r < R; ++r)
            stage_scales(a.scales + row(16 * r + (l >> 2)) * a.chunks, s0, a.chunks, scales + 16 * kScaleRow * r, l);
#pragma unroll
        for (int j = 0; j < T; ++j)
            stage_scales(a.xs + token(16 * j + (l >> 2)) * a.chunks, s0, a.chunks, scales + 16 * kScaleRow * (R + j), l);
        uint32_t sw_at = scales + kScaleRow * uint32_t(c), sx_at = scales + kScaleRow * uint32_t(16 * R + ct);
#pragma unroll 1
        for (int t = s0; t < s1; ++t, ++sw_at, ++sx_at) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads * (kDepth - 1)) : "memory");
            u32x4 w[R][2], x[T][2];
            uint32_t sw[R], sx[T];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int r = 0; r < R; ++r) w[r][e] = *reinterpret_cast<lds_u32x4*>(slot + (fw ^ (16u * e)) + 2048u * r);
#pragma unroll
                for (int j = 0; j < T; ++j) x[j][e] = *reinterpret_cast<lds_u32x4*>(slot + (fx ^ (16u * e)) + 2048u * j);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) sw[r] = *reinterpret_cast<lds_u8*>(sw_at + 16 * kScaleRow * r);
#pragma unroll
            for (int j = 0; j < T; ++j) sx[j] = *reinterpret_cast<lds_u8*>(sx_at + 16 * kScaleRow * j);
            // what the slot held is in registers before the ring's next chunk takes its place
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            load(t - c0 + kDepth, slot);
            slot = slot == ring + (kDepth - 1) * kSlot ? ring : slot + kSlot;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                bf8v wv[R];
#pragma unroll
                for (int r = 0; r < R; ++r) wv[r] = widen(w[r][h >> 1][2 * (h & 1)], w[r][h >> 1][2 * (h & 1) + 1], sw[r]);
#pragma unroll
                for (int j = 0; j < T; ++j) {
                    const bf8v xv = widen(x[j][h >> 1][2 * (h & 1)], x[j][h >> 1][2 * (h & 1) + 1], sx[j]);
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[r], xv, acc[r][j], 0, 0, 0);
                }
            }
        }
    }
    // no load may write LDS once its place is used otherwise, or another workgroup's
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    if (a.ks > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < R * T; ++i) *reinterpret_cast<lds_float4*>(ring + 1024u * i + 16u * l) = acc[i / T][i % T];
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (int i = 0; i < R * T; ++i)
            for (int p = 1; p < a.ks; ++p) acc[i / T][i % T] += *reinterpret_cast<lds_float4*>(ring + p * kWave + 1024u * i + 16u * l);
    }
    // lane (q, c) holds rows 4 q .. 4 q + 3 of a tile for token c
#pragma unroll
    for (int j = 0; j < T; ++j) {
        const int64_t m = m0 + 16 * j + c;
        if (m >= a.m) continue;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t n = n0 + 16 * r + 4 * q + e;
                if (n >= a.n) continue;
                if (a.y_dtype == TL_F32) static_cast<float*>(a.y)[m * a.n + n] = acc[r][j][e];
                else
                    static_cast<uint16_t*>(a.y)[m * a.n + n] =
                        uint16_t(a.y_dtype == TL_F16 ? f16_bits(acc[r][j][e]) : bf16_bits(acc[r][j][e]));
            }
    }
}

template <int R, int XI>
hipError_t launch(Args a, int64_t waves, hipStream_t stream) {
    const auto kernel = f8_gemv_kernel<R, XI>;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), 160 * 1024);
    if (e != hipSuccess) return e;
    const int64_t tiles = (a.n + 16 * R - 1) / (16 * R);
    constexpr int most = 160 * 1024 / wave_bytes<R, XI>();
    int64_t ks = (waves + tiles / 2) / tiles;
    ks = ks > 8 ? 8 : ks;
    ks = ks > most ? most : ks;
    ks = ks > a.chunks ? a.chunks : ks;
    a.ks = ks < 1 ? 1 : int(ks);
    const dim3 grid(unsigned(tiles), unsigned((a.m + 8 * XI - 1) / (8 * XI)));
    hipLaunchKernelGGL(kernel, grid, dim3(64 * a.ks), unsigned(a.ks * wave_bytes<R, XI>()), stream, a);
    return hipGetLastError();
}

}  // namespace

// More than 16 tokens come in blocks of 32 where the product is so small that the other
// kernels would cut K and add the parts in a second launch: up to one workgroup a compute
// unit and 64 chunks, sixteen a wave.  us in a graph, weights not in the caches, here and in
// the others' tiles with fp32 sums: 2048 x 2048 by 17, 64 tokens 6.1 8.2, 6.8 9.1;
// 1024 x 5120 by 17, 32, 64, 128 8.3 9.4, 9.6 9.7, 9.4 10.2, 9.5 10.9; 1024 x 7168 by 32,
// 128 10.5 11.5, 10.4 13.1; 2048 x 8192 by 32, 64 11.6 12.5, 11.4 13.6.  The others are
// ahead with 32 tokens and few rows (256 x 7168 10.2 9.9, 512 x 5120 9.3 8.4) and where
// little K needs no cut (512 x 512 4.7 4.5, 4096 x 640 by 32 6.0 5.6); of more workgroups
// (1024 x 7168 by 160 16.5 12.9, 1536 x 5120 by 80 13.0 11.2) and of longer rows (1024 x
// 10240 by 32, 64 14.3 11.6, 14.2 12.3).  Called one by one, with that second launch and
// its workspace, 16 x 2560 by 18 takes 11.4 there and 6.4 here.  The 8-bit instructions'
// sums would gain little on it: 1024 x 5120 by 32, 64 9.2, 10.1.
bool f8_gemv_fits(int64_t m, int64_t n, int64_t k) {
    return m <= 16 || (k <= 8192 && ((n + 15) / 16) * ((m + 31) / 32) <= 256);
}

// Waves share a tile until there are about 1024 (512 where each brings 16 tokens'
// activations too); from 320 tiles on, two tiles a wave share those.  Measured, us in
// a graph with 1 .. 8 waves a tile: 17408 x 5120 of one token 19.7 20.4 21.0 20.3
// .. 24, 5120 x 17408 36 25 21.1 21.3 .. 23, 1024 x 5120 14 8.6 7.0 6.2 6.0 6.2 ..;
// sixteen tokens, one and two tiles: 32003 x 5120 36.9 and 34.6, 5120 x 17408 27 and
// 25.4, 1024 x 5120 7.3 and 8.5.
hipError_t launch_f8_gemv(const uint8_t* codes, const uint8_t* scales, const uint8_t* x, const uint8_t* x_scales,
                          int64_t m, int64_t n, int64_t k, void* y, int y_dtype, hipStream_t stream) {
    const Args a = {codes, scales, x, x_scales, y, m, n, k, y_dtype, int(k / 128), 1};
    if (m <= 8) return launch<1, 1>(a, 1024, stream);
    if (m <= 16) return n >= 16 * 320 ? launch<2, 2>(a, 512, stream) : launch<1, 2>(a, 512, stream);
    return launch<1, 4>(a, 4 * ((n + 15) / 16), stream);
}

}  // namespace tl
