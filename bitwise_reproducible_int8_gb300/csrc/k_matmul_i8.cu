// k_matmul_i8.cu -- product of 8-bit codes with a scale for each row of both sides, in the three
// layouts of a linear's training step.
//
//   y_mn = (i2f(sum_k A(m, k) B(n, k)) (x) s_a[m]) (x) s_b[n], the integer sum exact
//
// As in k_fwd_tc.cu the codes go to tcgen05.mma kind::f16 (as fp16, exact), fp32 accumulators over
// slices of 512 terms (integers below 2^23, exact), the slices added up in int32.  What differs:
//   * the widening pass also transposes (a reduction over tokens has its operands the other way
//     round) and pads the rows, so any K, stride and layout reaches the tensor cores;
//   * two SMs work on one 256 x 256 tile (cta_group::2): each loads its 128 rows of A and half of B,
//     32 KB for 64 terms of K instead of 48 KB, because with one SM a tile of 128 x 256 the operands'
//     way from L2 bound the product, not the tensor pipe;
//   * the epilogue has a scale for each of its rows and columns.
// Products of few tokens are bound by the weights' bytes: up to 4 on the CUDA cores (k_mm_rows, k_mm_cols),
// up to 128 in k_matmul_few.cu.
//
// Measured, 16384 x 11264 x 2048 with fp32 results: 475 to 510 us (boards differ, and so does one board
// warm and cold), 25 of them the widened copies, beside 394 us of tensor work at cuBLAS's bf16 rate and
// 738 MB to store (with bf16 results 429 to 450); the input gradient's layout, 16384 x 2048 x 11264 by
// weights [K][N], 490 to 525 (394) and 16384 x 5632 x 2048 260 to 270 (197); 2048 x 5632 x 16384 with both
// sides transposed and added on: 281 to 294 us, 63 of them the copies.  What bounds it now is the way out: an
// accumulator is free again only once 16 warps have read it, and their results' stores take L2 from the
// operands.
//
// Roles in a CTA of the pair, as in k_fwd_tc.cu: warp 0 loads, warp 1 of the leading CTA issues the
// MMAs for both (warp 1 of the other holds its tensor memory), the others are the epilogue.  The
// leader's full barriers count both CTAs' bytes; an MMA's commit frees its stage, and hands over its
// accumulator, in both; both epilogues free the accumulator on the leader's barrier.  Every wait is
// bounded as there, with one outcome for a whole warp.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mm.cuh"
#include "pipeline.cuh"
#include "umma.cuh"

namespace repro {
namespace {

typedef unsigned long long u64;

// ---------------------------------------------------------------- operands to fp16

inline int64_t pad8(int64_t k) { return (k + 7) / 8 * 8; }
inline int64_t align256(int64_t b) { return (b + 255) & ~(int64_t)255; }

struct Widen {
    const int8_t* q;
    int64_t ld, rows, K, Kp;    // source rows of K (or, transposed, K rows of `rows`); pitch of the copy
    __half* out;
    const int8_t* end;          // behind the last code
    bool vec;                   // source rows on 8-byte (transposed: 16-byte) boundaries
};

// the `left` (at most 8) codes from p on, wherever p lies, 0 behind them: three words that cover them,
// shifted, where these lie within [lo, hi), else one by one
__device__ __forceinline__ uint2 codes8(const int8_t* p, int64_t left, const int8_t* lo, const int8_t* hi)
{
    uint32_t v[2] = {0, 0};
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3;
    if (left >= 8 && at >= reinterpret_cast<uintptr_t>(lo) && at + 12 <= reinterpret_cast<uintptr_t>(hi)) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(at);
        const uint32_t a = __ldg(q), b = __ldg(q + 1), c = __ldg(q + 2), s = 8 * (uint32_t)(reinterpret_cast<uintptr_t>(p) & 3);
        v[0] = __funnelshift_r(a, b, s);
        v[1] = __funnelshift_r(b, c, s);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left)
                v[e >> 2] |= (uint32_t)(uint8_t)p[e] << (8 * (e & 3));
    }
    return make_uint2(v[0], v[1]);
}

// rows of K codes to rows of Kp fp16, zeros behind K; 8 at a time
__global__ void __launch_bounds__(256)
k_mm_widen(const __grid_constant__ Widen w)
{
    pdl_wait();
    pdl_trigger();
    const int64_t per = w.Kp / 8, total = w.rows * per, step = (int64_t)gridDim.x * blockDim.x;
    const bool flat = w.vec && w.K == w.Kp && w.ld == w.K;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        uint2 c;
        if (flat) {
            c = __ldg(reinterpret_cast<const uint2*>(w.q) + i);
        } else {
            const int64_t r = i / per, k = 8 * (i - r * per);
            const int8_t* p = w.q + r * w.ld + k;
            if (w.vec && k + 8 <= w.K) {
                c = __ldg(reinterpret_cast<const uint2*>(p));
            } else {
                c = codes8(p, w.K - k, w.q, w.end);
            }
        }
        const uint2 a = widen4(c.x), b = widen4(c.y);
        reinterpret_cast<uint4*>(w.out)[i] = make_uint4(a.x, a.y, b.x, b.y);
    }
}

// where word c (4 rows) of term k lies in a tile of 128 x 32 words: rotated so that neither the 4
// terms of a warp's stores nor the 8 octets of terms of its loads meet in a bank
__device__ __forceinline__ int tile_word(int k, int c) { return 32 * k + ((c + 4 * (k >> 3) + (k & 3)) & 31); }

// K rows of codes to `rows` rows of Kp fp16, through tiles of 128 terms x 128 rows in shared memory
__global__ void __launch_bounds__(256)
k_mm_widen_t(const __grid_constant__ Widen w, int tiles_r)
{
    __shared__ uint32_t tile[128 * 32];
    const int tr = blockIdx.x % tiles_r;
    const int64_t k0 = (int64_t)(blockIdx.x / tiles_r) * 128, r0 = (int64_t)tr * 128;
    pdl_wait();
    pdl_trigger();
    const int c16 = threadIdx.x & 7;                 // 16 rows of a term
    const int64_t r = r0 + 16 * c16;
    const bool whole = w.vec && r + 16 <= w.rows && k0 + 128 <= w.K;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t k = k0 + (threadIdx.x >> 3) + 32 * i;
        const int8_t* p = w.q + k * w.ld + r;
        if (whole) {
            asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                         : "l"(p));
        } else {
            uint32_t x[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (k < w.K && r + e < w.rows)
                    x[e >> 2] |= (uint32_t)(uint8_t)p[e] << (8 * (e & 3));
            v[i] = make_uint4(x[0], x[1], x[2], x[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = (threadIdx.x >> 3) + 32 * i;
        tile[tile_word(k, 4 * c16)] = v[i].x;
        tile[tile_word(k, 4 * c16 + 1)] = v[i].y;
        tile[tile_word(k, 4 * c16 + 2)] = v[i].z;
        tile[tile_word(k, 4 * c16 + 3)] = v[i].w;
    }
    __syncthreads();
    // 8 terms of 4 rows a step: 8 neighbouring threads write 128 bytes of each of the rows
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int kk = 8 * (threadIdx.x & 7) + 64 * h, c = threadIdx.x >> 3;
        if (k0 + kk >= w.Kp)
            break;
        uint32_t in[8], t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            in[i] = tile[tile_word(kk + i, c)];
#pragma unroll
        for (int q = 0; q < 2; ++q) {   // 4 x 4 bytes transposed
            const uint32_t a = __byte_perm(in[4 * q], in[4 * q + 1], 0x5140), b = __byte_perm(in[4 * q], in[4 * q + 1], 0x7362);
            const uint32_t c2 = __byte_perm(in[4 * q + 2], in[4 * q + 3], 0x5140), d = __byte_perm(in[4 * q + 2], in[4 * q + 3], 0x7362);
            t[q] = __byte_perm(a, c2, 0x5410);
            t[2 + q] = __byte_perm(a, c2, 0x7632);
            t[4 + q] = __byte_perm(b, d, 0x5410);
            t[6 + q] = __byte_perm(b, d, 0x7632);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int64_t row = r0 + 4 * c + b;
            if (row < w.rows) {
                const uint2 x = widen4(t[2 * b]), y = widen4(t[2 * b + 1]);
                *reinterpret_cast<uint4*>(w.out + row * w.Kp + k0 + kk) = make_uint4(x.x, x.y, y.x, y.y);
            }
        }
    }
}

cudaError_t widen(const int8_t* q, int64_t ld, int64_t rows, int64_t K, bool t, __half* out, cudaStream_t st)
{
    const size_t b = t ? 16 : 8;
    Widen w = {q, ld, rows, K, pad8(K), out, q + (t ? (K - 1) * ld + rows : (rows - 1) * ld + K), reinterpret_cast<uintptr_t>(q) % b == 0 && ld % (int64_t)b == 0};
    count_launches(1);
    if (t) {
        const int tiles_r = (int)((rows + 127) / 128);
        return launch_pdl(k_mm_widen_t, dim3((unsigned)(tiles_r * ((K + 127) / 128))), dim3(256), 0, st, w, tiles_r);
    }
    const int64_t want = (rows * (w.Kp / 8) + 255) / 256, most = (int64_t)num_sms() * 8;
    return launch_pdl(k_mm_widen, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st, w);
}

// ---------------------------------------------------------------- any shape on the CUDA cores

constexpr int FT = 64, KW = 16;

__device__ __forceinline__ int word_of(const int8_t* p, int64_t ld, bool t, int64_t row, int64_t rows, int64_t k, int64_t K)
{
    uint32_t w = 0;
    if (row < rows)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i < K)
                w |= (uint32_t)(uint8_t)p[t ? (k + i) * ld + row : row * ld + k + i] << (8 * i);
    return (int)w;
}

template <typename Y>
__global__ void __launch_bounds__(256)
k_mm_any(const __grid_constant__ MatmulI8Args g, int64_t tiles_n)
{
    __shared__ __align__(16) int As[KW][FT + 4];
    __shared__ __align__(16) int Bs[KW][FT + 4];
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * FT, n0 = (int64_t)(blockIdx.x % tiles_n) * FT;
    int acc[4][4] = {};
    pdl_wait();
    for (int64_t k0 = 0; k0 < g.K; k0 += 4 * KW) {
        for (int e = tid; e < FT * KW; e += 256) {
            const int ra = g.a_t ? e % FT : e / KW, wa = g.a_t ? e / FT : e % KW;
            const int rb = g.b_t ? e % FT : e / KW, wb = g.b_t ? e / FT : e % KW;
            As[wa][ra] = word_of(g.a, g.a_ld, g.a_t, m0 + ra, g.M, k0 + 4 * wa, g.K);
            Bs[wb][rb] = word_of(g.b, g.b_ld, g.b_t, n0 + rb, g.N, k0 + 4 * wb, g.K);
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            const int4 a = *reinterpret_cast<const int4*>(&As[w][4 * ty]), b = *reinterpret_cast<const int4*>(&Bs[w][4 * tx]);
            const int av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __dp4a(av[i], bv[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + 4 * ty + i, n = n0 + 4 * tx + j;
            if (m < g.M && n < g.N)
                put(static_cast<Y*>(g.y) + m * g.y_ld + n,
                    scaled(acc[i][j], g.s_a, g.s_a ? flush(__ldg(g.s_a + m)) : 0.0f, g.s_b, g.s_b ? flush(__ldg(g.s_b + n)) : 0.0f),
                    g.accumulate);
        }
}

// ---------------------------------------------------------------- few rows of A: the weights' bytes

constexpr int RM = 8;    // rows of A a pass

// this lane's part of the sums over a row of B, 16 codes at a time, against up to R rows of A (out of L1)
template <int R> __device__ __forceinline__ void rows_by_16(const MatmulI8Args& g, const int8_t* a, const int8_t* b, int64_t m0, int lane, int (&acc)[R])
{
#pragma unroll 4
    for (int64_t k = 16 * lane; k < g.K; k += 512) {
        const int4 v = __ldg(reinterpret_cast<const int4*>(b + k));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (R > 1 && m0 + r >= g.M)
                break;
            const int4 x = __ldg(reinterpret_cast<const int4*>(a + r * g.a_ld + k));
            acc[r] = __dp4a(x.x, v.x, __dp4a(x.y, v.y, __dp4a(x.z, v.z, __dp4a(x.w, v.w, acc[r]))));
        }
    }
}

// four codes from p on, wherever p lies, out of the two words that cover them
__device__ __forceinline__ int word_at(const int8_t* p)
{
    const uint32_t s = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 3);
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p - s);
    return (int)__funnelshift_r(__ldg(q), __ldg(q + 1), 8 * s);
}

// The same for any K and rows on any byte.  Groups of 4 codes from the fourth code on, neighbouring lanes
// neighbouring groups, as far as the words that cover them lie inside the row; the 11 codes at most that
// are left at its ends one a lane.  U: groups a lane has in flight.  (16 codes a lane, byte by byte, took
// 200 us for 16 x 11264 x 2049, 25 for one token; this takes 65 and 15, where 17 tokens take 36 through the
// widened copies.)
template <int U, int R> __device__ __forceinline__ void rows_by_4(const MatmulI8Args& g, const int8_t* a, const int8_t* b, int64_t m0, int lane, int (&acc)[R])
{
    const int K = (int)g.K, G = K < 12 ? 0 : (K - 8) / 4;
    for (int i0 = lane; i0 - lane < G; i0 += 32 * U) {
        int v[U], k[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 32 * u;
            k[u] = 4 + 4 * min(i, G - 1);      // a group past the last is the last, times 0
            const int w = word_at(b + k[u]);
            v[u] = i < G ? w : 0;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (R > 1 && m0 + r >= g.M)
                break;
#pragma unroll
            for (int u = 0; u < U; ++u)
                acc[r] = __dp4a(word_at(a + r * g.a_ld + k[u]), v[u], acc[r]);
        }
    }
    const int k = lane < 4 ? lane : 4 * G + lane;
    if (lane < 12 && k < K) {
        const int v = __ldg(b + k);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (R > 1 && m0 + r >= g.M)
                break;
            acc[r] += v * __ldg(a + r * g.a_ld + k);
        }
    }
}

// A warp takes a row of B at a time.  U 0: rows of both on 16-byte boundaries and K a multiple of 16; else
// of rows_by_4.
template <typename Y, int R, int U>
__global__ void __launch_bounds__(128)
k_mm_rows(const __grid_constant__ MatmulI8Args g)
{
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), m0 = (int64_t)blockIdx.y * R;
    pdl_wait();
    if (n >= g.N)
        return;
    int acc[R] = {};
    const int8_t* b = g.b + n * g.b_ld;
    const int8_t* a = g.a + m0 * g.a_ld;
    if (U == 0)
        rows_by_16(g, a, b, m0, lane, acc);
    else
        rows_by_4<U == 0 ? 1 : U>(g, a, b, m0, lane, acc);
#pragma unroll
    for (int r = 0; r < R; ++r)
        acc[r] = __reduce_add_sync(0xffffffffu, acc[r]);
    int mine = acc[0];
#pragma unroll
    for (int r = 1; r < R; ++r)
        mine = lane == r ? acc[r] : mine;
    if (lane < R && m0 + lane < g.M)
        put(static_cast<Y*>(g.y) + (m0 + lane) * g.y_ld + n,
            scaled(mine, g.s_a, g.s_a ? flush(__ldg(g.s_a + m0 + lane)) : 0.0f, g.s_b, g.s_b ? flush(__ldg(g.s_b + n)) : 0.0f),
            g.accumulate);
}

template <typename Y> cudaError_t run_rows(const MatmulI8Args& g, cudaStream_t st)
{
    const bool vec = reinterpret_cast<uintptr_t>(g.a) % 16 == 0 && reinterpret_cast<uintptr_t>(g.b) % 16 == 0 &&
                     (g.M == 1 || g.a_ld % 16 == 0) && (g.N == 1 || g.b_ld % 16 == 0) && g.K % 16 == 0;
    const dim3 grid((unsigned)((g.N + 3) / 4), (unsigned)(g.M == 1 ? 1 : (g.M + RM - 1) / RM));
    count_launches(1);
    if (g.M == 1)   // 2048 x 5633 by 8 groups 19 us, by 4 22; 1001 x 1001 by 8 2.9, by 4 2.5
        return vec          ? launch_pdl(k_mm_rows<Y, 1, 0>, grid, dim3(128), 0, st, g)
               : g.K > 1024 ? launch_pdl(k_mm_rows<Y, 1, 8>, grid, dim3(128), 0, st, g)
                            : launch_pdl(k_mm_rows<Y, 1, 4>, grid, dim3(128), 0, st, g);
    return vec ? launch_pdl(k_mm_rows<Y, RM, 0>, grid, dim3(128), 0, st, g)
               : launch_pdl(k_mm_rows<Y, RM, 4>, grid, dim3(128), 0, st, g);
}

// The same against b = [K][N].  A CTA takes 512 columns of B (16 a lane) and a slab of its rows, 4 rows a
// warp at a time: 4 x 4 codes are turned in registers and go to dp4a with 4 codes of each of the R rows
// of A.  The warps' sums meet in shared memory, the slabs' in the workspace (exact in any order).
// 1 x 4096 x 4096 8 us, 4 x 2048 x 5632 13 us; the widened copies and a tile for 256 tokens take 26.
constexpr int CN = 512;          // columns of a CTA

template <int R>
__global__ void __launch_bounds__(256, 2)
k_mm_cols(const __grid_constant__ MatmulI8Args g, int* sums, int slab, int slabs)
{
    __shared__ int red[8][CN];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n0 = (int64_t)(blockIdx.x / slabs) * CN, n = n0 + 16 * lane;
    const int part = blockIdx.x % slabs;
    const int64_t lo = (int64_t)part * slab, hi = lo + slab < g.K ? lo + slab : g.K;
    pdl_wait();
    pdl_trigger();
    const bool words = reinterpret_cast<uintptr_t>(g.a) % 4 == 0 && (g.M == 1 || g.a_ld % 4 == 0);   // slabs start on 32
    int acc[R][16] = {};
#pragma unroll 2
    for (int64_t k = lo + 4 * warp; k < hi; k += 32) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (k + i < hi && n < g.N)   // N is a multiple of 16
                v[i] = __ldg(reinterpret_cast<const uint4*>(g.b + (k + i) * g.b_ld + n));
        }
        int a[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint32_t w = 0;
            const int8_t* p = g.a + r * g.a_ld + k;
            if (r < g.M) {
                if (words && k + 4 <= hi) {
                    w = __ldg(reinterpret_cast<const uint32_t*>(p));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (k + i < hi)
                            w |= (uint32_t)(uint8_t)__ldg(p + i) << (8 * i);
                }
            }
            a[r] = (int)w;
        }
        const uint32_t in[4][4] = {{v[0].x, v[1].x, v[2].x, v[3].x}, {v[0].y, v[1].y, v[2].y, v[3].y},
                                   {v[0].z, v[1].z, v[2].z, v[3].z}, {v[0].w, v[1].w, v[2].w, v[3].w}};
#pragma unroll
        for (int c = 0; c < 4; ++c) {   // 4 x 4 bytes transposed
            const uint32_t p = __byte_perm(in[c][0], in[c][1], 0x5140), q = __byte_perm(in[c][0], in[c][1], 0x7362);
            const uint32_t x = __byte_perm(in[c][2], in[c][3], 0x5140), y = __byte_perm(in[c][2], in[c][3], 0x7362);
            const uint32_t t[4] = {__byte_perm(p, x, 0x5410), __byte_perm(p, x, 0x7632), __byte_perm(q, y, 0x5410),
                                   __byte_perm(q, y, 0x7632)};
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[r][4 * c + e] = __dp4a((int)t[e], a[r], acc[r][4 * c + e]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (r >= g.M)
            break;
        if (r > 0)
            __syncthreads();
#pragma unroll
        for (int c = 0; c < 16; c += 4)
            *reinterpret_cast<int4*>(&red[warp][16 * lane + c]) = make_int4(acc[r][c], acc[r][c + 1], acc[r][c + 2], acc[r][c + 3]);
        __syncthreads();
        for (int c = threadIdx.x; c < CN; c += 256) {
            int s = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w)
                s += red[w][c];
            if (n0 + c < g.N)
                sums[((int64_t)part * g.M + r) * g.N + n0 + c] = s;
        }
    }
}

template <typename Y>
__global__ void __launch_bounds__(128)
k_mm_cols_join(const __grid_constant__ MatmulI8Args g, const int* sums, int slabs)
{
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x, m = i / g.N, n = i - m * g.N;
    pdl_wait();
    if (i >= g.M * g.N)
        return;
    int s = 0;
#pragma unroll 16
    for (int k = 0; k < slabs; ++k)
        s += __ldcg(sums + (int64_t)k * g.M * g.N + i);
    put(static_cast<Y*>(g.y) + m * g.y_ld + n,
        scaled(s, g.s_a, g.s_a ? flush(__ldg(g.s_a + m)) : 0.0f, g.s_b, g.s_b ? flush(__ldg(g.s_b + n)) : 0.0f), g.accumulate);
}

// rows of a slab: two CTAs on every SM, but 32 rows at least and 16 slabs at most, which one thread's
// loads can have in flight when it adds them up (with 32, 1 x 4096 x 4096 took 9.6 us).  152 SMs,
// whatever the device: the workspace's size depends on it
int cols_slab(int64_t N, int64_t K)
{
    const int64_t tiles = (N + CN - 1) / CN, want = std::min<int64_t>(std::max<int64_t>(2 * 152 / tiles, 1), 16);
    return (int)(((K + want - 1) / want + 31) / 32 * 32);
}

bool cols_of(int64_t M, int64_t K, bool a_t, bool b_t) { return M <= 4 && !a_t && b_t && K > 0; }

size_t cols_ws_bytes(int64_t M, int64_t N, int64_t K)
{
    const int slab = cols_slab(N, K);
    return (size_t)((K + slab - 1) / slab * M * N * 4);
}

cudaError_t run_cols(const MatmulI8Args& g, int* sums, cudaStream_t st)
{
    const int slab = cols_slab(g.N, g.K), slabs = (int)((g.K + slab - 1) / slab);
    const dim3 grid((unsigned)((g.N + CN - 1) / CN * slabs)), join((unsigned)((g.M * g.N + 127) / 128));
    count_launches(2);
    cudaError_t e = g.M == 1 ? launch_pdl(k_mm_cols<1>, grid, dim3(256), 0, st, g, sums, slab, slabs)
                             : launch_pdl(k_mm_cols<4>, grid, dim3(256), 0, st, g, sums, slab, slabs);
    if (e == cudaSuccess)
        e = g.y_type == 0 ? launch_pdl(k_mm_cols_join<float>, join, dim3(128), 0, st, g, static_cast<const int*>(sums), slabs)
                          : launch_pdl(k_mm_cols_join<__nv_bfloat16>, join, dim3(128), 0, st, g, static_cast<const int*>(sums), slabs);
    return e;
}

// ---------------------------------------------------------------- tensor cores, two SMs a tile

constexpr int HM = 128;                   // rows of a tile that one CTA of the pair holds
constexpr int TN = 256;
constexpr int TK = 64;                    // terms a stage: one 128-byte swizzle row of fp16
constexpr int SLICE_KB = 8;               // stages an exact slice: 8 * 64 = 512 terms
constexpr int STAGES = 5;
constexpr int HALF_BYTES = HM * TK * 2;   // 16 KB: a CTA's rows of A, and as much of B
constexpr int STAGE_BYTES = 2 * HALF_BYTES;
constexpr int NBUF = 2;                   // accumulators of 256 columns
constexpr uint32_t TMEM_COLS = 512;
constexpr int EPI_WARPS = 16;
constexpr int EW = TN / (EPI_WARPS / 4);  // columns of a tile that an epilogue warp holds of 32 rows
constexpr int STG_BYTES = 4096;          // an epilogue warp's 32 rows x 128 bytes on their way out
constexpr int THREADS = 64 + 32 * EPI_WARPS;

struct Smem {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t dfull[NBUF];
    uint64_t dempty[NBUF];
    uint64_t done;
    uint32_t tmem_base;
    int failed;
};
constexpr size_t SMEM_BYTES = 1024 + (size_t)STAGES * STAGE_BYTES + EPI_WARPS * STG_BYTES + 256;
static_assert(sizeof(Smem) <= 256 && SMEM_BYTES <= 227 * 1024, "fits one SM's shared memory");

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// true in one lane of a whole warp
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// the address of this CTA's variable in CTA `rank` of the pair
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(su32(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// an arrival on a barrier of either CTA.  What it orders are tensor memory's reads, which the
// tcgen05 fences around it order
__device__ __forceinline__ void arrive_at(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// a tile into this CTA's shared memory, its bytes counted on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(su32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t dtmem, uint64_t a, uint64_t b, uint32_t acc)
{
    // kind::f16: fp32 accumulator, fp16 A and B, both K-major, M = 256, N = 256
    constexpr uint32_t id = (1u << 4) | ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(2 * HM >> 4) << 24);
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtmem),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

// arrives on the barrier at this place in both CTAs once the MMAs issued so far are done
__device__ __forceinline__ void commit_pair(uint64_t* bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(su32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 16 accumulator columns into registers, not waited for
__device__ __forceinline__ void tmem_ask16(uint32_t taddr, uint32_t* v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

// waits for what was asked for; it names the registers, so that no use of them comes before it
__device__ __forceinline__ void tmem_got16(uint32_t* v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

// 32 rows x 128 bytes from shared memory (128-byte swizzle) to y; the tensor map clips what lies outside
__device__ __forceinline__ void store_block(const CUtensorMap* map, const void* src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(su32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// p: on 32 bytes.  (Two stores of 16: 256 x 256 x 16384 27.0 us against 23.6, 1024 x 1024 x 16384 61 against 56)
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]));
}

// whether a scale's products with whole numbers below 2^31, and with another such scale, need no
// flush: they are zero, or not below 2^-120
__device__ __forceinline__ bool ample(float s) { return !(fabsf(s) < 0x1p-60f) || s == 0.0f; }

// How a product is cut: whole tiles in rounds over the pairs of SMs; the tiles of a last round that
// would leave most pairs idle are cut along K instead (the integer sums are exact, so any cut gives
// the same bits) and their parts added up by k_mm_join.  A cut has to save four slices, what the
// parts' way through memory costs.
struct Plan {
    int tiles_m, tiles_n, pairs;
    int whole, split, items;    // tiles 0 .. whole - 1, then the rest in `split` parts each
};

Plan plan_of(int64_t M, int64_t N, int64_t K)
{
    Plan p;
    p.tiles_m = (int)((M + 2 * HM - 1) / (2 * HM));
    p.tiles_n = (int)((N + TN - 1) / TN);
    p.pairs = std::max(1, num_sms() / 2);
    const int tiles = p.tiles_m * p.tiles_n, rest = tiles % p.pairs, slices = (int)((K + TK * SLICE_KB - 1) / (TK * SLICE_KB));
    p.split = rest > 0 ? std::min(p.pairs / rest, slices) : 1;
    if (slices - (slices + p.split - 1) / p.split < 4)
        p.split = 1;
    p.whole = p.split > 1 ? tiles - rest : tiles;
    p.items = p.whole + (tiles - p.whole) * p.split;
    return p;
}

constexpr int64_t PART_BYTES = 2 * HM * TN * 4;
constexpr int64_t PART_ALIGN = 32;     // of the cut tiles' sums, in a workspace that starts on 16

struct PairArgs {
    MatmulI8Args g;
    Plan p;
    int K;
    bool y_tma;          // rows of y on 16-byte boundaries
    int* parts;          // the cut tiles' sums, [part][256][256], on a 32-byte boundary
    int* err;
};

// Tiles in groups of 8 rows of tiles, column by column within a group: the 76 tiles of a round then
// share 8 blocks of A and about 10 of B, which stay in L2 beside the output that streams through it
__host__ __device__ __forceinline__ void tile_at(const Plan& p, int tile, int& m0, int& n0)
{
    const int per = 8 * p.tiles_n, group = tile / per, in = tile - group * per;
    const int rows = p.tiles_m - 8 * group < 8 ? p.tiles_m - 8 * group : 8;
    n0 = (in / rows) * TN;
    m0 = (8 * group + in % rows) * 2 * HM;
}

// An item: its tile, its part (-1: a whole tile) and its stages of K
struct Item {
    int m0, n0, part, kb0, kb1;
};

__device__ __forceinline__ Item item_at(const PairArgs& a, int i)
{
    const int KB = (a.K + TK - 1) / TK;
    Item t;
    t.part = -1, t.kb0 = 0, t.kb1 = KB;
    int tile = i;
    if (i >= a.p.whole) {
        const int j = i - a.p.whole, q = j / a.p.split, s = j - q * a.p.split, NS = (KB + SLICE_KB - 1) / SLICE_KB;
        tile = a.p.whole + q;
        if (a.p.split > 1) {
            t.part = j;
            t.kb0 = SLICE_KB * (int)((int64_t)NS * s / a.p.split);
            t.kb1 = min(KB, SLICE_KB * (int)((int64_t)NS * (s + 1) / a.p.split));
        }
    }
    tile_at(a.p, tile, t.m0, t.n0);
    return t;
}

// A warp's 32 rows x EW columns: scaled, added to what is there, stored.  own: the columns' scales,
// two a lane.  They go through the warp's buffer in blocks of 128 bytes a row (chunk k of row r at
// k ^ (r mod 8)): rows on 16-byte boundaries by one tensor store a block, others row by row (9034 x
// 9034 x 64 bf16 114 us; 754 by a lane's own row).  (Straight to memory, 4 lanes to a row's line after
// a turn by shuffles, 16384 x 11264 x 2048 took 46 us longer, although the operands' ring then has two
// stages more; a lane's own 32 bytes at a time took 34 us longer still.)
template <typename Y>
__device__ __forceinline__ void finish(const PairArgs& p, const CUtensorMap* map, const uint32_t (&acc)[EW], uint8_t* stg, int lane,
                                       float sa, const float (&own)[2], int r0, int n)
{
    constexpr int W = 128 / (int)sizeof(Y), E = W / 8;
    const MatmulI8Args& g = p.g;
    Y* row = static_cast<Y*>(g.y) + (int64_t)(r0 + lane) * g.y_ld;
    const bool live = r0 + lane < g.M;
    const bool fast = __all_sync(0xffffffffu, ample(sa) && ample(own[0]) && ample(own[1]));
    const u64 sa2 = pack2(sa, sa), z = pack2(-0.0f, -0.0f);
#pragma unroll
    for (int b = 0; b < EW; b += W) {
        if (n + b >= g.N)   // warp-uniform
            break;
        float o[W];
#pragma unroll
        for (int e = 0; e < W; e += 2) {
            const int c = b + e, from = c >> 1;
            u64 v = pack2(__int2float_rn((int)acc[c]), __int2float_rn((int)acc[c + 1]));
            if (g.s_a)
                v = fmul2_rn(v, sa2);
            if (!fast)
                v = fadd2_ftz(v, z);
            if (g.s_b)
                v = fmul2_rn(v, pack2(__shfl_sync(0xffffffffu, own[0], from), __shfl_sync(0xffffffffu, own[1], from)));
            if (!fast)
                v = fadd2_ftz(v, z);
            unpack2(v, o[e], o[e + 1]);
        }
        // added to the old values here: a reduction in L2 would not flush subnormals
        if (sizeof(Y) == 4 && g.accumulate && live && p.y_tma) {
#pragma unroll
            for (int e = 0; e < W; e += 4) {
                const int c = n + b + e;
                if (c + 4 <= g.N) {
                    const float4 old = load4(reinterpret_cast<const float*>(row) + c);
                    o[e] = fadd_ftz(old.x, o[e]), o[e + 1] = fadd_ftz(old.y, o[e + 1]);
                    o[e + 2] = fadd_ftz(old.z, o[e + 2]), o[e + 3] = fadd_ftz(old.w, o[e + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c + i < g.N)
                            o[e + i] = fadd_ftz(to_f32<Y>(row[c + i]), o[e + i]);
                }
            }
        }
        if (lane == 0)   // the buffer's last store has read it
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k)   // 16 bytes a step
            store16(reinterpret_cast<Y*>(stg + lane * 128 + 16 * (k ^ (lane & 7))), o + E * k);
        if (p.y_tma) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                store_block(map, stg, n + b, r0);
            continue;
        }
        // rows off 16-byte boundaries: row by row, neighbouring lanes neighbouring elements; old values come
        // 4 rows at a time (one at a time, 119 x 119 x 68 took 31 us)
        __syncwarp();
        for (int i = 0; i < 32 && r0 + i < g.M; i += 4)
#pragma unroll
            for (int e = lane; e < W; e += 32) {
                Y* at = static_cast<Y*>(g.y) + (int64_t)(r0 + i) * g.y_ld + n + b + e;
                float old[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    old[j] = g.accumulate && n + b + e < g.N && r0 + i + j < g.M ? to_f32<Y>(at[j * g.y_ld]) : 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float v = to_f32<Y>(*reinterpret_cast<const Y*>(stg + (i + j) * 128 + 16 * ((e / E) ^ ((i + j) & 7)) + e % E * sizeof(Y)));
                    if (n + b + e < g.N && r0 + i + j < g.M)
                        at[j * g.y_ld] = from_f32<Y>(g.accumulate ? fadd_ftz(old[j], v) : v);
                }
            }
        __syncwarp();
    }
}

// hands an accumulator back to the leader's MMA thread
__device__ __forceinline__ void release(uint32_t bar, int lane)
{
    fence_before();
    __syncwarp();
    if (lane == 0)
        arrive_at(bar);
}

__device__ __forceinline__ void turn_buffer(int& d, uint32_t& ph)
{
    d ^= 1;
    ph ^= d == 0;
}
static_assert(NBUF == 2, "turn_buffer");

// a slice's columns on top of what a warp holds, as floats or as int32; the next 16 come while
// these are added
template <bool FLOAT> __device__ __forceinline__ void add_slice(uint32_t (&acc)[EW], uint32_t at)
{
    uint32_t v[2][16];
    tmem_ask16(at, v[0]);
#pragma unroll
    for (int c = 0; c < EW / 16; ++c) {
        tmem_got16(v[c & 1]);
        if (c < EW / 16 - 1)
            tmem_ask16(at + 16 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float x = __uint_as_float(v[c & 1][e]);
            uint32_t& y = acc[16 * c + e];
            y = FLOAT ? __float_as_uint(__fadd_rn(__uint_as_float(y), x)) : y + (uint32_t)__float2int_rn(x);
        }
    }
}

template <typename Y>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
k_mm_pair(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
          const __grid_constant__ CUtensorMap map_y, const __grid_constant__ PairArgs p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u);
    uint8_t* A = base;                                   // STAGES x 16 KB
    uint8_t* B = base + STAGES * HALF_BYTES;             // STAGES x 16 KB
    uint8_t* STG = base + STAGES * STAGE_BYTES;          // EPI_WARPS x 4 KB
    Smem* sm = reinterpret_cast<Smem*>(STG + EPI_WARPS * STG_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm->full[s], 1);
            mbar_init(&sm->empty[s], 1);
        }
        for (int d = 0; d < NBUF; ++d) {
            mbar_init(&sm->dfull[d], 1);
            mbar_init(&sm->dempty[d], 2 * EPI_WARPS);
        }
        mbar_init(&sm->done, 1);
        sm->failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map_b)) : "memory");
    }
    __syncwarp();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&sm->tmem_base)),
                     "r"(TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    const uint32_t tmem = sm->tmem_base;
    pdl_wait();

    // Warps 0 and 1 go through their loops whole and one lane issues: addresses and descriptors stay in
    // uniform registers.  With one lane in the loops the issuing thread took 620 cycles for a stage
    // whose MMAs take 512
    if (warp == 0) {
        const uint32_t bar0 = peer_addr(&sm->full[0], 0);
        bool ok = true;
        int s = 0, ph = 1;   // stage, and the parity whose end frees it (of a fresh barrier: at once)
        int filled = 0;
        for (int i = pair; i < p.p.items && ok && !__any_sync(0xffffffffu, *(volatile int*)&sm->failed); i += pairs) {
            const Item t = item_at(p, i);
            const int ya = t.m0 + (int)rank * HM, yb = t.n0 + (int)rank * HM;
            for (int kb = t.kb0; kb < t.kb1; ++kb) {
                if (!mbar_wait_warp(&sm->empty[s], (uint32_t)ph)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    if (rank == 0)
                        mbar_expect_tx(&sm->full[s], 2 * STAGE_BYTES);
                    tma_load_pair(A + s * HALF_BYTES, &map_a, kb * TK, ya, bar0 + 8 * s);
                    tma_load_pair(B + s * HALF_BYTES, &map_b, kb * TK, yb, bar0 + 8 * s);
                }
                filled = min(filled + 1, STAGES);
                if (++s == STAGES)
                    s = 0, ph ^= 1;
            }
        }
        const int s1 = s, ph1 = ph;
        // the leader sees both CTAs' last copies land before either can exit (cluster_sync below):
        // of the last `filled` stages, the newest first
        if (rank == 0)
            for (; filled > 0; --filled) {
                if (--s < 0)
                    s = STAGES - 1, ph ^= 1;
                if (!mbar_wait_warp(&sm->full[s], (uint32_t)(ph ^ 1)))
                    ok = false;
            }
        // and either CTA the arrivals of its own stages' last products, which come from the leader's
        // tensor core: none may be on its way into a CTA that has exited
        s = s1, ph = ph1;
        for (int k = 0; k < STAGES && ok; ++k) {
            ok = mbar_wait_warp(&sm->empty[s], (uint32_t)ph);
            if (++s == STAGES)
                s = 0, ph ^= 1;
        }
        if (!ok && lane == 0)
            sm->failed = 1;
    } else if (warp == 1) {
        if (rank == 0) {
            const uint64_t a0 = sdesc(su32(A)), b0 = sdesc(su32(B));
            bool ok = true;
            int s = 0, ph = 0, d = 0, dph = 1;   // stage and accumulator, and the parities to wait for
            for (int i = pair; i < p.p.items && ok; i += pairs) {
                const Item t = item_at(p, i);
                for (int kb = t.kb0; kb < t.kb1 && ok; kb += SLICE_KB) {   // a slice; a part starts with one
                    const int end = min(kb + SLICE_KB, t.kb1);
                    ok = mbar_wait_warp(&sm->dempty[d], (uint32_t)dph);
                    for (int j = kb; j < end && ok; ++j) {
                        ok = mbar_wait_warp(&sm->full[s], (uint32_t)ph);
                        if (!ok)
                            break;
                        fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < TK / 16; ++k)
                                mma_pair(tmem + (uint32_t)(d * TN), a0 + (uint32_t)(s * (HALF_BYTES >> 4) + 2 * k),
                                         b0 + (uint32_t)(s * (HALF_BYTES >> 4) + 2 * k), (j != kb || k != 0) ? 1u : 0u);
                            commit_pair(&sm->empty[s]);
                            if (j == end - 1)
                                commit_pair(&sm->dfull[d]);
                        }
                        __syncwarp();
                        if (++s == STAGES)
                            s = 0, ph ^= 1;
                    }
                    if (++d == NBUF)
                        d = 0, dph ^= 1;
                }
            }
            if (elect_one())
                commit_pair(&sm->done);
            __syncwarp();
            if (!ok && lane == 0)
                sm->failed = 1;
        }
    } else {
        // epilogue: rows m0 + 128 rank + 32 q + lane, columns n0 + EW h .. on.  The tensor core runs at
        // most two slices ahead, so a tile's way out has to be short: 16 warps
        const int q = warp & 3, h = (warp - 2) >> 2;
        const MatmulI8Args& g = p.g;
        const uint32_t lead = peer_addr(&sm->dempty[0], 0);
        const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(EW * h);
        bool ok = true;
        int d = 0;
        uint32_t ph = 0;   // accumulator, and the parity whose end fills it
        for (int i = pair; i < p.p.items && ok; i += pairs) {
            const Item t = item_at(p, i);
            const int nc = t.n0 + EW * h, r0 = t.m0 + (int)rank * HM + 32 * q;
            const int NS = (t.kb1 - t.kb0 + SLICE_KB - 1) / SLICE_KB;
            float sa = 0.0f, own[2] = {0.0f, 0.0f};
            if (g.s_a && r0 + lane < g.M)
                sa = flush(__ldg(g.s_a + r0 + lane));
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (g.s_b && nc + 2 * lane + e < g.N)
                    own[e] = flush(__ldg(g.s_b + nc + 2 * lane + e));
            // The first slice stays as it comes, the second is added as floats (together at most 2^24,
            // exact) and both become int32 once the accumulator is free: what stands between a tile's
            // way out and the next tile's third slice is then the loads alone
            uint32_t acc[EW];
            ok = mbar_wait_warp(&sm->dfull[d], ph);
            if (!ok)
                break;
            fence_after();
#pragma unroll
            for (int c = 0; c < EW; c += 16)
                tmem_ask16(at + (uint32_t)(d * TN + c), acc + c);
#pragma unroll
            for (int c = 0; c < EW; c += 16)
                tmem_got16(acc + c);
            release(lead + 8 * d, lane);
            turn_buffer(d, ph);
            if (NS > 1) {
                ok = mbar_wait_warp(&sm->dfull[d], ph);
                if (!ok)
                    break;
                fence_after();
                add_slice<true>(acc, at + (uint32_t)(d * TN));
                release(lead + 8 * d, lane);
                turn_buffer(d, ph);
            }
#pragma unroll
            for (int j = 0; j < EW; ++j)
                acc[j] = (uint32_t)__float2int_rn(__uint_as_float(acc[j]));
            for (int sl = 2; sl < NS && ok; ++sl) {
                ok = mbar_wait_warp(&sm->dfull[d], ph);
                if (!ok)
                    break;
                fence_after();
                add_slice<false>(acc, at + (uint32_t)(d * TN));
                release(lead + 8 * d, lane);
                turn_buffer(d, ph);
            }
            if (!ok)
                break;
            if (t.part >= 0) {
                int* out = p.parts + (int64_t)t.part * (2 * HM * TN) + (int64_t)((int)rank * HM + 32 * q + lane) * TN + EW * h;
#pragma unroll
                for (int c = 0; c < EW; c += 8) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] = acc[c + e];
                    store32(out + c, w);
                }
            } else if (r0 < g.M) {   // warp-uniform
                finish<Y>(p, &map_y, acc, STG + (warp - 2) * STG_BYTES, lane, sa, own, r0, nc);
            }
        }
        if (!ok && lane == 0)
            sm->failed = 1;
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    __syncwarp();
    fence_before();
    __syncthreads();
    // `done` arrives in both CTAs, by itself in each, once every MMA has completed: each waits for its own
    // (here, behind all other waits, where it is on its way already, so that the limit fits any product)
    if (warp == 1) {
        if (!mbar_wait_warp(&sm->done, 0) && lane == 0)
            sm->failed = 1;
        __syncwarp();
    }
    cluster_sync();   // no barrier, tile or tensor memory of either CTA is used past here
    if (warp == 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TMEM_COLS) : "memory");
    }
    if (threadIdx.x == 0 && sm->failed)
        atomicOr(p.err, kErrTimeoutBit);
}

// the cut tiles: the sum of a tile's parts, scaled.  A thread takes 4 columns of a row
template <typename Y>
__global__ void __launch_bounds__(256)
k_mm_join(const __grid_constant__ PairArgs p)
{
    pdl_wait();
    const MatmulI8Args& g = p.g;
    const int tile = blockIdx.x >> 6, e = (blockIdx.x & 63) * 256 + threadIdx.x;   // 64 CTAs a tile
    int m0, n0;
    tile_at(p.p, p.p.whole + tile, m0, n0);
    const int r = e >> 6, c = 4 * (e & 63);
    const int64_t m = m0 + r, n = n0 + c;
    if (m >= g.M || n >= g.N)
        return;
    const int* part = p.parts + (int64_t)tile * p.p.split * (2 * HM * TN) + r * TN + c;
    int4 s = *reinterpret_cast<const int4*>(part);
    for (int k = 1; k < p.p.split; ++k) {
        const int4 v = *reinterpret_cast<const int4*>(part + (int64_t)k * (2 * HM * TN));
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const int acc[4] = {s.x, s.y, s.z, s.w};
    const float sa = g.s_a ? flush(__ldg(g.s_a + m)) : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < g.N)
            put(static_cast<Y*>(g.y) + m * g.y_ld + n + i,
                scaled(acc[i], g.s_a, sa, g.s_b, g.s_b ? flush(__ldg(g.s_b + n + i)) : 0.0f), g.accumulate);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &qr) != cudaSuccess ||
            qr != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// rows of `cols` elements, `ld` apart; boxes of 128 bytes x box_rows, 128-byte swizzle
bool make_map(CUtensorMap* map, const void* p, CUtensorMapDataType type, int size, int64_t rows, int64_t cols, int64_t ld,
              int box_rows)
{
    const auto fn = encode_fn();
    if (!fn)
        return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * size};
    cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, type, 2, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Y>
cudaError_t run_pair(const MatmulI8Args& g, const __half* xa, const __half* xb, int* parts, cudaStream_t st)
{
    PairArgs p = {};
    p.g = g;
    p.p = plan_of(g.M, g.N, g.K);
    p.K = (int)g.K;
    p.parts = parts;
    p.err = device_error_word();
    if (!p.err)
        return cudaErrorInvalidValue;
    const int64_t Kp = pad8(g.K), y_ld = g.M == 1 ? (g.N + 7) / 8 * 8 : g.y_ld;
    p.y_tma = reinterpret_cast<uintptr_t>(g.y) % 16 == 0 && y_ld * (int64_t)sizeof(Y) % 16 == 0;
    CUtensorMap ma, mb, my;
    memset(&my, 0, sizeof(my));
    if (!make_map(&ma, xa, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, g.M, Kp, Kp, HM) ||
        !make_map(&mb, xb, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, g.N, Kp, Kp, HM) ||
        (p.y_tma && !make_map(&my, g.y, sizeof(Y) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              (int)sizeof(Y), g.M, g.N, y_ld, 32)))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(k_mm_pair<Y>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
    if (e != cudaSuccess)
        return e;
    const int pairs = std::min(p.p.items, p.p.pairs);
    e = launch_pdl(k_mm_pair<Y>, dim3((unsigned)(2 * pairs)), dim3(THREADS), SMEM_BYTES, st, ma, mb, my, p);
    count_launches(1);
    if (e == cudaSuccess && p.p.split > 1) {
        const int cut = (p.p.items - p.p.whole) / p.p.split;
        e = launch_pdl(k_mm_join<Y>, dim3((unsigned)(64 * cut)), dim3(256), 0, st, p);
        count_launches(1);
    }
    return e;
}

template <typename Y> cudaError_t run_any(const MatmulI8Args& g, cudaStream_t st)
{
    const int64_t tiles_n = (g.N + FT - 1) / FT, tiles = tiles_n * ((g.M + FT - 1) / FT);
    count_launches(1);
    return launch_pdl(k_mm_any<Y>, dim3((unsigned)tiles), dim3(256), 0, st, g, tiles_n);
}

bool aligned16(const MatmulI8Args& g)
{
    return reinterpret_cast<uintptr_t>(g.a) % 16 == 0 && reinterpret_cast<uintptr_t>(g.b) % 16 == 0 &&
           (g.M == 1 || g.a_ld % 16 == 0) && (g.N == 1 || g.b_ld % 16 == 0);
}

// Which kernel, for a = [M][K], b = [N][K] (times for N 11264, K 2048 out of HBM): up to 4 tokens the
// weights' bytes against each of them on the CUDA cores (1 token 7 us, 2 tokens 12, 4 tokens 15); up to 128 the
// weights widened on their way (k_matmul_few.cu: 5 tokens 13 us, 16 tokens 13, 64 tokens 21, 128 tokens
// 31, or 20 for N 2048 and K 5632); else a widened copy and pairs of SMs (31 us up to 256 tokens).  The CUDA
// cores also take up to 16 tokens where the tensor cores may not be used or rows are not aligned (K 2049: 1
// token 15 us, 4 tokens 27, 8 tokens 41, 16 tokens 65; 17 tokens by widened copies 36), and up to 4 by
// transposed weights (k_mm_cols).
bool small_of(int64_t M, bool a_t, bool b_t) { return M <= 16 && !a_t && !b_t; }
bool few_of(int64_t M, int64_t K, bool a_t, bool b_t) { return M > 4 && M <= 128 && !a_t && !b_t && K % 16 == 0 && K > 0; }

size_t pair_ws_bytes(int64_t M, int64_t N, int64_t K)
{
    const Plan p = plan_of(M, N, K);
    const int64_t parts = p.split > 1 ? p.items - p.whole : 0;
    return (size_t)(align256(2 * M * pad8(K)) + align256(2 * N * pad8(K)) + (parts > 0 ? parts * PART_BYTES + PART_ALIGN - 16 : 0));
}

} // namespace

size_t matmul_i8_ws_bytes(int64_t M, int64_t N, int64_t K, bool a_t, bool b_t)
{
    const size_t few = few_of(M, K, a_t, b_t) ? std::max<size_t>(matmul_few_ws_bytes(M, N, K), 16) : 0;
    const size_t cols = cols_of(M, K, a_t, b_t) ? cols_ws_bytes(M, N, K) : 0;
    return small_of(M, a_t, b_t) ? few : std::max({few, cols, pair_ws_bytes(M, N, K)});
}

cudaError_t launch_matmul_pair(const MatmulI8Args& g, void* ws, cudaStream_t st)
{
    __half* xa = static_cast<__half*>(ws);
    __half* xb = reinterpret_cast<__half*>(static_cast<uint8_t*>(ws) + align256(2 * g.M * pad8(g.K)));
    const uintptr_t behind = reinterpret_cast<uintptr_t>(xb) + align256(2 * g.N * pad8(g.K));
    int* parts = reinterpret_cast<int*>((behind + PART_ALIGN - 1) / PART_ALIGN * PART_ALIGN);
    cudaError_t e = widen(g.a, g.a_ld, g.M, g.K, g.a_t, xa, st);
    if (e == cudaSuccess)
        e = widen(g.b, g.b_ld, g.N, g.K, g.b_t, xb, st);
    if (e != cudaSuccess)
        return e;
    return g.y_type == 0 ? run_pair<float>(g, xa, xb, parts, st) : run_pair<__nv_bfloat16>(g, xa, xb, parts, st);
}

cudaError_t launch_matmul_i8(const MatmulI8Args& g, void* ws, bool tc, cudaStream_t st)
{
    if (tc && few_of(g.M, g.K, g.a_t, g.b_t) && aligned16(g))
        return launch_matmul_few(g, ws, st);
    if (small_of(g.M, g.a_t, g.b_t) && g.K > 0)
        return g.y_type == 0 ? run_rows<float>(g, st) : run_rows<__nv_bfloat16>(g, st);
    if (cols_of(g.M, g.K, g.a_t, g.b_t) && reinterpret_cast<uintptr_t>(g.b) % 16 == 0 && g.N % 16 == 0 &&
        (g.K == 1 || g.b_ld % 16 == 0))
        return run_cols(g, static_cast<int*>(ws), st);
    if (!tc || g.K == 0)
        return g.y_type == 0 ? run_any<float>(g, st) : run_any<__nv_bfloat16>(g, st);
    return launch_matmul_pair(g, ws, st);
}

} // namespace repro
