// k_quant_rows.cu -- 8-bit codes with a scale for each row or each column.
//
//   s = max |v| (/) 127, q = clamp(rne(v (/) s), -127, 127), v = x or x (x) mul
//
// Bound by HBM: the values in, a byte each out (5 bytes an element from fp32).  By rows: a row stays
// in its threads' registers between the maximum and the codes (32 elements a thread; what lies past
// 16,384 elements is read again, out of L2).  By columns: one pass takes the columns' maxima, the
// second reads the matrix again from its end, whose last part L2 (129 MB) still holds.  A maximum
// does not depend on its order, so the columns' may meet in atomics.
//
// Measured, 16384 x 5632: by rows fp32 67 us, 6.9 TB/s, which is its floor, bf16 54 us (floor 41; issue
// slots); by columns, where two passes have 122 and 68 us of bytes, fp32 127 us and bf16 105.  4099 x
// 2003 fp32 by columns with a multiplier (rows off 16-byte boundaries, so elements one by one) 22 us.
// 16384 x 11264 fp32 by rows 141 us, floor 136 (170 with 256 threads a row and a third of it read again).
#include "codes.cuh"
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace repro {
namespace {

// the larger of m and the magnitudes of four; a NaN is passed over
__device__ __forceinline__ float top4(float m, const float (&v)[4])
{
    return fmaxf(fmaxf(fmaxf(m, fabsf(v[0])), fmaxf(fabsf(v[1]), fabsf(v[2]))), fabsf(v[3]));
}

// Four elements of a row of D.  VEC (rows on 4-element boundaries, D a multiple of 4): the neighbours
// from element d.  Else elements d, d + hop, d + 2 hop and d + 3 hop, so that a warp's loads and
// stores of single elements are still of neighbours.
template <bool VEC, bool STREAM, typename T>
__device__ __forceinline__ void take4(const T* p, int d, int hop, int D, float (&v)[4])
{
    if (VEC) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (d < D)
            x = STREAM ? stream4(p + d) : load4(p + d);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = d + e * hop < D ? to_f32<T>(p[d + e * hop]) : 0.0f;
    }
}

template <bool VEC> __device__ __forceinline__ void put4(int8_t* p, int d, int hop, int D, uint32_t c)
{
    if (VEC) {
        if (d < D)
            *reinterpret_cast<uint32_t*>(p + d) = c;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e * hop < D)
                p[d + e * hop] = (int8_t)(c >> (8 * e));
    }
}

struct Kernel {
    QuantRowsArgs a;
    bool vec;               // x, q (and by rows mul) on 4-element boundaries, D a multiple of 4
    int tpr;                // threads of a row (rows)
    int tiles;              // column tiles (columns)
    int64_t slab;           // tokens of a slab (columns)
    unsigned* top;          // columns' maxima
};

// v (x) mul; without a multiplier v as it is: what is subnormal is flushed with the maximum, and beside
// a scale of 2^-67 or more, below which values are divided, it is nothing
__device__ __forceinline__ void times4(float (&v)[4], const float (&m)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = fmul_flush(flush(v[e]), flush(m[e]));
}

constexpr int G = 8;     // groups of 4 a thread holds of a row

// VEC: rows of x and q on 4-element boundaries, whole groups of 4 (and mul on 16 bytes): every load is
// issued before the first value is looked at.  (With a branch around each load, one was in flight at a
// time: 198 us for 16384 x 5632 fp32, 81 without.)
template <typename T, bool VEC, bool LONG, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
k_quant_tokens(const __grid_constant__ Kernel k)
{
    __shared__ unsigned red[2][16];
    const int tpr = k.tpr, per = blockDim.x / tpr, sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
    // group g of a thread: 4 neighbours from d0 + g hop on, or 4 elements tpr apart
    const int D = (int)k.a.D, d0 = VEC ? 4 * t : t, hop = 4 * tpr;
    int phase = 0;
    pdl_wait();
    pdl_trigger();
    for (int64_t i = (int64_t)blockIdx.x * per + sub; i - sub < k.a.n; i += (int64_t)gridDim.x * per) {
        const bool live = i < k.a.n;
        const int w = live ? D : 0;      // width of this thread's row
        const T* row = static_cast<const T*>(k.a.x) + i * k.a.x_ld;
        const float* mul = k.a.mul;
        float v[G][4];
#pragma unroll
        for (int g = 0; g < G; ++g)
            take4<VEC, true>(row, d0 + g * hop, tpr, w, v[g]);
        if (mul)
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float f[4];
                take4<VEC, false>(mul, d0 + g * hop, tpr, w, f);
                times4(v[g], f);
            }
        float top = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g)
            top = top4(top, v[g]);
        auto again = [&](int d, float (&x)[4]) {      // a group from memory
            take4<VEC, false>(row, d, tpr, w, x);
            if (mul) {
                float f[4];
                take4<VEC, false>(mul, d, tpr, w, f);
                times4(x, f);
            }
        };
        if (LONG)
            for (int d = d0 + G * hop; d < w; d += hop) {
                float x[4];
                again(d, x);
                top = top4(top, x);
            }
        unsigned m = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        if (tpr > 32) {   // one row a CTA
            if ((t & 31) == 0)
                red[phase][t >> 5] = m;
            __syncthreads();
            m = (t & 31) < (tpr >> 5) ? red[phase][t & 31] : 0u;
            m = __reduce_max_sync(0xffffffffu, m);
            phase ^= 1;
        }
        if (!live)
            continue;
        const CodeScale c = code_scale_of_max(__uint_as_float(m));
        int8_t* q = k.a.q + i * k.a.q_ld;
        const CodeScale all[4] = {c, c, c, c};
        unsigned divide = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint32_t o;
            divide |= (unsigned)!codes4(v[g], all, o) << g;
            put4<VEC>(q, d0 + g * hop, tpr, D, o);
        }
        // what has to be divided is read once more: kept in registers beside 8 inlined divisions, the
        // values left room for two rows on an SM instead of five
        for (; divide; divide &= divide - 1) {
            const int d = d0 + (__ffs(divide) - 1) * hop;
            float x[4];
            again(d, x);
            put4<VEC>(q, d, tpr, D, codes4_divided(x, all));
        }
        if (LONG)
            for (int d = d0 + G * hop; d < D; d += hop) {
                float x[4];
                again(d, x);
                uint32_t o;
                if (!codes4(x, all, o))
                    o = codes4_divided(x, all);
                put4<VEC>(q, d, tpr, D, o);
            }
        if (t == 0)
            k.a.scales[i] = c.s;
    }
}

constexpr int RUN = 8;   // tokens whose loads a warp has in flight by columns

// four columns of RUN tokens, 8 apart from token i on, times their multipliers; 0 past the last, `rows` of
// them being there
template <typename T, bool VEC>
__device__ __forceinline__ void take_run(const Kernel& k, const T* row, int64_t i, int rows, int d, float (&v)[RUN][4])
{
    const int64_t step = 8 * k.a.x_ld;
    float f[RUN];
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
        take4<VEC, false>(row, d, 32, u < rows ? (int)k.a.D : 0, v[u]);
        row += step;
        if (k.a.mul)
            f[u] = u < rows ? __ldg(k.a.mul + i + 8 * u) : 1.0f;
    }
    if (k.a.mul)
#pragma unroll
        for (int u = 0; u < RUN; ++u) {
            const float all[4] = {f[u], f[u], f[u], f[u]};
            times4(v[u], all);
        }
}

// a CTA: a tile of 128 columns of a slab of tokens, 8 warps taking every eighth token; a lane has 4
// neighbours of the tile (VEC) or every 32nd column
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 4)
k_column_max(const __grid_constant__ Kernel k)
{
    __shared__ unsigned red[8][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tile = blockIdx.x % k.tiles, at = VEC ? 4 * lane : lane, d = tile * 128 + at;
    const int64_t slab = blockIdx.x / k.tiles, lo = slab * k.slab, hi = min(lo + k.slab, k.a.n);
    pdl_wait();
    pdl_trigger();
    float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const T* row = static_cast<const T*>(k.a.x) + (lo + warp) * k.a.x_ld;
    for (int64_t i = lo + warp; i < hi; i += 8 * RUN, row += 8 * RUN * k.a.x_ld) {
        float v[RUN][4];
        take_run<T, VEC>(k, row, i, (int)((hi - i + 7) >> 3), d, v);
#pragma unroll
        for (int u = 0; u < RUN; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                m[e] = fmaxf(m[e], fabsf(v[u][e]));   // passes over NaN
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        red[warp][at + e * (VEC ? 1 : 32)] = __float_as_uint(m[e]);
    __syncthreads();
    if (threadIdx.x < 128) {
        unsigned x = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            x = max(x, red[w][threadIdx.x]);
        const int c = tile * 128 + threadIdx.x;
        if (c < k.a.D && x != 0)
            atomicMax(k.top + c, x);
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 4)
k_quant_columns(const __grid_constant__ Kernel k)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = (int)k.a.D;
    const int b = gridDim.x - 1 - blockIdx.x;      // the slabs read last come first
    const int tile = b % k.tiles, d = tile * 128 + (VEC ? 4 * lane : lane);
    const int64_t slab = b / k.tiles, lo = slab * k.slab, hi = min(lo + k.slab, k.a.n);
    pdl_wait();
    pdl_trigger();
    CodeScale c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int col = d + e * (VEC ? 1 : 32);
        c[e] = code_scale_of_max(__uint_as_float(col < D ? k.top[col] : 0u));
        if (slab == 0 && warp == 0 && col < D)
            k.a.scales[col] = c[e].s;
    }
    const T* row = static_cast<const T*>(k.a.x) + (lo + warp) * k.a.x_ld;
    int8_t* out = k.a.q + (lo + warp) * k.a.q_ld;
    for (int64_t i = lo + warp; i < hi; i += 8 * RUN) {
        const int rows = (int)((hi - i + 7) >> 3);
        float v[RUN][4];
        take_run<T, VEC>(k, row, i, rows, d, v);
        unsigned divide = 0;
        int8_t* to = out;
#pragma unroll
        for (int u = 0; u < RUN; ++u) {
            uint32_t q;
            divide |= (unsigned)(!codes4(v[u], c, q) && u < rows) << u;
            put4<VEC>(to, d, 32, u < rows ? D : 0, q);
            to += 8 * k.a.q_ld;
        }
        for (; divide; divide &= divide - 1) {     // read once more, as by rows
            const int u = __ffs(divide) - 1;
            float x[4];
            take4<VEC, false>(row + 8 * u * k.a.x_ld, d, 32, D, x);
            if (k.a.mul) {
                const float f = __ldg(k.a.mul + i + 8 * u), all[4] = {f, f, f, f};
                times4(x, all);
            }
            put4<VEC>(out + 8 * u * k.a.q_ld, d, 32, D, codes4_divided(x, c));
        }
        row += 8 * RUN * k.a.x_ld;
        out += 8 * RUN * k.a.q_ld;
    }
}

template <typename T> cudaError_t launch(Kernel& k, cudaStream_t st)
{
    const QuantRowsArgs& a = k.a;
    if (!a.columns) {
        const int64_t want = (a.D + 4 * G * 32 - 1) / (4 * G * 32);   // warps of a row
        k.tpr = 32 * (int)(want < 16 ? want : 16);
        const int threads = k.tpr == 32 ? 128 : k.tpr, per = threads / k.tpr;
        const int64_t ctas = (a.n + per - 1) / per, most = (int64_t)num_sms() * 64;
        count_launches(1);
        const dim3 grid((unsigned)(ctas < most ? ctas : most));
        const bool fits = a.D <= 4 * G * k.tpr;
#define GO(V, L, N) launch_pdl(k_quant_tokens<T, V, L, N>, grid, dim3(threads), 0, st, k)
        return threads <= 256 ? (k.vec ? GO(true, false, 256) : GO(false, false, 256))
               : fits         ? (k.vec ? GO(true, false, 512) : GO(false, false, 512))
                              : (k.vec ? GO(true, true, 512) : GO(false, true, 512));
#undef GO
    }
    k.tiles = (int)((a.D + 127) / 128);
    // slabs of a multiple of 64 tokens, about eight CTAs on every SM
    const int64_t want = (8 * (int64_t)num_sms() + k.tiles - 1) / k.tiles, tokens = (a.n + want - 1) / want;
    k.slab = tokens < 64 ? 64 : (tokens + 63) / 64 * 64;
    const int64_t slabs = (a.n + k.slab - 1) / k.slab;
    const dim3 grid((unsigned)(k.tiles * slabs));
    cudaError_t e = cudaMemsetAsync(k.top, 0, (size_t)a.D * 4, st);
    if (e == cudaSuccess)
        e = k.vec ? launch_pdl(k_column_max<T, true>, grid, dim3(256), 0, st, k)
                : launch_pdl(k_column_max<T, false>, grid, dim3(256), 0, st, k);
    if (e == cudaSuccess)
        e = k.vec ? launch_pdl(k_quant_columns<T, true>, grid, dim3(256), 0, st, k)
                : launch_pdl(k_quant_columns<T, false>, grid, dim3(256), 0, st, k);
    count_launches(2);
    return e;
}

} // namespace

size_t quant_rows_ws_bytes(int64_t n, int64_t D, bool columns) { return columns ? (size_t)D * 4 : 0; }

cudaError_t launch_quant_rows(const QuantRowsArgs& a, void* ws, cudaStream_t st)
{
    Kernel k = {};
    k.a = a;
    const bool bf = a.type != 0;
    k.vec = (bf ? rows4<__nv_bfloat16>(a.x, a.x_ld) : rows4<float>(a.x, a.x_ld)) && rows4<int8_t>(a.q, a.q_ld) && a.D % 4 == 0 &&
            (a.columns || reinterpret_cast<uintptr_t>(a.mul) % 16 == 0);
    k.top = static_cast<unsigned*>(ws);
    return bf ? launch<__nv_bfloat16>(k, st) : launch<float>(k, st);
}

} // namespace repro
