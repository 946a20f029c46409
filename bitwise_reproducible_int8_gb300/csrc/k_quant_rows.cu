// k_quant_rows.cu -- 8-bit codes with a scale for each row or each column.
//
//   s = max |v| (/) 127, q = clamp(rne(v (/) s), -127, 127), v = x or x (x) mul
//
// Bound by HBM: the values in, a byte each out (5 bytes an element from fp32).  By rows: a row stays
// in its threads' registers between the maximum and the codes (16 elements a thread; rows past
// 8,192 elements are read again, out of L2).  By columns: one pass takes the columns' maxima, the
// second reads the matrix again from its end, whose last part L2 (129 MB) still holds.  A maximum
// does not depend on its order, so the columns' may meet in atomics.
#include "codes.cuh"
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace repro {
namespace {

// |v| as an integer that orders as it does; 0 for a NaN, which the maximum passes over
__device__ __forceinline__ unsigned magnitude(float v)
{
    const unsigned m = __float_as_uint(v) & 0x7fffffffu;
    return m > 0x7f800000u ? 0u : m;
}

// four neighbours from element d of a row of D
template <typename T, bool STREAM> __device__ __forceinline__ void take4(const T* p, int64_t d, int64_t D, bool vec, float (&v)[4])
{
    if (vec && d + 4 <= D) {
        const float4 x = STREAM ? stream4(p + d) : load4(p + d);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = d + e < D ? to_f32<T>(p[d + e]) : 0.0f;
    }
}

__device__ __forceinline__ void put4(int8_t* p, int64_t d, int64_t D, bool vec, uint32_t c)
{
    if (vec && d + 4 <= D) {
        *reinterpret_cast<uint32_t*>(p + d) = c;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < D)
                p[d + e] = (int8_t)(c >> (8 * e));
    }
}

struct Kernel {
    QuantRowsArgs a;
    bool vec, qvec, mvec;   // x, q, mul on 4-element boundaries
    int tpr;                // threads of a row (rows)
    int tiles;              // column tiles (columns)
    int64_t slab;           // tokens of a slab (columns)
    unsigned* top;          // columns' maxima
};

template <typename T, bool STREAM>
__device__ __forceinline__ void values4(const Kernel& k, const T* p, int64_t d, float (&v)[4])
{
    take4<T, STREAM>(p, d, k.a.D, k.vec, v);
    if (k.a.mul) {
        float m[4];
        take4<float, false>(k.a.mul, d, k.a.D, k.mvec, m);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = fmul_flush(flush(v[e]), flush(m[e]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = flush(v[e]);
    }
}

// VEC: rows of x and q on 4-element boundaries, whole groups of 4 (and mul on 16 bytes): every load is
// issued before the first value is looked at.  (With a branch around each load, one was in flight at a
// time: 198 us against 81 for 16384 x 5632 fp32.)
template <typename T, bool VEC>
__global__ void __launch_bounds__(512)
k_quant_tokens(const __grid_constant__ Kernel k)
{
    __shared__ unsigned red[2][16];
    const int tpr = k.tpr, per = blockDim.x / tpr, sub = threadIdx.x / tpr, t = threadIdx.x - sub * tpr;
    const int64_t D = k.a.D;
    int phase = 0;
    pdl_wait();
    pdl_trigger();
    for (int64_t i0 = (int64_t)blockIdx.x * per; i0 < k.a.n; i0 += (int64_t)gridDim.x * per) {
        const int64_t i = i0 + sub;
        const bool live = i < k.a.n;
        const T* row = static_cast<const T*>(k.a.x) + i * k.a.x_ld;
        float v[4][4];
        unsigned m = 0;
        if (VEC) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int64_t d = 4 * ((int64_t)t + g * tpr);
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (live && d < D)
                    x = stream4(row + d);
                v[g][0] = x.x, v[g][1] = x.y, v[g][2] = x.z, v[g][3] = x.w;
            }
            if (k.a.mul) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int64_t d = 4 * ((int64_t)t + g * tpr);
                    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (d < D)
                        f = load4(k.a.mul + d);
                    v[g][0] = fmul_flush(flush(v[g][0]), flush(f.x)), v[g][1] = fmul_flush(flush(v[g][1]), flush(f.y));
                    v[g][2] = fmul_flush(flush(v[g][2]), flush(f.z)), v[g][3] = fmul_flush(flush(v[g][3]), flush(f.w));
                }
            } else {
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[g][e] = flush(v[g][e]);
            }
        } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int64_t d = 4 * ((int64_t)t + g * tpr);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[g][e] = 0.0f;
                if (live && d < D)
                    values4<T, true>(k, row, d, v[g]);
            }
        }
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                m = max(m, magnitude(v[g][e]));
        if (live)
            for (int64_t d = 4 * ((int64_t)t + 4 * tpr); d < D; d += 4 * tpr) {
                float w[4];
                values4<T, false>(k, row, d, w);
                m = max(max(max(m, magnitude(w[0])), max(magnitude(w[1]), magnitude(w[2]))), magnitude(w[3]));
            }
        m = __reduce_max_sync(0xffffffffu, m);
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
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int64_t d = 4 * ((int64_t)t + g * tpr);
            if (d < D)
                put4(q, d, D, VEC || k.qvec, codes4(v[g], c));
        }
        for (int64_t d = 4 * ((int64_t)t + 4 * tpr); d < D; d += 4 * tpr) {
            float w[4];
            values4<T, false>(k, row, d, w);
            put4(q, d, D, k.qvec, codes4(w, c));
        }
        if (t == 0)
            k.a.scales[i] = c.s;
    }
}

constexpr int RUN = 8;   // tokens whose loads a warp has in flight by columns

// four columns of RUN tokens, `step` apart, times their multipliers; 0 past the last
template <typename T, bool VEC>
__device__ __forceinline__ void take_run(const Kernel& k, int64_t i, int64_t hi, int step, int64_t d, float (&v)[RUN][4])
{
    const T* x = static_cast<const T*>(k.a.x);
    float f[RUN];
#pragma unroll
    for (int u = 0; u < RUN; ++u) {
        const int64_t r = i + u * step;
        f[u] = 1.0f;
        if (VEC) {
            float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < hi)
                w = load4(x + r * k.a.x_ld + d);
            v[u][0] = w.x, v[u][1] = w.y, v[u][2] = w.z, v[u][3] = w.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[u][e] = r < hi && d + e < k.a.D ? to_f32<T>(x[r * k.a.x_ld + d + e]) : 0.0f;
        }
        if (k.a.mul && r < hi)
            f[u] = __ldg(k.a.mul + r);
    }
#pragma unroll
    for (int u = 0; u < RUN; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[u][e] = fmul_flush(flush(v[u][e]), flush(f[u]));
}

// a CTA: 32 x 4 columns of a slab of tokens, 8 warps taking every eighth token
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
k_column_max(const __grid_constant__ Kernel k)
{
    __shared__ unsigned red[8][128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tile = blockIdx.x % k.tiles;
    const int64_t slab = blockIdx.x / k.tiles, d = (int64_t)tile * 128 + 4 * lane;
    const int64_t lo = slab * k.slab, hi = min(lo + k.slab, k.a.n);
    pdl_wait();
    pdl_trigger();
    unsigned m[4] = {0, 0, 0, 0};
    if (d < k.a.D)
        for (int64_t i = lo + warp; i < hi; i += 8 * RUN) {
            float v[RUN][4];
            take_run<T, VEC>(k, i, hi, 8, d, v);
#pragma unroll
            for (int u = 0; u < RUN; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    m[e] = max(m[e], magnitude(v[u][e]));
        }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        red[warp][4 * lane + e] = m[e];
    __syncthreads();
    if (threadIdx.x < 128) {
        unsigned x = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            x = max(x, red[w][threadIdx.x]);
        const int64_t c = (int64_t)tile * 128 + threadIdx.x;
        if (c < k.a.D && x != 0)
            atomicMax(k.top + c, x);
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
k_quant_columns(const __grid_constant__ Kernel k)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = gridDim.x - 1 - blockIdx.x;      // the slabs read last come first
    const int tile = b % k.tiles;
    const int64_t slab = b / k.tiles, d = (int64_t)tile * 128 + 4 * lane;
    const int64_t lo = slab * k.slab, hi = min(lo + k.slab, k.a.n);
    pdl_wait();
    pdl_trigger();
    if (d >= k.a.D)
        return;
    CodeScale c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        c[e] = code_scale_of_max(__uint_as_float(d + e < k.a.D ? k.top[d + e] : 0u));
        if (slab == 0 && warp == 0 && d + e < k.a.D)
            k.a.scales[d + e] = c[e].s;
    }
    for (int64_t i = lo + warp; i < hi; i += 8 * RUN) {
        float v[RUN][4];
        take_run<T, VEC>(k, i, hi, 8, d, v);
#pragma unroll
        for (int u = 0; u < RUN; ++u) {
            const int64_t r = i + 8 * u;
            if (r < hi)
                put4(k.a.q + r * k.a.q_ld, d, k.a.D, k.qvec, codes4_by(v[u], c));
        }
    }
}

template <typename T> cudaError_t launch(Kernel& k, cudaStream_t st)
{
    const QuantRowsArgs& a = k.a;
    if (!a.columns) {
        const int64_t want = (a.D + 511) / 512;             // warps of a row, 16 elements a lane
        k.tpr = 32 * (int)(want < 16 ? want : 16);
        const int threads = k.tpr == 32 ? 128 : k.tpr, per = threads / k.tpr;
        const int64_t ctas = (a.n + per - 1) / per, most = (int64_t)num_sms() * 64;
        count_launches(1);
        const dim3 grid((unsigned)(ctas < most ? ctas : most));
        return k.vec && k.qvec && a.D % 4 == 0 && (!a.mul || k.mvec)
                   ? launch_pdl(k_quant_tokens<T, true>, grid, dim3(threads), 0, st, k)
                   : launch_pdl(k_quant_tokens<T, false>, grid, dim3(threads), 0, st, k);
    }
    k.tiles = (int)((a.D + 127) / 128);
    // slabs of a multiple of 64 tokens, about eight CTAs on every SM
    const int64_t want = (8 * (int64_t)num_sms() + k.tiles - 1) / k.tiles, tokens = (a.n + want - 1) / want;
    k.slab = tokens < 64 ? 64 : (tokens + 63) / 64 * 64;
    const int64_t slabs = (a.n + k.slab - 1) / k.slab;
    const dim3 grid((unsigned)(k.tiles * slabs));
    cudaError_t e = cudaMemsetAsync(k.top, 0, (size_t)a.D * 4, st);
    const bool vec = k.vec && a.D % 4 == 0;
    if (e == cudaSuccess)
        e = vec ? launch_pdl(k_column_max<T, true>, grid, dim3(256), 0, st, k)
                : launch_pdl(k_column_max<T, false>, grid, dim3(256), 0, st, k);
    if (e == cudaSuccess)
        e = vec ? launch_pdl(k_quant_columns<T, true>, grid, dim3(256), 0, st, k)
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
    k.vec = bf ? rows4<__nv_bfloat16>(a.x, a.x_ld) : rows4<float>(a.x, a.x_ld);
    k.qvec = rows4<int8_t>(a.q, a.q_ld);
    k.mvec = a.mul && reinterpret_cast<uintptr_t>(a.mul) % 16 == 0;
    k.top = static_cast<unsigned*>(ws);
    return bf ? launch<__nv_bfloat16>(k, st) : launch<float>(k, st);
}

} // namespace repro
