// k_rowtree.cu -- the upper half of a canonical sum of rows: chunk partials
// (each a row of D floats) combined by the stride-doubling pairwise tree, and
// the debug scan of strided tensors.
//
// t_j += t_{j+s} for j a multiple of 2s: at every stride the pairs are
// independent, so a CTA gives 8 lanes to 32 columns and spreads the pairs over
// its 32 groups of lanes, with a barrier between strides.  The partial rows come
// straight out of L2.
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace repro {
namespace {

constexpr int RT_COLS = 32;       // columns per CTA step
constexpr int RT_WORKERS = 32;    // pairs at a time

__global__ void __launch_bounds__(256)
k_row_tree(const RowTree t, int colsegs)
{
    pdl_wait();
    const int64_t joins = t.joins ? *t.njoins : 1;
    const int lane = threadIdx.x & 7, worker = threadIdx.x >> 3;
    const float sc = flush(t.scale);
    for (int64_t item = blockIdx.x; item < joins * colsegs; item += gridDim.x) {
        const int64_t jn = item / colsegs;
        const int64_t c = (item - jn * colsegs) * RT_COLS + 4 * lane;
        const int4 j = t.joins ? t.joins[jn] : make_int4(0, (int)t.count, 0, 0);
        const bool live = c < t.D;
        // partial row of chunk k: see the slot rule of the chunk list (k_embed.cu)
        auto row = [&](int64_t k) {
            const int64_t slot = t.joins ? (k == 0 ? 2 * (int64_t)(j.x >> 6) + 1 : 2 * ((j.x + 64 * k) >> 6)) : k;
            return t.parts + slot * t.pitch + c;
        };
        const int64_t C = j.y;
        for (int64_t s = 1; s < C; s *= 2) {
            if (live)
                for (int64_t k = 2 * s * worker; k + s < C; k += 2 * s * RT_WORKERS) {
                    float* p = row(k);
                    const float4 x = load4(p), y = load4(row(k + s));
                    store4(p, make_float4(fadd_ftz(x.x, y.x), fadd_ftz(x.y, y.y), fadd_ftz(x.z, y.z),
                                          fadd_ftz(x.w, y.w)));
                }
            __syncthreads();
        }
        if (live && worker == 0) {
            const float4 x = load4(row(0));
            const float v[4] = {x.x, x.y, x.z, x.w};
            float* o = t.out + (int64_t)j.z * t.out_ld + c;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < t.D) {
                    const float r = fmul_flush(v[e], sc);
                    o[e] = t.accumulate ? fadd_ftz(o[e], r) : r;
                }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
k_check_rows(const T* __restrict__ p, int64_t n, int64_t D, int64_t ld, int* err)
{
    bool bad = false;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n * D; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / D;
        bad |= !(fabsf(to_f32<T>(p[r * ld + (i - r * D)])) <= 3.402823466e38f);
    }
    if (bad)
        atomicOr(err, kErrNonfiniteBit);
}

} // namespace

cudaError_t launch_row_tree(const RowTree& t, int max_ctas, cudaStream_t st)
{
    const int colsegs = (int)((t.D + RT_COLS - 1) / RT_COLS);
    const int grid = t.joins ? max_ctas : (colsegs < max_ctas ? colsegs : max_ctas);
    const cudaError_t e = launch_pdl(k_row_tree, dim3((unsigned)grid), dim3(256), 0, st, t, colsegs);
    count_launches(1);
    return e;
}

cudaError_t launch_check_finite_rows(const void* p, int type, int64_t n, int64_t D, int64_t ld, int* err,
                                     cudaStream_t st)
{
    const int64_t want = (n * D + 255) / 256, cap = (int64_t)num_sms() * 8;
    const unsigned grid = (unsigned)(want < 1 ? 1 : want < cap ? want : cap);
    if (type == 0)
        k_check_rows<float><<<grid, 256, 0, st>>>(static_cast<const float*>(p), n, D, ld, err);
    else
        k_check_rows<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(p), n, D, ld, err);
    count_launches(1);
    return cudaGetLastError();
}

} // namespace repro
