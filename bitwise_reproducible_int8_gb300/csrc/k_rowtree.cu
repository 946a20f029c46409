// k_rowtree.cu -- the upper half of a canonical sum of rows: chunk partials
// (each a row of D floats) combined by the stride-doubling pairwise tree, and
// the debug scan of strided tensors.
//
// t_j += t_{j+s} for j a multiple of 2s.  An aligned group of 16 chunks is a subtree:
// a worker loads its 16 rows at once and folds them in registers, so a tree over C
// chunks takes log16 C rounds over memory (out of L2) instead of log2 C, with 16
// loads in flight.  LANES lanes of 4 columns make a worker: a warp where many joins
// of few chunks over wide rows are to be done (the table's gradient), two lanes for
// one long join over a narrow row (the gains' gradients; with 8 lanes and one pair
// per worker and barrier, 4,096 chunks of 128 took 25 us).
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace repro {
namespace {

constexpr int FOLD = 16;   // chunks a worker folds at a time

template <int LANES>
__global__ void __launch_bounds__(256)
k_row_tree(const __grid_constant__ RowTree t, int colsegs)
{
    constexpr int WORKERS = 256 / LANES;
    pdl_wait();
    const int64_t joins = t.joins ? *t.njoins : t.jobs;
    const int lane = threadIdx.x % LANES, worker = threadIdx.x / LANES;
    const float sc = flush(t.scale);
    for (int64_t item = blockIdx.x; item < joins * colsegs; item += gridDim.x) {
        const int64_t jn = item / colsegs;
        const int64_t c = (item - jn * colsegs) * (4 * LANES) + 4 * lane;
        const int4 j = t.joins ? t.joins[jn] : make_int4(0, (int)t.count[jn != 0], 0, 0);
        float* parts = t.joins || jn == 0 ? t.parts[0] : t.parts[1];
        float* out = t.joins || jn == 0 ? t.out[0] : t.out[1];
        const bool live = c < t.D;
        // partial row of chunk k: see the slot rule of the chunk list (k_embed.cu)
        auto row = [&](int64_t k) {
            const int64_t slot = t.joins ? (k == 0 ? 2 * (int64_t)(j.x >> 6) + 1 : 2 * ((j.x + 64 * k) >> 6)) : k;
            return parts + slot * t.pitch + c;
        };
        const int64_t C = j.y;
        for (int64_t s = 1; s < C; s *= FOLD) {
            if (live)
                for (int64_t k = (int64_t)worker * FOLD * s; k < C; k += (int64_t)WORKERS * FOLD * s) {
                    float4 v[FOLD];
#pragma unroll
                    for (int i = 0; i < FOLD; ++i)   // -0 in place of a missing chunk leaves a sum as it is
                        v[i] = k + i * s < C ? load4(row(k + i * s)) : make_float4(-0.0f, -0.0f, -0.0f, -0.0f);
#pragma unroll
                    for (int w = 1; w < FOLD; w *= 2)
#pragma unroll
                        for (int i = 0; i < FOLD; i += 2 * w)
                            v[i] = make_float4(fadd_ftz(v[i].x, v[i + w].x), fadd_ftz(v[i].y, v[i + w].y),
                                               fadd_ftz(v[i].z, v[i + w].z), fadd_ftz(v[i].w, v[i + w].w));
                    store4(row(k), v[0]);
                }
            __syncthreads();
        }
        if (live && worker == 0) {
            const float4 x = load4(row(0));
            const float v[4] = {x.x, x.y, x.z, x.w};
            float* o = out + (int64_t)j.z * t.out_ld + c;
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
    const int cols = t.joins ? 128 : 8;
    const int colsegs = (int)((t.D + cols - 1) / cols);
    const int grid = t.joins ? max_ctas : (colsegs * t.jobs < max_ctas ? colsegs * t.jobs : max_ctas);
    const cudaError_t e = t.joins ? launch_pdl(k_row_tree<32>, dim3((unsigned)grid), dim3(256), 0, st, t, colsegs)
                                  : launch_pdl(k_row_tree<2>, dim3((unsigned)grid), dim3(256), 0, st, t, colsegs);
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
