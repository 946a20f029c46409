// k_blocknorm.cu -- RMS norms behind and before a block, its gate and the residual scales in one pass.
//
//   p = (y r1) gain_post, gated; h = x alpha + p beta; u = (h r2) gain_pre, r = 1 / sqrt(mean v^2 + eps)
//
// Bound by HBM: x and y in, h and u out (16 bytes an element in fp32).  A row stays in the registers
// of its threads between its sums (rows.cuh).  Measured: 16,384 x 2048 fp32 80 us, 6.7 TB/s, floor 79;
// 4096 x 8192 81 us; 8192 x 4096 bf16 53 us, floor 40.
#include "blocknorm.cuh"

namespace repro {
namespace {

__device__ __forceinline__ float rms_of(float S, const NormArgs& a)
{
    return flush(__fdiv_rn(1.0f, flush(__fsqrt_rn(fadd_ftz(mean_of(S, (float)a.D, a.inv), a.eps)))));
}

// 64 registers a thread: with 94, five rows of 2048 on an SM instead of eight, 8192 x 4096 fp32 took
// 93 us against 80.  TPR known: 16,384 x 2048 fp32 80 us against 85, 8192 x 4096 bf16 53 against 57; in
// fp32 from 4096 on the registers spill with it (4096 x 8192 86 us against 81), so there it is read.
template <typename T, typename U, int THREADS, int TPR, int G, int W>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
k_norm_fwd(const __grid_constant__ NormArgs a)
{
    __shared__ float red[4][64];
    int sub, phase = 0;
    const RowLane r = row_lane<THREADS, TPR>(a.D, a.tpr, sub);
    const int per = THREADS / r.tpr;
    const float alpha = flush(a.alpha), beta = flush(a.beta);
    pdl_wait();
    for (int64_t i = (int64_t)blockIdx.x * per + sub; i < a.n; i += (int64_t)gridDim.x * per) {
        u64 x[2 * G], w[2 * G];
        float r1 = 0.0f, r2 = 0.0f;
        if (a.y) {
            u64 y[2 * G];
            load_row<W, true>(static_cast<const T*>(a.y) + i * a.y_ld, r, y);
            load_row<W, false>(static_cast<const T*>(a.x) + i * a.x_ld, r, x);
            flush_row(y);
            if (a.post) {
                r1 = rms_of(tree_of_chains(chain_of<W>(y, y, r), r, red[sub], phase), a);
                mul_row(y, r1);
                if (a.gain_post) {
                    gain_row<W>(a.gain_post, r, w);
                    mul_row(y, w);
                }
            }
            if (a.gate) {
                if (a.gate_rows) {
                    load_row<W, true>(static_cast<const T*>(a.gate) + i * a.gate_ld, r, w);
                    flush_row(w);
                } else {
                    gain_row<W>(static_cast<const float*>(a.gate), r, w);
                }
                mul_row(y, w);
            }
            flush_row(x);
            const u64 al = pack2(alpha, alpha), be = pack2(beta, beta);
#pragma unroll
            for (int e = 0; e < 2 * G; ++e) {
                x[e] = fadd2_ftz(fmul2_rn(x[e], al), fmul2_rn(y[e], be));
                if (sizeof(T) == 2) {   // the norm reads the stream as it is stored
                    float p, q;
                    unpack2(x[e], p, q);
                    x[e] = pack2(to_f32<T>(from_f32<T>(p)), to_f32<T>(from_f32<T>(q)));
                }
            }
            store_row<W>(static_cast<T*>(a.h) + i * a.h_ld, r, x);
        } else {
            load_row<W, true>(static_cast<const T*>(a.x) + i * a.x_ld, r, x);
        }
        if (a.u) {
            flush_row(x);
            r2 = rms_of(tree_of_chains(chain_of<W>(x, x, r), r, red[sub], phase), a);
            mul_row(x, r2);
            if (a.gain_pre) {
                gain_row<W>(a.gain_pre, r, w);
                mul_row(x, w);
            }
            store_row<W>(static_cast<U*>(a.u) + i * a.u_ld, r, x);
        }
        if (a.stats && r.t == 0) {
            a.stats[2 * i] = r1;
            a.stats[2 * i + 1] = r2;
        }
    }
}

template <typename T, typename U> cudaError_t launch_fwd(const NormArgs& a, int threads, dim3 grid, cudaStream_t st)
{
    const int w = check_of(a);
#define RUN(N, TPR, G, W) launch_pdl(k_norm_fwd<T, U, N, TPR, G, W>, grid, dim3(threads), 0, st, a)
#define GO(N, TPR) (w == WHOLE ? RUN(N, TPR, 4, WHOLE) : w == GROUPS ? RUN(N, TPR, 4, GROUPS) : RUN(N, TPR, 4, ELEMENTS))
    if (a.D <= 128)
        return w != ELEMENTS ? RUN(128, 32, 1, GROUPS) : RUN(128, 32, 1, ELEMENTS);
    if (a.D <= 256)
        return w != ELEMENTS ? RUN(128, 32, 2, GROUPS) : RUN(128, 32, 2, ELEMENTS);
    constexpr bool KNOWN = sizeof(T) == 2;
    return a.tpr < 128      ? GO(128, 0)
           : threads == 128 ? GO(128, 128)
           : threads == 256 ? GO(256, (KNOWN ? 256 : 0))
           : threads == 512 ? GO(512, (KNOWN ? 512 : 0))
                            : GO(1024, (KNOWN ? 1024 : 0));
#undef GO
#undef RUN
}

} // namespace

cudaError_t launch_norm_fwd(NormArgs a, cudaStream_t st)
{
    set_up(a);
    int threads;
    const dim3 grid = grid_of(a, a.n, threads);
    if (a.type == 0)
        return a.u_type == 0 ? launch_fwd<float, float>(a, threads, grid, st) : launch_fwd<float, __nv_bfloat16>(a, threads, grid, st);
    return a.u_type == 0 ? launch_fwd<__nv_bfloat16, float>(a, threads, grid, st)
                         : launch_fwd<__nv_bfloat16, __nv_bfloat16>(a, threads, grid, st);
}

} // namespace repro
