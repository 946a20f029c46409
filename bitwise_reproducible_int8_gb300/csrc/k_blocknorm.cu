// k_blocknorm.cu -- RMS norms behind and before a block, its gate and the residual scales in
// one pass, and the backward with the gradients of gains and gate.
//
//   p = (y r1) gain_post, gated; h = x alpha + p beta; u = (h r2) gain_pre, r = 1 / sqrt(mean v^2 + eps)
//   back: g = dh + r2 (v - hn c), v = du gain_pre, hn = h r2, c = mean(v hn); dx = g alpha;
//         dy = r1 (w - yn c'), w = g beta gate gain_post, yn = y r1, c' = mean(w yn)
//
// Bound by HBM: x and y in, h and u out (16 bytes an element in fp32); backward du, dh, h, y in,
// dx, dy out (24).  A row stays in the registers of its threads between its sums (rows.cuh).
//
// The gradients that are sums over tokens: a group of the backward takes 16 consecutive tokens one
// after another and keeps its columns' sums in registers, so a chunk's order costs nothing, and
// writes one row of partial sums (1/16 of a stream of the pass, out of L2); k_rowtree.cu joins them.
#include "internal.h"
#include "launch.cuh"
#include "rows.cuh"

namespace repro {
namespace {

constexpr int CHUNK = 16;        // tokens a group of the backward sums: REPRO_NORM_CHUNK

__device__ __forceinline__ float rms_of(float S, const NormArgs& a)
{
    return flush(__fdiv_rn(1.0f, flush(__fsqrt_rn(fadd_ftz(mean_of(S, (float)a.D, a.inv), a.eps)))));
}

__device__ __forceinline__ RowLane lane_of(const NormArgs& a, int& sub)
{
    RowLane r;
    r.tpr = a.tpr;
    sub = threadIdx.x / a.tpr;
    r.t = threadIdx.x - sub * a.tpr;
    r.D = (int)a.D;
    r.bar = 1 + sub;
    r.vec = a.vec;
    return r;
}

template <bool FULL> __device__ __forceinline__ void gain16(const float* g, const RowLane& r, u64 (&v)[8])
{
    load_row16<FULL, false>(g, r, v);
    flush16(v);
}

template <typename T, typename U, int THREADS, bool FULL>
__global__ void __launch_bounds__(THREADS)
k_norm_fwd(const __grid_constant__ NormArgs a)
{
    __shared__ float red[4][64];
    int sub, phase = 0;
    const RowLane r = lane_of(a, sub);
    const int per = blockDim.x / a.tpr;
    const float alpha = flush(a.alpha), beta = flush(a.beta);
    pdl_wait();
    for (int64_t i = (int64_t)blockIdx.x * per + sub; i < a.n; i += (int64_t)gridDim.x * per) {
        u64 x[8], w[8];
        float r1 = 0.0f, r2 = 0.0f;
        if (a.y) {
            u64 y[8];
            load_row16<FULL, true>(static_cast<const T*>(a.y) + i * a.y_ld, r, y);
            load_row16<FULL, false>(static_cast<const T*>(a.x) + i * a.x_ld, r, x);
            flush16(y);
            if (a.post) {
                r1 = rms_of(tree_of_chains(chain16<FULL>(y, y, r), r, red[sub], phase), a);
                mul16(y, r1);
                if (a.gain_post) {
                    gain16<FULL>(a.gain_post, r, w);
                    mul16(y, w);
                }
            }
            if (a.gate) {
                if (a.gate_rows) {
                    load_row16<FULL, true>(static_cast<const T*>(a.gate) + i * a.gate_ld, r, w);
                    flush16(w);
                } else {
                    gain16<FULL>(static_cast<const float*>(a.gate), r, w);
                }
                mul16(y, w);
            }
            flush16(x);
            const u64 al = pack2(alpha, alpha), be = pack2(beta, beta);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = fadd2_ftz(fmul2_rn(x[e], al), fmul2_rn(y[e], be));
                if (sizeof(T) == 2) {   // the norm reads the stream as it is stored
                    float p, q;
                    unpack2(x[e], p, q);
                    x[e] = pack2(to_f32<T>(from_f32<T>(p)), to_f32<T>(from_f32<T>(q)));
                }
            }
            store_row16<FULL>(static_cast<T*>(a.h) + i * a.h_ld, r, x);
        } else {
            load_row16<FULL, true>(static_cast<const T*>(a.x) + i * a.x_ld, r, x);
        }
        if (a.u) {
            flush16(x);
            r2 = rms_of(tree_of_chains(chain16<FULL>(x, x, r), r, red[sub], phase), a);
            mul16(x, r2);
            if (a.gain_pre) {
                gain16<FULL>(a.gain_pre, r, w);
                mul16(x, w);
            }
            store_row16<FULL>(static_cast<U*>(a.u) + i * a.u_ld, r, x);
        }
        if (a.stats && r.t == 0) {
            a.stats[2 * i] = r1;
            a.stats[2 * i + 1] = r2;
        }
    }
}

// v <- scale (x) (v (-) (unit (x) c)), c = S(v (x) unit) (/) D
template <bool FULL>
__device__ __forceinline__ void norm_back(u64 (&v)[8], const u64 (&unit)[8], float scale, const NormArgs& a,
                                          const RowLane& r, float* red, int& phase)
{
    const float c = mean_of(tree_of_chains(chain16<FULL>(v, unit, r), r, red, phase), (float)a.D, a.inv);
    const u64 cc = pack2(-c, -c), sc = pack2(scale, scale), z = pack2(-0.0f, -0.0f);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = fadd2_ftz(fmul2_rn(sc, fadd2_ftz(v[e], fmul2_rn(unit[e], cc))), z);
}

// s (+) a (x) b, or the product alone for a chunk's first token
__device__ __forceinline__ void column_sum(u64 (&s)[8], const u64 (&a)[8], const u64 (&b)[8], bool first)
{
    const u64 z = pack2(-0.0f, -0.0f);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s[e] = fadd2_ftz(fmul2_rn(a[e], b[e]), first ? z : s[e]);
}

template <bool FULL>
__device__ __forceinline__ void store_parts(float* parts, int64_t chunk, int64_t pitch, const RowLane& r, const u64 (&s)[8])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int d = r.at(k);
        float4 v;
        unpack2(s[2 * k], v.x, v.y);
        unpack2(s[2 * k + 1], v.z, v.w);
        if (FULL || d < r.D)   // the pitch is a multiple of 4
            store4(parts + chunk * pitch + d, v);
    }
}

template <typename T, typename U, int THREADS, bool FULL>
__global__ void __launch_bounds__(THREADS)
k_norm_bwd(const __grid_constant__ NormArgs a)
{
    __shared__ float red[4][64];
    int sub, phase = 0;
    const RowLane r = lane_of(a, sub);
    const int per = blockDim.x / a.tpr;
    const float alpha = flush(a.alpha), beta = flush(a.beta);
    pdl_wait();
    pdl_trigger();
    const int64_t chunks = (a.n + CHUNK - 1) / CHUNK;
    for (int64_t ch = (int64_t)blockIdx.x * per + sub; ch < chunks; ch += (int64_t)gridDim.x * per) {
        u64 s_pre[8], s_post[8], s_gate[8];
        const int64_t lo = ch * CHUNK, hi = lo + CHUNK < a.n ? lo + CHUNK : a.n;
        for (int64_t i = lo; i < hi; ++i) {
            const bool first = i == lo;
            u64 g[8], unit[8], w[8];
            if (a.dh)
                load_row16<FULL, false>(static_cast<const T*>(a.dh) + i * a.dh_ld, r, g);
            if (a.du) {
                u64 v[8];
                load_row16<FULL, true>(static_cast<const U*>(a.du) + i * a.du_ld, r, v);
                load_row16<FULL, true>(static_cast<const T*>(a.hs) + i * a.hs_ld, r, unit);
                const float r2 = flush(a.stats[2 * i + 1]);
                flush16(v);
                flush16(unit);
                mul16(unit, r2);
                if (a.dgain_pre)
                    column_sum(s_pre, v, unit, first);
                if (a.gain_pre) {
                    gain16<FULL>(a.gain_pre, r, w);
                    mul16(v, w);
                }
                norm_back<FULL>(v, unit, r2, a, r, red[sub], phase);
                if (a.dh) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        g[e] = fadd2_ftz(g[e], v[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        g[e] = v[e];
                }
            } else {
                flush16(g);
            }
            if (!a.y) {
                store_row16<FULL>(static_cast<T*>(a.dx) + i * a.dx_ld, r, g);
                continue;
            }
            u64 o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = g[e];
            mul16(o, alpha);
            store_row16<FULL>(static_cast<T*>(a.dx) + i * a.dx_ld, r, o);
            mul16(g, beta);
            load_row16<FULL, true>(static_cast<const T*>(a.y) + i * a.y_ld, r, unit);
            const float r1 = flush(a.stats[2 * i]);
            flush16(unit);
            if (a.post)
                mul16(unit, r1);
            if (a.gate) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = unit[e];
                if (a.post && a.gain_post) {
                    gain16<FULL>(a.gain_post, r, w);
                    mul16(o, w);
                }
                if (a.gate_rows) {
                    mul16(o, g);
                    store_row16<FULL>(static_cast<T*>(a.dgate) + i * a.dgate_ld, r, o);
                    load_row16<FULL, true>(static_cast<const T*>(a.gate) + i * a.gate_ld, r, w);
                    flush16(w);
                } else {
                    column_sum(s_gate, g, o, first);
                    gain16<FULL>(static_cast<const float*>(a.gate), r, w);
                }
                mul16(g, w);
            }
            if (a.post) {
                if (a.dgain_post)
                    column_sum(s_post, g, unit, first);
                if (a.gain_post) {
                    gain16<FULL>(a.gain_post, r, w);
                    mul16(g, w);
                }
                norm_back<FULL>(g, unit, r1, a, r, red[sub], phase);
            }
            store_row16<FULL>(static_cast<T*>(a.dy) + i * a.dy_ld, r, g);
        }
        if (a.dgain_pre)
            store_parts<FULL>(a.parts[0], ch, a.pitch, r, s_pre);
        if (a.dgain_post)
            store_parts<FULL>(a.parts[1], ch, a.pitch, r, s_post);
        if (a.gate && !a.gate_rows)
            store_parts<FULL>(a.parts[2], ch, a.pitch, r, s_gate);
    }
}

inline int64_t pitch_of(int64_t D) { return (D + 3) / 4 * 4; }

bool rows4_or_none(const void* p, int64_t ld, size_t bytes)
{
    return !p || ((reinterpret_cast<uintptr_t>(p) % (4 * bytes)) == 0 && ld % 4 == 0);
}

void set_up(NormArgs& a)
{
    const size_t t = a.type == 0 ? 4 : 2, u = a.u_type == 0 ? 4 : 2;
    a.tpr = row_threads(a.D);
    a.inv = (a.D & (a.D - 1)) == 0 ? 1.0f / (float)a.D : 0.0f;
    a.vec = rows4_or_none(a.x, a.x_ld, t) && rows4_or_none(a.y, a.y_ld, t) && rows4_or_none(a.h, a.h_ld, t) &&
            rows4_or_none(a.u, a.u_ld, u) && rows4_or_none(a.dh, a.dh_ld, t) && rows4_or_none(a.du, a.du_ld, u) &&
            rows4_or_none(a.hs, a.hs_ld, t) && rows4_or_none(a.dx, a.dx_ld, t) && rows4_or_none(a.dy, a.dy_ld, t) &&
            (a.gate_rows ? rows4_or_none(a.gate, a.gate_ld, t) && rows4_or_none(a.dgate, a.dgate_ld, t)
                         : rows4_or_none(a.gate, 0, 4)) &&
            rows4_or_none(a.gain_post, 0, 4) && rows4_or_none(a.gain_pre, 0, 4);
}

template <typename T, typename U, bool BWD> cudaError_t launch(const NormArgs& a, cudaStream_t st)
{
    const bool full = a.vec && a.D == (int64_t)ROW_E * a.tpr;
    const int threads = a.tpr < 128 ? 128 : a.tpr;
    const int64_t items = BWD ? (a.n + CHUNK - 1) / CHUNK : a.n, per = threads / a.tpr;
    const int64_t ctas = (items + per - 1) / per, most = (int64_t)num_sms() * 64;
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    count_launches(1);
#define GO(N, F) (BWD ? launch_pdl(k_norm_bwd<T, U, N, F>, grid, dim3(threads), 0, st, a) \
                      : launch_pdl(k_norm_fwd<T, U, N, F>, grid, dim3(threads), 0, st, a))
    if (threads <= 256)
        return full ? GO(256, true) : GO(256, false);
    if (threads == 512)
        return full ? GO(512, true) : GO(512, false);
    return full ? GO(1024, true) : GO(1024, false);
#undef GO
}

template <bool BWD> cudaError_t dispatch(const NormArgs& a, cudaStream_t st)
{
    if (a.type == 0)
        return a.u_type == 0 ? launch<float, float, BWD>(a, st) : launch<float, __nv_bfloat16, BWD>(a, st);
    return a.u_type == 0 ? launch<__nv_bfloat16, float, BWD>(a, st) : launch<__nv_bfloat16, __nv_bfloat16, BWD>(a, st);
}

} // namespace

cudaError_t launch_norm_fwd(NormArgs a, cudaStream_t st)
{
    set_up(a);
    return dispatch<false>(a, st);
}

size_t norm_bwd_ws_bytes(int64_t n, int64_t D)
{
    return (size_t)((n + CHUNK - 1) / CHUNK) * (size_t)pitch_of(D) * 4 * 3;
}

cudaError_t launch_norm_bwd(NormArgs a, void* ws, cudaStream_t st)
{
    set_up(a);
    const int64_t chunks = (a.n + CHUNK - 1) / CHUNK;
    a.pitch = pitch_of(a.D);
    RowTree t = {};
    t.pitch = a.pitch;
    t.D = a.D;
    t.scale = 1.0f;
    t.accumulate = a.accumulate;
    float* out[3] = {a.dgain_pre, a.dgain_post, a.gate && !a.gate_rows ? static_cast<float*>(a.dgate) : nullptr};
    for (int k = 0; k < 3; ++k) {
        a.parts[k] = static_cast<float*>(ws) + k * chunks * a.pitch;
        if (out[k]) {
            t.parts[t.jobs] = a.parts[k];
            t.count[t.jobs] = chunks;
            t.out[t.jobs] = out[k];
            ++t.jobs;
        }
    }
    cudaError_t e = dispatch<true>(a, st);
    if (e == cudaSuccess && t.jobs > 0)
        e = launch_row_tree(t, num_sms() * 4, st);
    return e;
}

} // namespace repro
