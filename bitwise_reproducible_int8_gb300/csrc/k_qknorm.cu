// k_qknorm.cu -- RMS norm of every query and key head and the rotary position
// in one pass, and its backward.
//
//   r = 1 (/) sqrt((S (/) D) (+) eps), y_d = (x_d (x) r) (x) gain_d, then each pair
//   (a, b) turned by the position's angle.  Backward: turn the gradient back, then
//   dx_d = r (x) (u_d (-) (h_d (x) c1)) with h = x r, u = dy gain, c1 = S'(u h) / D.
//
// One read and one write of the heads (and the gradient): bound by HBM.  A head
// lies in the registers of 8, 16 or 32 lanes, 4, 8 or 16 consecutive elements
// each, so the norm's order (groups of 4, then the pairwise tree) is a chain in a
// lane and a butterfly over lanes, and no shared memory stands between the load
// and the store.  A pair's other half is in the same lane (neighbour pairs), at a
// fixed lane distance (halves, R / 2 a multiple of the lane's elements), or else
// fetched through shared memory (every other width or alignment).
//
// The gains' gradients are sums over all rows (token, head): a CTA of the backward
// owns one 64-row chunk, leaves dy (x) h of each row in shared memory and adds the
// columns up in row order; k_rowtree.cu combines the chunk rows.
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace repro {
namespace {

constexpr int INTER = 0, HALF = 1, GENERIC = 2;   // how a rotation partner is found


// the head's values in this lane: E elements from d0 on (0 past the width)
template <typename T, int E, bool VEC>
__device__ __forceinline__ void load_head(const T* p, int d0, int D, float (&x)[E])
{
    if (VEC) {
#pragma unroll
        for (int g = 0; g < E; g += 4)
            if (d0 + g < D) {
                const float4 v = load4(p + d0 + g);
                x[g] = v.x, x[g + 1] = v.y, x[g + 2] = v.z, x[g + 3] = v.w;
            } else {
                x[g] = x[g + 1] = x[g + 2] = x[g + 3] = 0.0f;
            }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[e] = d0 + e < D ? to_f32<T>(p[d0 + e]) : 0.0f;
    }
}

template <typename T, int E, bool VEC>
__device__ __forceinline__ void store_head(T* p, int d0, int D, const float (&x)[E])
{
    if (VEC) {
#pragma unroll
        for (int g = 0; g < E; g += 4)
            if (d0 + g < D)
                store4(p + d0 + g, make_float4(x[g], x[g + 1], x[g + 2], x[g + 3]));
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (d0 + e < D)
                p[d0 + e] = from_f32<T>(x[e]);
    }
}

// S of the terms a_e (x) b_e over the head: groups of 4 left to right, then the
// pairwise tree, first within the lane, then over its LPH lanes.  A term past the
// width counts as -0, which leaves every sum as it is.
template <int E, int LPH>
__device__ __forceinline__ float head_sum(const float (&a)[E], const float (&b)[E], int d0, int D)
{
    float g[E / 4];
#pragma unroll
    for (int k = 0; k < E / 4; ++k) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            p[e] = d0 + 4 * k + e < D ? fmul_rn(a[4 * k + e], b[4 * k + e]) : -0.0f;
        g[k] = fadd_ftz(fadd_ftz(fadd_ftz(p[0], p[1]), p[2]), p[3]);
    }
#pragma unroll
    for (int s = 1; s < E / 4; s *= 2)
#pragma unroll
        for (int k = 0; k + s < E / 4; k += 2 * s)
            g[k] = fadd_ftz(g[k], g[k + s]);
    float v = g[0];
#pragma unroll
    for (int s = 1; s < LPH; s *= 2)
        v = fadd_ftz(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

// v turned by the position's angle (BACK: turned back), in place.  d0 + e >= R is
// left alone.  cs: the position's row, R / 2 cosines then R / 2 sines.
template <int E, int LPH, int MODE, bool BACK>
__device__ __forceinline__ void rotate(float (&v)[E], const float* __restrict__ cs, int d0, int D, int R,
                                       bool inter, float* row)
{
    const int half = R >> 1;
    if (MODE == INTER) {
#pragma unroll
        for (int e = 0; e < E; e += 2)
            if (d0 + e < R) {
                const int j = (d0 + e) >> 1;
                const float c = flush(__ldg(cs + j)), s = flush(__ldg(cs + half + j));
                const float a = v[e], b = v[e + 1];
                const float as = fmul_rn(a, s), bs = fmul_rn(b, s);
                v[e] = fadd_ftz(fmul_rn(a, c), BACK ? bs : -bs);
                v[e + 1] = fadd_ftz(fmul_rn(b, c), BACK ? -as : as);
            }
    } else if (MODE == HALF) {
        const int lane = threadIdx.x & 31, step = half / E;
        const bool low = d0 < half, turns = d0 < R;
        const int other = turns ? (low ? lane + step : lane - step) : lane;
        float w[E];
#pragma unroll
        for (int e = 0; e < E; ++e)
            w[e] = __shfl_sync(0xffffffffu, v[e], other);
        if (turns) {
            const int j0 = low ? d0 : d0 - half;
            const bool minus = low != BACK;   // a: c y_a - s y_b (turned back: +); b the other way round
#pragma unroll
            for (int g = 0; g < E; g += 4) {
                const float4 c4 = __ldg(reinterpret_cast<const float4*>(cs + j0 + g));
                const float4 s4 = __ldg(reinterpret_cast<const float4*>(cs + half + j0 + g));
                const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float ws = fmul_rn(w[g + e], flush(s[e]));
                    v[g + e] = fadd_ftz(fmul_rn(v[g + e], flush(c[e])), minus ? -ws : ws);
                }
            }
        }
    } else {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (d0 + e < D)
                row[d0 + e] = v[e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = d0 + e;
            if (d < R) {
                const bool low = inter ? !(d & 1) : d < half;
                const int j = inter ? d >> 1 : (low ? d : d - half);
                const int o = inter ? d ^ 1 : (low ? d + half : d - half);
                const float ws = fmul_rn(row[o], flush(__ldg(cs + half + j)));
                v[e] = fadd_ftz(fmul_rn(v[e], flush(__ldg(cs + j))), low != BACK ? -ws : ws);
            }
        }
    }
}

__device__ __forceinline__ float rnorm(float S, float width, float eps)
{
    const float ms = fadd_ftz(flush(__fdiv_rn(S, width)), eps);
    return flush(__fdiv_rn(1.0f, flush(__fsqrt_rn(ms))));
}

// the row of the table for a token's position, or NULL (and the error word) when
// there is none
__device__ __forceinline__ const float* rope_row(const QkArgs& a, unsigned tok, bool report, bool& ok)
{
    ok = true;
    if (a.R == 0)
        return nullptr;
    const int64_t p = a.positions ? (int64_t)__ldg(a.positions + tok) : (int64_t)(tok % (unsigned)a.T);
    ok = p >= 0 && p < a.P;
    if (!ok && report)
        atomicOr(a.err, kErrIndexBit);
    return a.rope + (ok ? p : 0) * a.R;
}

template <typename T, int E, int LPH, int MODE>
__global__ void __launch_bounds__(256)
k_qk_fwd(const __grid_constant__ QkArgs a)
{
    constexpr int HPW = 32 / LPH;            // heads a warp holds
    constexpr int U = E >= 16 ? 1 : 16 / E;  // rows in flight per lane
    constexpr bool VEC = MODE != GENERIC;
    __shared__ float rows[MODE == GENERIC ? 8 * HPW * E * LPH : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = (int)a.D, R = (int)a.R, d0 = (lane % LPH) * E, sub = lane / LPH;
    const unsigned H = (unsigned)(a.t[0].H + a.t[1].H), total = (unsigned)a.n * H;
    const unsigned base = blockIdx.x * (8u * HPW * U) + (unsigned)(warp * HPW + sub);
    const float width = (float)D, eps = flush(a.eps);
    float x[U][E];
    unsigned tok[U], h[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const unsigned row = base + (unsigned)u * 8u * HPW;
        tok[u] = row / H;
        h[u] = row - tok[u] * H;
        if (row < total) {
            const bool is_q = h[u] < (unsigned)a.t[0].H;
            const QkTensor& t = is_q ? a.t[0] : a.t[1];
            const int64_t head = is_q ? h[u] : h[u] - (unsigned)a.t[0].H;
            load_head<T, E, VEC>(static_cast<const T*>(t.x) + (int64_t)tok[u] * t.ld + head * t.hs, d0, D, x[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const unsigned row = base + (unsigned)u * 8u * HPW;
        // lanes of one warp may hold rows on both sides of the end: all take part in the shuffles
        const bool live = row < total;
        if (__ballot_sync(0xffffffffu, live) == 0)
            break;
        const bool is_q = !live || h[u] < (unsigned)a.t[0].H;
        const QkTensor& t = is_q ? a.t[0] : a.t[1];
        const int64_t head = !live ? 0 : is_q ? h[u] : h[u] - (unsigned)a.t[0].H;
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[u][e] = live ? flush(x[u][e]) : 0.0f;
        const float r = rnorm(head_sum<E, LPH>(x[u], x[u], d0, D), width, eps);
#pragma unroll
        for (int e = 0; e < E; ++e)
            x[u][e] = fmul_flush(x[u][e], r);
        if (t.gain) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (d0 + e < D)
                    x[u][e] = fmul_flush(x[u][e], flush(__ldg(t.gain + d0 + e)));
        }
        bool ok;
        const float* cs = rope_row(a, live ? tok[u] : 0u, live && d0 == 0, ok);
        rotate<E, LPH, MODE, false>(x[u], cs, d0, D, R, a.interleaved,
                                    rows + (MODE == GENERIC ? (warp * HPW + sub) * E * LPH : 0));
        if (!ok) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[u][e] = 0.0f;
        }
        if (live) {
            float* o = t.out + ((int64_t)tok[u] * t.H + head) * D;
            if (D % 4 == 0)
                store_head<float, E, true>(o, d0, D, x[u]);
            else
                store_head<float, E, false>(o, d0, D, x[u]);
        }
    }
}

constexpr int CHUNK = 64;   // rows of a chunk of the gains' canonical sums

template <typename T, int E, int LPH, int MODE>
__global__ void __launch_bounds__(256)
k_qk_bwd(const __grid_constant__ QkArgs a, unsigned chunks_q, float* __restrict__ parts, int64_t pitch)
{
    constexpr int HPW = 32 / LPH;
    constexpr int U = E >= 8 ? 1 : 2;
    constexpr bool VEC = MODE != GENERIC;
    __shared__ float rows[MODE == GENERIC ? 8 * HPW * E * LPH : 1];
    extern __shared__ float terms[];   // [CHUNK][D] with a gain
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = (int)a.D, R = (int)a.R, d0 = (lane % LPH) * E, sub = lane / LPH;
    const bool is_q = blockIdx.x < chunks_q;
    const QkTensor& t = is_q ? a.t[0] : a.t[1];
    const unsigned chunk = is_q ? blockIdx.x : blockIdx.x - chunks_q;
    const unsigned H = (unsigned)t.H, total = (unsigned)a.n * H, first = chunk * CHUNK;
    const float width = (float)D, eps = flush(a.eps);
    const bool gain = t.gain != nullptr;
    float* srow = rows + (MODE == GENERIC ? (warp * HPW + sub) * E * LPH : 0);
    for (int k0 = 0; k0 < CHUNK; k0 += 8 * HPW * U) {
        float x[U][E], dy[U][E];
        unsigned tok[U], h[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned row = first + (unsigned)(k0 + u * 8 * HPW + warp * HPW + sub);
            tok[u] = row / H;
            h[u] = row - tok[u] * H;
            if (row < total) {
                load_head<T, E, VEC>(static_cast<const T*>(t.x) + (int64_t)tok[u] * t.ld + (int64_t)h[u] * t.hs,
                                     d0, D, x[u]);
                const float* g = t.dout + (int64_t)row * D;
                if (D % 4 == 0)
                    load_head<float, E, true>(g, d0, D, dy[u]);
                else
                    load_head<float, E, false>(g, d0, D, dy[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned row = first + (unsigned)(k0 + u * 8 * HPW + warp * HPW + sub);
            const bool live = row < total;
            if (__ballot_sync(0xffffffffu, live) == 0)
                break;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x[u][e] = live ? flush(x[u][e]) : 0.0f;
                dy[u][e] = live ? flush(dy[u][e]) : 0.0f;
            }
            const float r = rnorm(head_sum<E, LPH>(x[u], x[u], d0, D), width, eps);
            bool ok;
            const float* cs = rope_row(a, live ? tok[u] : 0u, live && d0 == 0, ok);
            rotate<E, LPH, MODE, true>(dy[u], cs, d0, D, R, a.interleaved, srow);
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[u][e] = fmul_flush(x[u][e], r);   // h
            if (gain) {
                const int at = (int)(row - first) * D;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (live && d0 + e < D) {
                        terms[at + d0 + e] = ok ? fmul_flush(dy[u][e], x[u][e]) : 0.0f;
                        dy[u][e] = fmul_flush(dy[u][e], flush(__ldg(t.gain + d0 + e)));
                    }
            }
            const float c1 = flush(__fdiv_rn(head_sum<E, LPH>(dy[u], x[u], d0, D), width));
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float v = fadd_ftz(dy[u][e], -fmul_flush(x[u][e], c1));
                x[u][e] = ok ? fmul_flush(r, v) : 0.0f;
            }
            if (live)
                store_head<T, E, VEC>(static_cast<T*>(t.dx) + (int64_t)tok[u] * t.dx_ld + (int64_t)h[u] * t.dx_hs,
                                      d0, D, x[u]);
        }
    }
    if (gain) {
        __syncthreads();
        const int L = total - first < CHUNK ? (int)(total - first) : CHUNK;
        for (int d = threadIdx.x; d < D; d += 256) {
            float s = terms[d];
#pragma unroll 8
            for (int k = 1; k < L; ++k)
                s = fadd_ftz(s, terms[k * D + d]);
            parts[(int64_t)blockIdx.x * pitch + d] = s;
        }
    }
}

unsigned chunks_of(int64_t rows) { return (unsigned)((rows + CHUNK - 1) / CHUNK); }

// how partners are found, given everything that is loaded four at a time
template <typename T> int mode_of(const QkArgs& a, int E, bool back)
{
    bool vec = a.D % 4 == 0;
    for (const QkTensor& t : a.t)
        if (t.H > 0) {
            vec = vec && rows4<T>(t.x, t.ld) && t.hs % 4 == 0;
            if (back)
                vec = vec && rows4<T>(t.dx, t.dx_ld) && t.dx_hs % 4 == 0;
        }
    if (!vec)
        return GENERIC;
    if (a.interleaved || a.R == 0)
        return INTER;
    return (a.R / 2) % E == 0 ? HALF : GENERIC;
}

// calls f(E, LPH) as compile-time constants for the head width: up to 128
// elements 4 per lane in 8, 16 or 32 lanes, wider ones 8 or 16 per lane
template <typename F> cudaError_t by_width(int64_t D, F f)
{
    if (D <= 32)
        return f(std::integral_constant<int, 4>(), std::integral_constant<int, 8>());
    if (D <= 64)
        return f(std::integral_constant<int, 4>(), std::integral_constant<int, 16>());
    if (D <= 128)
        return f(std::integral_constant<int, 4>(), std::integral_constant<int, 32>());
    if (D <= 256)
        return f(std::integral_constant<int, 8>(), std::integral_constant<int, 32>());
    return f(std::integral_constant<int, 16>(), std::integral_constant<int, 32>());
}

template <typename T> cudaError_t fwd_typed(const QkArgs& a, cudaStream_t st)
{
    return by_width(a.D, [&](auto e, auto l) {
        constexpr int E = decltype(e)::value, LPH = decltype(l)::value;
        constexpr int per = 8 * (32 / LPH) * (E >= 16 ? 1 : 16 / E);
        const int64_t total = a.n * (a.t[0].H + a.t[1].H);
        const unsigned grid = (unsigned)((total + per - 1) / per);
        const int m = mode_of<T>(a, E, false);
        if (m == INTER)
            k_qk_fwd<T, E, LPH, INTER><<<grid, 256, 0, st>>>(a);
        else if (m == HALF)
            k_qk_fwd<T, E, LPH, HALF><<<grid, 256, 0, st>>>(a);
        else
            k_qk_fwd<T, E, LPH, GENERIC><<<grid, 256, 0, st>>>(a);
        count_launches(1);
        return cudaGetLastError();
    });
}

template <typename T> cudaError_t bwd_typed(const QkArgs& a, float* parts, int64_t pitch, cudaStream_t st)
{
    return by_width(a.D, [&](auto e, auto l) {
        constexpr int E = decltype(e)::value, LPH = decltype(l)::value;
        const unsigned cq = chunks_of(a.n * a.t[0].H), ck = chunks_of(a.n * a.t[1].H);
        const bool gain = a.t[0].gain || a.t[1].gain;
        const size_t smem = gain ? (size_t)CHUNK * a.D * 4 : 0;
        const int m = mode_of<T>(a, E, true);
        auto go = [&](auto kernel) {
            if (smem > 32 * 1024) {
                const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                           (int)smem);
                if (r != cudaSuccess)
                    return r;
            }
            kernel<<<cq + ck, 256, smem, st>>>(a, cq, parts, pitch);
            count_launches(1);
            return cudaGetLastError();
        };
        return m == INTER ? go(k_qk_bwd<T, E, LPH, INTER>)
               : m == HALF ? go(k_qk_bwd<T, E, LPH, HALF>) : go(k_qk_bwd<T, E, LPH, GENERIC>);
    });
}

} // namespace

cudaError_t launch_qk_fwd(const QkArgs& a, cudaStream_t st)
{
    return a.type == 0 ? fwd_typed<float>(a, st) : fwd_typed<__nv_bfloat16>(a, st);
}

size_t qk_bwd_ws_bytes(int64_t n, int64_t Hq, int64_t Hkv, int64_t D)
{
    return ((size_t)chunks_of(n * Hq) + chunks_of(n * Hkv)) * (size_t)((D + 3) & ~3LL) * 4;
}

cudaError_t launch_qk_bwd(const QkArgs& a, void* ws, cudaStream_t st)
{
    const int64_t pitch = (a.D + 3) & ~3LL;
    float* parts = static_cast<float*>(ws);
    cudaError_t e = a.type == 0 ? bwd_typed<float>(a, parts, pitch, st) : bwd_typed<__nv_bfloat16>(a, parts, pitch, st);
    for (int x = 0; x < 2 && e == cudaSuccess; ++x) {
        const QkTensor& t = a.t[x];
        if (!t.gain || t.H == 0)
            continue;
        RowTree r;
        r.parts = parts;
        r.pitch = pitch;
        r.joins = nullptr;
        r.njoins = nullptr;
        r.count = chunks_of(a.n * t.H);
        r.D = a.D;
        r.out = t.dgain;
        r.out_ld = a.D;
        r.scale = 1.0f;
        r.accumulate = a.accumulate;
        if (x == 1)
            r.parts += (int64_t)chunks_of(a.n * a.t[0].H) * pitch;
        e = launch_row_tree(r, num_sms(), st);
    }
    return e;
}

} // namespace repro
