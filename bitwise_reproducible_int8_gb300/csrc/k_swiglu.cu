// k_swiglu.cu -- gated activation with an 8-bit copy of its inputs, and its backward out of
// that copy (or out of the inputs).
//
//   a = g sig(g) up;  dg = da up sig(g) (1 + g sig(-g)), dup = da g sig(g)
//   sig(g), sig(-g) = w, e w in g's order, e = exp_r(-|g|), w = 1 / (1 + e): one e^x and one
//   reciprocal serve both and neither loses bits by a difference from 1
//
// Bound by HBM, with the FP32 pipe close behind: 14 bytes a pair either way in fp32 (8 in, 4 out and
// 2.06 of codes and scales; backward 4 + 2.06 in, 8 out) where keeping the inputs themselves would
// take 20 in the backward.  A warp takes a group of 128 pairs: a lane 4 neighbours of either, the
// group's scales from two warp-wide maxima.
#include "codes.cuh"
#include "elem.cuh"
#include "expr.cuh"
#include "internal.h"
#include "launch.cuh"

namespace repro {
namespace {

constexpr int GROUP = 128;

struct Kernel {
    SwigluArgs s;
    int64_t G, items;      // groups of a row, of all rows
    bool vec, avec;        // gu (dgu) and a (da) on 4-element boundaries, F too
};

template <typename T> __device__ __forceinline__ void take4(const T* p, int64_t d, int64_t F, bool vec, float (&v)[4])
{
    if (vec && d + 4 <= F) {
        const float4 x = stream4(p + d);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = d + e < F ? to_f32<T>(p[d + e]) : 0.0f;
    }
}

template <typename T> __device__ __forceinline__ void put4(T* p, int64_t d, int64_t F, bool vec, const float (&v)[4])
{
    if (vec && d + 4 <= F) {
        store4(p + d, make_float4(v[0], v[1], v[2], v[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < F)
                p[d + e] = from_f32<T>(v[e]);
    }
}

// sig(g) and sig(-g) of four
__device__ __forceinline__ void sigmoids(const float (&g)[4], float (&sig)[4], float (&rest)[4])
{
    float e[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2)
        unpack2(exp_r2(pack2(-fabsf(g[i]), -fabsf(g[i + 1]))), e[i], e[i + 1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float w = __frcp_rn(fadd_ftz(1.0f, e[i])), ew = fmul_flush(e[i], w);
        sig[i] = g[i] >= 0.0f ? w : ew;
        rest[i] = g[i] >= 0.0f ? ew : w;
    }
}

__device__ __forceinline__ unsigned magnitude(float v)
{
    const unsigned m = __float_as_uint(v) & 0x7fffffffu;
    return m > 0x7f800000u ? 0u : m;   // a NaN is passed over
}

// the group's codes and scale
__device__ __forceinline__ void keep(const float (&v)[4], int8_t* codes, float* scale, int lane)
{
    const unsigned m = max(max(magnitude(v[0]), magnitude(v[1])), max(magnitude(v[2]), magnitude(v[3])));
    const CodeScale c = code_scale_of_max(__uint_as_float(__reduce_max_sync(0xffffffffu, m)));
    reinterpret_cast<uint32_t*>(codes)[lane] = codes4(v, c);
    if (lane == 0)
        *scale = c.s;
}

template <typename T, typename A, bool KEEP>
__global__ void __launch_bounds__(256)
k_swiglu_fwd(const __grid_constant__ Kernel k)
{
    const int lane = threadIdx.x & 31;
    const int64_t F = k.s.F, step = (int64_t)gridDim.x * 8;
    pdl_wait();
    for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < k.items; it += step) {
        const int64_t i = it / k.G, gr = it - i * k.G, d = gr * GROUP + 4 * lane;
        const T* row = static_cast<const T*>(k.s.gu) + i * k.s.gu_ld;
        float g[4], u[4], sig[4], rest[4];
        take4<T>(row, d, F, k.vec, g);
        take4<T>(row + F, d, F, k.vec, u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            g[e] = flush(g[e]), u[e] = flush(u[e]);
        if (KEEP) {
            const int64_t at = 2 * i * k.G + gr;
            keep(g, k.s.codes + at * GROUP, k.s.scales + at, lane);
            keep(u, k.s.codes + (at + k.G) * GROUP, k.s.scales + at + k.G, lane);
        }
        sigmoids(g, sig, rest);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            g[e] = fmul_flush(fmul_flush(g[e], sig[e]), u[e]);
        put4<A>(static_cast<A*>(k.s.a) + i * k.s.a_ld, d, F, k.avec, g);
    }
}

__device__ __forceinline__ void decode(const int8_t* codes, float s, int lane, float (&v)[4])
{
    const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes) + lane);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = dequant((int)(int8_t)(c >> (8 * e)), s);
}

template <typename T, typename A, bool KEPT>
__global__ void __launch_bounds__(256)
k_swiglu_bwd(const __grid_constant__ Kernel k)
{
    const int lane = threadIdx.x & 31;
    const int64_t F = k.s.F, step = (int64_t)gridDim.x * 8;
    pdl_wait();
    for (int64_t it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); it < k.items; it += step) {
        const int64_t i = it / k.G, gr = it - i * k.G, d = gr * GROUP + 4 * lane;
        float g[4], u[4], da[4], sig[4], rest[4];
        take4<A>(static_cast<const A*>(k.s.da) + i * k.s.a_ld, d, F, k.avec, da);
        if (KEPT) {
            const int64_t at = 2 * i * k.G + gr;
            decode(k.s.codes + at * GROUP, flush(__ldg(k.s.scales + at)), lane, g);
            decode(k.s.codes + (at + k.G) * GROUP, flush(__ldg(k.s.scales + at + k.G)), lane, u);
        } else {
            const T* row = static_cast<const T*>(k.s.gu) + i * k.s.gu_ld;
            take4<T>(row, d, F, k.vec, g);
            take4<T>(row + F, d, F, k.vec, u);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                g[e] = flush(g[e]), u[e] = flush(u[e]);
        }
        sigmoids(g, sig, rest);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = flush(da[e]);
            const float dg = fmul_flush(fmul_flush(fmul_flush(x, u[e]), sig[e]), fadd_ftz(1.0f, fmul_rn(g[e], rest[e])));
            u[e] = fmul_flush(x, fmul_flush(g[e], sig[e]));
            g[e] = dg;
        }
        T* out = static_cast<T*>(k.s.dgu) + i * k.s.dgu_ld;
        put4<T>(out, d, F, k.vec, g);
        put4<T>(out + F, d, F, k.vec, u);
    }
}

template <typename T> bool vec_of(const void* p, int64_t ld, int64_t F)
{
    return !p || (rows4<T>(p, ld) && F % 4 == 0);
}

template <typename T, typename A> cudaError_t launch(Kernel& k, bool fwd, cudaStream_t st)
{
    const SwigluArgs& s = k.s;
    k.vec = vec_of<T>(s.gu, s.gu_ld, s.F) && vec_of<T>(s.dgu, s.dgu_ld, s.F);
    k.avec = vec_of<A>(fwd ? s.a : s.da, s.a_ld, s.F);
    const int64_t ctas = (k.items + 7) / 8, most = (int64_t)num_sms() * 32;
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    count_launches(1);
    if (fwd)
        return s.codes ? launch_pdl(k_swiglu_fwd<T, A, true>, grid, dim3(256), 0, st, k)
                       : launch_pdl(k_swiglu_fwd<T, A, false>, grid, dim3(256), 0, st, k);
    return s.codes ? launch_pdl(k_swiglu_bwd<T, A, true>, grid, dim3(256), 0, st, k)
                   : launch_pdl(k_swiglu_bwd<T, A, false>, grid, dim3(256), 0, st, k);
}

cudaError_t dispatch(const SwigluArgs& a, bool fwd, cudaStream_t st)
{
    Kernel k = {};
    k.s = a;
    k.G = (a.F + GROUP - 1) / GROUP;
    k.items = a.n * k.G;
    if (a.type == 0)
        return a.a_type == 0 ? launch<float, float>(k, fwd, st) : launch<float, __nv_bfloat16>(k, fwd, st);
    return a.a_type == 0 ? launch<__nv_bfloat16, float>(k, fwd, st) : launch<__nv_bfloat16, __nv_bfloat16>(k, fwd, st);
}

} // namespace

cudaError_t launch_swiglu_fwd(const SwigluArgs& a, cudaStream_t st) { return dispatch(a, true, st); }
cudaError_t launch_swiglu_bwd(const SwigluArgs& a, cudaStream_t st) { return dispatch(a, false, st); }

} // namespace repro
