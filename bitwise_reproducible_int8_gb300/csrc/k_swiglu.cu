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
// Measured, 16,384 x 5632 fp32: forward 204 us, 6.4 TB/s, backward 193 us, 6.7 TB/s, floor 191 each.  In
// bf16 instructions bound it (forward 194 us, 114 without the copy, floors 110 and 82; backward 166).  Backward out
// of the inputs 268 us in fp32, floor 272, 159 in bf16, floor 136.
#include "codes.cuh"
#include "elem.cuh"
#include "expr.cuh"
#include "internal.h"
#include "launch.cuh"

namespace repro {
namespace {

typedef unsigned long long u64;

constexpr int GROUP = 128;
constexpr int RUN = 2;       // neighbouring groups of a row a warp takes at a time

struct Kernel {
    SwigluArgs s;
    int64_t G, R, items;   // groups of a row; runs of RUN of them, of a row and of all rows
    int64_t rows, runs;    // how far a warp steps: so many rows and runs
};

// four neighbours from element d of F; VEC: on a boundary of 4 elements, F a multiple of 4
template <bool VEC, typename T> __device__ __forceinline__ void take4(const T* p, int64_t d, int64_t F, float (&v)[4])
{
    if (VEC) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (d < F)
            x = stream4(p + d);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = d + e < F ? to_f32<T>(p[d + e]) : 0.0f;
    }
}

template <bool VEC, typename T> __device__ __forceinline__ void put4(T* p, int64_t d, int64_t F, const float (&v)[4])
{
    if (VEC) {
        if (d < F)
            store4(p + d, make_float4(v[0], v[1], v[2], v[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < F)
                p[d + e] = from_f32<T>(v[e]);
    }
}

__device__ __forceinline__ u64 mul_flush2(u64 a, u64 b) { return fadd2_ftz(fmul2_rn(a, b), pack2(-0.0f, -0.0f)); }
__device__ __forceinline__ u64 flush2(u64 a) { return fadd2_ftz(a, pack2(-0.0f, -0.0f)); }

// RN(1 / d) for d in [1, 2]: the hardware's reciprocal (within 2^-23) and one Newton step, which is
// correctly rounded by Markstein's theorem (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990) but for a significand of all ones; equal to the division for
// every float of the interval, that one included (all 2^23 + 1 compared)
__device__ __forceinline__ float reciprocal(float d)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return __fmaf_rn(r, __fmaf_rn(-d, r, 1.0f), r);
}

// sig(g), and with REST sig(-g), of two
template <bool REST> __device__ __forceinline__ u64 sigmoids(u64 g, u64& rest)
{
    float g0, g1, d0, d1;
    unpack2(g, g0, g1);
    const u64 e = exp_r2_neg(-fabsf(g0), -fabsf(g1));
    unpack2(fadd2_ftz(e, pack2(1.0f, 1.0f)), d0, d1);
    const float w0 = reciprocal(d0), w1 = reciprocal(d1);
    float s0, s1;
    unpack2(mul_flush2(e, pack2(w0, w1)), s0, s1);
    const bool up0 = g0 >= 0.0f, up1 = g1 >= 0.0f;
    if (REST)
        rest = pack2(up0 ? s0 : w0, up1 ? s1 : w1);
    return pack2(up0 ? w0 : s0, up1 ? w1 : s1);
}

// the largest magnitude of a group.  Subnormals are not flushed one by one: it is, and beside a scale
// of 2^-67 or more, below which values are divided, they are nothing
__device__ __forceinline__ unsigned top_of(const float (&v)[4])
{
    const float m = fmaxf(fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fabsf(v[2])), fabsf(v[3])), 0.0f);   // passes over NaN
    return __reduce_max_sync(0xffffffffu, __float_as_uint(m));
}

__device__ __forceinline__ uint32_t codes_of(const float (&v)[4], const CodeScale& c)
{
    const CodeScale all[4] = {c, c, c, c};
    uint32_t q;
    if (!codes4(v, all, q))
        q = codes4_divided(v, all);
    return q;
}

// codes and scale of a group
__device__ __forceinline__ void keep(const float (&v)[4], uint32_t* codes, float* scale, int lane)
{
    const CodeScale c = code_scale_of_max(__uint_as_float(top_of(v)));
    *codes = codes_of(v, c);
    if (lane == 0)
        *scale = c.s;
}

// The runs a warp takes: every so many, without a division for each
struct Walk {
    int64_t it, i, run;   // run of all, row, run of the row

    __device__ __forceinline__ Walk(const Kernel& k)
    {
        it = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
        i = it / k.R;
        run = it - i * k.R;
    }
    __device__ __forceinline__ void next(const Kernel& k)
    {
        it += (int64_t)gridDim.x * 8;
        i += k.rows;
        run += k.runs;
        if (run >= k.R) {
            run -= k.R;
            ++i;
        }
    }
};

template <typename T, typename A, bool KEEP, bool VEC>
__global__ void __launch_bounds__(256, KEEP ? 6 : 4)
k_swiglu_fwd(const __grid_constant__ Kernel k)
{
    const int lane = threadIdx.x & 31;
    const int64_t F = k.s.F;
    pdl_wait();
    pdl_trigger();
    for (Walk w(k); w.it < k.items; w.next(k)) {
        const int64_t gr = RUN * w.run, d = gr * GROUP + 4 * lane;
        const T* row = static_cast<const T*>(k.s.gu) + w.i * k.s.gu_ld;
        A* out = static_cast<A*>(k.s.a) + w.i * k.s.a_ld;
        float g[RUN][4], u[RUN][4];
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
            take4<VEC>(row, d + r * GROUP, F, g[r]);
            take4<VEC>(row + F, d + r * GROUP, F, u[r]);
        }
        const int64_t at = 2 * w.i * k.G + gr;
        uint32_t* const codes = reinterpret_cast<uint32_t*>(k.s.codes + at * GROUP) + lane;
        float* const scales = k.s.scales + at;
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
            if (r > 0 && gr + r >= k.G)
                break;
            if (KEEP) {
                keep(g[r], codes + r * (GROUP / 4), scales + r, lane);
                keep(u[r], codes + (k.G + r) * (GROUP / 4), scales + k.G + r, lane);
            }
#pragma unroll
            for (int e = 0; e < 4; e += 2) {   // a subnormal g is flushed with its product, sig being at most 1
                const u64 gg = pack2(g[r][e], g[r][e + 1]);
                u64 none;
                const u64 a = mul_flush2(mul_flush2(gg, sigmoids<false>(gg, none)), flush2(pack2(u[r][e], u[r][e + 1])));
                unpack2(a, g[r][e], g[r][e + 1]);
            }
            put4<VEC>(out, d + r * GROUP, F, g[r]);
        }
    }
}

// two neighbours of a group: from its codes, or as they are
__device__ __forceinline__ u64 decode(uint32_t c, int e, float s)
{
    return mul_flush2(pack2(__int2float_rn((int)(int8_t)(c >> (8 * e))), __int2float_rn((int)(int8_t)(c >> (8 * e + 8)))), pack2(s, s));
}

template <typename T, typename A, bool KEPT, bool VEC>
__global__ void __launch_bounds__(256, 4)
k_swiglu_bwd(const __grid_constant__ Kernel k)
{
    const int lane = threadIdx.x & 31;
    const int64_t F = k.s.F;
    pdl_wait();
    pdl_trigger();
    for (Walk w(k); w.it < k.items; w.next(k)) {
        const int64_t gr = RUN * w.run, d = gr * GROUP + 4 * lane, at = 2 * w.i * k.G + gr;
        float g[RUN][4], u[RUN][4], da[RUN][4], sg[RUN], su[RUN];
        uint32_t cg[RUN], cu[RUN];
        const A* in = static_cast<const A*>(k.s.da) + w.i * k.s.a_ld;
        const T* row = static_cast<const T*>(k.s.gu) + w.i * k.s.gu_ld;
        T* out = static_cast<T*>(k.s.dgu) + w.i * k.s.dgu_ld;
        const uint32_t* codes = reinterpret_cast<const uint32_t*>(k.s.codes + at * GROUP) + lane;
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
            take4<VEC>(in, d + r * GROUP, F, da[r]);
            if (KEPT) {
                const bool live = r == 0 || gr + r < k.G;
                cg[r] = live ? __ldg(codes + r * (GROUP / 4)) : 0u;
                cu[r] = live ? __ldg(codes + (k.G + r) * (GROUP / 4)) : 0u;
                sg[r] = live ? flush(__ldg(k.s.scales + at + r)) : 0.0f;
                su[r] = live ? flush(__ldg(k.s.scales + at + k.G + r)) : 0.0f;
            } else {
                take4<VEC>(row, d + r * GROUP, F, g[r]);
                take4<VEC>(row + F, d + r * GROUP, F, u[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
            if (r > 0 && gr + r >= k.G)
                break;
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const u64 gg = KEPT ? decode(cg[r], e, sg[r]) : flush2(pack2(g[r][e], g[r][e + 1]));
                const u64 uu = KEPT ? decode(cu[r], e, su[r]) : flush2(pack2(u[r][e], u[r][e + 1]));
                const u64 x = flush2(pack2(da[r][e], da[r][e + 1]));
                u64 rest;
                const u64 sig = sigmoids<true>(gg, rest);
                const u64 slope = fadd2_ftz(fmul2_rn(gg, rest), pack2(1.0f, 1.0f));
                unpack2(mul_flush2(mul_flush2(mul_flush2(x, uu), sig), slope), g[r][e], g[r][e + 1]);
                unpack2(mul_flush2(x, mul_flush2(gg, sig)), u[r][e], u[r][e + 1]);
            }
            put4<VEC>(out, d + r * GROUP, F, g[r]);
            put4<VEC>(out + F, d + r * GROUP, F, u[r]);
        }
    }
}

template <typename T> bool vec_of(const void* p, int64_t ld, int64_t F)
{
    return !p || (rows4<T>(p, ld) && F % 4 == 0);
}

template <typename T, typename A> cudaError_t launch(Kernel& k, bool fwd, cudaStream_t st)
{
    const SwigluArgs& s = k.s;
    const bool vec = vec_of<T>(s.gu, s.gu_ld, s.F) && vec_of<T>(s.dgu, s.dgu_ld, s.F) && vec_of<A>(fwd ? s.a : s.da, s.a_ld, s.F);
    const int64_t ctas = (k.items + 7) / 8, most = (int64_t)num_sms() * 32;
    const dim3 grid((unsigned)(ctas < most ? ctas : most));
    const int64_t step = 8 * (int64_t)grid.x;
    k.rows = step / k.R;
    k.runs = step - k.rows * k.R;
    count_launches(1);
#define GO(F) (s.codes ? (vec ? launch_pdl(F<T, A, true, true>, grid, dim3(256), 0, st, k) \
                              : launch_pdl(F<T, A, true, false>, grid, dim3(256), 0, st, k)) \
                       : (vec ? launch_pdl(F<T, A, false, true>, grid, dim3(256), 0, st, k) \
                              : launch_pdl(F<T, A, false, false>, grid, dim3(256), 0, st, k)))
    return fwd ? GO(k_swiglu_fwd) : GO(k_swiglu_bwd);
#undef GO
}

cudaError_t dispatch(const SwigluArgs& a, bool fwd, cudaStream_t st)
{
    Kernel k = {};
    k.s = a;
    k.G = (a.F + GROUP - 1) / GROUP;
    k.R = (k.G + RUN - 1) / RUN;
    k.items = a.n * k.R;
    if (a.type == 0)
        return a.a_type == 0 ? launch<float, float>(k, fwd, st) : launch<float, __nv_bfloat16>(k, fwd, st);
    return a.a_type == 0 ? launch<__nv_bfloat16, float>(k, fwd, st) : launch<__nv_bfloat16, __nv_bfloat16>(k, fwd, st);
}

} // namespace

cudaError_t launch_swiglu_fwd(const SwigluArgs& a, cudaStream_t st) { return dispatch(a, true, st); }
cudaError_t launch_swiglu_bwd(const SwigluArgs& a, cudaStream_t st) { return dispatch(a, false, st); }

} // namespace repro
