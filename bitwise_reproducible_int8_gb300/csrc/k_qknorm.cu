// k_qknorm.cu -- RMS norm of every query and key head and the rotary position
// in one pass, and its backward.
//
//   r = 1 (/) sqrt((S (/) D) (+) eps), y_d = (x_d (x) r) (x) gain_d, then each pair
//   (a, b) turned by the position's angle.  Backward: turn the gradient back, then
//   dx_d = r (x) (u_d (-) (h_d (x) c1)) with h = x r, u = dy gain, c1 = S'(u h) / D.
//
// One read and one write of the heads (and the gradient): bound by HBM, and close
// behind by the instructions issued.  A head lies in the registers of 8, 16 or 32
// lanes, so the norm's order (groups of 4, then the pairwise tree) is a chain in a
// lane, an exchange over lanes and a few sums in a lane; only partners that lie in
// other lanes pass through shared memory.  Two rows a lane share the exchanges and the
// root and division of the norm; the arithmetic is on packed pairs.  16,384 tokens of 16 + 4
// heads of 128, fp32: forward 52.4 us, 6.4 TB/s (0.96 of a copy's); backward with gains 88 us,
// 5.7 TB/s (0.86; 5 us of it the gains' tree).  With 4 elements a lane, a row at a time, these were
// 108 and 213 us: 265 warp instructions a row in the forward, now 101.  bf16 heads, 8,192 tokens:
// 30 us forward, 46 us backward with gains, 37 without (fp32 31 and 49 with gains): as many
// instructions over fewer bytes, 0.63 and 0.54 of a copy's rate.
//
// The gains' gradients are sums over all rows (token, head): a CTA of the backward
// owns one 64-row chunk, leaves dy (x) h of each row in shared memory and adds the
// columns up in row order; k_rowtree.cu combines the chunk rows.
#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace repro {
namespace {

typedef unsigned long long u64;

// How a rotation partner is found.  SPLIT: heads of 64, 128, 256 or 512 elements turned
// whole, by halves: both members of a pair lie in one lane, with one set of cosines and
// sines for them.  INTER: neighbour pairs (or no turn): in the lane.  HALF: by halves,
// R / 2 a multiple of 4: groups of 4 through shared memory.  GENERIC: any other R by
// halves, and rows off 4-element boundaries: single elements through shared memory.
constexpr int INTER = 0, HALF = 1, GENERIC = 2, SPLIT = 3;

// First element of group g of 4 in lane l of a head's LPH: neighbouring lanes hold
// neighbouring groups, so a load of 16 bytes a lane takes whole lines.  (With E
// consecutive elements in a lane each of its loads took half or a quarter of every
// sector: 321 us against 126 for 16 + 4 heads
// of 512, 8,192 tokens.)
template <int LPH> __device__ __forceinline__ int group(int l, int g) { return 4 * (l + g * LPH); }

// two neighbours on a two-element boundary
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p)
{
    const unsigned v = *reinterpret_cast<const unsigned*>(p);
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void store2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b)
{
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

// the head's values in this lane (0 past the width), w elements at a time: 4, or in GENERIC
// 4, 2 or 1, whatever width, strides and start allow
template <typename T, int E, int LPH, int MODE>
__device__ __forceinline__ void load_head(const T* p, int l, int D, int w, float (&x)[E])
{
#pragma unroll
    for (int g = 0; g < E / 4; ++g) {
        const int d = group<LPH>(l, g);
        if (MODE != GENERIC || w == 4) {
            if (MODE == SPLIT || d < D) {
                const float4 v = stream4(p + d);
                x[4 * g] = v.x, x[4 * g + 1] = v.y, x[4 * g + 2] = v.z, x[4 * g + 3] = v.w;
            }
        } else if (w == 2) {
#pragma unroll
            for (int e = 0; e < 4; e += 2)
                if (d + e < D) {
                    const float2 v = load2(p + d + e);
                    x[4 * g + e] = v.x, x[4 * g + e + 1] = v.y;
                }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < D)
                    x[4 * g + e] = to_f32<T>(p[d + e]);
        }
    }
}

template <typename T, int E, int LPH, int MODE>
__device__ __forceinline__ void store_head(T* p, int l, int D, int w, const float (&x)[E])
{
#pragma unroll
    for (int g = 0; g < E / 4; ++g) {
        const int d = group<LPH>(l, g);
        if (MODE != GENERIC || w == 4) {
            if (MODE == SPLIT || d < D)
                store4(p + d, make_float4(x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]));
        } else if (w == 2) {
#pragma unroll
            for (int e = 0; e < 4; e += 2)
                if (d + e < D)
                    store2(p + d + e, x[4 * g + e], x[4 * g + e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < D)
                    p[d + e] = from_f32<T>(x[4 * g + e]);
        }
    }
}

// In-lane part of S of the terms a_e (x) b_e: each group of 4 left to right.  A term
// past the width counts as -0, which leaves every sum as it is.
template <int E, int LPH, int MODE>
__device__ __forceinline__ void lane_sum(const u64 (&a)[E / 2], const u64 (&b)[E / 2], int l, int D, float* out)
{
#pragma unroll
    for (int k = 0; k < E / 4; ++k) {
        float p[4];
        unpack2(fmul2_rn(a[2 * k], b[2 * k]), p[0], p[1]);
        unpack2(fmul2_rn(a[2 * k + 1], b[2 * k + 1]), p[2], p[3]);
        const int d = group<LPH>(l, k);
        if (MODE == GENERIC) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = d + e < D ? p[e] : -0.0f;
        }
        out[k] = fadd_ftz(fadd_ftz(fadd_ftz(p[0], p[1]), p[2]), p[3]);
        if (MODE == INTER || MODE == HALF)
            out[k] = d < D ? out[k] : -0.0f;
    }
}

// The pairwise tree over the groups of U rows at once, G sums a row in a lane: over the
// lanes first, then over a row's sums, as the groups' order has it.  At the first levels
// a lane keeps half of the sums it still has and hands its partner the others, so 4 sums
// take 6 exchanges instead of 20, and every row's sum ends up in lanes of its own:
// lane_of<U>(u) holds row u.
template <int U, int LPH, int G> __device__ __forceinline__ float rows_tree(const float* S, int lane)
{
    constexpr unsigned ALL = 0xffffffffu;
    constexpr int N = U * G;
    float v;
    int s = 1;
    if (N == 4) {
        const bool hi = lane & 1, hi2 = lane & 2;
        const float a = fadd_ftz(hi ? S[2] : S[0], __shfl_xor_sync(ALL, hi ? S[0] : S[2], 1));
        const float b = fadd_ftz(hi ? S[3] : S[1], __shfl_xor_sync(ALL, hi ? S[1] : S[3], 1));
        v = fadd_ftz(hi2 ? b : a, __shfl_xor_sync(ALL, hi2 ? a : b, 2));
        s = 4;
    } else if (N == 2) {
        const bool hi = lane & 1;
        v = fadd_ftz(hi ? S[1] : S[0], __shfl_xor_sync(ALL, hi ? S[0] : S[1], 1));
        s = 2;
    } else {
        v = S[0];
    }
#pragma unroll
    for (; s < LPH; s *= 2)
        v = fadd_ftz(v, __shfl_xor_sync(ALL, v, s));
    static_assert(G == 1 || N == 4, "sum 2 b0 + b1 is in lanes with bits b0 and b1");
    if (G >= 2)
        v = fadd_ftz(v, __shfl_xor_sync(ALL, v, 2));
    if (G == 4)
        v = fadd_ftz(v, __shfl_xor_sync(ALL, v, 1));
    return v;
}

template <int U> __device__ __forceinline__ int lane_of(int u)
{
    return U == 4 ? (u >> 1) | ((u & 1) << 1) : u;
}

// S (/) D; by an exact product where D is a power of two
__device__ __forceinline__ float over_width(float S, float width, float inv)
{
    return inv != 0.0f ? fmul_flush(S, inv) : flush(__fdiv_rn(S, width));
}

__device__ __forceinline__ float rnorm(float S, float width, float inv, float eps)
{
    return flush(__fdiv_rn(1.0f, flush(__fsqrt_rn(fadd_ftz(over_width(S, width, inv), eps)))));
}

// the turn of a position for this lane's elements: out_e = v_e c_e + w_e s_e, w_e the
// other member of the pair, s_e with its sign (BACK: the turn undone).  SPLIT: of the
// lower half's elements; the upper half's s is the negative.
template <int E, int LPH, int MODE, bool BACK>
__device__ __forceinline__ void load_turn(u64 (&c)[E / 2], u64 (&s)[E / 2], const float* __restrict__ cs, int l,
                                          int R, bool inter)
{
    const int half = R >> 1;
    const u64 z = pack2(-0.0f, -0.0f);
#pragma unroll
    for (int g = 0; g < (MODE == SPLIT ? E / 8 : E / 4); ++g) {
        const int d = group<LPH>(l, g);
        if (MODE == SPLIT || (MODE == HALF && d < R)) {
            const bool low = MODE == SPLIT || d < half, minus = low != BACK;
            const int j = low ? d : d - half;
            const float4 a = __ldg(reinterpret_cast<const float4*>(cs + j));
            const float4 b = __ldg(reinterpret_cast<const float4*>(cs + half + j));
            c[2 * g] = fadd2_ftz(pack2(a.x, a.y), z);
            c[2 * g + 1] = fadd2_ftz(pack2(a.z, a.w), z);
            s[2 * g] = fadd2_ftz(minus ? pack2(-b.x, -b.y) : pack2(b.x, b.y), z);
            s[2 * g + 1] = fadd2_ftz(minus ? pack2(-b.z, -b.w) : pack2(b.z, b.w), z);
            if (MODE == SPLIT) {
                s[E / 4 + 2 * g] = fmul2_rn(s[2 * g], pack2(-1.0f, -1.0f));
                s[E / 4 + 2 * g + 1] = fmul2_rn(s[2 * g + 1], pack2(-1.0f, -1.0f));
            }
        }
        if (MODE == INTER) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (d + 2 * i < R) {
                    const float a = __ldg(cs + d / 2 + i), b = __ldg(cs + half + d / 2 + i);
                    c[2 * g + i] = fadd2_ftz(pack2(a, a), z);
                    s[2 * g + i] = fadd2_ftz(BACK ? pack2(b, -b) : pack2(-b, b), z);
                }
        }
        if (MODE == GENERIC) {
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                float cc[2] = {0.0f, 0.0f}, ss[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = d + e + i;
                    if (k < R) {
                        const bool low = inter ? i == 0 : k < half;
                        const int j = inter ? k >> 1 : (low ? k : k - half);
                        cc[i] = __ldg(cs + j);
                        ss[i] = __ldg(cs + half + j);
                        ss[i] = low != BACK ? -ss[i] : ss[i];
                    }
                }
                c[2 * g + e / 2] = fadd2_ftz(pack2(cc[0], cc[1]), z);
                s[2 * g + e / 2] = fadd2_ftz(pack2(ss[0], ss[1]), z);
            }
        }
    }
}

// v turned in place; elements from R on are left alone
template <int E, int LPH, int MODE>
__device__ __forceinline__ void turn(u64 (&v)[E / 2], const u64 (&c)[E / 2], const u64 (&s)[E / 2], int l, int D,
                                     int R, bool inter, float* row)
{
    if (MODE == SPLIT) {   // the first half of the lane's pairs is of the lower half
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
            const u64 a = v[i], b = v[E / 4 + i];
            v[i] = fadd2_ftz(fmul2_rn(a, c[i]), fmul2_rn(b, s[i]));
            v[E / 4 + i] = fadd2_ftz(fmul2_rn(b, c[i]), fmul2_rn(a, s[E / 4 + i]));
        }
        return;
    }
    const int half = R >> 1;
    float x[E], y[E];
#pragma unroll
    for (int i = 0; i < E; i += 2)
        unpack2(v[i / 2], x[i], x[i + 1]);
    if (MODE == INTER) {
#pragma unroll
        for (int i = 0; i < E; ++i)
            y[i] = x[i ^ 1];
    } else if (MODE == HALF) {
        __syncwarp();
#pragma unroll
        for (int g = 0; g < E / 4; ++g) {
            const int d = group<LPH>(l, g);
            if (d < R)
                *reinterpret_cast<float4*>(row + d) = make_float4(x[4 * g], x[4 * g + 1], x[4 * g + 2], x[4 * g + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int g = 0; g < E / 4; ++g) {
            const int d = group<LPH>(l, g);
            float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (d < R)
                w = *reinterpret_cast<const float4*>(row + (d < half ? d + half : d - half));
            y[4 * g] = w.x, y[4 * g + 1] = w.y, y[4 * g + 2] = w.z, y[4 * g + 3] = w.w;
        }
    } else {   // element d at (d mod 4) E LPH / 4 + d / 4: lanes side by side at any distance
        constexpr unsigned Q = E * LPH / 4;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (group<LPH>(l, i / 4) + i % 4 < R)
                row[i % 4 * Q + l + i / 4 * LPH] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int d = group<LPH>(l, i / 4) + i % 4;
            const unsigned o = inter ? d ^ 1 : d < half ? d + half : d - half;
            y[i] = d < R ? row[o % 4 * Q + o / 4] : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const int d = group<LPH>(l, i / 2) + i % 2 * 2;
        const u64 t = fadd2_ftz(fmul2_rn(v[i], c[i]), fmul2_rn(pack2(y[2 * i], y[2 * i + 1]), s[i]));
        v[i] = d < R ? t : v[i];   // R is even
    }
}

// the table's row for a token's position; its first row and ok = false (and the
// error word) when there is none
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

// Rows (token, head) of one tensor, U consecutive ones per LPH lanes: where their
// data lies, and which begin another token than the row before.
template <int U> struct Rows {
    unsigned tok[U];
    bool live[U], turned[U];   // turned: the position differs from the row before
    int64_t at[U];             // offset of the row in the strided tensor

    __device__ __forceinline__ void locate(unsigned row, unsigned total, unsigned H, int64_t ld, int64_t hs)
    {
        unsigned t = row / H, h = row - t * H;
        int64_t o = (int64_t)t * ld + (int64_t)h * hs;
        const int64_t wrap = ld - (int64_t)(H - 1) * hs;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            tok[u] = t;
            live[u] = row + u < total;
            turned[u] = u == 0 || h == 0;
            at[u] = o;
            const bool last = ++h == H;
            h = last ? 0 : h;
            t += last;
            o += last ? wrap : hs;
        }
    }
};

// a row's values from memory as packed pairs (0 for rows past the end)
template <typename T, int E, int LPH, int MODE>
__device__ __forceinline__ void load_row(const T* p, bool live, int l, int D, int w, u64 (&v)[E / 2])
{
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        x[e] = 0.0f;
    if (live)
        load_head<T, E, LPH, MODE>(p, l, D, w, x);
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
        v[i] = pack2(x[2 * i], x[2 * i + 1]);
}

template <typename T, int E, int LPH, int MODE>
__device__ __forceinline__ void store_row(T* p, int l, int D, int w, const u64 (&v)[E / 2])
{
    float x[E];
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
        unpack2(v[i], x[2 * i], x[2 * i + 1]);
    store_head<T, E, LPH, MODE>(p, l, D, w, x);
}

template <int N> __device__ __forceinline__ void mul_flush(u64 (&v)[N], const u64 (&w)[N])
{
    const u64 z = pack2(-0.0f, -0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = fadd2_ftz(fmul2_rn(v[i], w[i]), z);
}

template <int N> __device__ __forceinline__ void mul_flush(u64 (&v)[N], float w)
{
    const u64 z = pack2(-0.0f, -0.0f), ww = pack2(w, w);
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = fadd2_ftz(fmul2_rn(v[i], ww), z);
}

template <int N> __device__ __forceinline__ void flush_row(u64 (&v)[N])
{
    const u64 z = pack2(-0.0f, -0.0f);
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = fadd2_ftz(v[i], z);
}

// this lane's gains, flushed
template <int E, int LPH> __device__ __forceinline__ void load_gain(const float* gain, int l, int D, u64 (&g)[E / 2])
{
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int d = group<LPH>(l, e / 4) + e % 4;
        x[e] = gain && d < D ? __ldg(gain + d) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
        g[i] = pack2(x[2 * i], x[2 * i + 1]);
    flush_row(g);
}

__host__ __device__ constexpr int fwd_rows(int E) { return E == 4 ? 4 : E == 8 ? 2 : 1; }

template <typename T, int E, int LPH, int MODE>
__global__ void __launch_bounds__(256)
k_qk_fwd(const __grid_constant__ QkArgs a, unsigned blocks_q)
{
    constexpr int HPW = 32 / LPH;   // heads a warp holds
    constexpr int U = fwd_rows(E);
    constexpr int G = E / 4;        // groups of 4 a lane holds of a row
    constexpr int ROW = MODE == HALF || MODE == GENERIC ? E * LPH + (HPW > 1 ? LPH : 0) : 0;   // of a head, shared
    __shared__ __align__(16) float rows[ROW ? 8 * HPW * ROW : 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = (int)a.D, R = (int)a.R, l = lane % LPH, sub = lane / LPH;
    float* srow = rows + (warp * HPW + sub) * ROW;
    const int dense = D % 4 == 0 ? 4 : D % 2 == 0 ? 2 : 1;   // of rows without gaps
    const bool is_q = blockIdx.x < blocks_q;
    const QkTensor& t = is_q ? a.t[0] : a.t[1];
    const unsigned block = is_q ? blockIdx.x : blockIdx.x - blocks_q;
    const unsigned H = (unsigned)t.H, total = (unsigned)a.n * H;
    const unsigned row0 = ((block * 8 + warp) * HPW + sub) * U;
    Rows<U> at;
    at.locate(row0, total, H, t.ld, t.hs);
    u64 x[U][E / 2];
#pragma unroll
    for (int u = 0; u < U; ++u)
        load_row<T, E, LPH, MODE>(static_cast<const T*>(t.x) + at.at[u], at.live[u], l, D, a.w, x[u]);
    if (__ballot_sync(0xffffffffu, at.live[0]) == 0)
        return;
    u64 c[E / 2] = {}, s[E / 2] = {}, g[E / 2];
    bool ok;
    const float* cs = rope_row(a, at.live[0] ? at.tok[0] : 0u, at.live[0] && l == 0, ok);
    load_turn<E, LPH, MODE, false>(c, s, cs, l, R, a.interleaved);
    load_gain<E, LPH>(t.gain, l, D, g);
    float S[G * U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        flush_row(x[u]);
        lane_sum<E, LPH, MODE>(x[u], x[u], l, D, S + G * u);
    }
    const float r = rnorm(rows_tree<U, LPH, G>(S, lane), (float)D, a.inv, flush(a.eps));
#pragma unroll
    for (int u = 0; u < U; ++u) {
        mul_flush(x[u], __shfl_sync(0xffffffffu, r, lane_of<U>(u), LPH));
        if (t.gain)
            mul_flush(x[u], g);
        if (u > 0 && at.turned[u] && at.live[u]) {
            cs = rope_row(a, at.tok[u], l == 0, ok);
            load_turn<E, LPH, MODE, false>(c, s, cs, l, R, a.interleaved);
        }
        turn<E, LPH, MODE>(x[u], c, s, l, D, R, a.interleaved, srow);
        if (!ok) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i)
                x[u][i] = 0ull;
        }
        if (at.live[u]) {
            float* o = t.out + (int64_t)(row0 + u) * D;
            store_row<float, E, LPH, MODE>(o, l, D, dense, x[u]);
        }
    }
}

constexpr int CHUNK = 64;   // rows of a chunk of the gains' canonical sums
__host__ __device__ constexpr int bwd_rows(int E) { return E == 16 ? 1 : 2; }
// warps of a CTA: the terms of heads past 256 leave room for one CTA or two an SM (16 + 4
// heads of 512, 8,192 tokens: 262 us with 8 warps, 192 with 16)
__host__ __device__ constexpr int bwd_warps(int E) { return E == 16 ? 16 : 8; }

template <typename T, int E, int LPH, int MODE>
__global__ void __launch_bounds__(32 * bwd_warps(E), E == 16 ? 1 : 3)
k_qk_bwd(const __grid_constant__ QkArgs a, unsigned chunks_q, float* __restrict__ parts, int64_t pitch)
{
    constexpr int HPW = 32 / LPH;
    constexpr int U = bwd_rows(E), W = bwd_warps(E);
    constexpr int G = E / 4;        // groups of 4 a lane holds of a row
    constexpr int PER = CHUNK / (W * HPW);   // consecutive rows of the chunk per LPH lanes
    constexpr int ROW = MODE == HALF || MODE == GENERIC ? E * LPH + (HPW > 1 ? LPH : 0) : 0;   // of a head, shared
    __shared__ __align__(16) float rows[ROW ? W * HPW * ROW : 4];
    extern __shared__ float terms[];   // [CHUNK][D] with a gain
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = (int)a.D, R = (int)a.R, l = lane % LPH, sub = lane / LPH;
    float* srow = rows + (warp * HPW + sub) * ROW;
    const int dense = D % 4 == 0 ? 4 : D % 2 == 0 ? 2 : 1;   // of rows without gaps
    const bool is_q = blockIdx.x < chunks_q;
    const QkTensor& t = is_q ? a.t[0] : a.t[1];
    const unsigned chunk = is_q ? blockIdx.x : blockIdx.x - chunks_q;
    const unsigned H = (unsigned)t.H, total = (unsigned)a.n * H, first = chunk * CHUNK;
    const float width = (float)D, eps = flush(a.eps);
    const bool gain = t.gain != nullptr;
    pdl_trigger();   // the gains' tree may be launched; it waits for this grid
    u64 g[E / 2];
    load_gain<E, LPH>(t.gain, l, D, g);
#pragma unroll 1
    for (int k0 = 0; k0 < PER; k0 += U) {
        const unsigned row0 = first + (unsigned)((warp * HPW + sub) * PER + k0);
        Rows<U> at;
        at.locate(row0, total, H, t.ld, t.hs);
        if (__ballot_sync(0xffffffffu, at.live[0]) == 0)
            break;
        u64 x[U][E / 2], dy[U][E / 2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            load_row<T, E, LPH, MODE>(static_cast<const T*>(t.x) + at.at[u], at.live[u], l, D, a.w, x[u]);
            const float* p = t.dout + (int64_t)(row0 + u) * D;
            load_row<float, E, LPH, MODE>(p, at.live[u], l, D, dense, dy[u]);
        }
        u64 c[E / 2] = {}, s[E / 2] = {};
        bool ok[U];
        const float* cs = rope_row(a, at.live[0] ? at.tok[0] : 0u, at.live[0] && l == 0, ok[0]);
        load_turn<E, LPH, MODE, true>(c, s, cs, l, R, a.interleaved);
        float S[G * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            flush_row(x[u]);
            lane_sum<E, LPH, MODE>(x[u], x[u], l, D, S + G * u);
        }
        const float r = rnorm(rows_tree<U, LPH, G>(S, lane), width, a.inv, eps);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u > 0) {
                ok[u] = ok[u - 1];
                if (at.turned[u] && at.live[u]) {
                    cs = rope_row(a, at.tok[u], l == 0, ok[u]);
                    load_turn<E, LPH, MODE, true>(c, s, cs, l, R, a.interleaved);
                }
            }
            flush_row(dy[u]);
            turn<E, LPH, MODE>(dy[u], c, s, l, D, R, a.interleaved, srow);
            mul_flush(x[u], __shfl_sync(0xffffffffu, r, lane_of<U>(u), LPH));   // h
            if (gain) {
                u64 p[E / 2];
#pragma unroll
                for (int i = 0; i < E / 2; ++i)
                    p[i] = dy[u][i];
                mul_flush(p, x[u]);
                if (!ok[u]) {
#pragma unroll
                    for (int i = 0; i < E / 2; ++i)
                        p[i] = 0ull;
                }
                if (at.live[u]) {
                    float* o = terms + (row0 + u - first) * D;
                    store_row<float, E, LPH, MODE>(o, l, D, dense, p);
                }
                mul_flush(dy[u], g);
            }
            lane_sum<E, LPH, MODE>(dy[u], x[u], l, D, S + G * u);
        }
        const float c1 = over_width(rows_tree<U, LPH, G>(S, lane), width, a.inv);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float ru = __shfl_sync(0xffffffffu, r, lane_of<U>(u), LPH);
            const float cu = __shfl_sync(0xffffffffu, c1, lane_of<U>(u), LPH);
            const u64 nc = pack2(-cu, -cu);
#pragma unroll
            for (int i = 0; i < E / 2; ++i)
                x[u][i] = fadd2_ftz(dy[u][i], fmul2_rn(x[u][i], nc));
            mul_flush(x[u], ru);
            if (!ok[u]) {
#pragma unroll
                for (int i = 0; i < E / 2; ++i)
                    x[u][i] = 0ull;
            }
        }
        Rows<U> to;
        to.locate(row0, total, H, t.dx_ld, t.dx_hs);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (to.live[u])
                store_row<T, E, LPH, MODE>(static_cast<T*>(t.dx) + to.at[u], l, D, a.w, x[u]);
    }
    if (gain) {
        __syncthreads();
        const int L = total - first < CHUNK ? (int)(total - first) : CHUNK;
        for (int d = threadIdx.x; d < D; d += 32 * W) {
            float s = terms[d];
#pragma unroll 8
            for (int k = 1; k < L; ++k)
                s = fadd_ftz(s, terms[k * D + d]);
            parts[(int64_t)blockIdx.x * pitch + d] = s;
        }
    }
}

unsigned chunks_of(int64_t rows) { return (unsigned)((rows + CHUNK - 1) / CHUNK); }

// elements that may be loaded and stored at a time: 4, 2 or 1
template <typename T> int width_of(const QkArgs& a, bool back)
{
    auto whole = [&](int64_t w) {
        bool ok = a.D % w == 0;
        for (const QkTensor& t : a.t)
            if (t.H > 0) {
                ok = ok && reinterpret_cast<uintptr_t>(t.x) % (w * sizeof(T)) == 0 && t.ld % w == 0 && t.hs % w == 0;
                if (back)
                    ok = ok && reinterpret_cast<uintptr_t>(t.dx) % (w * sizeof(T)) == 0 && t.dx_ld % w == 0 &&
                         t.dx_hs % w == 0;
            }
        return ok;
    };
    return whole(4) ? 4 : whole(2) ? 2 : 1;
}

// how partners are found
int mode_of(const QkArgs& a, int E, int LPH)
{
    if (a.w != 4)
        return GENERIC;
    if (a.interleaved || a.R == 0)
        return INTER;
    if (E >= 8 && a.R == a.D && a.D == E * LPH)
        return SPLIT;
    return a.R % 8 == 0 ? HALF : GENERIC;
}

// calls f(E, LPH) as compile-time constants for the head width
template <typename F> cudaError_t by_width(int64_t D, F f)
{
    if (D <= 32)
        return f(std::integral_constant<int, 4>(), std::integral_constant<int, 8>());
    if (D <= 64)
        return f(std::integral_constant<int, 8>(), std::integral_constant<int, 8>());
    if (D <= 128)
        return f(std::integral_constant<int, 8>(), std::integral_constant<int, 16>());
    if (D <= 256)
        return f(std::integral_constant<int, 8>(), std::integral_constant<int, 32>());
    return f(std::integral_constant<int, 16>(), std::integral_constant<int, 32>());
}

template <typename T> cudaError_t fwd_typed(QkArgs a, cudaStream_t st)
{
    a.w = width_of<T>(a, false);
    return by_width(a.D, [&](auto e, auto l) {
        constexpr int E = decltype(e)::value, LPH = decltype(l)::value;
        constexpr int per = 8 * (32 / LPH) * fwd_rows(E);
        const unsigned bq = (unsigned)((a.n * a.t[0].H + per - 1) / per);
        const unsigned grid = bq + (unsigned)((a.n * a.t[1].H + per - 1) / per);
        const int m = mode_of(a, E, LPH);
        if (m == INTER)
            k_qk_fwd<T, E, LPH, INTER><<<grid, 256, 0, st>>>(a, bq);
        else if (m == HALF)
            k_qk_fwd<T, E, LPH, HALF><<<grid, 256, 0, st>>>(a, bq);
        else if (m == GENERIC)
            k_qk_fwd<T, E, LPH, GENERIC><<<grid, 256, 0, st>>>(a, bq);
        else if constexpr (E >= 8)
            k_qk_fwd<T, E, LPH, SPLIT><<<grid, 256, 0, st>>>(a, bq);
        count_launches(1);
        return cudaGetLastError();
    });
}

template <typename T> cudaError_t bwd_typed(QkArgs a, float* parts, int64_t pitch, cudaStream_t st)
{
    a.w = width_of<T>(a, true);
    return by_width(a.D, [&](auto e, auto l) {
        constexpr int E = decltype(e)::value, LPH = decltype(l)::value;
        const unsigned cq = chunks_of(a.n * a.t[0].H), ck = chunks_of(a.n * a.t[1].H);
        const bool gain = a.t[0].gain || a.t[1].gain;
        const size_t smem = gain ? (size_t)CHUNK * a.D * 4 : 0;
        const int m = mode_of(a, E, LPH);
        // the limit is the variant's widest head's, so that calls of other widths in other host
        // threads set the same
        constexpr int most = CHUNK * E * LPH * 4;
        auto go = [&](auto kernel) {
            if (gain && most > 32 * 1024) {
                const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
                if (r != cudaSuccess)
                    return r;
            }
            kernel<<<cq + ck, 32 * bwd_warps(E), smem, st>>>(a, cq, parts, pitch);
            count_launches(1);
            return cudaGetLastError();
        };
        if (m == INTER)
            return go(k_qk_bwd<T, E, LPH, INTER>);
        if (m == HALF)
            return go(k_qk_bwd<T, E, LPH, HALF>);
        if constexpr (E >= 8)
            if (m == SPLIT)
                return go(k_qk_bwd<T, E, LPH, SPLIT>);
        return go(k_qk_bwd<T, E, LPH, GENERIC>);
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
    RowTree r = {};
    for (int x = 0; x < 2; ++x) {
        const QkTensor& t = a.t[x];
        if (!t.gain || t.H == 0)
            continue;
        r.parts[r.jobs] = parts + (x == 1 ? (int64_t)chunks_of(a.n * a.t[0].H) * pitch : 0);
        r.count[r.jobs] = chunks_of(a.n * t.H);
        r.out[r.jobs++] = t.dgain;
    }
    if (e != cudaSuccess || r.jobs == 0)
        return e;
    r.pitch = pitch;
    r.D = a.D;
    r.out_ld = a.D;
    r.scale = 1.0f;
    r.accumulate = a.accumulate;
    return launch_row_tree(r, num_sms(), st);
}

} // namespace repro
