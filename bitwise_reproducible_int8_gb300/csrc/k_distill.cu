// k_distill.cu -- loss of a student's logits against a teacher's top logits (with
// the label's cross entropy and the log-partition penalty), and the logits'
// gradient.
//
//   u = z / tau, q = softmax(u), p = the teacher's weights over its K entries
//   loss = w_kd tau^2 sum p_k (ln p_k - ln q_idx_k) + w_ce (lse(z) - z_label) + w_z lse(z)^2
//   dz   = g (w_kd tau (P q - p) + (w_ce + 2 w_z lse(z)) softmax(z) - w_ce [label])
//
// The forward reads the logits once, the backward reads them and writes the
// gradient: bytes bound both at binary32, and the e^x of every logit (about 20
// unfused operations) comes close to the bytes' time there and above it for bf16.
// So e^x is 2^t with a plain rounded product t = x log2 e (the argument is a
// difference from the maximum: its large values weigh nothing) and a degree-6
// polynomial, on packed pairs.
//
// Order: the row is cut into blocks of 1024 logits; a warp holds a block in
// registers (32 per lane), so the block's exact maximum and then its sum come
// from one read, with no running rescale.  128 chains per block and the pairwise
// tree over them: chain j mod 128 puts a chain's terms into one lane whether the
// lane loads single elements (lane, lane + 32, ..: rows of any alignment) or four
// neighbours.  k_distill_rows joins the blocks' (maximum, sum) pairs per row, so
// few rows over a long vocabulary still spread over the card.
#include <math_constants.h>

#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace repro {
namespace {

typedef unsigned long long u64;

constexpr int BLK = 1024;          // logits per block
constexpr int PER = BLK / 32;      // per lane
constexpr int STATS = 8;
constexpr float LOG2E = 0x1.715476p+0f;   // RN(1 / ln 2)

// which sums a call needs
constexpr int ONE = 0;      // tau = 1: one sum serves all terms
constexpr int SOFT = 1;     // tau != 1, only the softened softmax
constexpr int BOTH = 2;     // tau != 1 and the softmax of z itself

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ u64 dup2(float v) { return pack2(v, v); }

// e^x of a packed pair, x <= 0 (a NaN stays a NaN): t = x (x) log2 e, k = rint(t) by
// adding and subtracting 1.5 * 2^23, f = t (-) k, the degree-6 minimax polynomial
// of 2^f on [-1/2, 1/2] (relative error 2.6e-9, constant term 1; by the exchange
// algorithm of Remez, rounded to binary32) in Horner form, times 2^k; 0 below
// t = -125, so nothing here is subnormal
__device__ __forceinline__ u64 exp_neg2(u64 x)
{
    const u64 z = dup2(-0.0f), big = dup2(0x1.8p23f), nbig = dup2(-0x1.8p23f);
    const u64 t = fadd2_ftz(fmul2_rn(x, dup2(LOG2E)), z);
    const u64 m = fadd2_ftz(t, big);
    const u64 k = fadd2_ftz(m, nbig);
    float k0, k1, m0, m1, t0, t1;
    unpack2(k, k0, k1);
    const u64 f = fadd2_ftz(t, pack2(-k0, -k1));
    u64 p = dup2(0x1.470b5p-13f);
    p = fadd2_ftz(fmul2_rn(p, f), dup2(0x1.5f7278p-10f));
    p = fadd2_ftz(fmul2_rn(p, f), dup2(0x1.3b270ep-7f));
    p = fadd2_ftz(fmul2_rn(p, f), dup2(0x1.c6ae72p-5f));
    p = fadd2_ftz(fmul2_rn(p, f), dup2(0x1.ebfbe2p-3f));
    p = fadd2_ftz(fmul2_rn(p, f), dup2(0x1.62e432p-1f));
    p = fadd2_ftz(fmul2_rn(p, f), dup2(1.0f));
    unpack2(m, m0, m1);
    unpack2(t, t0, t1);
    // the low bits of 1.5 * 2^23 + k are k: shifted into the exponent of 1.0
    const u64 s = pack2(__int_as_float((__float_as_int(m0) << 23) + 0x3f800000),
                        __int_as_float((__float_as_int(m1) << 23) + 0x3f800000));
    float r0, r1;
    unpack2(fmul2_rn(p, s), r0, r1);
    return pack2(t0 < -125.0f ? 0.0f : r0, t1 < -125.0f ? 0.0f : r1);
}

__device__ __forceinline__ float exp_neg(float x)
{
    float a, b;
    unpack2(exp_neg2(pack2(x, -0.0f)), a, b);
    return a;
}

// ln of a positive finite binary32 value, in binary64: x = m 2^e, m in
// [sqrt(1/2), sqrt(2)), ln m = 2 atanh(s), s = (m - 1) / (m + 1), by the power
// series to s^21; NaN for anything else.  The compiler's contraction is off.
__device__ double ln_d(float x)
{
    if (!(x > 0.0f) || x > 3.402823466e38f)
        return CUDART_NAN;
    int e;
    double m = frexp((double)x, &e);
    if (m < 0.70710678118654752440) {
        m *= 2.0;
        e -= 1;
    }
    const double s = (m - 1.0) / (m + 1.0), w = s * s;
    double p = 1.0 / 21.0;
#pragma unroll
    for (int k = 19; k >= 1; k -= 2)
        p = p * w + 1.0 / (double)k;
    return (double)e * 0.69314718055994530942 + (2.0 * s) * p;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int s = 1; s < 32; s *= 2)
        v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

__device__ __forceinline__ float warp_tree(float v)
{
#pragma unroll
    for (int s = 1; s < 32; s *= 2)
        v = fadd_ftz(v, __shfl_xor_sync(0xffffffffu, v, s));
    return v;
}

__device__ __forceinline__ double warp_tree(double v)
{
#pragma unroll
    for (int s = 1; s < 32; s *= 2)
        v = v + __shfl_xor_sync(0xffffffffu, v, s);
    return v;
}

// Element of the block in slot i of this lane.  Rows on 4-element boundaries:
// four neighbours per load; else single elements.  Either way slots i, i + 4, ..
// of a lane are one chain (element mod 128), ascending.
template <bool VEC> __device__ __forceinline__ int element(int i, int lane)
{
    return VEC ? (i >> 2) * 128 + 4 * lane + (i & 3) : 32 * i + lane;
}

// the lane's logits of the block at p, `len` of them in the block; -infinity past it
template <typename T, bool VEC>
__device__ __forceinline__ void load_block(const T* p, int len, int lane, float (&x)[PER])
{
    if (VEC) {
        // rows on 4-element boundaries may still end inside a group
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const int e = element<true>(i, lane);
            if (e + 4 <= len) {
                const float4 v = load4(p + e);
                x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    x[i + c] = e + c < len ? to_f32<T>(p[e + c]) : -CUDART_INF_F;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = element<false>(i, lane);
            x[i] = e < len ? to_f32<T>(p[e]) : -CUDART_INF_F;
        }
    }
}

// sum over the block of e(x_i (x) it (-) Mu): four chains per lane, then the tree
// over the 128 chains in their order
template <bool VEC, bool SCALE>
__device__ __forceinline__ float block_sum(const float (&x)[PER], float it, float Mu)
{
    const u64 nm = dup2(-Mu), sc = dup2(it), z = dup2(-0.0f);
    u64 a = dup2(0.0f), b = dup2(0.0f);
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
        u64 v = pack2(x[i], x[i + 1]), w = pack2(x[i + 2], x[i + 3]);
        v = SCALE ? fmul2_rn(fadd2_ftz(v, z), sc) : v;
        w = SCALE ? fmul2_rn(fadd2_ftz(w, z), sc) : w;
        a = fadd2_ftz(a, exp_neg2(fadd2_ftz(v, nm)));
        b = fadd2_ftz(b, exp_neg2(fadd2_ftz(w, nm)));
    }
    float s0, s1, s2, s3;
    unpack2(a, s0, s1);
    unpack2(b, s2, s3);
    if (VEC)   // chain 4 lane + c: neighbours first
        return warp_tree(fadd_ftz(fadd_ftz(s0, s1), fadd_ftz(s2, s3)));
    // chain 32 c + lane: lanes first
    return fadd_ftz(fadd_ftz(warp_tree(s0), warp_tree(s1)), fadd_ftz(warp_tree(s2), warp_tree(s3)));
}

template <typename T, int SUMS, bool VEC>
__global__ void __launch_bounds__(256)
k_distill_blocks(const T* __restrict__ z, int64_t z_ld, int64_t V, int64_t nblk, int64_t items, float it,
                 float2* __restrict__ ms, float* __restrict__ s1)
{
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= items)
        return;
    const int64_t row = item / nblk, blk = item - row * nblk;
    const int len = (int)(V - blk * BLK < BLK ? V - blk * BLK : BLK);
    float x[PER];
    load_block<T, VEC>(z + row * z_ld + blk * BLK, len, lane, x);
    float m = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        m = max_nan(m, x[i]);
    m = warp_max(m);
    m = flush(m);
    m = m == 0.0f ? 0.0f : m;
    const bool none = m == -CUDART_INF_F;
    float s = 0.0f, o = 0.0f;
    if (!none) {
        s = block_sum<VEC, SUMS != ONE>(x, it, fmul_flush(m, it));
        if (SUMS == BOTH)
            o = block_sum<VEC, false>(x, 1.0f, m);
    }
    if (lane == 0) {
        ms[item] = make_float2(m, s);
        if (SUMS == BOTH)
            s1[item] = o;
    }
}

struct RowArgs {
    const void* t_idx;
    const void* t_val;
    int t_type;
    const void* labels;
    int index_bytes;
    int64_t n, V, K, nblk;
    float it, tau, w_kd, w_ce, w_z;
    bool logprobs;
    const float2* ms;
    const float* s1;
    float* loss;
    float* stats;
    int* err;
};

// one warp per row: joins the blocks, forms the teacher's weights and the loss
template <typename T, int SUMS>
__global__ void __launch_bounds__(128)
k_distill_rows(const T* __restrict__ z, int64_t z_ld, const RowArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= a.n)
        return;
    const float2* ms = a.ms + row * a.nblk;
    float M = -CUDART_INF_F;
    for (int64_t b = lane; b < a.nblk; b += 32)
        M = max_nan(M, ms[b].x);
    M = warp_max(M);
    M = M == 0.0f ? 0.0f : M;
    const float Mu = fmul_flush(M, a.it);
    const bool none = M == -CUDART_INF_F;
    float l = 0.0f, l1 = 0.0f;
    if (!none) {
        for (int64_t b = lane; b < a.nblk; b += 32) {
            const float2 v = ms[b];
            l = fadd_ftz(l, fmul_rn(v.y, exp_neg(fadd_ftz(fmul_rn(v.x, a.it), -Mu))));
            if (SUMS == BOTH)
                l1 = fadd_ftz(l1, fmul_rn(a.s1[row * a.nblk + b], exp_neg(fadd_ftz(v.x, -M))));
        }
        l = warp_tree(l);
        l1 = SUMS == BOTH ? warp_tree(l1) : l;
    }
    if (SUMS == SOFT)
        l1 = 0.0f;
    // the teacher's weights
    float* st = a.stats + row * (STATS + a.K);
    float* p = st + STATS;
    auto value = [&](int64_t k, int64_t& j) {   // a_k, and the column or -1
        j = load_index(a.t_idx, a.index_bytes, row * a.K + k);
        if (j >= a.V)
            atomicOr(a.err, kErrIndexBit);
        if (j < 0 || j >= a.V) {
            j = -1;
            return -CUDART_INF_F;
        }
        const float t = a.t_type == 0 ? static_cast<const float*>(a.t_val)[row * a.K + k]
                                      : __bfloat162float(static_cast<const __nv_bfloat16*>(a.t_val)[row * a.K + k]);
        return a.logprobs ? flush(t) : fmul_flush(flush(t), a.it);
    };
    float mt = -CUDART_INF_F;
    int64_t j;
    if (a.logprobs) {
        mt = 0.0f;
    } else {
        for (int64_t k = lane; k < a.K; k += 32)
            mt = max_nan(mt, value(k, j));
        mt = warp_max(mt);
        mt = mt == 0.0f ? 0.0f : mt;
    }
    float lt = 0.0f, P = 0.0f;
    if (mt == -CUDART_INF_F) {
        for (int64_t k = lane; k < a.K; k += 32)
            p[k] = 0.0f;
    } else {
        for (int64_t k = lane; k < a.K; k += 32) {
            const float e = exp_neg(fadd_ftz(value(k, j), -mt));
            lt = fadd_ftz(lt, e);
            p[k] = e;
        }
        lt = warp_tree(lt);
        if (a.logprobs) {
            P = lt;
            lt = 1.0f;
        } else {
            P = lt == lt ? 1.0f : lt;
        }
    }
    const double lse_t = none ? 0.0 : (double)Mu + ln_d(l);
    const double lse1 = none || SUMS == SOFT ? 0.0 : (double)M + ln_d(l1);
    double v = 0.0;
    if (mt != -CUDART_INF_F) {
        const double cst = none ? 0.0 : lse_t - ((double)mt + ln_d(lt));
        double sum = 0.0;
        for (int64_t k = lane; k < a.K; k += 32) {
            float w = p[k];
            if (!a.logprobs) {
                w = flush(__fdiv_rn(w, lt));
                p[k] = w;
            }
            if (w != 0.0f && !none && a.w_kd != 0.0f) {
                const float ak = value(k, j);
                const float u = fmul_flush(flush(to_f32<T>(z[row * z_ld + j])), a.it);
                sum = sum + (double)w * (((double)ak - (double)u) + cst);
            }
        }
        if (!none && a.w_kd != 0.0f)
            v = ((double)a.w_kd * ((double)a.tau * (double)a.tau)) * warp_tree(sum);
    }
    if (lane == 0) {
        if (a.w_ce != 0.0f) {
            const int64_t lab = load_index(a.labels, a.index_bytes, row);
            if (lab >= a.V)
                atomicOr(a.err, kErrIndexBit);
            else if (lab >= 0 && !none)
                v = v + (double)a.w_ce * (lse1 - (double)flush(to_f32<T>(z[row * z_ld + lab])));
        }
        if (a.w_z != 0.0f && !none)
            v = v + (double)a.w_z * (lse1 * lse1);
        a.loss[row] = flush(__double2float_rn(v));
        st[0] = M;
        st[1] = l;
        st[2] = none ? M : flush(__double2float_rn(lse_t));
        st[3] = l1;
        st[4] = SUMS == SOFT ? 0.0f : none ? M : flush(__double2float_rn(lse1));
        st[5] = mt;
        st[6] = lt;
        st[7] = P;
    }
}

struct BwdArgs {
    const void* t_idx;
    const void* labels;
    int index_bytes;
    int64_t V, K, nblk, items;
    float it, tau, w_kd, w_ce, w_z;
    const float* stats;
    const float* g;
    int64_t g_stride;
};

// v at block element e, if this lane has it: `slot` and `own` are uniform
__device__ __forceinline__ void subtract_at(float (&v)[PER], int slot, bool mine, float c)
{
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (i == slot && mine)
            v[i] = fadd_ftz(v[i], -c);
}

template <typename T, int SUMS, bool VEC>
__global__ void __launch_bounds__(256)
k_distill_bwd(const T* z, int64_t z_ld, T* dz, int64_t dz_ld, const BwdArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= a.items)
        return;
    const int64_t row = item / a.nblk, blk = item - row * a.nblk, lo = blk * BLK;
    const int len = (int)(a.V - lo < BLK ? a.V - lo : BLK);
    float x[PER];
    load_block<T, VEC>(z + row * z_ld + lo, len, lane, x);
    const float* st = a.stats + row * (STATS + a.K);
    const float M = st[0], l = st[1], l1 = st[3], lse1 = st[4], P = st[7];
    const float g = flush(a.g[row * a.g_stride]);
    int64_t lab = -1;
    if (a.w_ce != 0.0f) {
        lab = load_index(a.labels, a.index_bytes, row);
        lab = lab < a.V ? lab : -1;
    }
    const float gk = fmul_flush(fmul_flush(g, a.w_kd), a.tau);
    const float ca = fmul_flush(gk, P);
    const float cb = fmul_flush(g, fadd_ftz(lab >= 0 ? a.w_ce : 0.0f,
                                            fmul_rn(fmul_flush(2.0f, a.w_z), a.w_z != 0.0f ? lse1 : 0.0f)));
    const float qa = flush(__fdiv_rn(SUMS == ONE ? fadd_ftz(ca, cb) : ca, l));
    const float qb = SUMS == BOTH ? flush(__fdiv_rn(cb, l1)) : 0.0f;
    const bool none = M == -CUDART_INF_F;
    const float Mu = fmul_flush(M, a.it);
    const u64 zero = dup2(-0.0f), nu = dup2(-Mu), nm = dup2(-M), sc = dup2(a.it), wa = dup2(qa), wb = dup2(qb);
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
        const u64 v = pack2(x[i], x[i + 1]);
        const u64 u = SUMS == ONE ? v : fmul2_rn(fadd2_ftz(v, zero), sc);
        u64 d = fadd2_ftz(fmul2_rn(exp_neg2(fadd2_ftz(u, nu)), wa), zero);
        if (SUMS == BOTH)
            d = fadd2_ftz(d, fmul2_rn(exp_neg2(fadd2_ftz(v, nm)), wb));
        unpack2(d, x[i], x[i + 1]);
    }
    // the teacher's entries and the label inside this block, entry by entry
    auto take = [&](int64_t e, float c) {
        const int el = (int)e;
        const int slot = VEC ? (el >> 7) * 4 + (el & 3) : el >> 5;
        const int own = VEC ? (el >> 2) & 31 : el & 31;
        subtract_at(x, slot, lane == own, c);
    };
    if (a.w_kd != 0.0f)
        for (int64_t k0 = 0; k0 < a.K; k0 += 32) {
            int64_t e = -1;
            if (k0 + lane < a.K)
                e = load_index(a.t_idx, a.index_bytes, row * a.K + k0 + lane) - lo;
            unsigned hits = __ballot_sync(0xffffffffu, e >= 0 && e < len);
            if (hits == 0)
                continue;
            const float c = e >= 0 && e < len ? fmul_flush(gk, st[STATS + k0 + lane]) : 0.0f;
            while (hits) {
                const int src = __ffs(hits) - 1;
                hits &= hits - 1;
                take(__shfl_sync(0xffffffffu, (int)e, src), __shfl_sync(0xffffffffu, c, src));
            }
        }
    if (lab >= lo && lab < lo + len)
        take(lab - lo, fmul_flush(g, a.w_ce));
    if (none) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            x[i] = 0.0f;
    }
    T* out = dz + row * dz_ld + lo;
    if (VEC) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            const int e = element<true>(i, lane);
            if (e + 4 <= len) {
                store4(out + e, make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (e + c < len)
                        out[e + c] = from_f32<T>(x[i + c]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = element<false>(i, lane);
            if (e < len)
                out[e] = from_f32<T>(x[i]);
        }
    }
}

int64_t blocks_of(int64_t V) { return (V + BLK - 1) / BLK; }

int sums_of(const DistillArgs& a)
{
    return a.tau == 1.0f ? ONE : a.w_ce != 0.0f || a.w_z != 0.0f ? BOTH : SOFT;
}

// calls f(SUMS) as a compile-time constant
template <typename F> cudaError_t by_sums(int sums, F f)
{
    if (sums == ONE)
        return f(std::integral_constant<int, ONE>());
    if (sums == SOFT)
        return f(std::integral_constant<int, SOFT>());
    return f(std::integral_constant<int, BOTH>());
}

template <typename T> cudaError_t fwd_typed(const DistillArgs& a, void* ws, cudaStream_t st)
{
    const T* z = static_cast<const T*>(a.z);
    const int64_t nblk = blocks_of(a.V), items = a.n * nblk;
    const float it = 1.0f / a.tau;
    float2* ms = static_cast<float2*>(ws);
    float* s1 = reinterpret_cast<float*>(ms + items);
    const bool vec = rows4<T>(a.z, a.z_ld);
    RowArgs r;
    r.t_idx = a.t_idx;
    r.t_val = a.t_val;
    r.t_type = a.t_type;
    r.labels = a.labels;
    r.index_bytes = a.index_bytes;
    r.n = a.n;
    r.V = a.V;
    r.K = a.K;
    r.nblk = nblk;
    r.it = it;
    r.tau = a.tau;
    r.w_kd = a.w_kd;
    r.w_ce = a.w_ce;
    r.w_z = a.w_z;
    r.logprobs = a.logprobs;
    r.ms = ms;
    r.s1 = s1;
    r.loss = a.loss;
    r.stats = a.stats;
    r.err = a.err;
    return by_sums(sums_of(a), [&](auto s) {
        constexpr int SUMS = decltype(s)::value;
        const unsigned grid = (unsigned)((items + 7) / 8);
        if (vec)
            k_distill_blocks<T, SUMS, true><<<grid, 256, 0, st>>>(z, a.z_ld, a.V, nblk, items, it, ms, s1);
        else
            k_distill_blocks<T, SUMS, false><<<grid, 256, 0, st>>>(z, a.z_ld, a.V, nblk, items, it, ms, s1);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
        e = launch_pdl(k_distill_rows<T, SUMS>, dim3((unsigned)((a.n + 3) / 4)), dim3(128), 0, st, z, a.z_ld, r);
        count_launches(2);
        return e;
    });
}

template <typename T> cudaError_t bwd_typed(const DistillArgs& a, cudaStream_t st)
{
    const T* z = static_cast<const T*>(a.z);
    T* dz = static_cast<T*>(a.dz);
    BwdArgs b;
    b.t_idx = a.t_idx;
    b.labels = a.labels;
    b.index_bytes = a.index_bytes;
    b.V = a.V;
    b.K = a.K;
    b.nblk = blocks_of(a.V);
    b.items = a.n * b.nblk;
    b.it = 1.0f / a.tau;
    b.tau = a.tau;
    b.w_kd = a.w_kd;
    b.w_ce = a.w_ce;
    b.w_z = a.w_z;
    b.stats = a.stats;
    b.g = a.g;
    b.g_stride = a.g_stride;
    const bool vec = rows4<T>(a.z, a.z_ld) && rows4<T>(a.dz, a.dz_ld);
    return by_sums(sums_of(a), [&](auto s) {
        constexpr int SUMS = decltype(s)::value;
        const unsigned grid = (unsigned)((b.items + 7) / 8);
        if (vec)
            k_distill_bwd<T, SUMS, true><<<grid, 256, 0, st>>>(z, a.z_ld, dz, a.dz_ld, b);
        else
            k_distill_bwd<T, SUMS, false><<<grid, 256, 0, st>>>(z, a.z_ld, dz, a.dz_ld, b);
        count_launches(1);
        return cudaGetLastError();
    });
}

} // namespace

size_t distill_ws_bytes(int64_t n, int64_t V) { return (size_t)(n * blocks_of(V)) * 12; }

cudaError_t launch_distill_fwd(const DistillArgs& a, void* ws, cudaStream_t st)
{
    return a.z_type == 0 ? fwd_typed<float>(a, ws, st) : fwd_typed<__nv_bfloat16>(a, ws, st);
}

cudaError_t launch_distill_bwd(const DistillArgs& a, cudaStream_t st)
{
    return a.z_type == 0 ? bwd_typed<float>(a, st) : bwd_typed<__nv_bfloat16>(a, st);
}

} // namespace repro
