// k_distill.cu -- loss of a student's logits against a teacher's top logits (with
// the label's cross entropy and the log-partition penalty), and the logits'
// gradient.
//
//   u = z / tau, q = softmax(u), p = the teacher's weights over its K entries
//   loss = w_kd tau^2 sum p_k (ln p_k - ln q_idx_k) + w_ce (lse(z) - z_label) + w_z lse(z)^2
//   dz   = g (w_kd tau (P q - p) + (w_ce + 2 w_z lse(z)) softmax(z) - w_ce [label])
//
// The forward reads the logits once, the backward reads them and writes the
// gradient: bytes bound both at binary32, and the e^x of every logit (about 12
// unfused operations) comes close to the bytes' time there and above it for bf16.
// So e^x is 2^t with a plain rounded product t = x log2 e (the argument is a
// difference from the maximum: its large values weigh nothing), 32 powers of two
// that the lanes of a warp hold and a degree-2 polynomial, on packed pairs.
//
// Order: the row is cut into blocks of 1024 logits; a warp holds a block in
// registers (32 per lane), so the block's exact maximum and then its sum come
// from one read, with no running rescale.  128 chains per block and the pairwise
// tree over them: chain j mod 128 puts a chain's terms into one lane whether the
// lane loads single elements (lane, lane + 32, ..: rows of any alignment) or four
// neighbours.  The blocks' (maximum, sum) pairs of a row are joined once all are
// there, in the same CTA when there are rows enough for a CTA to own its rows
// (k_distill_fwd), else by a second kernel, so that few rows over a long
// vocabulary still spread over the card (k_distill_blocks, k_distill_rows).  What a row
// needs of the teacher does not wait for its blocks and is done beside them.
//
// Rows may hold what masks and half-precision teachers leave there: a NaN or an infinity beside
// empty entries, the type's lowest value throughout, products by 1 / tau that overflow.
// What those take is kept off the ordinary rows' path (far_row, join_apart).
//
// 8192 x 32768 fp32 with 64 entries a row: forward 168 us at tau 1 (6.4 TB/s, 0.96 of a
// copy's), 188 us at tau 2 with labels; backward 312 us (6.9 TB/s).  4096 x 32768 bf16:
// forward 89 us (0.45 of a copy's rate: the FP32 pipe is active half of the time, HBM a third; a
// warp loads its block, waits and then computes, so the two add up), backward 114 us (94
// with one entry a row; FP32 pipe 57 %, HBM 62 %).  As cross entropy and z-loss without a teacher
// 8192 x 32768 takes 171 and 309 us in fp32, 161 and 177 us in bf16.
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
constexpr int BOTH = 2;     // tau != 1 and the softmax of z itself: a second e^x per logit,
constexpr int SQR1 = 3;     // .. or for tau = 2 the square of the first,
constexpr int SQR2 = 4;     // .. or for tau = 4 its fourth power

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ u64 dup2(float v) { return pack2(v, v); }

// e^x for x <= 0 (a NaN stays a NaN): t = x (x) log2 e; k / 32 = t rounded to a multiple
// of 1/32 by adding and subtracting 1.5 * 2^18, f = t (-) k / 32; the degree-2 minimax
// polynomial of 2^f on [-1/64, 1/64] (relative error 5.4e-8, constant term 1; by the
// exchange algorithm of Remez, rounded to binary32) in Horner form, times
// T[k mod 32] 2^floor(k / 32), T[j] = RN(2^(j / 32)); 0 where floor(k / 32) < -125.
//   The coefficients below are doubled and the power halved, both exact, so that its
// bits are (floor(k / 32) + 126) << 23 down to -125, and -126, where smaller t are
// clamped, gives a factor that is zero or subnormal: the flushing product reads 0.
// 126 is part of the number added, so the sum's low 12 bits are the exponent over the
// table's index.  The table lies in the warp's lanes, entry j in lane j, and the
// exchange that fetches an entry takes just those five bits of its index.  Against a
// degree-6 polynomial without a table (8192 x 32768 bf16: forward 192 us, backward
// 240 us) this has 7 fewer operations per logit on the pipe that bounds these kernels.
__device__ const unsigned kPow32[32] = {   // the fractions of T[j]
    0x000000, 0x02cd87, 0x05aac3, 0x08980f, 0x0b95c2, 0x0ea43a, 0x11c3d3, 0x14f4f0,
    0x1837f0, 0x1b8d3a, 0x1ef532, 0x227043, 0x25fed7, 0x29a15b, 0x2d583f, 0x3123f6,
    0x3504f3, 0x38fbaf, 0x3d08a4, 0x412c4d, 0x45672a, 0x49b9be, 0x4e248c, 0x52a81e,
    0x5744fd, 0x5bfbb8, 0x60ccdf, 0x65b907, 0x6ac0c7, 0x6fe4ba, 0x75257d, 0x7a83b3};

constexpr float BIG = 0x1.8p18f + 126.0f;

__device__ __forceinline__ unsigned lane_pow() { return __ldg(kPow32 + (threadIdx.x & 31)); }

__device__ __forceinline__ float power_of(float m, unsigned fraction)
{
    return __uint_as_float(((__float_as_uint(m) << 18) & 0x7f800000u) | fraction);
}

__device__ __forceinline__ u64 mul2_ftz(u64 a, u64 b)
{
    u64 r;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Sums of such e(x): neither they nor their terms are ever subnormal, so an addition
// without flushing has the same bits.  It is used on purpose: the assembler was seen to
// fuse mul.rn.ftz.f32x2 with a following add.rn.ftz.f32x2 (a sum one unit off the
// oracle's), explicit rounding or not; where only one of the two flushes it cannot.
__device__ __forceinline__ u64 add2_plain(u64 a, u64 b)
{
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// a packed pair, clamped t and the polynomial; m returns the rounded sum
__device__ __forceinline__ u64 exp_poly2(u64 x, u64& m)
{
    float t0, t1;
    unpack2(fmul2_rn(x, dup2(LOG2E)), t0, t1);   // subnormal t: consumed by flushing sums only
    const u64 t = pack2(max_nan(t0, -126.0f), max_nan(t1, -126.0f));
    m = fadd2_ftz(t, dup2(BIG));
    // -k / 32 = BIG - m: the product by -1 and the difference are exact, so nothing is fused
    // here that rounds; it saves a negation
    const u64 f = fadd2_ftz(t, ffma2_rn(m, dup2(-1.0f), dup2(BIG)));
    const u64 p = fadd2_ftz(fmul2_rn(dup2(0x1.ebfeacp-2f), f), dup2(0x1.62e586p+0f));
    return fadd2_ftz(fmul2_rn(p, f), dup2(2.0f));
}

// every lane of the warp takes part; `pow` is the lane's entry of the table
__device__ __forceinline__ u64 exp_neg2(u64 x, unsigned pow)
{
    u64 m;
    float m0, m1;
    const u64 p = exp_poly2(x, m);
    unpack2(m, m0, m1);
    const unsigned f0 = __shfl_sync(0xffffffffu, pow, __float_as_int(m0));
    const unsigned f1 = __shfl_sync(0xffffffffu, pow, __float_as_int(m1));
    return mul2_ftz(p, pack2(power_of(m0, f0), power_of(m1, f1)));
}

// the same for lanes that go their own ways
__device__ __forceinline__ float exp_neg(float x)
{
    u64 m;
    float m0, m1, p0, p1;
    unpack2(exp_poly2(pack2(x, x), m), p0, p1);
    unpack2(m, m0, m1);
    const u64 s = dup2(power_of(m0, __ldg(kPow32 + (__float_as_uint(m0) & 31u))));
    unpack2(mul2_ftz(dup2(p0), s), p0, p1);
    return flush(p0);   // (keeps the product apart from the caller's additions)
}

// the softmax-of-z term from the softened one, e(x)^tau by squaring
template <int SUMS> __device__ __forceinline__ u64 power2(u64 e)
{
    const u64 z = dup2(-0.0f);
    u64 q = fadd2_ftz(fmul2_rn(e, e), z);
    if (SUMS == SQR2)
        q = fadd2_ftz(fmul2_rn(q, q), z);
    return q;
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
    if (len == BLK) {   // all but a row's last block: no bounds
        const T* q = p + (VEC ? 4 * lane : lane);
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
            if (VEC) {
                const float4 v = stream4(q + 32 * i);
                x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    x[i + c] = to_f32<T>(q[32 * (i + c)]);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = element<VEC>(i, lane);
        x[i] = e < len ? to_f32<T>(p[e]) : -CUDART_INF_F;
    }
}

// Whether differences from m are taken before they are scaled: m (x) it is infinite although m
// is not (tau below 1 and a row, block or list masked by the type's lowest value), so that
// the difference of the products would be a NaN.
__device__ __forceinline__ bool overflows(float m, float mu)
{
    return fabsf(mu) == CUDART_INF_F && fabsf(m) < CUDART_INF_F;
}

// which sums' products can do that
template <int SUMS> constexpr bool SCALED = SUMS == SOFT || SUMS == BOTH;

// the tree over a block's 128 chains: this lane's four, in slots i mod 4
template <bool VEC> __device__ __forceinline__ float chains_tree(u64 a, u64 b)
{
    float s0, s1, s2, s3;
    unpack2(a, s0, s1);
    unpack2(b, s2, s3);
    if (VEC)   // chain 4 lane + c: neighbours first
        return warp_tree(fadd_ftz(fadd_ftz(s0, s1), fadd_ftz(s2, s3)));
    // chain 32 c + lane: lanes first
    return fadd_ftz(fadd_ftz(warp_tree(s0), warp_tree(s1)), fadd_ftz(warp_tree(s2), warp_tree(s3)));
}

// maximum of one block and the sums over it of e(z_i (x) it (-) m (x) it) and, where the
// call needs it, of e(z_i (-) m)
template <typename T, int SUMS, bool VEC>
__device__ __forceinline__ void block_stats(const T* p, int len, int lane, unsigned pow, float it, float& m, float& s,
                                            float& s1)
{
    float x[PER];
    load_block<T, VEC>(p, len, lane, x);
    float t = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        t = max_nan(t, x[i]);
    t = flush(warp_max(t));
    m = t == 0.0f ? 0.0f : t;
    s = s1 = 0.0f;
    if (m == -CUDART_INF_F)
        return;
    const u64 nu = dup2(-fmul_flush(m, it)), nm = dup2(-m), sc = dup2(it);
    u64 a = dup2(0.0f), b = dup2(0.0f), a1 = a, b1 = b;
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
        const u64 v = pack2(x[i], x[i + 1]), w = pack2(x[i + 2], x[i + 3]);
        // a subnormal logit is not flushed before it is scaled: it is far below half a step
        // of any maximum that e(.) can tell from 0
        const u64 ev = exp_neg2(fadd2_ftz(SUMS == ONE ? v : fmul2_rn(v, sc), nu), pow);
        const u64 ew = exp_neg2(fadd2_ftz(SUMS == ONE ? w : fmul2_rn(w, sc), nu), pow);
        a = add2_plain(a, ev);
        b = add2_plain(b, ew);
        if (SUMS >= BOTH) {
            a1 = add2_plain(a1, SUMS == BOTH ? exp_neg2(fadd2_ftz(v, nm), pow) : power2<SUMS>(ev));
            b1 = add2_plain(b1, SUMS == BOTH ? exp_neg2(fadd2_ftz(w, nm), pow) : power2<SUMS>(ew));
        }
    }
    s = chains_tree<VEC>(a, b);
    if (SUMS >= BOTH)
        s1 = chains_tree<VEC>(a1, b1);
}

// a row's teacher: the sums of p_k (a_k - u_k) and of p_k, maximum, sum and P; `ref` not
// infinite: the first sum is of differences from the maximum and from that logit's u
struct Teacher {
    double sum, weight;
    float mt, lt, P, ref;
};

struct FwdArgs {
    const void* t_idx;
    const void* t_val;
    int t_type;
    const void* labels;
    int index_bytes;
    int n, V, K, nblk;
    float it, tau, w_kd, w_ce, w_z;
    bool logprobs;
    float2* ms;      // [n][nblk] block maxima and sums
    float* s1;       // [n][nblk]
    Teacher* teachers;   // [n], where a CTA does not own its rows
    float* loss;
    float* stats;
    int* err;
};

template <typename T, int SUMS, bool VEC>
__device__ __forceinline__ void do_block(const T* z, int64_t z_ld, const FwdArgs& a, int row, int blk, int lane,
                                         unsigned pow)
{
    const int lo = blk * BLK;
    float m, s, s1;
    block_stats<T, SUMS, VEC>(z + (int64_t)row * z_ld + lo, min(a.V - lo, BLK), lane, pow, a.it, m, s, s1);
    if (lane == 0) {
        const int64_t at = (int64_t)row * a.nblk + blk;
        // where m (x) it overflows the sum is a NaN: +0 under a row's finite maximum, which
        // such a block adds nothing to; else join_apart forms it again
        a.ms[at] = make_float2(m, SCALED<SUMS> && fabsf(m) < CUDART_INF_F && s != s ? 0.0f : s);
        if (SUMS >= BOTH)
            a.s1[at] = s1;
    }
}

constexpr int WARPS = 8;
constexpr int FWD_CTAS = 5;
constexpr int MAX_ROWS = 8;   // rows a CTA joins at a time

// asks L2 for `count` elements from p on, a 128-byte line a lane
template <typename T> __device__ __forceinline__ void fetch_ahead(const T* p, int count, int lane)
{
    const int e = lane * (128 / (int)sizeof(T));
    if (e < count)
        asm volatile("prefetch.global.L2 [%0];" :: "l"(p + e));
}

struct RowShared {
    Teacher t[MAX_ROWS];
    float M[MAX_ROWS], l[MAX_ROWS], l1[MAX_ROWS];
    double ln[3][MAX_ROWS];
    int next;   // block handed out
};

// t_k of an entry, and its column (-1, and -infinity: empty)
__device__ __forceinline__ float teacher(const FwdArgs& a, int64_t at, int& j)
{
    const int64_t c = load_index(a.t_idx, a.index_bytes, at);
    if (c >= a.V)
        atomicOr(a.err, kErrIndexBit);
    j = c < 0 || c >= a.V ? -1 : (int)c;
    if (j < 0)
        return -CUDART_INF_F;
    return flush(a.t_type == 0 ? static_cast<const float*>(a.t_val)[at]
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(a.t_val)[at]));
}

// a_k from t_k
__device__ __forceinline__ float weighed(const FwdArgs& a, float t) { return a.logprobs ? t : fmul_flush(t, a.it); }

// From here on a value is far from zero: binary64 holds its sum with a logarithm no better
// than to 2^-23, and the loss takes differences first.
constexpr float FAR = 0x1p30f;

// |v| < FAR (by its bits: a binary64 comparison costs the SM 16 cycles a warp)
__device__ __forceinline__ bool below_far(double v) { return (__double2hiint(v) & 0x7fffffff) < 0x41d00000; }

// v (x) it for the loss's binary64 terms: in binary64 itself where binary32 overflows
__device__ __forceinline__ double wide_mul(float v, float it)
{
    const float p = fmul_flush(v, it);
    return overflows(v, p) ? (double)v * (double)it : (double)p;
}

// What a row's loss needs of the teacher, by one warp: the weights p_k, and in binary64
// the sums of p_k (a_k - u_k) and of p_k.  None of it waits for the row's blocks:
//   sum p_k (ln p_k - ln q_k) = sum p_k (a_k - u_k) + (lse(u) - (m + ln lt)) sum p_k,
// and far from zero sum p_k ((a_k - m) - (u_k - u_ref)) + ((lse(u) - u_ref) - ln lt) sum p_k.
template <typename T>
__device__ void teacher_row(const T* zr, const FwdArgs& a, int64_t row, Teacher* out)
{
    const int lane = threadIdx.x & 31;
    float* p = a.stats + row * (STATS + a.K) + STATS;
    float mt = a.logprobs ? 0.0f : -CUDART_INF_F, lt = 0.0f, P = 0.0f;
    double sum = 0.0, weight = 0.0;
    int j;
    if (!a.logprobs) {
        for (int k = lane; k < a.K; k += 32)
            mt = max_nan(mt, weighed(a, teacher(a, row * a.K + k, j)));
        mt = warp_max(mt);
        mt = mt == 0.0f ? 0.0f : mt;
    }
    float most = 0.0f;   // the largest t_k, where its product by it may have overflowed
    if (fabsf(mt) == CUDART_INF_F) {
        most = -CUDART_INF_F;
        for (int k = lane; k < a.K; k += 32)
            most = max_nan(most, teacher(a, row * a.K + k, j));
        most = warp_max(most);
    }
    const bool apart = overflows(most, mt);
    if (mt == -CUDART_INF_F && !apart) {
        for (int k = lane; k < a.K; k += 32)
            p[k] = 0.0f;
    } else {
        for (int k = lane; k < a.K; k += 32) {
            const float t = teacher(a, row * a.K + k, j);
            const float x = apart ? fmul_flush(fadd_ftz(t, -most), a.it) : fadd_ftz(weighed(a, t), -mt);
            // a log-probability may be anything the caller has; e(.) has no powers from 2^128 on
            float e = x > 88.0f ? CUDART_INF_F : exp_neg(x);
            e = j >= 0 ? e : 0.0f;   // an empty entry weighs nothing, whatever the maximum is
            lt = fadd_ftz(lt, e);
            p[k] = e;
        }
        lt = warp_tree(lt);
        P = a.logprobs ? lt : lt == lt ? 1.0f : lt;
        lt = a.logprobs ? 1.0f : lt;
        for (int k = lane; k < a.K; k += 32) {
            const float ak = weighed(a, teacher(a, row * a.K + k, j));
            if (j < 0)   // its +0 stays: over a sum that is no number it would be one no more
                continue;
            float w = p[k];
            if (!a.logprobs) {
                w = flush(__fdiv_rn(w, lt));
                p[k] = w;
            }
            if (w != 0.0f && a.w_kd != 0.0f) {
                const float u = fmul_flush(flush(to_f32<T>(zr[j])), a.it);
                sum = sum + (double)w * ((double)ak - (double)u);
                weight = weight + (double)w;
            }
        }
        if (a.w_kd != 0.0f) {
            // both trees at once: after the first level the even lanes have the one, the odd
            // lanes the other (6 binary64 additions instead of 10)
            const bool odd = lane & 1;
            double v = (odd ? weight : sum) + __shfl_xor_sync(0xffffffffu, odd ? sum : weight, 1);
#pragma unroll
            for (int s = 2; s < 32; s *= 2)
                v = v + __shfl_xor_sync(0xffffffffu, v, s);
            sum = __shfl_sync(0xffffffffu, v, 0);
            weight = __shfl_sync(0xffffffffu, v, 1);
        }
    }
    if (lane == 0)
        *out = {sum, weight, mt, lt, P, CUDART_INF_F};
}

// A block's sum of e((z_i (-) m) (x) it), for rows whose maximum overflows when scaled: they
// are rare, so the block is read again (ahead of block_stats's own sums this cost those
// registers: 8192 x 32768 fp32 at tau 1.5 with labels 278 us instead of 267).  The order is
// block_stats's for either way of loading.
template <typename T> __device__ float block_apart(const T* p, int len, float it, float m)
{
    const int lane = threadIdx.x & 31;
    const unsigned pow = lane_pow();
    u64 s[2] = {dup2(0.0f), dup2(0.0f)};
#pragma unroll 1
    for (int i = 0; i < PER; i += 4) {
        float d[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int e = element<false>(i + c, lane);
            d[c] = e < len ? fadd_ftz(to_f32<T>(p[e]), -m) : -CUDART_INF_F;
        }
        s[0] = add2_plain(s[0], exp_neg2(fmul2_rn(pack2(d[0], d[1]), dup2(it)), pow));
        s[1] = add2_plain(s[1], exp_neg2(fmul2_rn(pack2(d[2], d[3]), dup2(it)), pow));
    }
    return chains_tree<false>(s[0], s[1]);
}

// lane's chain of the sum over the blocks of such a row, M its maximum (in line 276 us for the
// bf16 rows of those sizes, out of line 273)
template <typename T>
__device__ __noinline__ float join_apart(const T* zr, const float2* ms, int nblk, int V, float it, float M)
{
    const int lane = threadIdx.x & 31;
    float l = 0.0f;
#pragma unroll 1
    for (int b = 0; b < nblk; ++b) {
        const float2 v = ms[b];
        const float f = exp_neg(fmul_rn(fadd_ftz(v.x, -M), it));
        float s = v.y;
        if (f != 0.0f && overflows(v.x, fmul_flush(v.x, it)))
            s = block_apart<T>(zr + b * BLK, min(V - b * BLK, BLK), it, v.x);
        if (lane == (b & 31))
            l = fadd_ftz(l, fmul_rn(s, f));
    }
    return l;
}

// A row far from zero (masked by the type's lowest value throughout): its teacher's sum anew, of
// p_k ((a_k - m) - (u_k - u_ref)), ref the largest logit that has weight.
template <typename T> __device__ __noinline__ void far_row(const T* zr, const FwdArgs& a, int64_t row, Teacher* out)
{
    const int lane = threadIdx.x & 31;
    const float ta = a.logprobs ? 1.0f : a.it;
    const float* p = a.stats + row * (STATS + a.K) + STATS;
    int j;
    float ref = -CUDART_INF_F, most = a.logprobs ? 0.0f : -CUDART_INF_F;
    for (int k = lane; k < a.K; k += 32) {
        const float t = teacher(a, row * a.K + k, j);
        most = a.logprobs ? most : max_nan(most, t);
        if (j >= 0 && p[k] != 0.0f)
            ref = max_nan(ref, flush(to_f32<T>(zr[j])));
    }
    ref = warp_max(ref);
    if (!(fabsf(ref) < CUDART_INF_F))
        return;
    const double m = wide_mul(warp_max(most), ta), c = wide_mul(ref, a.it);
    double sum = 0.0;
    for (int k = lane; k < a.K; k += 32) {
        const float t = teacher(a, row * a.K + k, j);
        if (j >= 0 && p[k] != 0.0f)
            sum = sum + (double)p[k] * ((wide_mul(t, ta) - m) - (wide_mul(flush(to_f32<T>(zr[j])), a.it) - c));
    }
#pragma unroll
    for (int s = 1; s < 32; s *= 2)
        sum = sum + __shfl_xor_sync(0xffffffffu, sum, s);
    if (lane == 0) {
        out->sum = sum;
        out->ref = ref;
    }
}

// joins the blocks of rows [r0, r0 + cnt) and forms the losses.  A warp per row, but the
// logarithms: binary64 runs at 1/64 of the binary32 rate here whether one lane needs
// it or 32, so one warp takes all of the CTA's, a lane each.
template <typename T, int SUMS>
__device__ void finish_rows(const T* z, int64_t z_ld, const FwdArgs& a, int r0, int cnt, Teacher* teachers,
                            RowShared& sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int r = warp; r < cnt; r += WARPS) {
        const int64_t row = r0 + r;
        const float2* ms = a.ms + row * a.nblk;
        float M = -CUDART_INF_F;
        for (int b = lane; b < a.nblk; b += 32)
            M = max_nan(M, ms[b].x);
        M = warp_max(M);
        M = M == 0.0f ? 0.0f : M;
        const float Mu = fmul_flush(M, a.it);
        float l = 0.0f, l1 = 0.0f;
        if (M != -CUDART_INF_F) {
            for (int b = lane; b < a.nblk; b += 32) {
                const float2 v = ms[b];
                l = fadd_ftz(l, fmul_rn(v.y, exp_neg(fadd_ftz(fmul_rn(v.x, a.it), -Mu))));
                if (SUMS >= BOTH)
                    l1 = fadd_ftz(l1, fmul_rn(a.s1[row * a.nblk + b], exp_neg(fadd_ftz(v.x, -M))));
            }
            if (SCALED<SUMS> && overflows(M, Mu))
                l = join_apart(z + row * z_ld, ms, a.nblk, a.V, a.it, M);
            l = warp_tree(l);
            l1 = SUMS >= BOTH ? warp_tree(l1) : SUMS == ONE ? l : 0.0f;
        }
        const Teacher* t = teachers + r;
        if (a.w_kd != 0.0f && t->lt != 0.0f && !(fabsf(t->mt) < FAR && below_far(t->sum)))
            far_row(z + row * z_ld, a, row, teachers + r);
        if (lane == 0) {
            sh.M[r] = M;
            sh.l[r] = l;
            sh.l1[r] = l1;
        }
    }
    __syncthreads();
    if (threadIdx.x >= 32)
        return;
    if (lane < 3 * MAX_ROWS) {
        const int which = lane / MAX_ROWS, r = lane % MAX_ROWS;
        if (r < cnt)
            sh.ln[which][r] = ln_d(which == 0 ? sh.l[r] : which == 1 ? sh.l1[r] : teachers[r].lt);
    }
    __syncwarp();
    if (lane >= cnt)
        return;
    const int r = lane;
    const int64_t row = r0 + r;
    const T* zr = z + row * z_ld;
    const float M = sh.M[r];
    const Teacher t = teachers[r];
    const bool none = M == -CUDART_INF_F;
    const double Mu = SCALED<SUMS> ? wide_mul(M, a.it) : (double)fmul_flush(M, a.it);
    const double lse_t = none ? 0.0 : Mu + sh.ln[0][r];
    const double lse1 = none || SUMS == SOFT ? 0.0 : (double)M + sh.ln[1][r];
    double v = 0.0;
    if (!none && a.w_kd != 0.0f && t.lt != 0.0f) {   // 0: no teacher
        double rest = lse_t - ((double)t.mt + sh.ln[2][r]);
        if (t.ref != CUDART_INF_F)
            rest = ((Mu - wide_mul(t.ref, a.it)) + sh.ln[0][r]) - sh.ln[2][r];
        v = ((double)a.w_kd * ((double)a.tau * (double)a.tau)) * (t.sum + rest * t.weight);
    }
    if (a.w_ce != 0.0f) {
        const int64_t lab = load_index(a.labels, a.index_bytes, row);
        if (lab >= a.V)
            atomicOr(a.err, kErrIndexBit);
        else if (lab >= 0 && !none) {
            const double zl = (double)flush(to_f32<T>(zr[lab]));
            v = v + (double)a.w_ce * (fabsf(M) < FAR ? lse1 - zl : ((double)M - zl) + sh.ln[1][r]);
        }
    }
    if (a.w_z != 0.0f && !none)
        v = v + (double)a.w_z * (lse1 * lse1);
    float* st = a.stats + row * (STATS + a.K);
    a.loss[row] = flush(__double2float_rn(v));
    st[0] = M;
    st[1] = sh.l[r];
    st[2] = none ? M : flush(__double2float_rn(lse_t));
    st[3] = sh.l1[r];
    st[4] = SUMS == SOFT ? 0.0f : none ? M : flush(__double2float_rn(lse1));
    st[5] = t.mt;
    st[6] = t.lt;
    st[7] = t.P;
}

// a CTA owns `rows` rows: the teacher's part by a warp each, the rows' blocks by all
// warps as they come free, then the losses
template <typename T, int SUMS, bool VEC>
__global__ void __launch_bounds__(32 * WARPS, FWD_CTAS)
k_distill_fwd(const T* z, int64_t z_ld, const __grid_constant__ FwdArgs a, int rows)
{
    __shared__ RowShared sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned pow = lane_pow();
    const int r0 = blockIdx.x * rows, cnt = min(rows, a.n - r0), items = cnt * a.nblk;
    if (threadIdx.x == 0)
        sh.next = 0;
    __syncthreads();
    if (warp < cnt)
        teacher_row(z + (int64_t)(r0 + warp) * z_ld, a, r0 + warp, &sh.t[warp]);
    for (;;) {
        int i = 0;
        if (lane == 0)
            i = atomicAdd(&sh.next, 1);
        i = __shfl_sync(0xffffffffu, i, 0);
        if (i >= items)
            break;
        const int r = i / a.nblk;
        do_block<T, SUMS, VEC>(z, z_ld, a, r0 + r, i - r * a.nblk, lane, pow);
    }
    __syncthreads();
    finish_rows<T, SUMS>(z, z_ld, a, r0, cnt, sh.t, sh);
}

// the same work spread over the card: the first `tctas` CTAs take the teacher's part of a
// row per warp, the others a block per warp; k_distill_rows joins them
template <typename T, int SUMS, bool VEC>
__global__ void __launch_bounds__(32 * WARPS)
k_distill_blocks(const T* z, int64_t z_ld, const __grid_constant__ FwdArgs a, int tctas)
{
    const int warp = threadIdx.x >> 5;
    if (blockIdx.x < tctas) {
        const int row = blockIdx.x * WARPS + warp;
        if (row < a.n)
            teacher_row(z + (int64_t)row * z_ld, a, row, a.teachers + row);
        return;
    }
    const int item = (blockIdx.x - tctas) * WARPS + warp;
    if (item >= a.n * a.nblk)
        return;
    const int row = item / a.nblk;
    do_block<T, SUMS, VEC>(z, z_ld, a, row, item - row * a.nblk, threadIdx.x & 31, lane_pow());
}

template <typename T, int SUMS>
__global__ void __launch_bounds__(32 * WARPS)
k_distill_rows(const T* z, int64_t z_ld, const __grid_constant__ FwdArgs a)
{
    __shared__ RowShared sh;
    pdl_wait();
    const int r0 = blockIdx.x * MAX_ROWS;
    finish_rows<T, SUMS>(z, z_ld, a, r0, min(MAX_ROWS, a.n - r0), a.teachers + r0, sh);
}

struct BwdArgs {
    const void* t_idx;
    const void* labels;
    int index_bytes;
    int V, K, nblk, groups, items, per, mask;
    float it, tau, w_kd, w_ce, w_z;
    const float* stats;
    const float* g;
    int64_t g_stride;
};

constexpr int BWD_CTAS = 4;
constexpr int LIST = 128;          // teacher entries in its pieces that a warp of the backward lists
constexpr int FEW = 3;             // entries in a piece that are taken one by one
constexpr int BPER = 16;           // logits per lane and piece of the backward
constexpr int BBLK = 32 * BPER;

// A piece of a row.  The order of the elements does not matter in the backward.  LINES,
// where z and dz start equally far past a 128-byte line: a row's pieces are cut at
// lines, and all but the row's ends move 16 bytes a lane and whole lines by the warp,
// whatever the vocabulary's remainder: with W = 16 / sizeof(T), slot i of a lane is
// element 32 W (i / W) + W lane + i mod W.  Otherwise element 32 i + lane.  Elements
// outside [0, V) are -infinity.
template <typename T, bool LINES> __device__ __forceinline__ int piece_element(int i, int lane)
{
    constexpr int W = 16 / sizeof(T);
    return LINES ? 32 * W * (i / W) + W * lane + i % W : 32 * i + lane;
}

template <typename T, bool LINES>
__device__ __forceinline__ void load_piece(const T* p, int lo, int V, int lane, float (&x)[BPER])
{
    constexpr int W = 16 / sizeof(T);
    if (LINES && lo >= 0 && lo + BBLK <= V) {
        const T* q = p + lo + W * lane;
#pragma unroll
        for (int i = 0; i < BPER; i += W)
            load16(q + 32 * i, x + i);
        return;
    }
#pragma unroll
    for (int i = 0; i < BPER; ++i) {
        const int e = lo + piece_element<T, LINES>(i, lane);
        x[i] = e >= 0 && e < V ? to_f32<T>(p[e]) : -CUDART_INF_F;
    }
}

template <typename T, bool LINES>
__device__ __forceinline__ void store_piece(T* p, int lo, int V, int lane, const float (&x)[BPER])
{
    constexpr int W = 16 / sizeof(T);
    if (LINES && lo >= 0 && lo + BBLK <= V) {
        T* q = p + lo + W * lane;
#pragma unroll
        for (int i = 0; i < BPER; i += W)
            store16(q + 32 * i, x + i);
        return;
    }
#pragma unroll
    for (int i = 0; i < BPER; ++i) {
        const int e = lo + piece_element<T, LINES>(i, lane);
        if (e >= 0 && e < V)
            p[e] = from_f32<T>(x[i]);
    }
}

// One warp takes `per` consecutive pieces of a row, so that what belongs to the row
// (statistics, coefficients and their divisions) is done once.  Pieces of 16 logits a
// lane leave registers for 32 warps per SM, which is what covers the loads.
template <typename T, int SUMS, bool LINES, bool LONG>
__global__ void __launch_bounds__(32 * WARPS, BWD_CTAS)
k_distill_bwd(const T* z, int64_t z_ld, T* dz, int64_t dz_ld, const __grid_constant__ BwdArgs a)
{
    __shared__ float pieces[WARPS][BBLK], weights[WARPS][LONG ? LIST : 1];
    __shared__ int columns[WARPS][LONG ? LIST : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = blockIdx.x * WARPS + warp;
    if (item >= a.items)
        return;
    const int row = item / a.groups, first = (item - row * a.groups) * a.per;
    const T* zr = z + row * z_ld;
    T* dr = dz + row * dz_ld;
    const int shift = LINES ? (int)((reinterpret_cast<uintptr_t>(zr) / sizeof(T)) & a.mask) : 0;
    const unsigned pow = lane_pow();
    float x[BPER];
    load_piece<T, LINES>(zr, first * BBLK - shift, a.V, lane, x);   // on its way while the row's numbers come
    const float* st = a.stats + (int64_t)row * (STATS + a.K);
    const float M = st[0], l = st[1], l1 = st[3], lse1 = st[4], P = st[7];
    const float g = flush(a.g[row * a.g_stride]);
    int lab = -1;
    if (a.w_ce != 0.0f) {
        const int64_t t = load_index(a.labels, a.index_bytes, row);
        lab = t >= 0 && t < a.V ? (int)t : -1;
    }
    const int K = a.w_kd != 0.0f ? a.K : 0;
    auto column = [&](int k) {
        const int64_t j = k < K ? load_index(a.t_idx, a.index_bytes, (int64_t)row * a.K + k) : -1;
        return j >= 0 && j < a.V ? (int)j : -1;
    };
    int col0 = column(lane), col1 = K > 32 ? column(lane + 32) : -1;   // on their way, too
    float p0 = 0.0f, p1 = 0.0f;
    if (!LONG) {
        p0 = col0 >= 0 ? st[STATS + lane] : 0.0f;
        p1 = col1 >= 0 ? st[STATS + lane + 32] : 0.0f;
    }
    const float gk = fmul_flush(fmul_flush(g, a.w_kd), a.tau);
    const float ca = a.w_kd != 0.0f ? fmul_flush(gk, P) : gk;   // P may be a NaN that no one asked for
    const float cb = fmul_flush(g, fadd_ftz(lab >= 0 ? a.w_ce : 0.0f,
                                            fmul_rn(fmul_flush(2.0f, a.w_z), a.w_z != 0.0f ? lse1 : 0.0f)));
    const float qa = flush(__fdiv_rn(SUMS == ONE ? fadd_ftz(ca, cb) : ca, l));
    const float qb = SUMS >= BOTH ? flush(__fdiv_rn(cb, l1)) : 0.0f;
    const float Mu = fmul_flush(M, a.it);
    const bool apart = SCALED<SUMS> && overflows(M, Mu);
    const u64 zero = dup2(-0.0f), nu = dup2(apart ? -0.0f : -Mu), nm = dup2(apart ? -0.0f : -M), sc = dup2(a.it),
              wa = dup2(qa), wb = dup2(qb);
    const int last = min(first + a.per, a.nblk);
    int listed = 0;
    if (M == -CUDART_INF_F) {   // nothing in the row: no gradient
#pragma unroll
        for (int i = 0; i < BPER; ++i)
            x[i] = 0.0f;
        for (int blk = first; blk < last; ++blk)
            store_piece<T, LINES>(dr, blk * BBLK - shift, a.V, lane, x);
        return;
    }
    const float cl = lab >= 0 ? fmul_flush(g, a.w_ce) : 0.0f;
    for (int blk = first; blk < last; ++blk) {
        const int lo = blk * BBLK - shift;
        if (lo >= a.V)
            break;
        if (blk > first)
            load_piece<T, LINES>(zr, lo, a.V, lane, x);
        if (blk + 1 < last)
            fetch_ahead(zr + lo + BBLK, min(a.V - lo - BBLK, BBLK), lane);
        if (apart) {
#pragma unroll
            for (int i = 0; i < BPER; ++i)
                x[i] = fadd_ftz(x[i], -M);
        }
#pragma unroll
        for (int i = 0; i < BPER; i += 2) {
            const u64 v = pack2(x[i], x[i + 1]);
            const u64 e = exp_neg2(fadd2_ftz(SUMS == ONE ? v : fmul2_rn(v, sc), nu), pow);
            u64 d = fmul2_rn(e, wa);
            if (SUMS >= BOTH)
                d = fadd2_ftz(d, fmul2_rn(SUMS == BOTH ? exp_neg2(fadd2_ftz(v, nm), pow) : power2<SUMS>(e), wb));
            else
                d = fadd2_ftz(d, zero);
            unpack2(d, x[i], x[i + 1]);
        }
        // the teacher's entries and the label inside this piece, entry by entry
        const int lo0 = max(lo, 0), end = lo + BBLK;
        const bool inl = lab >= lo0 && lab < end;
        if (LONG && blk == first) {
            // the teacher's entries in the warp's pieces, in order: most pieces have few or none
            const int from = max(lo, 0), to = min(a.V, (last * BBLK) - shift);
            for (int k0 = 0; k0 < K; k0 += 32) {
                const int j = k0 == 0 ? col0 : k0 == 32 ? col1 : column(k0 + lane);
                const bool in = j >= from && j < to;
                const unsigned m = __ballot_sync(0xffffffffu, in);
                const int at = listed + __popc(m & ((1u << lane) - 1u));
                if (in && at < LIST) {
                    columns[warp][at] = j;
                    weights[warp][at] = st[STATS + k0 + lane];
                }
                listed += __popc(m);
            }
            __syncwarp();
            col0 = lane < min(listed, LIST) ? columns[warp][lane] : -1;
            p0 = col0 >= 0 ? weights[warp][lane] : 0.0f;
        }
        auto within = [&](int j) { return j >= lo0 && j < end; };
        // entry k0 + lane: of the row, or of the list where that has all of them
        const int entries = !LONG || listed > LIST ? K : listed;
        auto entry = [&](int k0, int& j, float& p) {
            j = k0 == 0 ? col0 : col1;
            p = k0 == 0 ? p0 : p1;
            if (LONG && listed > LIST) {
                j = column(k0 + lane);
                p = within(j) ? st[STATS + k0 + lane] : 0.0f;
            } else if (LONG && k0 > 0) {
                j = k0 + lane < listed ? columns[warp][k0 + lane] : -1;
                p = j >= 0 ? weights[warp][k0 + lane] : 0.0f;
            }
        };
        int hits = 0;
        for (int k0 = 0; k0 < entries; k0 += 32) {
            int j;
            float p;
            entry(k0, j, p);
            hits += __popc(__ballot_sync(0xffffffffu, within(j)));
        }
        if (hits > FEW) {
            // through shared memory, 32 entries at a time, those of one column after one another
            float* piece = pieces[warp];
            auto place = [&](int e) {
                constexpr int W = 16 / sizeof(T);
                return LINES ? 32 * (e / (32 * W) * W + e % W) + (e / W & 31) : e;
            };
#pragma unroll
            for (int i = 0; i < BPER; ++i)
                piece[32 * i + lane] = x[i];
            __syncwarp();
            for (int k0 = 0; k0 < entries; k0 += 32) {
                int j;
                float p;
                entry(k0, j, p);
                if (__ballot_sync(0xffffffffu, within(j)) == 0)
                    continue;
                const int at = within(j) ? place(j - lo) : -1 - lane;
                const unsigned same = __match_any_sync(0xffffffffu, at);
                const int turn = __popc(same & ((1u << lane) - 1u));
                const int turns = __reduce_max_sync(0xffffffffu, turn);
                for (int t = 0; t <= turns; ++t) {
                    if (within(j) && turn == t)
                        piece[at] = fadd_ftz(piece[at], -fmul_flush(gk, p));
                    __syncwarp();
                }
            }
            if (inl && lane == 0)
                piece[place(lab - lo)] = fadd_ftz(piece[place(lab - lo)], -cl);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < BPER; ++i)
                x[i] = piece[32 * i + lane];
            __syncwarp();
        } else if (hits > 0 || inl) {
            auto take = [&](int e, float c) {   // (a branch on the slot would put x in local memory)
                constexpr int W = 16 / sizeof(T);
                const int slot = LINES ? e / (32 * W) * W + e % W : e >> 5;
                const int own = LINES ? e / W & 31 : e & 31;
#pragma unroll
                for (int i = 0; i < BPER; ++i)
                    if (i == slot && lane == own)
                        x[i] = fadd_ftz(x[i], -c);
            };
            for (int k0 = 0; hits > 0; k0 += 32) {
                int j;
                float p;
                entry(k0, j, p);
                unsigned in = __ballot_sync(0xffffffffu, within(j));
                hits -= __popc(in);
                while (in) {
                    const int src = __ffs(in) - 1;
                    in &= in - 1;
                    take(__shfl_sync(0xffffffffu, j - lo, src), fmul_flush(gk, __shfl_sync(0xffffffffu, p, src)));
                }
            }
            if (inl)
                take(lab - lo, cl);
        }
        store_piece<T, LINES>(dr, lo, a.V, lane, x);
    }
}

int64_t blocks_of(int64_t V) { return (V + BLK - 1) / BLK; }

int sums_of(const DistillArgs& a)
{
    if (a.tau == 1.0f)
        return ONE;
    if (a.w_ce == 0.0f && a.w_z == 0.0f)
        return SOFT;
    return a.tau == 2.0f ? SQR1 : a.tau == 4.0f ? SQR2 : BOTH;
}

// calls f(SUMS) as a compile-time constant
template <typename F> cudaError_t by_sums(int sums, F f)
{
    switch (sums) {
    case ONE: return f(std::integral_constant<int, ONE>());
    case SOFT: return f(std::integral_constant<int, SOFT>());
    case BOTH: return f(std::integral_constant<int, BOTH>());
    case SQR1: return f(std::integral_constant<int, SQR1>());
    default: return f(std::integral_constant<int, SQR2>());
    }
}

template <typename T> cudaError_t fwd_typed(const DistillArgs& a, void* ws, cudaStream_t st)
{
    const T* z = static_cast<const T*>(a.z);
    const int64_t nblk = blocks_of(a.V), items = a.n * nblk;
    const bool vec = rows4<T>(a.z, a.z_ld);
    FwdArgs r;
    r.t_idx = a.t_idx;
    r.t_val = a.t_val;
    r.t_type = a.t_type;
    r.labels = a.labels;
    r.index_bytes = a.index_bytes;
    r.n = (int)a.n;
    r.V = (int)a.V;
    r.K = (int)a.K;
    r.nblk = (int)nblk;
    r.it = 1.0f / a.tau;
    r.tau = a.tau;
    r.w_kd = a.w_kd;
    r.w_ce = a.w_ce;
    r.w_z = a.w_z;
    r.logprobs = a.logprobs;
    r.teachers = static_cast<Teacher*>(ws);
    r.ms = reinterpret_cast<float2*>(r.teachers + a.n);
    r.s1 = reinterpret_cast<float*>(r.ms + items);
    r.loss = a.loss;
    r.stats = a.stats;
    r.err = a.err;
    // rows per CTA: two of at least 8 blocks (8192 x 32768: one row 205 us, two 193, four 200),
    // more of shorter ones; from four CTAs per SM on a CTA owns its rows (the other way 217 us)
    const int rows = nblk >= 8 ? 2 : nblk >= 4 ? 4 : MAX_ROWS;
    const bool owned = (a.n + rows - 1) / rows >= 4 * num_sms();
    return by_sums(sums_of(a), [&](auto s) {
        constexpr int SUMS = decltype(s)::value;
        if (owned) {
            const unsigned grid = (unsigned)((a.n + rows - 1) / rows);
            if (vec)
                k_distill_fwd<T, SUMS, true><<<grid, 32 * WARPS, 0, st>>>(z, a.z_ld, r, rows);
            else
                k_distill_fwd<T, SUMS, false><<<grid, 32 * WARPS, 0, st>>>(z, a.z_ld, r, rows);
            count_launches(1);
            return cudaGetLastError();
        }
        const int tctas = (int)((a.n + WARPS - 1) / WARPS);
        const unsigned grid = (unsigned)((items + WARPS - 1) / WARPS) + tctas;
        if (vec)
            k_distill_blocks<T, SUMS, true><<<grid, 32 * WARPS, 0, st>>>(z, a.z_ld, r, tctas);
        else
            k_distill_blocks<T, SUMS, false><<<grid, 32 * WARPS, 0, st>>>(z, a.z_ld, r, tctas);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
        e = launch_pdl(k_distill_rows<T, SUMS>, dim3((unsigned)((a.n + MAX_ROWS - 1) / MAX_ROWS)), dim3(32 * WARPS),
                       0, st, z, a.z_ld, r);
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
    b.V = (int)a.V;
    b.K = (int)a.K;
    b.it = 1.0f / a.tau;
    b.tau = a.tau;
    b.w_kd = a.w_kd;
    b.w_ce = a.w_ce;
    b.w_z = a.w_z;
    b.stats = a.stats;
    b.g = a.g;
    b.g_stride = a.g_stride;
    // pieces begin on 128-byte lines where z and dz agree on them
    const int64_t line = 128 / sizeof(T);
    const bool lines = (reinterpret_cast<uintptr_t>(a.z) - reinterpret_cast<uintptr_t>(a.dz)) % 128 == 0 &&
                       (a.z_ld - a.dz_ld) % line == 0;
    b.mask = lines ? (int)line - 1 : 0;
    b.nblk = (int)((a.V + b.mask + BBLK - 1) / BBLK);
    // eight pieces a warp once that leaves every scheduler several warps (1021 x 130001 bf16 with
    // pieces of 1024: one a warp 264 us, two 251, four 240)
    b.per = a.n * b.nblk >= (int64_t)num_sms() * 256 ? 8 : 1;
    b.groups = (b.nblk + b.per - 1) / b.per;
    b.items = (int)(a.n * b.groups);
    return by_sums(sums_of(a), [&](auto s) {
        constexpr int SUMS = decltype(s)::value;
        const unsigned grid = (unsigned)((b.items + WARPS - 1) / WARPS);
        auto go = [&](auto kernel) { kernel<<<grid, 32 * WARPS, 0, st>>>(z, a.z_ld, dz, a.dz_ld, b); };
        if (lines)
            a.K > 64 ? go(k_distill_bwd<T, SUMS, true, true>) : go(k_distill_bwd<T, SUMS, true, false>);
        else
            a.K > 64 ? go(k_distill_bwd<T, SUMS, false, true>) : go(k_distill_bwd<T, SUMS, false, false>);
        count_launches(1);
        return cudaGetLastError();
    });
}

} // namespace

size_t distill_ws_bytes(int64_t n, int64_t V) { return (size_t)(n * blocks_of(V)) * 12 + (size_t)n * sizeof(Teacher); }

cudaError_t launch_distill_fwd(const DistillArgs& a, void* ws, cudaStream_t st)
{
    return a.z_type == 0 ? fwd_typed<float>(a, ws, st) : fwd_typed<__nv_bfloat16>(a, ws, st);
}

cudaError_t launch_distill_bwd(const DistillArgs& a, cudaStream_t st)
{
    return a.z_type == 0 ? bwd_typed<float>(a, st) : bwd_typed<__nv_bfloat16>(a, st);
}

} // namespace repro
