/*
 * oracle.c -- plain CPU statement of the bitwise-reproducible int8 QAT linear
 * layer (forward, backward) and of the fixed-order gradient reduction.
 *
 * TEST INFRASTRUCTURE ONLY: see oracle.h for who may load it, for the
 * arithmetic model and for the canonical reduction order.  Nothing here is
 * blocked, fused or reordered beyond what those definitions state; loops over
 * independent output elements may run on several threads, which changes no
 * bit because every element's own sequence of operations is fixed.
 *
 * Build: cc -O2 -std=c11 -ffp-contract=off -fno-fast-math
 *           -fexcess-precision=standard [-fopenmp] -fPIC -shared oracle.c -lm
 */
#include "oracle.h"

#include <float.h>
#include <math.h>
#include <stdlib.h>
#include <string.h>

#ifdef _OPENMP
#include <omp.h>
#endif

/* ------------------------------------------------------------------------ */
/* Elementary operations.  [P4] "How it works": subnormals are flushed on     */
/* every backend; a*b+c is never contracted.  Operands are flushed first      */
/* (denormals-are-zero), the IEEE result is formed by the host's binary32     */
/* unit in its default round-to-nearest-even mode, then a subnormal result is */
/* flushed.                                                                   */
/* ------------------------------------------------------------------------ */

float oracle_flush(float x)
{
    if (x != 0.0f && fabsf(x) < FLT_MIN)
        return copysignf(0.0f, x);
    return x;
}

float oracle_add(float a, float b)
{
    float r = oracle_flush(a) + oracle_flush(b);
    return oracle_flush(r);
}

float oracle_mul(float a, float b)
{
    float r = oracle_flush(a) * oracle_flush(b);
    return oracle_flush(r);
}

float oracle_div(float a, float b)
{
    float r = oracle_flush(a) / oracle_flush(b);
    return oracle_flush(r);
}

float oracle_sqrt(float a)
{
    float r = sqrtf(oracle_flush(a)); /* IEEE 754 requires correct rounding */
    return oracle_flush(r);
}

float oracle_i2f(int64_t v)
{
    return (float)v; /* round to nearest even in the default mode */
}

/* [P4] "How to use": int8 weights and activations.  The quantiser is
 * q = clamp(round_half_even(x (/) s), -qmax, qmax) with q_max = 127, so -128
 * is never produced.  Special cases: a zero (or flushed) scale maps every
 * element to 0; a NaN quotient maps to 0; +-Inf clamps to +-qmax. */
int oracle_quant_one(float x, float s, int qmax)
{
    float sf = oracle_flush(s);
    if (sf == 0.0f)
        return 0;
    float v = oracle_div(x, sf);
    if (v != v)
        return 0;
    float r = rintf(v); /* integral value, ties to even (default mode) */
    if (r > (float)qmax)
        return qmax;
    if (r < -(float)qmax)
        return -qmax;
    return (int)r;
}

/* ------------------------------------------------------------------------ */
/* Canonical sum: chunks of 64 summed left to right (seeded with the chunk's  */
/* first term), chunk partials combined by the stride-doubling pairwise tree. */
/* ------------------------------------------------------------------------ */

float oracle_canon_sum(const float* p, int64_t L)
{
    if (L <= 0)
        return 0.0f;
    int64_t C = (L + ORACLE_CHUNK - 1) / ORACLE_CHUNK;
    float* t = (float*)malloc((size_t)C * sizeof(float));
    for (int64_t c = 0; c < C; ++c) {
        int64_t lo = c * ORACLE_CHUNK;
        int64_t hi = lo + ORACLE_CHUNK;
        if (hi > L)
            hi = L;
        float a = p[lo];
        for (int64_t i = lo + 1; i < hi; ++i)
            a = oracle_add(a, p[i]);
        t[c] = a;
    }
    for (int64_t s = 1; s < C; s *= 2)
        for (int64_t j = 0; j + s < C; j += 2 * s)
            t[j] = oracle_add(t[j], t[j + s]);
    float r = t[0];
    free(t);
    return r;
}

/* ------------------------------------------------------------------------ */
/* A1 / A2: scales.                                                           */
/* mode 0 (weights, [P4] "How to use" and "Premises and limits": the step    */
/*   size is re-pinned from the weights every optimiser step as              */
/*   2*mean(|w|)/sqrt(q_max)):                                               */
/*     S = canon(|w_0|, ..., |w_{n-1}|); mean = S (/) i2f(n);                 */
/*     s_w = (2 (x) mean) (/) sqrt(i2f(q_max)).                               */
/* mode 1 (activations): s_x = max_i |x_i| (/) i2f(q_max); max is exact.      */
/* ------------------------------------------------------------------------ */

float oracle_wscale(const float* x, int64_t n, int mode, int qmax)
{
    if (mode == 0) {
        float* a = (float*)malloc((size_t)(n > 0 ? n : 1) * sizeof(float));
        for (int64_t i = 0; i < n; ++i)
            a[i] = fabsf(x[i]); /* clears the sign bit: exact */
        float S = oracle_canon_sum(a, n);
        free(a);
        float mean = oracle_div(S, oracle_i2f(n));
        return oracle_div(oracle_mul(2.0f, mean), oracle_sqrt(oracle_i2f(qmax)));
    }
    float m = 0.0f;
    for (int64_t i = 0; i < n; ++i) {
        float v = fabsf(oracle_flush(x[i]));
        if (v > m)
            m = v;
    }
    return oracle_div(m, oracle_i2f(qmax));
}

void oracle_quant_i8(const float* x, int64_t n, float s, int qmax, int8_t* q)
{
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i)
        q[i] = (int8_t)oracle_quant_one(x[i], s, qmax);
}

/* ------------------------------------------------------------------------ */
/* A5: forward.  The int8 x int8 products and their sum are exact integers,  */
/* so the accumulation order cannot matter; the dequantisation is two        */
/* unfused multiplies, left to right: (i2f(acc) (x) s_x) (x) s_w.            */
/* ------------------------------------------------------------------------ */

int64_t oracle_int_dot(const int8_t* xq, const int8_t* wq, int64_t m, int64_t n,
                       int64_t K)
{
    int64_t acc = 0;
    for (int64_t k = 0; k < K; ++k)
        acc += (int64_t)xq[m * K + k] * (int64_t)wq[n * K + k];
    return acc;
}

static float fwd_one(const int8_t* xq, const int8_t* wq, float s_x, float s_w,
                     int64_t m, int64_t n, int64_t K)
{
    int64_t acc = oracle_int_dot(xq, wq, m, n, K);
    return oracle_mul(oracle_mul(oracle_i2f(acc), s_x), s_w);
}

void oracle_linear_fwd(const int8_t* xq, const int8_t* wq, float s_x, float s_w,
                       float* y, int64_t M, int64_t N, int64_t K)
{
#pragma omp parallel for schedule(static)
    for (int64_t m = 0; m < M; ++m)
        for (int64_t n = 0; n < N; ++n)
            y[m * N + n] = fwd_one(xq, wq, s_x, s_w, m, n, K);
}

void oracle_linear_fwd_at(const int8_t* xq, const int8_t* wq, float s_x, float s_w,
                          int64_t M, int64_t N, int64_t K,
                          const int64_t* idx_m, const int64_t* idx_n, int64_t cnt,
                          float* out)
{
    (void)M;
    (void)N;
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < cnt; ++i)
        out[i] = fwd_one(xq, wq, s_x, s_w, idx_m[i], idx_n[i], K);
}

/* ------------------------------------------------------------------------ */
/* A6-A8: backward in fp32.  The dequantised operands are recomputed from    */
/* int8 (W^ = i2f(Wq) (x) s_w, X^ = i2f(Xq) (x) s_x); each output is the      */
/* canonical sum of its rounded products in increasing reduction index.      */
/* ------------------------------------------------------------------------ */

static float dx_one(const float* dy, const int8_t* wq, float s_w, int64_t m, int64_t k,
                    int64_t N, int64_t K, float* terms)
{
    for (int64_t n = 0; n < N; ++n) {
        float w_hat = oracle_mul(oracle_i2f(wq[n * K + k]), s_w);
        terms[n] = oracle_mul(dy[m * N + n], w_hat);
    }
    return oracle_canon_sum(terms, N);
}

static float dw_one(const float* dy, const int8_t* xq, float s_x, int64_t n, int64_t k,
                    int64_t M, int64_t N, int64_t K, float* terms)
{
    for (int64_t m = 0; m < M; ++m) {
        float x_hat = oracle_mul(oracle_i2f(xq[m * K + k]), s_x);
        terms[m] = oracle_mul(dy[m * N + n], x_hat);
    }
    return oracle_canon_sum(terms, M);
}

void oracle_linear_bwd_dx(const float* dy, const int8_t* wq, float s_w, float* dx,
                          int64_t M, int64_t N, int64_t K)
{
#pragma omp parallel
    {
        float* terms = (float*)malloc((size_t)(N > 0 ? N : 1) * sizeof(float));
#pragma omp for schedule(static)
        for (int64_t m = 0; m < M; ++m)
            for (int64_t k = 0; k < K; ++k)
                dx[m * K + k] = dx_one(dy, wq, s_w, m, k, N, K, terms);
        free(terms);
    }
}

void oracle_linear_bwd_dw(const float* dy, const int8_t* xq, float s_x, float* dw,
                          int64_t M, int64_t N, int64_t K)
{
#pragma omp parallel
    {
        float* terms = (float*)malloc((size_t)(M > 0 ? M : 1) * sizeof(float));
#pragma omp for schedule(static)
        for (int64_t n = 0; n < N; ++n)
            for (int64_t k = 0; k < K; ++k)
                dw[n * K + k] = dw_one(dy, xq, s_x, n, k, M, N, K, terms);
        free(terms);
    }
}

void oracle_linear_bwd_dx_at(const float* dy, const int8_t* wq, float s_w,
                             int64_t M, int64_t N, int64_t K,
                             const int64_t* idx_m, const int64_t* idx_k, int64_t cnt,
                             float* out)
{
    (void)M;
#pragma omp parallel
    {
        float* terms = (float*)malloc((size_t)(N > 0 ? N : 1) * sizeof(float));
#pragma omp for schedule(static)
        for (int64_t i = 0; i < cnt; ++i)
            out[i] = dx_one(dy, wq, s_w, idx_m[i], idx_k[i], N, K, terms);
        free(terms);
    }
}

void oracle_linear_bwd_dw_at(const float* dy, const int8_t* xq, float s_x,
                             int64_t M, int64_t N, int64_t K,
                             const int64_t* idx_n, const int64_t* idx_k, int64_t cnt,
                             float* out)
{
#pragma omp parallel
    {
        float* terms = (float*)malloc((size_t)(M > 0 ? M : 1) * sizeof(float));
#pragma omp for schedule(static)
        for (int64_t i = 0; i < cnt; ++i)
            out[i] = dw_one(dy, xq, s_x, idx_n[i], idx_k[i], M, N, K, terms);
        free(terms);
    }
}

/* ------------------------------------------------------------------------ */
/* A9: micro-batch accumulation, level 1 of the audit's three-level          */
/* reduction ([P4] "Premises and limits"): one elementwise add per           */
/* micro-batch, in micro-batch order.                                        */
/* ------------------------------------------------------------------------ */

void oracle_grad_accum(float* acc, const float* g, int64_t n)
{
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i)
        acc[i] = oracle_add(acc[i], g[i]);
}

/* ------------------------------------------------------------------------ */
/* Level 2: the intra-node reduce-scatter is replayed as a running sum in one */
/* loop over virtual ranks in mesh order, so only one partial is resident     */
/* ([P4] "Premises and limits"): a left fold in shard order, first partial    */
/* taken as it is.                                                            */
/* ------------------------------------------------------------------------ */

void oracle_running_sum(const float* const* parts, int S, int64_t n, float* out)
{
    if (S < 1)
        return;
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i) {
        float a = parts[0][i];
        for (int s = 1; s < S; ++s)
            a = oracle_add(a, parts[s][i]);
        out[i] = a;
    }
}

/* ------------------------------------------------------------------------ */
/* A10: TreeFold ([P4] "Premises and limits": the replica all-reduce is      */
/* replayed by folding partials in the pairing order of the cluster's        */
/* recursive-doubling all-reduce).  For R not a power of two the pre-step of */
/* the recursive-doubling all-reduce of Thakur, Rabenseifner and Gropp       */
/* (IJHPCA 2005) is used: with p' the largest power of two <= R and          */
/* r = R - p', ranks 2i and 2i+1 (i < r) combine first; then p' survivors    */
/* exchange with partner (rank XOR d) for d = 1, 2, ..., p'/2.  The lower    */
/* rank's operand is written first (bits do not depend on it: IEEE addition  */
/* commutes).                                                                */
/* ------------------------------------------------------------------------ */

static int pow2_floor(int R)
{
    int p = 1;
    while (p * 2 <= R)
        p *= 2;
    return p;
}

/* runs the exchange; v must hold room for p' values; returns p' */
static int rd_allreduce(const float* vals, int R, float* v)
{
    int p2 = pow2_floor(R);
    int r = R - p2;
    for (int i = 0; i < r; ++i)
        v[i] = oracle_add(vals[2 * i], vals[2 * i + 1]);
    for (int i = r; i < p2; ++i)
        v[i] = vals[r + i];
    float nv[64];
    for (int d = 1; d < p2; d *= 2) {
        for (int j = 0; j < p2; ++j) {
            int q = j ^ d;
            nv[j] = (j < q) ? oracle_add(v[j], v[q]) : oracle_add(v[q], v[j]);
        }
        memcpy(v, nv, (size_t)p2 * sizeof(float));
    }
    return p2;
}

float oracle_treefold_one(const float* vals, int R)
{
    float v[64];
    if (R < 1 || R > 64)
        return NAN;
    rd_allreduce(vals, R, v);
    return v[0];
}

void oracle_treefold_all_ranks(const float* vals, int R, float* rank_out)
{
    float v[64];
    if (R < 1 || R > 64)
        return;
    int p2 = rd_allreduce(vals, R, v);
    int r = R - p2;
    for (int q = 0; q < R; ++q) {
        int newrank = (q < 2 * r) ? q / 2 : q - r;
        rank_out[q] = v[newrank];
    }
}

void oracle_treefold(const float* const* parts, int R, int64_t n, float* out)
{
    if (R < 1 || R > 64)
        return;
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i) {
        float vals[64];
        for (int r = 0; r < R; ++r)
            vals[r] = parts[r][i];
        out[i] = oracle_treefold_one(vals, R);
    }
}

/* ------------------------------------------------------------------------ */
/* Optimiser step (see oracle.h for the fixed operation order).               */
/* ------------------------------------------------------------------------ */

float oracle_sumsq(const float* g, int64_t n)
{
    float* t = (float*)malloc((size_t)(n > 0 ? n : 1) * sizeof(float));
    for (int64_t i = 0; i < n; ++i)
        t[i] = oracle_mul(g[i], g[i]);
    float S = oracle_canon_sum(t, n);
    free(t);
    return oracle_flush(S);
}

float oracle_pow_t(float b, int64_t t)
{
    float r = 1.0f, base = b;
    while (t > 0) {
        if (t & 1)
            r = oracle_mul(r, base);
        base = oracle_mul(base, base);
        t >>= 1;
    }
    return r;
}

float oracle_clip_coef(float sumsq, float max_norm)
{
    float norm = oracle_sqrt(sumsq);
    float coef = oracle_div(max_norm, oracle_add(norm, 1e-6f));
    return coef < 1.0f ? coef : 1.0f;
}

void oracle_adamw_step(float* p, float* m, float* v, const float* g, int64_t n, float sumsq,
                       const oracle_adamw_hparams* hp, int64_t t)
{
    const float coef = oracle_clip_coef(sumsq, hp->max_norm);
    const float one_b1 = oracle_add(1.0f, -hp->beta1);
    const float one_b2 = oracle_add(1.0f, -hp->beta2);
    const float bc1 = oracle_add(1.0f, -oracle_pow_t(hp->beta1, t));
    const float bc2 = oracle_add(1.0f, -oracle_pow_t(hp->beta2, t));
    const float decay = oracle_add(1.0f, -oracle_mul(hp->lr, hp->weight_decay));
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i) {
        const float gc = oracle_mul(g[i], coef);
        const float mi = oracle_add(oracle_mul(hp->beta1, m[i]), oracle_mul(one_b1, gc));
        const float vi = oracle_add(oracle_mul(hp->beta2, v[i]),
                                    oracle_mul(one_b2, oracle_mul(gc, gc)));
        const float mh = oracle_div(mi, bc1);
        const float vh = oracle_div(vi, bc2);
        const float den = oracle_add(oracle_sqrt(vh), hp->eps);
        const float upd = oracle_mul(hp->lr, oracle_div(mh, den));
        p[i] = oracle_add(oracle_mul(p[i], decay), -upd);
        m[i] = mi;
        v[i] = vi;
    }
}

/* ------------------------------------------------------------------------ */
/* Attention with int8 P.V ([P4] "How to use": inside flash attention the    */
/* P.V product runs on int8 while the QK^T logits and the softmax stay in    */
/* high precision; the attention backward accumulates dQ in 64-bit fixed     */
/* point).  The pages fix no operation order; the readings taken here:       */
/*   logits  s_ij = canon_d(q_id (x) k_jd) (x) c, c = 1 (/) sqrt(D);         */
/*   keys    j in [lo_i, i], lo_i = max(0, i - W + 1) for a sliding window  */
/*           of W tokens, 0 for W = 0 (full causal); GQA: query head h      */
/*           reads kv head h / (Hq / Hkv);                                   */
/*   m_i     = max_j s_ij (exact, so the softmax is taken in two passes);    */
/*   p_ij    = exp_r(s_ij (-) m_i), l_i = canon_j(p_ij) over j ascending;    */
/*   int8 P  P_ij = clamp(rint(p_ij (x) 127), 0, 127); V = V_q with scale s_v;*/
/*   o_id    = (i2f(sum_j P_ij V_q,jd) (x) s_v) (/) (l_i (x) 127), the       */
/*           integer sum exact.                                              */
/* Layout: q, o [B][T][Hq][D]; k, v [B][T][Hkv][D]; m, l [B][T][Hq].         */
/* ------------------------------------------------------------------------ */

/* e^x: range reduction of Cody and Waite ("Software Manual for the          */
/* Elementary Functions", 1980) with ln 2 split as C1 + C2, C1 = 355/512     */
/* (exact in 9 bits, so k (x) C1 is exact), then the degree-7 Taylor         */
/* polynomial of e^r in Horner form with binary32 coefficients RN(1/n!),     */
/* then the exact scaling by 2^k; every operation rounded and flushed.       */
#define EXP_LOG2E 0x1.715476p+0f   /* RN(1/ln 2) */
#define EXP_C1 0x1.63p-1f            /* 355/512 */
#define EXP_C2 -0x1.bd0106p-13f      /* RN(ln 2 - 355/512) */

float oracle_exp(float x)
{
    const float kf = nearbyintf(oracle_mul(x, EXP_LOG2E)); /* ties to even */
    const float r = oracle_add(oracle_add(x, -oracle_mul(kf, EXP_C1)), -oracle_mul(kf, EXP_C2));
    /* RN(1/n!), n = 0..7 */
    static const float c[8] = {1.0f, 1.0f, 0.5f, 0x1.555556p-3f, 0x1.555556p-5f, 0x1.111112p-7f,
                               0x1.6c16c2p-10f, 0x1.a01a02p-13f};
    float p = c[7];
    for (int n = 6; n >= 0; --n)
        p = oracle_add(oracle_mul(p, r), c[n]);
    if (kf < -126.0f)
        return 0.0f;
    if (kf > 254.0f)
        return INFINITY; /* 2^k alone overflows, whatever p is (so e^+inf = +inf) */
    if (kf != kf)
        return kf; /* NaN */
    return oracle_flush(ldexpf(p, (int)kf));
}

static float attn_c(int64_t D)
{
    return oracle_div(1.0f, oracle_sqrt((float)D));
}

static int64_t attn_lo(int64_t i, int64_t W)
{
    return (W > 0 && i - W + 1 > 0) ? i - W + 1 : 0;
}

static float attn_logit(const float* q, const float* k, int64_t b, int64_t i, int64_t j,
                        int64_t h, int64_t g, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                        float c, float* tmp)
{
    const float* qi = q + ((b * T + i) * Hq + h) * D;
    const float* kj = k + ((b * T + j) * Hkv + g) * D;
    for (int64_t d = 0; d < D; ++d)
        tmp[d] = oracle_mul(qi[d], kj[d]);
    return oracle_mul(oracle_canon_sum(tmp, D), c);
}

int oracle_attn_quant_p(float p)
{
    float r = nearbyintf(oracle_mul(p, 127.0f));
    if (r != r)
        return 0; /* NaN: the clamp's lower bound */
    if (r > 127.0f)
        r = 127.0f;
    if (r < 0.0f)
        r = 0.0f;
    return (int)r;
}

/* one query row: o[D], m, l */
static void attn_fwd_row(const float* q, const float* k, const int8_t* vq, float s_v,
                         int64_t b, int64_t i, int64_t h, int64_t T, int64_t Hq, int64_t Hkv,
                         int64_t D, int64_t W, float* o, float* m_out, float* l_out)
{
    const int64_t g = h / (Hq / Hkv), lo = attn_lo(i, W), n = i - lo + 1;
    const float c = attn_c(D);
    float* s = (float*)malloc((size_t)n * sizeof(float));
    float* tmp = (float*)malloc((size_t)(D > n ? D : n) * sizeof(float));
    int64_t* acc = (int64_t*)calloc((size_t)D, sizeof(int64_t));
    float m = -INFINITY; /* the maximum of no logit */
    for (int64_t t = 0; t < n; ++t) {
        s[t] = attn_logit(q, k, b, i, lo + t, h, g, T, Hq, Hkv, D, c, tmp);
        if (s[t] > m) /* a NaN logit never compares greater: it is passed over */
            m = s[t];
    }
    if (m == 0.0f)
        m = 0.0f; /* a zero maximum is stored as +0 */
    for (int64_t t = 0; t < n; ++t) {
        const float p = oracle_exp(oracle_add(s[t], -m));
        tmp[t] = p;
        const int pq = oracle_attn_quant_p(p);
        const int8_t* vj = vq + ((b * T + lo + t) * Hkv + g) * D;
        for (int64_t d = 0; d < D; ++d)
            acc[d] += (int64_t)pq * vj[d];
    }
    const float l = oracle_canon_sum(tmp, n);
    const float den = oracle_mul(l, 127.0f);
    for (int64_t d = 0; d < D; ++d)
        o[d] = oracle_div(oracle_mul(oracle_i2f(acc[d]), s_v), den);
    *m_out = m;
    *l_out = l;
    free(s);
    free(tmp);
    free(acc);
}

void oracle_attn_fwd(const float* q, const float* k, const int8_t* vq, float s_v, float* o,
                     float* mrow, float* lrow, int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                     int64_t D, int64_t W)
{
#pragma omp parallel for schedule(dynamic, 16)
    for (int64_t r = 0; r < B * T * Hq; ++r) {
        const int64_t h = r % Hq, bi = r / Hq, i = bi % T, b = bi / T;
        attn_fwd_row(q, k, vq, s_v, b, i, h, T, Hq, Hkv, D, W, o + r * D, mrow + r, lrow + r);
    }
}

void oracle_attn_fwd_rows(const float* q, const float* k, const int8_t* vq, float s_v,
                          const int64_t* rows, int64_t nrows, float* o, float* mrow,
                          float* lrow, int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                          int64_t D, int64_t W)
{
#pragma omp parallel for schedule(dynamic, 1)
    for (int64_t t = 0; t < nrows; ++t) {
        const int64_t r = rows[t];
        const int64_t h = r % Hq, bi = r / Hq, i = bi % T, b = bi / T;
        attn_fwd_row(q, k, vq, s_v, b, i, h, T, Hq, Hkv, D, W, o + t * D, mrow + t, lrow + t);
    }
}

/* Backward (straight-through for both quantisations):                        */
/*   a_ij  = p_ij (/) l_i, p_ij recomputed as in the forward from m_i;        */
/*   V^_jd = i2f(V_q,jd) (x) s_v;  Dr_i = canon_d(dO_id (x) O_id);            */
/*   dA_ij = canon_d(dO_id (x) V^_jd);  dS_ij = a_ij (x) (dA_ij (-) Dr_i);    */
/*   dQ_id = (fix2f(sum over key tiles t of fx(T_t))) (x) c, where T_t is the */
/*     left-to-right sum over the valid keys j of the 64-aligned key tile t   */
/*     of dS_ij (x) k_jd (seeded with the first such term), fx(x) = the       */
/*     nearest int64 to x * 2^48 (ties to even, saturating, NaN to 0) and     */
/*     fix2f(A) = flush(i2f(A) * 2^-48): the tile partials are accumulated in */
/*     64-bit fixed point, exactly and in any order (the int64 sum wraps      */
/*     modulo 2^64 where saturated partials overflow it);                     */
/*   dK_jd = (fold) (x) c and dV_jd = (fold), where the terms dS_ij (x) q_id  */
/*     (dK) and a_ij (x) dO_id (dV) run over the query heads h of kv head g   */
/*     in ascending order and, within a head, over the valid queries i;       */
/*     they are grouped by 64-aligned query tile, each group summed left to   */
/*     right from its first term, and the group partials folded left in      */
/*     (head, tile) order.                                                    */
#define ATTN_FIX_BITS 48
#define ATTN_TILE 64

int64_t oracle_attn_fx(float x)
{
    const double v = nearbyint((double)oracle_flush(x) * 281474976710656.0); /* exact */
    if (v != v)
        return 0; /* NaN */
    if (v >= 9223372036854775807.0)
        return INT64_MAX;
    if (v <= -9223372036854775808.0)
        return INT64_MIN;
    return (int64_t)v;
}

float oracle_attn_fix2f(int64_t a)
{
    return oracle_flush(oracle_i2f(a) * (1.0f / 281474976710656.0f)); /* exact but for the flush */
}

static float attn_drow(const float* o, const float* dout, int64_t r, int64_t D, float* tmp)
{
    for (int64_t d = 0; d < D; ++d)
        tmp[d] = oracle_mul(dout[r * D + d], o[r * D + d]);
    return oracle_canon_sum(tmp, D);
}

/* a_ij and dS_ij for one (query row, key) pair */
static void attn_pair(const float* q, const float* k, const int8_t* vq, float s_v,
                      const float* dout, const float* mrow, const float* lrow, float drow,
                      int64_t b, int64_t i, int64_t j, int64_t h, int64_t g, int64_t T,
                      int64_t Hq, int64_t Hkv, int64_t D, float c, float* tmp, float* a_out,
                      float* ds_out)
{
    const int64_t r = (b * T + i) * Hq + h;
    const float s = attn_logit(q, k, b, i, j, h, g, T, Hq, Hkv, D, c, tmp);
    const float a = oracle_div(oracle_exp(oracle_add(s, -mrow[r])), lrow[r]);
    const int8_t* vj = vq + ((b * T + j) * Hkv + g) * D;
    for (int64_t d = 0; d < D; ++d)
        tmp[d] = oracle_mul(dout[r * D + d], oracle_mul(oracle_i2f(vj[d]), s_v));
    const float dA = oracle_canon_sum(tmp, D);
    *a_out = a;
    *ds_out = oracle_mul(a, oracle_add(dA, -drow));
}

static void attn_dq_row(const float* q, const float* k, const int8_t* vq, float s_v,
                        const float* o, const float* dout, const float* mrow, const float* lrow,
                        int64_t b, int64_t i, int64_t h, int64_t T, int64_t Hq, int64_t Hkv,
                        int64_t D, int64_t W, float* dq)
{
    const int64_t g = h / (Hq / Hkv), lo = attn_lo(i, W), r = (b * T + i) * Hq + h;
    const float c = attn_c(D);
    float* tmp = (float*)malloc((size_t)D * sizeof(float));
    float* part = (float*)malloc((size_t)D * sizeof(float));
    uint64_t* acc = (uint64_t*)calloc((size_t)D, sizeof(uint64_t)); /* wraps modulo 2^64 */
    const float drow = attn_drow(o, dout, r, D, tmp);
    for (int64_t t0 = (lo / ATTN_TILE) * ATTN_TILE; t0 <= i; t0 += ATTN_TILE) {
        const int64_t jb = t0 > lo ? t0 : lo, je = t0 + ATTN_TILE - 1 < i ? t0 + ATTN_TILE - 1 : i;
        for (int64_t j = jb; j <= je; ++j) {
            float a, ds;
            attn_pair(q, k, vq, s_v, dout, mrow, lrow, drow, b, i, j, h, g, T, Hq, Hkv, D, c,
                      tmp, &a, &ds);
            const float* kj = k + ((b * T + j) * Hkv + g) * D;
            for (int64_t d = 0; d < D; ++d) {
                const float t = oracle_mul(ds, kj[d]);
                part[d] = j == jb ? t : oracle_add(part[d], t);
            }
        }
        for (int64_t d = 0; d < D; ++d)
            acc[d] += (uint64_t)oracle_attn_fx(part[d]);
    }
    for (int64_t d = 0; d < D; ++d) {
        int64_t a;
        memcpy(&a, &acc[d], sizeof a); /* the two's-complement value */
        dq[d] = oracle_mul(oracle_attn_fix2f(a), c);
    }
    free(tmp);
    free(part);
    free(acc);
}

static void attn_dkdv_row(const float* q, const float* k, const int8_t* vq, float s_v,
                          const float* o, const float* dout, const float* mrow,
                          const float* lrow, int64_t b, int64_t j, int64_t g, int64_t T,
                          int64_t Hq, int64_t Hkv, int64_t D, int64_t W, float* dk, float* dv)
{
    const int64_t G = Hq / Hkv;
    const float c = attn_c(D);
    const int64_t ihi = (W > 0 && j + W - 1 < T - 1) ? j + W - 1 : T - 1;
    float* tmp = (float*)malloc((size_t)D * sizeof(float));
    float* pk = (float*)malloc((size_t)D * sizeof(float));
    float* pv = (float*)malloc((size_t)D * sizeof(float));
    float* fk = (float*)malloc((size_t)D * sizeof(float));
    float* fv = (float*)malloc((size_t)D * sizeof(float));
    int first_group = 1;
    for (int64_t hh = 0; hh < G; ++hh) {
        const int64_t h = g * G + hh;
        for (int64_t t0 = (j / ATTN_TILE) * ATTN_TILE; t0 <= ihi; t0 += ATTN_TILE) {
            const int64_t ib = t0 > j ? t0 : j;
            const int64_t ie = t0 + ATTN_TILE - 1 < ihi ? t0 + ATTN_TILE - 1 : ihi;
            for (int64_t i = ib; i <= ie; ++i) {
                const int64_t r = (b * T + i) * Hq + h;
                const float drow = attn_drow(o, dout, r, D, tmp);
                float a, ds;
                attn_pair(q, k, vq, s_v, dout, mrow, lrow, drow, b, i, j, h, g, T, Hq, Hkv, D,
                          c, tmp, &a, &ds);
                const float* qi = q + r * D;
                const float* di = dout + r * D;
                for (int64_t d = 0; d < D; ++d) {
                    const float tk = oracle_mul(ds, qi[d]);
                    const float tv = oracle_mul(a, di[d]);
                    pk[d] = i == ib ? tk : oracle_add(pk[d], tk);
                    pv[d] = i == ib ? tv : oracle_add(pv[d], tv);
                }
            }
            for (int64_t d = 0; d < D; ++d) {
                fk[d] = first_group ? pk[d] : oracle_add(fk[d], pk[d]);
                fv[d] = first_group ? pv[d] : oracle_add(fv[d], pv[d]);
            }
            first_group = 0;
        }
    }
    for (int64_t d = 0; d < D; ++d) {
        dk[d] = oracle_mul(fk[d], c);
        dv[d] = fv[d];
    }
    free(tmp);
    free(pk);
    free(pv);
    free(fk);
    free(fv);
}

void oracle_attn_bwd(const float* q, const float* k, const int8_t* vq, float s_v, const float* o,
                     const float* dout, const float* mrow, const float* lrow, float* dq, float* dk,
                     float* dv, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                     int64_t W)
{
#pragma omp parallel for schedule(dynamic, 4)
    for (int64_t r = 0; r < B * T * Hq; ++r) {
        const int64_t h = r % Hq, bi = r / Hq, i = bi % T, b = bi / T;
        attn_dq_row(q, k, vq, s_v, o, dout, mrow, lrow, b, i, h, T, Hq, Hkv, D, W, dq + r * D);
    }
#pragma omp parallel for schedule(dynamic, 4)
    for (int64_t r = 0; r < B * T * Hkv; ++r) {
        const int64_t g = r % Hkv, bj = r / Hkv, j = bj % T, b = bj / T;
        attn_dkdv_row(q, k, vq, s_v, o, dout, mrow, lrow, b, j, g, T, Hq, Hkv, D, W, dk + r * D,
                      dv + r * D);
    }
}

/* sampled rows: dq for query rows qrows[] (flat (b, i, h) indices), dk/dv for
 * key rows krows[] (flat (b, j, g) indices) */
void oracle_attn_bwd_rows(const float* q, const float* k, const int8_t* vq, float s_v,
                          const float* o, const float* dout, const float* mrow,
                          const float* lrow, const int64_t* qrows, int64_t nq, float* dq,
                          const int64_t* krows, int64_t nk, float* dk, float* dv, int64_t B,
                          int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t W)
{
#pragma omp parallel for schedule(dynamic, 1)
    for (int64_t t = 0; t < nq; ++t) {
        const int64_t r = qrows[t];
        const int64_t h = r % Hq, bi = r / Hq, i = bi % T, b = bi / T;
        attn_dq_row(q, k, vq, s_v, o, dout, mrow, lrow, b, i, h, T, Hq, Hkv, D, W, dq + t * D);
    }
#pragma omp parallel for schedule(dynamic, 1)
    for (int64_t t = 0; t < nk; ++t) {
        const int64_t r = krows[t];
        const int64_t g = r % Hkv, bj = r / Hkv, j = bj % T, b = bj / T;
        attn_dkdv_row(q, k, vq, s_v, o, dout, mrow, lrow, b, j, g, T, Hq, Hkv, D, W, dk + t * D,
                      dv + t * D);
    }
}

int oracle_threads(void)
{
#ifdef _OPENMP
    return omp_get_max_threads();
#else
    return 1;
#endif
}

/* threads for the parallel loops over output elements from now on (n >= 1);
 * no element's sequence of operations depends on it */
void oracle_set_threads(int n)
{
#ifdef _OPENMP
    if (n >= 1)
        omp_set_num_threads(n);
#else
    (void)n;
#endif
}

/* ------------------------------------------------------------------------ */
/* The operators around the decoder blocks: token embedding, per-head norm of */
/* queries and keys with the position rotation, and the loss against a        */
/* teacher's top logits.  The pages name the model's parts and fix no order;  */
/* the definitions are those of include/repro.h.                              */
/* ------------------------------------------------------------------------ */

/* pairwise tree with stride doubling over n values, in place; n = 0 gives +0 */
static float tree_inplace(float* t, int64_t n)
{
    for (int64_t s = 1; s < n; s *= 2)
        for (int64_t j = 0; j + s < n; j += 2 * s)
            t[j] = oracle_add(t[j], t[j + s]);
    return n > 0 ? t[0] : 0.0f;
}

/* ---- embedding ---------------------------------------------------------- */

void oracle_embed_fwd(const float* W, const int8_t* Wq, float s_w, const int64_t* tok, int64_t n,
                      int64_t V, int64_t D, float scale, int64_t pad, float* out)
{
    for (int64_t i = 0; i < n; ++i) {
        const int ok = tok[i] >= 0 && tok[i] < V && tok[i] != pad;
        for (int64_t d = 0; d < D; ++d) {
            float w = 0.0f;
            if (ok)
                w = W ? oracle_flush(W[tok[i] * D + d]) : oracle_mul((float)Wq[tok[i] * D + d], s_w);
            out[i * D + d] = ok ? oracle_mul(w, scale) : 0.0f;
        }
    }
}

void oracle_embed_bwd(const float* dout, const int64_t* tok, int64_t n, int64_t V, int64_t D,
                      float scale, int64_t pad, int accumulate, float* dW)
{
#pragma omp parallel
    {
        float* terms = (float*)malloc(sizeof(float) * (size_t)(n > 0 ? n : 1));
        int64_t* rows = (int64_t*)malloc(sizeof(int64_t) * (size_t)(n > 0 ? n : 1));
#pragma omp for schedule(dynamic, 16)
        for (int64_t v = 0; v < V; ++v) {
            int64_t L = 0;
            for (int64_t i = 0; i < n; ++i)
                if (tok[i] == v && v != pad)
                    rows[L++] = i;
            for (int64_t d = 0; d < D; ++d) {
                for (int64_t j = 0; j < L; ++j)
                    terms[j] = dout[rows[j] * D + d];
                float* w = dW + v * D + d;
                if (L > 0) {
                    const float g = oracle_mul(oracle_canon_sum(terms, L), scale);
                    *w = accumulate ? oracle_add(*w, g) : g;
                } else if (!accumulate) {
                    *w = 0.0f;
                }
            }
        }
        free(terms);
        free(rows);
    }
}

/* ---- norm of every head and the rotation -------------------------------- */

/* groups of 4 consecutive terms left to right, the group sums by the tree */
static float sum4_tree(const float* t, int64_t D)
{
    float g[128];
    const int64_t G = (D + 3) / 4;
    for (int64_t k = 0; k < G; ++k) {
        float s = oracle_flush(t[4 * k]);
        for (int64_t d = 4 * k + 1; d < D && d < 4 * k + 4; ++d)
            s = oracle_add(s, t[d]);
        g[k] = s;
    }
    return tree_inplace(g, G);
}

static float head_rnorm(const float* x, int64_t D, float eps)
{
    float t[512];
    for (int64_t d = 0; d < D; ++d)
        t[d] = oracle_mul(x[d], x[d]);
    return oracle_div(1.0f, oracle_sqrt(oracle_add(oracle_div(sum4_tree(t, D), (float)D), eps)));
}

/* the two members of rotation pair j */
static void pair_of(int64_t j, int64_t R, int interleaved, int64_t* a, int64_t* b)
{
    *a = interleaved ? 2 * j : j;
    *b = interleaved ? 2 * j + 1 : j + R / 2;
}

void oracle_qk_fwd(const float* x, const float* rope, const int32_t* pos, int64_t P, const float* gain,
                   float eps, int interleaved, int64_t n, int64_t H, int64_t D, int64_t R, float* out)
{
#pragma omp parallel for schedule(static)
    for (int64_t u = 0; u < n * H; ++u) {
        const float* xr = x + u * D;
        float* o = out + u * D;
        const int64_t p = pos[u / H];
        if (p < 0 || p >= P) {
            for (int64_t d = 0; d < D; ++d)
                o[d] = 0.0f;
            continue;
        }
        const float r = head_rnorm(xr, D, eps);
        for (int64_t d = 0; d < D; ++d) {
            o[d] = oracle_mul(xr[d], r);
            if (gain)
                o[d] = oracle_mul(o[d], gain[d]);
        }
        for (int64_t j = 0; j < R / 2; ++j) {
            int64_t a, b;
            pair_of(j, R, interleaved, &a, &b);
            const float c = rope[p * R + j], s = rope[p * R + R / 2 + j], ya = o[a], yb = o[b];
            o[a] = oracle_add(oracle_mul(ya, c), -oracle_mul(yb, s));
            o[b] = oracle_add(oracle_mul(yb, c), oracle_mul(ya, s));
        }
    }
}

/* dx, and dg (when gain) = canonical sum over the rows (token, head) ascending */
void oracle_qk_bwd(const float* dout, const float* x, const float* rope, const int32_t* pos, int64_t P,
                   const float* gain, float eps, int interleaved, int64_t n, int64_t H, int64_t D,
                   int64_t R, float* dx, float* dg, int accumulate)
{
    float* gt = gain ? (float*)malloc(sizeof(float) * (size_t)(n * H * D + 1)) : NULL;
#pragma omp parallel for schedule(static)
    for (int64_t u = 0; u < n * H; ++u) {
        const float *xr = x + u * D, *dr = dout + u * D;
        const int64_t p = pos[u / H];
        float dy[512], xh[512], t[512];
        if (p < 0 || p >= P) {
            for (int64_t d = 0; d < D; ++d) {
                dx[u * D + d] = 0.0f;
                if (gt)
                    gt[d * n * H + u] = 0.0f;
            }
            continue;
        }
        const float r = head_rnorm(xr, D, eps);
        for (int64_t d = 0; d < D; ++d) {
            dy[d] = oracle_flush(dr[d]);
            xh[d] = oracle_mul(xr[d], r);
        }
        for (int64_t j = 0; j < R / 2; ++j) {
            int64_t a, b;
            pair_of(j, R, interleaved, &a, &b);
            const float c = rope[p * R + j], s = rope[p * R + R / 2 + j], da = dr[a], db = dr[b];
            dy[a] = oracle_add(oracle_mul(da, c), oracle_mul(db, s));
            dy[b] = oracle_add(oracle_mul(db, c), -oracle_mul(da, s));
        }
        for (int64_t d = 0; d < D; ++d) {
            if (gt)
                gt[d * n * H + u] = oracle_mul(dy[d], xh[d]);
            if (gain)
                dy[d] = oracle_mul(dy[d], gain[d]);
            t[d] = oracle_mul(dy[d], xh[d]);
        }
        const float c1 = oracle_div(sum4_tree(t, D), (float)D);
        for (int64_t d = 0; d < D; ++d)
            dx[u * D + d] = oracle_mul(r, oracle_add(dy[d], -oracle_mul(xh[d], c1)));
    }
    if (gt) {
        for (int64_t d = 0; d < D; ++d) {
            const float s = oracle_canon_sum(gt + d * n * H, n * H);
            dg[d] = accumulate ? oracle_add(dg[d], s) : s;
        }
        free(gt);
    }
}

/* ---- loss against a teacher's top logits -------------------------------- */

#define DISTILL_BLOCK 1024
#define DISTILL_CHAINS 128
#define DISTILL_STATS 8

/* 2^t for t <= 0: t = k / 32 + f, k = rint(32 t); the degree-2 minimax polynomial
 * of 2^f on [-1/64, 1/64] (relative error 5.4e-8, constant term 1; coefficients by
 * the exchange algorithm of Remez, rounded to binary32) times RN(2^((k mod 32) / 32))
 * 2^floor(k / 32); 0 where floor(k / 32) < -125 */
float oracle_exp2_neg(float t)
{
    static const float c[3] = {1.0f, 0x1.62e586p-1f, 0x1.ebfeacp-3f};
    if (t != t)
        return t;
    if (t < -126.0f)
        return 0.0f;
    const float k32 = nearbyintf(oracle_mul(32.0f, t));
    const int k = (int)floorf(k32 / 32.0f), j = (int)k32 - 32 * k;
    if (k < -125)
        return 0.0f;
    const float f = oracle_add(t, -(k32 / 32.0f));
    float p = c[2];
    for (int i = 1; i >= 0; --i)
        p = oracle_add(oracle_mul(p, f), c[i]);
    return oracle_mul(p, ldexpf((float)exp2((double)j / 32.0), k));
}

/* e^x for x <= 0 */
static float exp_neg(float x) { return oracle_exp2_neg(oracle_mul(x, EXP_LOG2E)); }

/* ln of a positive binary32 value in binary64: x = m 2^e with m in
 * [sqrt(1/2), sqrt(2)), ln m = 2 atanh((m - 1) / (m + 1)) by its power series
 * to the 21st power, in Horner form; NaN for anything else */
double oracle_ln(float x)
{
    if (!(x > 0.0f) || x > FLT_MAX)
        return (double)NAN;
    int e;
    double m = frexp((double)x, &e); /* [1/2, 1) */
    if (m < 0.70710678118654752440) {
        m *= 2.0;
        e -= 1;
    }
    const double s = (m - 1.0) / (m + 1.0), w = s * s;
    double p = 1.0 / 21.0;
    for (int k = 19; k >= 1; k -= 2)
        p = p * w + 1.0 / (double)k;
    return (double)e * 0.69314718055994530942 + (2.0 * s) * p;
}

static float max_nan(float a, float b)
{
    if (a != a || b != b)
        return NAN;
    if (a == 0.0f && b == 0.0f)
        return 0.0f;
    return a > b ? a : b;
}

/* chain i sums the terms j = i (mod chains) ascending from +0; tree over chains */
static float chains_sum(const float* t, int64_t n, int chains)
{
    float s[DISTILL_CHAINS];
    for (int i = 0; i < chains; ++i) {
        s[i] = 0.0f;
        for (int64_t j = i; j < n; j += chains)
            s[i] = oracle_add(s[i], t[j]);
    }
    return tree_inplace(s, chains);
}

static double chains_sum_d(const double* t, int64_t n, int chains)
{
    double s[DISTILL_CHAINS];
    for (int i = 0; i < chains; ++i) {
        s[i] = 0.0;
        for (int64_t j = i; j < n; j += chains)
            s[i] += t[j];
    }
    for (int st = 1; st < chains; st *= 2)
        for (int j = 0; j + st < chains; j += 2 * st)
            s[j] += s[j + st];
    return s[0];
}

/* x (x) it (-) m (x) it, the argument of e(.); the difference first where m (x) it overflows */
static float scaled_diff(float x, float m, float it)
{
    const float mu = oracle_mul(m, it);
    if (isinf(mu) && !isinf(m))
        return oracle_mul(oracle_add(x, -m), it);
    return oracle_add(oracle_mul(x, it), -mu);
}

/* the softmax-of-z term e^(z - m) from the softened one where tau is 2 or 4 */
static float term_power(float e, float tau)
{
    e = oracle_mul(e, e);
    return tau == 4.0f ? oracle_mul(e, e) : e;
}

/* max and sum of e^(it z - it max) over a row, block by block; with tau 2 or 4 (and
 * it = 1 / tau) the blocks' sums are of e^(z - max) as a power of that, joined with it = 1 */
static float row_sum(const float* z, int64_t V, float it, float tau, float* mx)
{
    const int64_t C = (V + DISTILL_BLOCK - 1) / DISTILL_BLOCK;
    float* S = (float*)malloc(sizeof(float) * (size_t)C);
    float* M = (float*)malloc(sizeof(float) * (size_t)C);
    float t[DISTILL_BLOCK], m = -INFINITY;
    for (int64_t c = 0; c < C; ++c) {
        const int64_t lo = c * DISTILL_BLOCK, n = V - lo < DISTILL_BLOCK ? V - lo : DISTILL_BLOCK;
        M[c] = -INFINITY;
        for (int64_t j = 0; j < n; ++j)
            M[c] = max_nan(M[c], oracle_flush(z[lo + j]));
        M[c] = M[c] == 0.0f ? 0.0f : M[c]; /* a zero maximum is +0 */
        for (int64_t j = 0; j < n; ++j)
            t[j] = exp_neg(scaled_diff(z[lo + j], M[c], it));
        if (tau != 0.0f)
            for (int64_t j = 0; j < n; ++j)
                t[j] = term_power(t[j], tau);
        S[c] = M[c] == -INFINITY ? 0.0f : chains_sum(t, n, DISTILL_CHAINS);
        m = max_nan(m, M[c]);
    }
    m = m == 0.0f ? 0.0f : m;
    *mx = m;
    float l = 0.0f;
    if (tau != 0.0f)
        it = 1.0f;
    if (m != -INFINITY) {
        for (int64_t c = 0; c < C; ++c)
            S[c] = oracle_mul(S[c], exp_neg(scaled_diff(M[c], m, it)));
        l = chains_sum(S, C, 32);
    }
    free(S);
    free(M);
    return l;
}

/* v (x) it for the loss's binary64 terms: in binary64 itself where binary32 overflows */
static double wide_mul(float v, float it)
{
    const float p = oracle_mul(v, it);
    return isinf(p) && !isinf(v) ? (double)v * (double)it : (double)p;
}

/* whether entry j names a logit of the row */
static int in_row(int64_t j, int64_t V) { return j >= 0 && j < V; }

void oracle_distill_fwd(const float* z, int64_t n, int64_t V, const int64_t* idx, const float* tl,
                        int64_t K, const int64_t* label, float tau, float w_kd, float w_ce, float w_z,
                        int logprobs, float* loss, float* stats)
{
    const float it = oracle_div(1.0f, tau);
#pragma omp parallel for schedule(dynamic, 1)
    for (int64_t r = 0; r < n; ++r) {
        const float* zr = z + r * V;
        float* st = stats + r * (DISTILL_STATS + K);
        float* p = st + DISTILL_STATS;
        float mz, m1;
        const int power = tau == 2.0f || tau == 4.0f;
        const float l = row_sum(zr, V, it, 0.0f, &mz);
        const float l1 = power ? row_sum(zr, V, it, tau, &m1) : row_sum(zr, V, 1.0f, 0.0f, &m1);
        /* the teacher's weights; t_k, or a_k = t_k (x) it */
        const float ta = logprobs ? 1.0f : it;
        float most = -INFINITY, mt, lt = 0.0f, P = 0.0f;
        float* t = (float*)malloc(sizeof(float) * (size_t)(K + 1));
        for (int64_t k = 0; k < K; ++k) {
            t[k] = in_row(idx[r * K + k], V) ? oracle_flush(tl[r * K + k]) : -INFINITY;
            most = max_nan(most, t[k]);
        }
        if (logprobs)
            most = 0.0f;
        mt = oracle_mul(most, ta);
        mt = mt == 0.0f ? 0.0f : mt;
        double* term = (double*)malloc(sizeof(double) * (size_t)(K + 1));
        if (most == -INFINITY) {
            for (int64_t k = 0; k < K; ++k)
                p[k] = 0.0f;
        } else {
            for (int64_t k = 0; k < K; ++k) {
                const float x = scaled_diff(t[k], most, ta);
                p[k] = !in_row(idx[r * K + k], V) ? 0.0f : x > 88.0f ? INFINITY : exp_neg(x);
            }
            lt = chains_sum(p, K, 32);
            if (logprobs) {
                P = lt;
                lt = 1.0f;
            } else {
                for (int64_t k = 0; k < K; ++k)
                    if (in_row(idx[r * K + k], V)) /* an empty entry's weight stays +0 */
                        p[k] = oracle_div(p[k], lt);
                P = lt == lt ? 1.0f : lt;
            }
        }
        const double Mu = wide_mul(mz, it), ln_l = oracle_ln(l), ln_l1 = oracle_ln(l1);
        const double lse_t = Mu + ln_l, lse1 = (double)mz + ln_l1;
        double v = 0.0;
        if (mz != -INFINITY) {
            if (w_kd != 0.0f && most != -INFINITY) {
                float ref = -INFINITY; /* the largest logit that has weight */
                for (int64_t k = 0; k < K; ++k) {
                    term[k] = 0.0;
                    if (p[k] != 0.0f) {
                        const float zk = oracle_flush(zr[idx[r * K + k]]);
                        term[k] = (double)p[k] * ((double)oracle_mul(t[k], ta) - (double)oracle_mul(zk, it));
                        ref = max_nan(ref, zk);
                    }
                }
                double sum = chains_sum_d(term, K, 32), rest = lse_t - ((double)mt + oracle_ln(lt));
                if (isfinite(ref) && !(fabsf(mt) < 0x1p30f && fabs(sum) < 0x1p30)) {
                    /* far from zero: differences from the largest on both sides */
                    for (int64_t k = 0; k < K; ++k)
                        if (p[k] != 0.0f)
                            term[k] = (double)p[k] * ((wide_mul(t[k], ta) - wide_mul(most, ta)) -
                                                      (wide_mul(zr[idx[r * K + k]], it) - wide_mul(ref, it)));
                    sum = chains_sum_d(term, K, 32);
                    rest = ((Mu - wide_mul(ref, it)) + ln_l) - oracle_ln(lt);
                }
                for (int64_t k = 0; k < K; ++k)
                    term[k] = (double)p[k];
                v = ((double)w_kd * ((double)tau * (double)tau)) * (sum + rest * chains_sum_d(term, K, 32));
            }
            if (w_ce != 0.0f && in_row(label[r], V)) {
                const double zl = (double)oracle_flush(zr[label[r]]);
                v = v + (double)w_ce * (fabsf(mz) < 0x1p30f ? lse1 - zl : ((double)mz - zl) + ln_l1);
            }
            if (w_z != 0.0f)
                v = v + (double)w_z * (lse1 * lse1);
        }
        const int need1 = w_ce != 0.0f || w_z != 0.0f || tau == 1.0f;
        loss[r] = oracle_flush((float)v);
        st[0] = mz;
        st[1] = l;
        st[2] = mz == -INFINITY ? mz : oracle_flush((float)lse_t);
        st[3] = need1 ? l1 : 0.0f;
        st[4] = !need1 ? 0.0f : mz == -INFINITY ? mz : oracle_flush((float)lse1);
        st[5] = mt;
        st[6] = lt;
        st[7] = P;
        free(t);
        free(term);
    }
}

void oracle_distill_bwd(const float* z, int64_t n, int64_t V, const int64_t* idx, int64_t K,
                        const int64_t* label, const float* stats, const float* g, int64_t g_stride,
                        float tau, float w_kd, float w_ce, float w_z, float* dz)
{
    const float it = oracle_div(1.0f, tau);
#pragma omp parallel for schedule(dynamic, 1)
    for (int64_t r = 0; r < n; ++r) {
        const float *zr = z + r * V, *st = stats + r * (DISTILL_STATS + K), *p = st + DISTILL_STATS;
        float* d = dz + r * V;
        if (st[0] == -INFINITY) {
            for (int64_t j = 0; j < V; ++j)
                d[j] = 0.0f;
            continue;
        }
        const float gr = g[r * g_stride];
        const int lab = w_ce != 0.0f && label[r] >= 0 && label[r] < V;
        const float gk = oracle_mul(oracle_mul(gr, w_kd), tau);
        const float a = w_kd != 0.0f ? oracle_mul(gk, st[7]) : gk;
        const float b = oracle_mul(gr, oracle_add(lab ? w_ce : 0.0f,
                                                  oracle_mul(oracle_mul(2.0f, w_z), w_z != 0.0f ? st[4] : 0.0f)));
        const int two = tau != 1.0f && (w_ce != 0.0f || w_z != 0.0f);
        const float ca = tau == 1.0f ? oracle_div(oracle_add(a, b), st[1]) : oracle_div(a, st[1]);
        const float cb = two ? oracle_div(b, st[3]) : 0.0f;
        for (int64_t j = 0; j < V; ++j) {
            const float e = exp_neg(scaled_diff(zr[j], st[0], it));
            d[j] = oracle_mul(e, ca);
            if (two)
                d[j] = oracle_add(d[j], oracle_mul(tau == 2.0f || tau == 4.0f ? term_power(e, tau)
                                                                              : exp_neg(oracle_add(zr[j], -st[0])), cb));
        }
        if (w_kd != 0.0f)
            for (int64_t k = 0; k < K; ++k) {
                const int64_t j = idx[r * K + k];
                if (j >= 0 && j < V)
                    d[j] = oracle_add(d[j], -oracle_mul(gk, p[k]));
            }
        if (lab)
            d[label[r]] = oracle_add(d[label[r]], -oracle_mul(gr, w_ce));
    }
}

/* ------------------------------------------------------------------------ */
/* Norms around a block, codes by row or column, their product, the gated     */
/* activation (definitions and orders: include/repro.h).                      */
/* ------------------------------------------------------------------------ */

#define NORM_CHUNK 8
#define SWIGLU_GROUP 128

/* to bf16 and back: nearest, ties to even; a NaN stays one */
float oracle_bf16(float x)
{
    uint32_t b;
    if (x != x)
        return x;
    memcpy(&b, &x, 4);
    b = (b + 0x7fffu + ((b >> 16) & 1u)) & 0xffff0000u;
    memcpy(&x, &b, 4);
    return x;
}

/* S(t): groups of 4 left to right into C ascending chains, the chains by the tree */
static float norm_sum(const float* t, int64_t D)
{
    int64_t C = 32;
    while (16 * C < D)
        C *= 2;
    const int64_t G = (D + 3) / 4, used = G < C ? G : C;
    float* s = (float*)malloc((size_t)used * sizeof(float));
    for (int64_t g = 0; g < G; ++g) {
        float a = t[4 * g];
        for (int64_t d = 4 * g + 1; d < 4 * g + 4 && d < D; ++d)
            a = oracle_add(a, t[d]);
        s[g % C] = g < C ? a : oracle_add(s[g % C], a);
    }
    for (int64_t w = 1; w < used; w *= 2)
        for (int64_t j = 0; j + w < used; j += 2 * w)
            s[j] = oracle_add(s[j], s[j + w]);
    const float r = s[0];
    free(s);
    return r;
}

static float norm_rms(const float* v, int64_t D, float eps, float* tmp)
{
    for (int64_t d = 0; d < D; ++d)
        tmp[d] = oracle_mul(v[d], v[d]);
    return oracle_div(1.0f, oracle_sqrt(oracle_add(oracle_div(norm_sum(tmp, D), (float)D), eps)));
}

void oracle_block_norm_fwd(const float* x, const float* y, const float* gate, int gate_rows,
                           const float* gp, const float* gn, float alpha, float beta, float eps,
                           int64_t n, int64_t D, int post, int want_u, int h_bf16, float* h, float* u,
                           float* stats)
{
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i) {
        float* tmp = (float*)malloc((size_t)D * sizeof(float));
        float* row = (float*)malloc((size_t)D * sizeof(float));
        float r1 = 0.0f, r2 = 0.0f;
        if (y && post)
            r1 = norm_rms(y + i * D, D, eps, tmp);
        for (int64_t d = 0; d < D; ++d) {
            float v = x[i * D + d];
            if (y) {
                float p = y[i * D + d];
                if (post)
                    p = oracle_mul(p, r1);
                if (post && gp)
                    p = oracle_mul(p, gp[d]);
                if (gate)
                    p = oracle_mul(p, gate[gate_rows ? i * D + d : d]);
                v = oracle_add(oracle_mul(v, alpha), oracle_mul(p, beta));
                if (h_bf16)
                    v = oracle_bf16(v);
                h[i * D + d] = v;
            }
            row[d] = v;
        }
        if (want_u) {
            r2 = norm_rms(row, D, eps, tmp);
            for (int64_t d = 0; d < D; ++d) {
                const float v = oracle_mul(row[d], r2);
                u[i * D + d] = gn ? oracle_mul(v, gn[d]) : v;
            }
        }
        stats[2 * i] = r1;
        stats[2 * i + 1] = r2;
        free(tmp);
        free(row);
    }
}

/* sum over the rows of terms [n][D], chunk by chunk, into out (or added to it) */
static void norm_columns(const float* terms, int64_t n, int64_t D, int accumulate, float* out)
{
    const int64_t C = (n + NORM_CHUNK - 1) / NORM_CHUNK;
#pragma omp parallel for schedule(static)
    for (int64_t d = 0; d < D; ++d) {
        float* t = (float*)malloc((size_t)(C > 0 ? C : 1) * sizeof(float));
        t[0] = 0.0f;
        for (int64_t i = 0; i < n; ++i) {
            const float v = terms[i * D + d];
            t[i / NORM_CHUNK] = i % NORM_CHUNK == 0 ? v : oracle_add(t[i / NORM_CHUNK], v);
        }
        for (int64_t w = 1; w < C; w *= 2)
            for (int64_t j = 0; j + w < C; j += 2 * w)
                t[j] = oracle_add(t[j], t[j + w]);
        out[d] = accumulate ? oracle_add(out[d], t[0]) : t[0];
        free(t);
    }
}

/* r (x) (v (-) (unit (x) (S(v (x) unit) (/) D))) of one row */
static void norm_back(const float* v, const float* unit, float r, int64_t D, float* tmp, float* out)
{
    for (int64_t d = 0; d < D; ++d)
        tmp[d] = oracle_mul(v[d], unit[d]);
    const float c = oracle_div(norm_sum(tmp, D), (float)D);
    for (int64_t d = 0; d < D; ++d)
        out[d] = oracle_mul(r, oracle_add(v[d], -oracle_mul(unit[d], c)));
}

void oracle_block_norm_bwd(const float* dh, const float* du, const float* h, const float* y,
                           const float* gate, int gate_rows, const float* gp, const float* gn,
                           const float* stats, float alpha, float beta, int64_t n, int64_t D, int post,
                           int accumulate, float* dx, float* dy, float* dgate, float* dgp, float* dgn)
{
    const size_t bytes = (size_t)(n * D > 0 ? n * D : 1) * sizeof(float);
    float *tn = (float*)malloc(bytes), *tp = (float*)malloc(bytes), *tg = (float*)malloc(bytes);
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i) {
        const size_t rb = (size_t)D * sizeof(float);
        float *tmp = (float*)malloc(rb), *v = (float*)malloc(rb), *unit = (float*)malloc(rb), *g = (float*)malloc(rb);
        const float r1 = stats[2 * i], r2 = stats[2 * i + 1];
        for (int64_t d = 0; d < D; ++d)
            g[d] = dh ? oracle_flush(dh[i * D + d]) : 0.0f;
        if (du) {
            for (int64_t d = 0; d < D; ++d) {
                const float u = du[i * D + d];
                unit[d] = oracle_mul(h[i * D + d], r2);
                v[d] = gn ? oracle_mul(u, gn[d]) : oracle_flush(u);
                tn[i * D + d] = oracle_mul(u, unit[d]);
            }
            norm_back(v, unit, r2, D, tmp, v);
            for (int64_t d = 0; d < D; ++d)
                g[d] = dh ? oracle_add(g[d], v[d]) : v[d];
        }
        for (int64_t d = 0; d < D; ++d)
            dx[i * D + d] = y ? oracle_mul(g[d], alpha) : g[d];
        if (y) {
            for (int64_t d = 0; d < D; ++d) {
                const float yv = oracle_flush(y[i * D + d]);
                unit[d] = post ? oracle_mul(yv, r1) : yv;
                const float p = post && gp ? oracle_mul(unit[d], gp[d]) : unit[d];
                const float b = oracle_mul(g[d], beta);
                if (gate) {
                    (gate_rows ? dgate : tg)[i * D + d] = oracle_mul(b, p);
                    v[d] = oracle_mul(b, gate[gate_rows ? i * D + d : d]);
                } else {
                    v[d] = b;
                }
            }
            if (post) {
                for (int64_t d = 0; d < D; ++d) {
                    tp[i * D + d] = oracle_mul(v[d], unit[d]);
                    if (gp)
                        v[d] = oracle_mul(v[d], gp[d]);
                }
                norm_back(v, unit, r1, D, tmp, dy + i * D);
            } else {
                memcpy(dy + i * D, v, rb);
            }
        }
        free(tmp);
        free(v);
        free(unit);
        free(g);
    }
    if (dgn)
        norm_columns(tn, n, D, accumulate, dgn);
    if (dgp)
        norm_columns(tp, n, D, accumulate, dgp);
    if (gate && !gate_rows)
        norm_columns(tg, n, D, accumulate, dgate);
    free(tn);
    free(tp);
    free(tg);
}

void oracle_quant_rows(const float* x, const float* mul, int64_t n, int64_t D, int columns, int8_t* q,
                       float* scales)
{
    const int64_t R = columns ? D : n, L = columns ? n : D;
#pragma omp parallel for schedule(static)
    for (int64_t r = 0; r < R; ++r) {
        float m = 0.0f;
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t j = 0; j < L; ++j) {
                const int64_t at = columns ? j * D + r : r * D + j;
                const float v = mul ? oracle_mul(x[at], mul[j]) : oracle_flush(x[at]);
                if (pass)
                    q[at] = (int8_t)oracle_quant_one(v, scales[r], 127);
                else if (fabsf(v) > m)
                    m = fabsf(v);
            }
            if (!pass)
                scales[r] = oracle_div(m, oracle_i2f(127));
        }
    }
}

void oracle_matmul_i8(const int8_t* a, const int8_t* b, const float* s_a, const float* s_b, int64_t M,
                      int64_t N, int64_t K, int a_t, int b_t, int accumulate, float* y)
{
#pragma omp parallel for schedule(static)
    for (int64_t m = 0; m < M; ++m)
        for (int64_t j = 0; j < N; ++j) {
            int64_t acc = 0;
            for (int64_t k = 0; k < K; ++k)
                acc += (int64_t)a[a_t ? k * M + m : m * K + k] * b[b_t ? k * N + j : j * K + k];
            float v = oracle_i2f(acc);
            if (s_a)
                v = oracle_mul(v, s_a[m]);
            if (s_b)
                v = oracle_mul(v, s_b[j]);
            y[m * N + j] = accumulate ? oracle_add(y[m * N + j], v) : v;
        }
}

/* sig(g) and sig(-g) from one e^-|g| and one reciprocal */
static void sigmoids(float g, float* sig, float* rest)
{
    const float e = oracle_exp(-fabsf(oracle_flush(g)));
    const float w = oracle_div(1.0f, oracle_add(1.0f, e)), ew = oracle_mul(e, w);
    *sig = g >= 0.0f ? w : ew;
    *rest = g >= 0.0f ? ew : w;
}

void oracle_swiglu_fwd(const float* gu, int64_t n, int64_t F, float* a, int8_t* codes, float* scales)
{
    const int64_t G = (F + SWIGLU_GROUP - 1) / SWIGLU_GROUP;
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i) {
        for (int64_t j = 0; j < F; ++j) {
            const float g = gu[2 * i * F + j], up = gu[(2 * i + 1) * F + j];
            float sig, rest;
            sigmoids(g, &sig, &rest);
            a[i * F + j] = oracle_mul(oracle_mul(g, sig), up);
        }
        for (int64_t h = 0; codes && h < 2 * G; ++h) {
            const float* v = gu + (2 * i + h / G) * F;
            const int64_t lo = h % G * SWIGLU_GROUP, hi = lo + SWIGLU_GROUP < F ? lo + SWIGLU_GROUP : F;
            float m = 0.0f;
            for (int64_t j = lo; j < hi; ++j)
                if (fabsf(oracle_flush(v[j])) > m)
                    m = fabsf(oracle_flush(v[j]));
            const float s = scales[2 * G * i + h] = oracle_div(m, oracle_i2f(127));
            int8_t* c = codes + (2 * G * i + h) * SWIGLU_GROUP;
            for (int64_t j = 0; j < SWIGLU_GROUP; ++j)
                c[j] = lo + j < hi ? (int8_t)oracle_quant_one(v[lo + j], s, 127) : 0;
        }
    }
}

void oracle_swiglu_bwd(const float* da, const float* gu, const int8_t* codes, const float* scales,
                       int64_t n, int64_t F, float* dgu)
{
    const int64_t G = (F + SWIGLU_GROUP - 1) / SWIGLU_GROUP;
#pragma omp parallel for schedule(static)
    for (int64_t i = 0; i < n; ++i)
        for (int64_t j = 0; j < F; ++j) {
            float v[2], sig, rest;
            for (int h = 0; h < 2; ++h) {
                const int64_t at = (2 * i + h) * G + j / SWIGLU_GROUP;
                v[h] = gu ? gu[(2 * i + h) * F + j]
                          : oracle_mul(oracle_i2f(codes[at * SWIGLU_GROUP + j % SWIGLU_GROUP]), scales[at]);
            }
            sigmoids(v[0], &sig, &rest);
            const float d = da[i * F + j];
            dgu[2 * i * F + j] = oracle_mul(oracle_mul(oracle_mul(d, v[1]), sig),
                                            oracle_add(1.0f, oracle_mul(v[0], rest)));
            dgu[(2 * i + 1) * F + j] = oracle_mul(d, oracle_mul(v[0], sig));
        }
}
