// k_blocknorm_bwd.cu -- the block norm's backward with the gradients of gains and gate.
//
//   g = dh + r2 (v - hn c), v = du gain_pre, hn = h r2, c = mean(v hn); dx = g alpha;
//   dy = r1 (w - yn c'), w = g beta gate gain_post, yn = y r1, c' = mean(w yn)
//
// Bound by HBM: du, dh, h, y in, dx, dy out (24 bytes an element in fp32).  Measured: 16,384 x 2048 fp32
// 133 us, 6.1 TB/s, floor 119; from 4096 on (143 us at 8192 x 4096, 161 at 4096 x 8192; bf16 115, floor
// 59) one row's two sums and their barriers stand alone on an SM and its latency shows.
//
// The gradients that are sums over tokens: a group of the backward takes 8 consecutive tokens one
// after another and keeps its columns' sums in registers, so a chunk's order costs nothing, and
// writes one row of partial sums (1/8 of a stream of the pass, most of it in L2; with chunks of 16, 2.25
// rounds over the card, it took 7 us more); k_rowtree.cu joins them.
// A few tokens would leave most of the card idle that way, and 8 rows one after another are all
// latency: then a group takes one token and writes its terms, and k_norm_fold adds the chunks up
// (1023 x 1001 bf16 with a gate per channel: 17 us, 79 in chunks of 16).
#include "blocknorm.cuh"

namespace repro {
namespace {

constexpr int CHUNK = 8;        // tokens of a chunk of the sums over tokens: REPRO_NORM_CHUNK

// v <- scale (x) (v (-) (unit (x) c)), c = S(v (x) unit) (/) D
template <int W, int G2>
__device__ __forceinline__ void norm_back(u64 (&v)[G2], const u64 (&unit)[G2], float scale, const NormArgs& a,
                                          const RowLane& r, float* red, int& phase)
{
    const float c = mean_of(tree_of_chains(chain_of<W>(v, unit, r), r, red, phase), (float)a.D, a.inv);
    const u64 cc = pack2(-c, -c), sc = pack2(scale, scale), z = pack2(-0.0f, -0.0f);
#pragma unroll
    for (int e = 0; e < G2; ++e)
        v[e] = fadd2_ftz(fmul2_rn(sc, fadd2_ftz(v[e], fmul2_rn(unit[e], cc))), z);
}

// s (+) a (x) b
template <int G2> __device__ __forceinline__ void column_sum(u64 (&s)[G2], const u64 (&a)[G2], const u64 (&b)[G2])
{
#pragma unroll
    for (int e = 0; e < G2; ++e)
        s[e] = fadd2_ftz(fmul2_rn(a[e], b[e]), s[e]);
}

template <int W, int G2>
__device__ __forceinline__ void store_parts(float* parts, int64_t chunk, int64_t pitch, const RowLane& r, const u64 (&s)[G2])
{
#pragma unroll
    for (int k = 0; k < G2 / 2; ++k) {
        const int d = r.at(k);
        float4 v;
        unpack2(s[2 * k], v.x, v.y);
        unpack2(s[2 * k + 1], v.z, v.w);
        if (W == WHOLE || d < r.D)   // the pitch is a multiple of 4
            store4(parts + chunk * pitch + d, v);
    }
}

// AHEAD: the next token's row is asked for as soon as this one's is taken, through shared memory (a
// row of each stream on its way for every group on an SM); else loads where values are needed.
// CHANNEL: a gate that is one row, whose sums take 16 more registers.  Three groups of 128 threads an
// SM at 168 registers; with four at 128 the kernel spills.
template <typename T, int THREADS, int TPR, int G, bool AHEAD, int W, bool CHANNEL>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 384 / THREADS : 1)
k_norm_bwd(const __grid_constant__ NormArgs a)
{
    extern __shared__ __align__(16) uint8_t slots[];
    __shared__ float red[4][64];
    int sub, phase = 0;
    const RowLane r = row_lane<THREADS, TPR>(a.D, a.tpr, sub);
    const int per = THREADS / r.tpr;
    const float alpha = flush(a.alpha), beta = flush(a.beta);
    // slots of du, h, dh, y and the gate's rows
    const size_t st = G * sizeof(Four<T>) * THREADS;
    Four<T>* const s_h = reinterpret_cast<Four<T>*>(slots);
    Four<T>* const s_dh = reinterpret_cast<Four<T>*>(slots + st);
    Four<T>* const s_y = reinterpret_cast<Four<T>*>(slots + 2 * st);
    Four<T>* const s_gate = reinterpret_cast<Four<T>*>(slots + 3 * st);
    void* const s_du = slots + (a.gate_rows ? 4 : 3) * st;
    const bool gates = !CHANNEL && a.gate;
    auto row_t = [&](const void* p, int64_t ld, int64_t i) { return static_cast<const T*>(p) + i * ld; };
    auto ask_norm = [&](int64_t i) {      // what the norm before the block needs of token i
        if (a.du) {
            if (a.u_type == 0)
                ask_row<W, G>(static_cast<Four<float>*>(s_du), static_cast<const float*>(a.du) + i * a.du_ld, r, a.piece_u);
            else
                ask_row<W, G>(static_cast<Four<__nv_bfloat16>*>(s_du), static_cast<const __nv_bfloat16*>(a.du) + i * a.du_ld, r, a.piece_u);
            ask_row<W, G>(s_h, row_t(a.hs, a.hs_ld, i), r, a.piece);
        }
        asked();
    };
    auto ask_rest = [&](int64_t i) {
        if (a.dh)
            ask_row<W, G>(s_dh, row_t(a.dh, a.dh_ld, i), r, a.piece);
        if (a.y)
            ask_row<W, G>(s_y, row_t(a.y, a.y_ld, i), r, a.piece);
        if (gates)
            ask_row<W, G>(s_gate, row_t(a.gate, a.gate_ld, i), r, a.piece);
        asked();
    };
    pdl_wait();
    pdl_trigger();
    const int64_t chunks = (a.n + a.chunk - 1) / a.chunk;
    for (int64_t ch = (int64_t)blockIdx.x * per + sub; ch < chunks; ch += (int64_t)gridDim.x * per) {
        u64 s_pre[2 * G], s_post[2 * G], s_chan[2 * G];
        const int64_t lo = ch * a.chunk, hi = lo + a.chunk < a.n ? lo + a.chunk : a.n;
#pragma unroll
        for (int e = 0; e < 2 * G; ++e)   // -0 (+) v is v
            s_pre[e] = s_post[e] = s_chan[e] = pack2(-0.0f, -0.0f);
        if (AHEAD) {
            ask_norm(lo);
            ask_rest(lo);
        }
        float next1 = __ldg(a.stats + 2 * lo), next2 = __ldg(a.stats + 2 * lo + 1);
        for (int64_t i = lo; i < hi; ++i) {
            const float r1 = flush(next1), r2 = flush(next2);
            if (i + 1 < hi) {
                next1 = __ldg(a.stats + 2 * (i + 1));
                next2 = __ldg(a.stats + 2 * (i + 1) + 1);
            }
            u64 g[2 * G], v[2 * G], unit[2 * G], w[2 * G];
            if (AHEAD)
                wait_asked<1>();
            if (a.du) {
                if (!AHEAD) {
                    if (a.u_type == 0)
                        load_row<W, true>(static_cast<const float*>(a.du) + i * a.du_ld, r, v);
                    else
                        load_row<W, true>(static_cast<const __nv_bfloat16*>(a.du) + i * a.du_ld, r, v);
                    load_row<W, true>(row_t(a.hs, a.hs_ld, i), r, unit);
                } else {
                    if (a.u_type == 0)
                        take_row<W>(static_cast<const Four<float>*>(s_du), r, v);
                    else
                        take_row<W>(static_cast<const Four<__nv_bfloat16>*>(s_du), r, v);
                    take_row<W>(s_h, r, unit);
                }
                flush_row(v);
                flush_row(unit);
                mul_row(unit, r2);
                if (a.dgain_pre)
                    column_sum(s_pre, v, unit);
                if (a.gain_pre) {
                    gain_row<W>(a.gain_pre, r, w);
                    mul_row(v, w);
                }
            }
            if (AHEAD) {
                if (i + 1 < hi)
                    ask_norm(i + 1);
                else
                    asked();
            }
            if (a.du)
                norm_back<W>(v, unit, r2, a, r, red[sub], phase);
            if (AHEAD)
                wait_asked<1>();
            if (a.dh) {
                if (!AHEAD)
                    load_row<W, false>(row_t(a.dh, a.dh_ld, i), r, g);
                else
                    take_row<W>(s_dh, r, g);
                flush_row(g);
                if (a.du)
#pragma unroll
                    for (int e = 0; e < 2 * G; ++e)
                        g[e] = fadd2_ftz(g[e], v[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 2 * G; ++e)
                    g[e] = v[e];
            }
            if (!a.y) {
                store_row<W>(static_cast<T*>(a.dx) + i * a.dx_ld, r, g);
                if (AHEAD) {
                    if (i + 1 < hi)
                        ask_rest(i + 1);
                    else
                        asked();
                }
                continue;
            }
#pragma unroll
            for (int e = 0; e < 2 * G; ++e)
                v[e] = g[e];
            mul_row(v, alpha);
            store_row<W>(static_cast<T*>(a.dx) + i * a.dx_ld, r, v);
            mul_row(g, beta);
            if (!AHEAD)
                load_row<W, true>(row_t(a.y, a.y_ld, i), r, unit);
            else
                take_row<W>(s_y, r, unit);
            if (gates) {
                if (!AHEAD)
                    load_row<W, true>(row_t(a.gate, a.gate_ld, i), r, w);
                else
                    take_row<W>(s_gate, r, w);
                flush_row(w);
            }
            if (AHEAD) {
                if (i + 1 < hi)
                    ask_rest(i + 1);
                else
                    asked();
            }
            flush_row(unit);
            if (a.post)
                mul_row(unit, r1);
            if (CHANNEL || gates) {
#pragma unroll
                for (int e = 0; e < 2 * G; ++e)
                    v[e] = unit[e];
                if (a.post && a.gain_post) {
                    u64 gp[2 * G];
                    gain_row<W>(a.gain_post, r, gp);
                    mul_row(v, gp);
                }
                if (gates) {
                    mul_row(v, g);
                    store_row<W>(static_cast<T*>(a.dgate) + i * a.dgate_ld, r, v);
                } else {
                    column_sum(s_chan, g, v);
                    gain_row<W>(static_cast<const float*>(a.gate), r, w);
                }
                mul_row(g, w);
            }
            if (a.post) {
                if (a.dgain_post)
                    column_sum(s_post, g, unit);
                if (a.gain_post) {
                    gain_row<W>(a.gain_post, r, w);
                    mul_row(g, w);
                }
                norm_back<W>(g, unit, r1, a, r, red[sub], phase);
            }
            store_row<W>(static_cast<T*>(a.dy) + i * a.dy_ld, r, g);
        }
        if (a.dgain_pre)
            store_parts<W>(a.parts[0], ch, a.pitch, r, s_pre);
        if (a.dgain_post)
            store_parts<W>(a.parts[1], ch, a.pitch, r, s_post);
        if (CHANNEL)
            store_parts<W>(a.parts[2], ch, a.pitch, r, s_chan);
    }
}

// chunks of terms, one row a token, to rows of partial sums; a thread has 4 columns of a chunk
struct Fold {
    const float* terms[3];
    float* parts[3];
    int64_t n, chunks, pitch;
    int segs;            // CTAs of a chunk
};

__global__ void __launch_bounds__(128)
k_norm_fold(const __grid_constant__ Fold f)
{
    pdl_wait();
    pdl_trigger();
    const int64_t per = f.chunks * f.segs, job = blockIdx.x / per, in = blockIdx.x - job * per, ch = in / f.segs;
    const int64_t c = 4 * ((in - ch * f.segs) * 128 + threadIdx.x), lo = ch * CHUNK;
    if (c >= f.pitch)
        return;
    const float* t = f.terms[job] + lo * f.pitch + c;
    float4 v[CHUNK];
#pragma unroll
    for (int i = 0; i < CHUNK; ++i)   // -0 in place of a missing token leaves a sum as it is
        v[i] = lo + i < f.n ? load4(t + i * f.pitch) : make_float4(-0.0f, -0.0f, -0.0f, -0.0f);
#pragma unroll
    for (int i = 1; i < CHUNK; ++i)
        v[0] = make_float4(fadd_ftz(v[0].x, v[i].x), fadd_ftz(v[0].y, v[i].y), fadd_ftz(v[0].z, v[i].z), fadd_ftz(v[0].w, v[i].w));
    store4(f.parts[job] + ch * f.pitch + c, v[0]);
}

// Few tokens: up to 2^21 elements, where the terms' way through L2 (16 MB for two sums) takes less than
// the rows of a chunk one after another, or chunks for less than half of the groups that run at once
// (three CTAs of 128 threads on an SM, one of more; 152 SMs, whatever the device, as the rule sets the
// workspace's size).  300 x 7296 fp32 26 us, 35 in chunks, bf16 24 and 40; 600 x 7296, at the border, 41 and
// 37, bf16 37 and 40; in chunks above it: 788 x 7296 38 us, 52 by tokens, 11000 x 3000 174 and 326.
inline bool by_tokens(int64_t n, int64_t D)
{
    const int tpr = row_threads(D);
    const int64_t at_once = (int64_t)152 * (tpr <= 128 ? 3 * (128 / tpr) : 1);
    return n > 1 && n <= (int64_t)1 << 21 && (n * D <= (int64_t)1 << 21 || 2 * ((n + CHUNK - 1) / CHUNK) < at_once);
}

inline int64_t pitch_of(int64_t D) { return (D + 3) / 4 * 4; }

// the pieces that every row of the backward can be copied by
void set_pieces(NormArgs& a)
{
    const int t = a.type == 0 ? 4 : 2, u = a.u_type == 0 ? 4 : 2;
    a.piece = 4;
    const struct {
        const void* p;
        int64_t ld;
    } rows[4] = {{a.hs, a.hs_ld}, {a.dh, a.dh_ld}, {a.y, a.y_ld}, {a.gate_rows ? a.gate : nullptr, a.gate_ld}};
    for (const auto& r : rows)
        if (r.p) {
            const int e = piece_of(r.p, r.ld, a.D, t);
            a.piece = e < a.piece ? e : a.piece;
        }
    a.piece_u = a.du ? piece_of(a.du, a.du_ld, a.D, u) : 4;
}

template <typename T, int N, int TPR, int G, bool AHEAD, int W> cudaError_t run_bwd(const NormArgs& a, dim3 grid, cudaStream_t st)
{
    const auto k = a.gate && !a.gate_rows ? k_norm_bwd<T, N, TPR, G, AHEAD, W, true> : k_norm_bwd<T, N, TPR, G, AHEAD, W, false>;
    const size_t smem = AHEAD ? (size_t)N * 4 * G * ((a.gate_rows ? 4 : 3) * sizeof(T) + (a.u_type == 0 ? 4 : 2)) : 0;
    if (smem > 40 * 1024) {   // static shared memory counts too
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(k, grid, dim3(N), smem, st, a);
}

template <typename T, int N, int TPR, int G = 4> cudaError_t pick_bwd(const NormArgs& a, dim3 grid, cudaStream_t st)
{
    if (a.piece == 0 || a.piece_u == 0)
        return run_bwd<T, N, TPR, G, false, ELEMENTS>(a, grid, st);
    const int w = check_of(a);
    if (G < 4)
        return w != ELEMENTS ? run_bwd<T, N, TPR, G, true, GROUPS>(a, grid, st) : run_bwd<T, N, TPR, G, true, ELEMENTS>(a, grid, st);
    return w == WHOLE ? run_bwd<T, N, TPR, 4, true, WHOLE>(a, grid, st) : w == GROUPS ? run_bwd<T, N, TPR, G, true, GROUPS>(a, grid, st)
                                                                              : run_bwd<T, N, TPR, G, true, ELEMENTS>(a, grid, st);
}

template <typename T> cudaError_t launch_bwd(NormArgs& a, int64_t items, cudaStream_t st)
{
    int threads;
    const dim3 grid = grid_of(a, items, threads);
    return a.D <= 128       ? pick_bwd<T, 128, 32, 1>(a, grid, st)
           : a.D <= 256     ? pick_bwd<T, 128, 32, 2>(a, grid, st)
           : a.tpr < 128    ? pick_bwd<T, 128, 0>(a, grid, st)
           : threads == 128 ? pick_bwd<T, 128, 128>(a, grid, st)
           : threads == 256 ? pick_bwd<T, 256, 256>(a, grid, st)
           : threads == 512 ? pick_bwd<T, 512, 512>(a, grid, st)
           : check_of(a) == ELEMENTS ? run_bwd<T, 1024, 1024, 4, false, ELEMENTS>(a, grid, st)   // the slots of 1,024 threads would not fit
                                     : run_bwd<T, 1024, 1024, 4, false, GROUPS>(a, grid, st);
}

} // namespace

size_t norm_bwd_ws_bytes(int64_t n, int64_t D)
{
    return (size_t)((n + CHUNK - 1) / CHUNK + (by_tokens(n, D) ? n : 0)) * (size_t)pitch_of(D) * 4 * 3;
}

cudaError_t launch_norm_bwd(NormArgs a, void* ws, cudaStream_t st)
{
    set_up(a);
    const int64_t chunks = (a.n + CHUNK - 1) / CHUNK;
    a.pitch = pitch_of(a.D);
    float* const out[3] = {a.dgain_pre, a.dgain_post, a.gate && !a.gate_rows ? static_cast<float*>(a.dgate) : nullptr};
    const bool sums = out[0] || out[1] || out[2], single = !sums || by_tokens(a.n, a.D);
    a.chunk = single ? 1 : CHUNK;
    set_pieces(a);
    float* const parts = static_cast<float*>(ws);
    RowTree t = {};
    t.pitch = a.pitch;
    t.D = a.D;
    t.scale = 1.0f;
    t.accumulate = a.accumulate;
    Fold f = {};
    f.n = a.n;
    f.chunks = chunks;
    f.pitch = a.pitch;
    f.segs = (int)((a.pitch + 511) / 512);
    for (int k = 0; k < 3; ++k)
        if (out[k]) {
            t.parts[t.jobs] = f.parts[t.jobs] = parts + t.jobs * chunks * a.pitch;
            t.count[t.jobs] = chunks;
            t.out[t.jobs] = out[k];
            a.parts[k] = t.parts[t.jobs];
            if (single) {
                a.parts[k] = parts + (3 * chunks + t.jobs * a.n) * a.pitch;
                f.terms[t.jobs] = a.parts[k];
            }
            ++t.jobs;
        }
    const int64_t items = single ? a.n : chunks;
    cudaError_t e = a.type == 0 ? launch_bwd<float>(a, items, st) : launch_bwd<__nv_bfloat16>(a, items, st);
    if (e == cudaSuccess && sums && single) {
        e = launch_pdl(k_norm_fold, dim3((unsigned)(t.jobs * chunks * f.segs)), dim3(128), 0, st, f);
        count_launches(1);
    }
    if (e == cudaSuccess && sums)
        e = launch_row_tree(t, num_sms() * 4, st);
    return e;
}

} // namespace repro
