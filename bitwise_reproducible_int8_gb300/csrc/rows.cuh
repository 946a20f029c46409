// rows.cuh -- rows held in the registers of a group of threads, 16 elements each.
//
// A row of D <= 16384 elements belongs to TPR threads, TPR the smallest power of two from
// 32 on with 16 TPR >= D: thread t holds the groups of 4 neighbours t, t + TPR, t + 2 TPR
// and t + 3 TPR, so that neighbouring threads load neighbouring 16 bytes, and the row's sum
// has the order that these threads can add in: a thread's groups are one chain of S, the
// tree over the chains is five exchanges inside a warp, one trip through shared memory and
// up to five exchanges over the warps.  Rows of up to 128 and 256 elements leave a thread one or two
// groups, and what is not there is not in the code either (G; G2 is twice that, its arrays' length):
// 200,000 x 128 bf16 forward 64 us against 168, backward 119 against 269.
// (Half a chain a thread, twice the threads at half the
// registers: the norm's backward at 16,384 x 2048 took 139 us against 133.)
#pragma once

#include "elem.cuh"

namespace repro {

typedef unsigned long long u64;

// threads of a row's group
inline int row_threads(int64_t D)
{
    int t = 32;
    while (16 * (int64_t)t < D)
        t *= 2;
    return t;
}

// Where a thread stands in its row's group.  What is known when a kernel is compiled becomes offsets of
// its loads: with TPR read from the arguments the backward took 203 us at 4096 x 8192 instead of 163.
struct RowLane {
    int t, tpr, D;      // thread in the group, threads of the group, width
    int threads;        // of the CTA
    int bar;            // named barrier of the group
    __device__ __forceinline__ int at(int k) const { return 4 * (t + k * tpr); }   // first element of group k
};

// TPR: threads of the row, or 0 where `tpr` says it
template <int THREADS, int TPR> __device__ __forceinline__ RowLane row_lane(int64_t D, int tpr, int& sub)
{
    RowLane r;
    r.threads = THREADS;
    r.tpr = TPR == 0 ? tpr : TPR;
    sub = TPR == THREADS ? 0 : threadIdx.x / r.tpr;
    r.t = threadIdx.x - sub * r.tpr;
    r.D = (int)D;
    r.bar = 1 + sub;
    return r;
}

__device__ __forceinline__ void group_barrier(const RowLane& r)
{
    asm volatile("bar.sync %0, %1;" ::"r"(r.bar), "r"(r.tpr) : "memory");
}

// What a row's width leaves to check.  WHOLE: D = 16 TPR, rows on 4-element boundaries: nothing.
// GROUPS: the boundaries and D a multiple of 4: whether a group is there.  ELEMENTS: each element.
constexpr int ELEMENTS = 0, GROUPS = 1, WHOLE = 2;

// What lies past D reads as 0.
template <int W, bool STREAM, int G2, typename T>
__device__ __forceinline__ void load_row(const T* p, const RowLane& r, u64 (&v)[G2])
{
#pragma unroll
    for (int k = 0; k < G2 / 2; ++k) {
        const int d = r.at(k);
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (W != ELEMENTS) {
            if (W == WHOLE || d < r.D)
                x = STREAM ? stream4(p + d) : load4(p + d);
        } else {
            x.x = d < r.D ? to_f32<T>(p[d]) : 0.0f;
            x.y = d + 1 < r.D ? to_f32<T>(p[d + 1]) : 0.0f;
            x.z = d + 2 < r.D ? to_f32<T>(p[d + 2]) : 0.0f;
            x.w = d + 3 < r.D ? to_f32<T>(p[d + 3]) : 0.0f;
        }
        v[2 * k] = pack2(x.x, x.y);
        v[2 * k + 1] = pack2(x.z, x.w);
    }
}

template <int W, int G2, typename T>
__device__ __forceinline__ void store_row(T* p, const RowLane& r, const u64 (&v)[G2])
{
#pragma unroll
    for (int k = 0; k < G2 / 2; ++k) {
        const int d = r.at(k);
        float4 x;
        unpack2(v[2 * k], x.x, x.y);
        unpack2(v[2 * k + 1], x.z, x.w);
        if (W != ELEMENTS) {
            if (W == WHOLE || d < r.D)
                store4(p + d, x);
        } else {
            if (d < r.D)
                p[d] = from_f32<T>(x.x);
            if (d + 1 < r.D)
                p[d + 1] = from_f32<T>(x.y);
            if (d + 2 < r.D)
                p[d + 2] = from_f32<T>(x.z);
            if (d + 3 < r.D)
                p[d + 3] = from_f32<T>(x.w);
        }
    }
}

// A thread's share of a row on its way through shared memory: asked for early, taken when it is needed.
// Each thread copies and reads its own elements only, so no barrier stands between; group k of
// thread t lies at k threads + t.  piece (ELEMENTS): elements copied at a time, 4, 2 or 1, whatever the
// rows' boundaries and width allow (a copy has 4 bytes at least).
template <typename T> struct alignas(4 * sizeof(T)) Four {
    T v[4];
};

template <int BYTES> __device__ __forceinline__ void copy_async(void* to, const void* from)
{
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(from), "n"(BYTES) : "memory");
}

template <int W, int G, typename T>
__device__ __forceinline__ void ask_row(Four<T>* slot, const T* p, const RowLane& r, int piece)
{
    constexpr int SZ = (int)sizeof(T);
#pragma unroll
    for (int k = 0; k < G; ++k) {
        const int d = r.at(k);
        T* to = slot[k * r.threads + threadIdx.x].v;
        if (W != ELEMENTS) {
            if (W == WHOLE || d < r.D)
                copy_async<4 * SZ>(to, p + d);
        } else if (piece == 4) {
            if (d < r.D)
                copy_async<4 * SZ>(to, p + d);
        } else if (SZ == 2 || piece == 2) {
#pragma unroll
            for (int e = 0; e < 4; e += 2)
                if (d + e < r.D)
                    copy_async<2 * SZ>(to + e, p + d + e);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (d + e < r.D)
                    copy_async<SZ == 4 ? 4 : 8>(to + e, p + d + e);   // fp32 alone comes here
        }
    }
}

template <int W, int G2, typename T> __device__ __forceinline__ void take_row(const Four<T>* slot, const RowLane& r, u64 (&v)[G2])
{
#pragma unroll
    for (int k = 0; k < G2 / 2; ++k) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (W != GROUPS || r.at(k) < r.D)
            x = load4(slot[k * r.threads + threadIdx.x].v);
        if (W == ELEMENTS) {
            const int left = r.D - r.at(k);
            x.x = left > 0 ? x.x : 0.0f, x.y = left > 1 ? x.y : 0.0f, x.z = left > 2 ? x.z : 0.0f, x.w = left > 3 ? x.w : 0.0f;
        }
        v[2 * k] = pack2(x.x, x.y);
        v[2 * k + 1] = pack2(x.z, x.w);
    }
}

// elements at a time that rows of `size` bytes an element, `ld` apart, can be copied by; 0: none
inline int piece_of(const void* p, int64_t ld, int64_t D, int size)
{
    for (int e = 4; e * size >= 4; e /= 2)
        if (reinterpret_cast<uintptr_t>(p) % (e * size) == 0 && ld % e == 0 && D % e == 0)
            return e;
    return 0;
}

__device__ __forceinline__ void asked() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void wait_asked() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

template <int G2> __device__ __forceinline__ void flush_row(u64 (&v)[G2])
{
    const u64 z = pack2(-0.0f, -0.0f);
#pragma unroll
    for (int i = 0; i < G2; ++i)
        v[i] = fadd2_ftz(v[i], z);
}

// v (x) w, flushed (both operands flushed already)
template <int G2> __device__ __forceinline__ void mul_row(u64 (&v)[G2], const u64 (&w)[G2])
{
    const u64 z = pack2(-0.0f, -0.0f);
#pragma unroll
    for (int i = 0; i < G2; ++i)
        v[i] = fadd2_ftz(fmul2_rn(v[i], w[i]), z);
}

template <int G2> __device__ __forceinline__ void mul_row(u64 (&v)[G2], float w)
{
    const u64 z = pack2(-0.0f, -0.0f), ww = pack2(w, w);
#pragma unroll
    for (int i = 0; i < G2; ++i)
        v[i] = fadd2_ftz(fmul2_rn(v[i], ww), z);
}

// this thread's chain of S(a (x) b); terms past the width count as -0, which leaves a sum alone
template <int W, int G2>
__device__ __forceinline__ float chain_of(const u64 (&a)[G2], const u64 (&b)[G2], const RowLane& r)
{
    float g[G2 / 2];
#pragma unroll
    for (int k = 0; k < G2 / 2; ++k) {
        float p[4];
        unpack2(fmul2_rn(a[2 * k], b[2 * k]), p[0], p[1]);
        unpack2(fmul2_rn(a[2 * k + 1], b[2 * k + 1]), p[2], p[3]);
        if (W == ELEMENTS) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = r.at(k) + e < r.D ? p[e] : -0.0f;
        }
        g[k] = fadd_ftz(fadd_ftz(fadd_ftz(p[0], p[1]), p[2]), p[3]);
        if (W == GROUPS)
            g[k] = r.at(k) < r.D ? g[k] : -0.0f;
    }
#pragma unroll
    for (int k = 1; k < G2 / 2; ++k)
        g[0] = fadd_ftz(g[0], g[k]);
    return g[0];
}

// the tree over the group's chains, the same bits in every thread.  red: 64 floats of the
// group in shared memory, used in halves by turns (phase), so that one barrier a sum is enough
__device__ __forceinline__ float tree_of_chains(float v, const RowLane& r, float* red, int& phase)
{
    constexpr unsigned ALL = 0xffffffffu;
#pragma unroll
    for (int s = 1; s < 32; s *= 2)
        v = fadd_ftz(v, __shfl_xor_sync(ALL, v, s));
    if (r.tpr == 32)
        return v;
    const int lane = r.t & 31, warps = r.tpr >> 5;
    float* half = red + 32 * phase;
    phase ^= 1;
    if (lane == 0)
        half[r.t >> 5] = v;
    group_barrier(r);
    v = lane < warps ? half[lane] : -0.0f;
#pragma unroll
    for (int s = 1; s < 32; s *= 2)
        if (s < warps)
            v = fadd_ftz(v, __shfl_xor_sync(ALL, v, s));
    return __shfl_sync(ALL, v, 0);
}

// S (/) D; by an exact product where D is a power of two (inv = 1 / D, else 0)
__device__ __forceinline__ float mean_of(float S, float width, float inv)
{
    return inv != 0.0f ? fmul_flush(S, inv) : flush(__fdiv_rn(S, width));
}

} // namespace repro
