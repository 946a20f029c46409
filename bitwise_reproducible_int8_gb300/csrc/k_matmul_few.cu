// k_matmul_few.cu -- the product of codes for few tokens (5 to 128): Y = X W^T bound by the weights'
// bytes, on the tensor cores without a widened copy of the weights.
//
// A CTA takes 128 weights' rows (output channels) and one exact slice of K (512 terms).  The weights
// are the M side of tcgen05.mma (128 rows), the tokens the N side (32, 64 or 128), so that few tokens
// cost few MMAs; both go from memory through registers, widened there, into swizzled shared
// memory.  A block of 64 terms of a row is 4 threads' 16 bytes; each thread has four blocks on their
// way at a time, so a CTA keeps 32 KB of weights in flight, and three CTAs (of up to 64 tokens) an SM.
//
// Every slice of a tile leaves its int32 sums in the workspace; k_mm_few_join adds them up, exact in
// any order, and scales them.  (Atomic additions into one sum took 53 us for 128 x 11264 x 2048, the
// last CTA of a tile adding up its parts 64 us.)  64 x 11264 x 2048 takes 21 us and
// 16 x 11264 x 2048 13 us; a widened copy of the weights and tiles for 256 tokens 27 us each: five
// bytes moved for each of the weights, and most of the MMAs on nothing.
#include "common.cuh"
#include "internal.h"
#include "launch.cuh"
#include "mm.cuh"
#include "pipeline.cuh"
#include "umma.cuh"

namespace repro {
namespace {

constexpr int ROWS = 128;               // output channels of a CTA
constexpr int TK = 64, BLOCKS = 8;      // terms a block, blocks a slice
constexpr int SLICE = TK * BLOCKS;
constexpr int STAGES = 3;
constexpr int AHEAD = 4;                // blocks whose codes a thread has on their way
constexpr int A_BYTES = ROWS * TK * 2;
constexpr int THREADS = 256;

struct FewArgs {
    MatmulI8Args g;
    int parts;            // slices of K
    int* sums;            // [tile][part][M][128]
    int* err;
};

// kind::f16 with fp16 operands, both K-major, fp32 accumulator, M = 128, N = MT
template <int MT> __device__ __forceinline__ void mma_half(uint32_t dtmem, uint64_t a, uint64_t b, uint32_t acc)
{
    constexpr uint32_t id = (1u << 4) | ((uint32_t)(MT >> 3) << 17) | ((uint32_t)(ROWS >> 4) << 24);
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(dtmem),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

// MT: tokens, rounded up to 32, 64 or 128
template <typename Y, int MT>
__global__ void __launch_bounds__(THREADS, MT <= 64 ? 3 : 2)
k_mm_few(const __grid_constant__ FewArgs p)
{
    constexpr int STAGE = A_BYTES + MT * TK * 2;
    constexpr int COLS = MT / 2;        // tokens that a warp takes out of tensor memory
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t empty[STAGES], done;
    __shared__ uint32_t tmem_base;
    __shared__ int failed;
    uint8_t* base = smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u);
    const MatmulI8Args& g = p.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile = blockIdx.x / p.parts, part = blockIdx.x - tile * p.parts;
    const int64_t n0 = (int64_t)tile * ROWS, k0 = (int64_t)part * SLICE;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s)
            mbar_init(&empty[s], 1);
        mbar_init(&done, 1);
        failed = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&tmem_base)), "r"(MT)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base;
    pdl_wait();
    pdl_trigger();

    // this thread's rows: every 64th of the weights' and of the tokens' from `first` on, 16 codes of
    // each block from 16 `chunk` on
    constexpr int WR = ROWS / 64, TR = (MT + 63) / 64;
    const int first = tid >> 2, chunk = tid & 3;
    const int64_t at = k0 + 16 * chunk;
    const int8_t* src[WR + TR];
    int left[WR + TR];             // terms from src on that exist
#pragma unroll
    for (int i = 0; i < WR + TR; ++i) {
        const int64_t row = i < WR ? n0 + first + 64 * i : first + 64 * (i - WR);
        const bool live = row < (i < WR ? g.N : g.M) && at < g.K;
        src[i] = (i < WR ? g.b + row * g.b_ld : g.a + row * g.a_ld) + at;
        left[i] = live ? (int)(g.K - at) : 0;
    }
    uint4 v[AHEAD][WR + TR];
    auto ask = [&](int b, uint4 (&x)[WR + TR]) {
#pragma unroll
        for (int i = 0; i < WR + TR; ++i) {
            x[i] = make_uint4(0, 0, 0, 0);
            if (TK * b < left[i])
                x[i] = __ldg(reinterpret_cast<const uint4*>(src[i] + TK * b));
        }
    };
#pragma unroll
    for (int b = 0; b < AHEAD; ++b)
        ask(b, v[b]);
    const int64_t terms = g.K - k0 < SLICE ? g.K - k0 : SLICE;
    const int blocks = (int)((terms + TK - 1) / TK);
    bool ok = true;
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
        if (b < blocks) {                      // the same for every thread
            const int s = b % STAGES;
            uint8_t* A = base + s * STAGE;
            if (b >= STAGES && ok)
                ok = mbar_wait_warp(&empty[s], ((b / STAGES) - 1) & 1);
#pragma unroll
            for (int i = 0; i < WR + TR; ++i) {
                const int r = first + 64 * (i < WR ? i : i - WR);
                if (i >= WR && r >= MT)
                    continue;
                // 16-byte chunks 2 chunk and 2 chunk + 1 of row r, at chunk ^ (r mod 8)
                uint8_t* to = (i < WR ? A : A + A_BYTES) + r * 128;
                const uint4 c = v[b % AHEAD][i];
                const uint2 w0 = widen4(c.x), w1 = widen4(c.y), w2 = widen4(c.z), w3 = widen4(c.w);
                *reinterpret_cast<uint4*>(to + 16 * ((2 * chunk) ^ (r & 7))) = make_uint4(w0.x, w0.y, w1.x, w1.y);
                *reinterpret_cast<uint4*>(to + 16 * ((2 * chunk + 1) ^ (r & 7))) = make_uint4(w2.x, w2.y, w3.x, w3.y);
            }
            if (b + AHEAD < BLOCKS)
                ask(b + AHEAD, v[b % AHEAD]);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            fence_before();
            __syncthreads();
            if (tid == 0) {
                fence_after();
                const uint64_t a0 = sdesc(su32(A)), b0 = sdesc(su32(A + A_BYTES));
#pragma unroll
                for (int k = 0; k < TK / 16; ++k)
                    mma_half<MT>(tmem, a0 + 2 * k, b0 + 2 * k, (b != 0 || k != 0) ? 1u : 0u);
                mma_commit(&empty[s]);
                if (b == blocks - 1)
                    mma_commit(&done);
            }
        }
    }
    if (!mbar_wait_warp(&done, 0))
        ok = false;
    if (!ok)
        failed = 1;
    fence_after();
    // lane = output channel, column = token
    const int q = warp & 3, m0 = COLS * (warp >> 2);
    const int64_t n = n0 + 32 * q + lane;
    int acc[COLS];
#pragma unroll
    for (int c = 0; c < COLS; c += 8) {
        uint32_t x[8];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                     : "r"(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(m0 + c)));
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7])
                     :
                     : "memory");
#pragma unroll
        for (int e = 0; e < 8; ++e)
            acc[c + e] = __float2int_rn(__uint_as_float(x[e]));
    }
    fence_before();
    const float sb = g.s_b && n < g.N ? flush(__ldg(g.s_b + n)) : 0.0f;
    Y* y = static_cast<Y*>(g.y);
    if (p.parts == 1) {
#pragma unroll
        for (int c = 0; c < COLS; ++c)
            if (m0 + c < g.M && n < g.N)
                put(y + (int64_t)(m0 + c) * g.y_ld + n,
                    scaled(acc[c], g.s_a, g.s_a ? flush(__ldg(g.s_a + m0 + c)) : 0.0f, g.s_b, sb), g.accumulate);
    } else {
        const int64_t step = (int64_t)g.M * ROWS;             // of a part
        int* sums = p.sums + (int64_t)tile * p.parts * step + (int64_t)m0 * ROWS + 32 * q + lane;
#pragma unroll
        for (int c = 0; c < COLS; ++c)
            if (m0 + c < g.M)
                sums[part * step + c * ROWS] = acc[c];
    }
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(MT) : "memory");
    }
    if (tid == 0 && failed)
        atomicOr(p.err, kErrTimeoutBit);
}

// outputs of the parts' sums; a thread has 4 neighbouring channels of a token
template <typename Y>
__global__ void __launch_bounds__(256)
k_mm_few_join(const __grid_constant__ FewArgs p, int64_t total)
{
    const MatmulI8Args& g = p.g;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (i >= total)
        return;
    const int64_t tm = i >> 5, tile = tm / g.M, m = tm - tile * g.M, n = tile * ROWS + 4 * (i & 31), step = g.M * ROWS;
    const int4* at = reinterpret_cast<const int4*>(p.sums + tile * p.parts * step + m * ROWS) + (i & 31);
    int4 s = make_int4(0, 0, 0, 0);
#pragma unroll 8
    for (int k = 0; k < p.parts; ++k) {
        const int4 x = __ldcg(at + k * (step / 4));
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    const int acc[4] = {s.x, s.y, s.z, s.w};
    const float sa = g.s_a ? flush(__ldg(g.s_a + m)) : 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n + e < g.N)
            put(static_cast<Y*>(g.y) + m * g.y_ld + n + e,
                scaled(acc[e], g.s_a, sa, g.s_b, g.s_b ? flush(__ldg(g.s_b + n + e)) : 0.0f), g.accumulate);
}

inline int parts_of(int64_t K) { return (int)((K + SLICE - 1) / SLICE); }
inline int64_t tiles_of(int64_t N) { return (N + ROWS - 1) / ROWS; }

template <typename Y, int MT> cudaError_t run(const FewArgs& p, cudaStream_t st)
{
    const size_t smem = 1024 + STAGES * (A_BYTES + MT * TK * 2);
    cudaError_t e = cudaFuncSetAttribute(k_mm_few<Y, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = launch_pdl(k_mm_few<Y, MT>, dim3((unsigned)(tiles_of(p.g.N) * p.parts)), dim3(THREADS), smem, st, p);
    count_launches(1);
    if (e == cudaSuccess && p.parts > 1) {
        const int64_t total = tiles_of(p.g.N) * p.g.M * (ROWS / 4);
        e = launch_pdl(k_mm_few_join<Y>, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, p, total);
        count_launches(1);
    }
    return e;
}

template <typename Y> cudaError_t pick(const FewArgs& p, cudaStream_t st)
{
    return p.g.M <= 32 ? run<Y, 32>(p, st) : p.g.M <= 64 ? run<Y, 64>(p, st) : run<Y, 128>(p, st);
}

} // namespace

size_t matmul_few_ws_bytes(int64_t M, int64_t N, int64_t K)
{
    return parts_of(K) > 1 ? (size_t)(tiles_of(N) * parts_of(K) * M * ROWS * 4) : 0;
}

cudaError_t launch_matmul_few(const MatmulI8Args& g, void* ws, cudaStream_t st)
{
    const FewArgs p = {g, parts_of(g.K), static_cast<int*>(ws), device_error_word()};
    if (!p.err)
        return cudaErrorInvalidValue;
    return g.y_type == 0 ? pick<float>(p, st) : pick<__nv_bfloat16>(p, st);
}

} // namespace repro
