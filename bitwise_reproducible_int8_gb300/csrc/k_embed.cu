// k_embed.cu -- token embedding with a scale, and the table's gradient in a
// fixed order.
//
// Forward: out_i = W[tok_i] (x) scale.  One read of the distinct rows, one write
// of n x D: bound by HBM.  A warp takes a 512-column piece of one row, four
// 4-element groups per lane in flight, so that a wide row spreads over several
// warps and few tokens over many SMs.  16,384 tokens of 2048 out of 32768 x 2048:
// 31.3 us, 5.8 TB/s (0.86 of a copy's).
//
// Backward: dW_v = canonical sum over {i : tok_i = v}, i ascending, of dout_i,
// (x) scale.  An atomic add per element would be shorter and its order, so its
// bits, would change from run to run; here the positions are sorted by token
// (stably, so ascending within a token) and every table element is summed by one
// thread in the canonical order:
//   1. k_embed_sort: one cluster of 8 CTAs sorts (token, position) by 8 bits a
//      pass and marks where chunks of up to 64 positions begin.  The other clusters
//      of the same launch zero the table rows that no token names (each marks its
//      own rows' tokens in a bitmap first), so the sort hides behind the part of the
//      write that needs no order.  Few tokens: k_embed_rank, every token's place by
//      counting, over the whole card and without passes.
//   2. k_embed_sum: the rows in sorted order as one stream per warp and piece of the
//      columns, left to right from each chunk's first term; a token's only chunk is
//      scaled and stored, others leave their partial row in the workspace.
//   3. k_row_tree (k_rowtree.cu): the pairwise tree over a token's partial rows;
//      only launched when n > 64, below which no token can have two chunks.
// 16,384 tokens (text-like frequencies) into 32768 x 2048: 83 to 86 us, 4.8 TB/s: 41 us
// zeroing beside the sort, 36 summing (rows read in sorted order, 4.9 TB/s), 7 the tree;
// added into an existing gradient 67 us, 301 tokens 10 us.  With bf16 gradient rows, loads of 8
// bytes a lane, 123 and 98 us.
#include <cooperative_groups.h>

#include <atomic>

#include "elem.cuh"
#include "internal.h"
#include "launch.cuh"

namespace cg = cooperative_groups;

namespace repro {
namespace {

typedef unsigned long long u64;

// ---------------------------------------------------------------- forward

constexpr int EF_U = 4;            // 4-element groups per lane
constexpr int EF_COLS = 32 * 4 * EF_U;

__device__ __forceinline__ float4 table4(const float* p, float) { return flush4(load4(p)); }
__device__ __forceinline__ float4 table4(const __nv_bfloat16* p, float) { return flush4(load4(p)); }
__device__ __forceinline__ float4 table4(const int8_t* p, float s)
{
    const char4 q = *reinterpret_cast<const char4*>(p);
    return make_float4(dequant((signed char)q.x, s), dequant((signed char)q.y, s),
                       dequant((signed char)q.z, s), dequant((signed char)q.w, s));
}
__device__ __forceinline__ float table1(const float* p, float) { return flush(*p); }
__device__ __forceinline__ float table1(const __nv_bfloat16* p, float) { return flush(__bfloat162float(*p)); }
__device__ __forceinline__ float table1(const int8_t* p, float s) { return dequant(*p, s); }

template <typename TT, typename TO, bool VEC>
__global__ void __launch_bounds__(256)
k_embed_fwd(const TT* __restrict__ table, int64_t table_ld, const float* __restrict__ s_w,
            const void* __restrict__ tokens, int index_bytes, int64_t n, int64_t V, int64_t D,
            float scale, int64_t pad, TO* __restrict__ out, int64_t out_ld, int segs, int* err)
{
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (item >= n * segs)
        return;
    const int64_t row = item / segs;
    const int64_t c0 = (item - row * segs) * EF_COLS;
    const int64_t tok = load_index(tokens, index_bytes, row);
    const bool ok = tok >= 0 && tok < V && tok != pad;
    if (!ok && tok != pad && c0 == 0 && lane == 0)
        atomicOr(err, kErrIndexBit);
    const float sw = s_w ? flush(*s_w) : 0.0f;
    const float sc = flush(scale);
    const TT* src = table + (ok ? tok : 0) * table_ld;
    TO* dst = out + row * out_ld;
    if (VEC) {
        float4 v[EF_U];
#pragma unroll
        for (int u = 0; u < EF_U; ++u) {
            const int64_t c = c0 + 4 * (lane + 32 * u);
            if (c < D)
                v[u] = ok ? table4(src + c, sw) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int u = 0; u < EF_U; ++u) {
            const int64_t c = c0 + 4 * (lane + 32 * u);
            if (c < D) {
                float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (ok)
                    r = make_float4(fmul_flush(v[u].x, sc), fmul_flush(v[u].y, sc),
                                    fmul_flush(v[u].z, sc), fmul_flush(v[u].w, sc));
                store4(dst + c, r);
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < 4 * EF_U; ++u) {
            const int64_t c = c0 + lane + 32 * u;
            if (c < D)
                dst[c] = from_f32<TO>(ok ? fmul_flush(table1(src + c, sw), sc) : 0.0f);
        }
    }
}

// ---------------------------------------------------------------- sort

constexpr int SORT_CTAS = 8;      // CTAs of the sorting cluster
constexpr int SORT_NT = 1024;
constexpr int SORT_W = SORT_NT / 32;
constexpr int DIGITS = 256;
constexpr int ZERO_BYTES = 16384; // zeroed shared memory that bulk copies read
constexpr int ZERO_WARPS = 8;     // warps whose first lane issues them
// what begins at a sorted index: a chunk with a partial row (>= 0), a token's only
// chunk, nothing (inside a chunk), or no token at all (padding, out of range: the end)
constexpr int WHOLE = -1, MIDDLE = -2, NOTHING = -3;

struct SortArgs {
    const void* tokens;
    int index_bytes;
    int n, V;
    int passes;
    int64_t pad;
    uint2* a;            // (token, position), written by passes 0, 2, ..
    uint2* b;            // .. and by passes 1, 3
    int2* seg;           // [V] first and one past the last sorted index of a named token
    int* counts;         // tokens with several chunks
    int4* order;         // [n] {position, token, what begins here, the token's positions}
    float* table;        // rows to zero, or NULL
    int64_t table_ld;
    int64_t D;
    bool vec;            // the table's rows begin on 16 bytes
    int* err;
};

struct SortSmem {
    unsigned hist[SORT_W][DIGITS];   // per warp, then its running offsets
    unsigned total[DIGITS];          // this CTA's digit counts (read by the cluster)
    unsigned warp_total[DIGITS / 32];
};

__device__ __forceinline__ unsigned sort_key(const SortArgs& a, int i, bool report)
{
    const int64_t t = load_index(a.tokens, a.index_bytes, i);
    if (t >= 0 && t < a.V && t != a.pad)
        return (unsigned)t;
    if (report && t != a.pad)
        atomicOr(a.err, kErrIndexBit);
    return (unsigned)a.V;
}

__device__ __forceinline__ uint2 ld_pair(const uint2* p) { return __ldcg(p); }
__device__ __forceinline__ unsigned ld_tok(const uint2* s, int i) { return __ldcg(&s[i].x); }

__device__ void sort_cluster(const SortArgs& a, SortSmem& sm)
{
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // each warp owns a run of 32-element rounds, so that (CTA, warp, round, lane) is position order
    const int rounds = (a.n + SORT_CTAS * SORT_NT - 1) / (SORT_CTAS * SORT_NT);
    const int base = (rank * SORT_W + warp) * rounds * 32;
    if (rank == 0 && tid == 0)
        a.counts[0] = 0;
    const uint2* src = nullptr;
    uint2* dst = a.a;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = 8 * pass;
        for (int i = tid; i < SORT_W * DIGITS; i += SORT_NT)
            (&sm.hist[0][0])[i] = 0;
        __syncthreads();
        for (int r = 0; r < rounds; ++r) {
            const int i = base + 32 * r + lane;
            const bool in = i < a.n;
            const unsigned key = !in ? 0u : pass == 0 ? sort_key(a, i, true) : ld_tok(src, i);
            const unsigned d = in ? (key >> shift) & (DIGITS - 1) : (unsigned)DIGITS;
            const unsigned same = __match_any_sync(0xffffffffu, d);
            if (in && lane == __ffs(same) - 1)
                sm.hist[warp][d] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        if (tid < DIGITS) {
            unsigned run = 0;
            for (int w = 0; w < SORT_W; ++w) {
                const unsigned c = sm.hist[w][tid];
                sm.hist[w][tid] = run;
                run += c;
            }
            sm.total[tid] = run;
        }
        cluster.sync();
        if (tid < DIGITS) {
            unsigned before = 0, all = 0;
            for (int r = 0; r < SORT_CTAS; ++r) {
                const unsigned c = cluster.map_shared_rank(&sm, r)->total[tid];
                before += r < rank ? c : 0u;
                all += c;
            }
            // exclusive scan of the digit counts: within warps, then over the 8 warps
            unsigned inc = all;
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o)
                    inc += up;
            }
            if (lane == 31)
                sm.warp_total[warp] = inc;
            asm volatile("bar.sync 1, 256;" ::: "memory");   // the eight warps that hold the digits
            unsigned off = 0;
            for (int w = 0; w < warp; ++w)
                off += sm.warp_total[w];
            const unsigned start = inc - all + off + before;
            for (int w = 0; w < SORT_W; ++w)
                sm.hist[w][tid] += start;
        }
        __syncthreads();
        for (int r = 0; r < rounds; ++r) {
            const int i = base + 32 * r + lane;
            const bool in = i < a.n;
            uint2 kv = make_uint2(0u, 0u);
            if (in)
                kv = pass == 0 ? make_uint2(sort_key(a, i, false), (unsigned)i) : ld_pair(src + i);
            const unsigned d = in ? (kv.x >> shift) & (DIGITS - 1) : (unsigned)DIGITS;
            const unsigned same = __match_any_sync(0xffffffffu, d);
            unsigned at = 0;
            if (in)
                at = sm.hist[warp][d] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (in) {
                dst[at] = kv;
                if (lane == __ffs(same) - 1)
                    sm.hist[warp][d] += __popc(same);
            }
            __syncwarp();
        }
        __threadfence();
        cluster.sync();   // the scattered pairs are visible to the cluster, and total[] free again
        src = dst;
        dst = dst == a.a ? a.b : a.a;
    }
    // where every named token's positions begin and end
    for (int i = rank * SORT_NT + tid; i < a.n; i += SORT_CTAS * SORT_NT) {
        const unsigned key = ld_tok(src, i);
        if (key >= (unsigned)a.V)
            continue;
        if (i == 0 || ld_tok(src, i - 1) != key)
            a.seg[key].x = i;
        if (i == a.n - 1 || ld_tok(src, i + 1) != key)
            a.seg[key].y = i + 1;
    }
    __threadfence();
    cluster.sync();
    // sorted index i begins a chunk when it is a multiple of 64 past its token's first
    for (int i = rank * SORT_NT + tid; i < a.n; i += SORT_CTAS * SORT_NT) {
        const uint2 kv = ld_pair(src + i);
        int what = NOTHING, length = 0;
        if (kv.x < (unsigned)a.V) {
            const int2 g = __ldcg(&a.seg[kv.x]);
            const bool several = g.y - g.x > 64;
            what = MIDDLE;
            // a partial row of its own: in a run of 64 sorted indexes at most one chunk of a
            // token with several starts that is its first, and at most one that is not
            if (((i - g.x) & 63) == 0)
                what = several ? 2 * (i >> 6) + (g.x == i ? 1 : 0) : WHOLE;
            length = g.y - g.x;
        }
        a.order[i] = make_int4((int)kv.y, (int)kv.x, what, length);
    }
}

// zeroes the table rows in [v0, v1) whose bit is not set, by all of the CTA's threads; `zero`
// is ZERO_BYTES of shared memory.  Where rows lie on 16 bytes the copy engine writes them
// out of zeroed shared memory, one instruction a row (268 MB at 6.2 TB/s, as plain stores from
// all threads); zero_wait() is due before the CTA ends.  Leaving part of this to the
// sums' kernel made the call longer: 84 -> 94 us with 96 MB written here, 89 with 140.
__device__ void zero_unnamed(const SortArgs& a, const unsigned* bits, float4* zero, int v0, int v1)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    if (!a.vec) {
        for (int v = v0 + warp; v < v1; v += threads / 32) {
            if (bits[(v - v0) >> 5] >> ((v - v0) & 31) & 1u)
                continue;
            float* row = a.table + (int64_t)v * a.table_ld;
            for (int64_t c = lane; c < a.D; c += 32)
                row[c] = 0.0f;
        }
        return;
    }
    for (int i = tid; i < ZERO_BYTES / 16; i += threads)
        zero[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    const unsigned src = (unsigned)__cvta_generic_to_shared(zero);
    if (warp < ZERO_WARPS && lane == 0) {
        for (int v = v0 + warp; v < v1; v += ZERO_WARPS) {
            if (bits[(v - v0) >> 5] >> ((v - v0) & 31) & 1u)
                continue;
            char* row = reinterpret_cast<char*>(a.table + (int64_t)v * a.table_ld);
            for (int64_t o = 0; o < a.D * 4; o += ZERO_BYTES) {
                const unsigned len = (unsigned)(a.D * 4 - o < ZERO_BYTES ? a.D * 4 - o : ZERO_BYTES);
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                             :: "l"(row + o), "r"(src), "r"(len) : "memory");
            }
        }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// until this thread's copies have read shared memory and written their rows
__device__ __forceinline__ void zero_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// zeroes the table rows in [v0, v1) that no token names
__device__ void zero_rows(const SortArgs& a, unsigned* bits, int v0, int v1)
{
    const int tid = threadIdx.x;
    const int words = (v1 - v0 + 31) / 32;
    for (int i = tid; i < words; i += SORT_NT)
        bits[i] = 0u;
    __syncthreads();
    for (int i0 = tid; i0 < a.n; i0 += 8 * SORT_NT) {
        int64_t t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            t[u] = i0 + u * SORT_NT < a.n ? load_index(a.tokens, a.index_bytes, i0 + u * SORT_NT) : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (t[u] >= v0 && t[u] < v1 && t[u] != a.pad)
                atomicOr(&bits[(t[u] - v0) >> 5], 1u << ((t[u] - v0) & 31));
    }
    __syncthreads();
    zero_unnamed(a, bits, reinterpret_cast<float4*>(bits + ((words + 31) & ~31)), v0, v1);
    zero_wait();
}

__global__ void __cluster_dims__(SORT_CTAS, 1, 1) __launch_bounds__(SORT_NT, 1)
k_embed_sort(const SortArgs a)
{
    extern __shared__ __align__(128) unsigned dyn[];
    pdl_trigger();   // the sums may be launched; they wait for this grid
    if (blockIdx.x < SORT_CTAS) {
        sort_cluster(a, *reinterpret_cast<SortSmem*>(dyn));
    } else {
        const int ctas = gridDim.x - SORT_CTAS, c = blockIdx.x - SORT_CTAS;
        const int per = (a.V + ctas - 1) / ctas;
        const int64_t v0 = (int64_t)c * per, v1 = v0 + per < a.V ? v0 + per : a.V;
        if (v0 < v1)
            zero_rows(a, dyn, (int)v0, (int)v1);
    }
}

// ---------------------------------------------------------------- order of few tokens

constexpr int RANK_NT = 512;
constexpr int RANK_W = RANK_NT / 32;
// Up to this many tokens are put in order by counting, alone and beside the zeroing of a
// table (by counting against by passes, 32768 x 2048, us: added into a gradient 301 tokens
// 10 and 19, 4096 31 and 36, 8192 51 and 40; into a new one 2048 63 and 63, 4096 70 and 66)
constexpr int RANKED = 4096, RANKED_NEW = 2048;

// A CTA takes 32 tokens, a lane each, and counts against all n how many are smaller and
// how many equal, before it and in all; its warps share the n.  That is the token's
// place, its chunk and its segment's length at once, with nothing to wait for.  Every CTA
// also has its share of the table rows to zero, which the copy engine does meanwhile.
__global__ void __launch_bounds__(RANK_NT)
k_embed_rank(const SortArgs a, int ranks, int per)
{
    extern __shared__ __align__(128) unsigned dyn[];
    __shared__ int sums[RANK_W][3][32];
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0 && tid == 0)
        a.counts[0] = 0;
    const int padded = (a.n + 127) & ~127, words = (per + 31) / 32;
    unsigned* bits = dyn + padded;
    for (int i = tid; i < padded; i += RANK_NT)   // past the end: larger than every key
        dyn[i] = i < a.n ? sort_key(a, i, blockIdx.x == 0) : 0xffffffffu;
    for (int i = tid; i < words; i += RANK_NT)
        bits[i] = 0u;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * per;
    const int v0 = (int)(first < a.V ? first : a.V), v1 = (int)(first + per < a.V ? first + per : a.V);
    if (v0 < v1) {
        for (int i = tid; i < a.n; i += RANK_NT)
            if ((int)dyn[i] >= v0 && (int)dyn[i] < v1)
                atomicOr(&bits[((int)dyn[i] - v0) >> 5], 1u << (((int)dyn[i] - v0) & 31));
        __syncthreads();
        zero_unnamed(a, bits, reinterpret_cast<float4*>(bits + ((words + 31) & ~31)), v0, v1);
    }
    if (blockIdx.x >= ranks) {
        zero_wait();
        return;
    }
    const int i0 = blockIdx.x * 32, i = i0 + lane;
    const unsigned own = i < a.n ? dyn[i] : 0u;
    int less = 0, upto = 0, before = 0;   // smaller; smaller or equal; equal and earlier
    for (int j = 4 * warp; j < padded; j += 4 * RANK_W) {
        const uint4 k = *reinterpret_cast<const uint4*>(dyn + j);
        const unsigned q[4] = {k.x, k.y, k.z, k.w};
        int l = 0, u = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            l += q[e] < own;
            u += q[e] <= own;
        }
        less += l;
        upto += u;
        if (j < i0) {
            before += u - l;
        } else if (j < i0 + 32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                before += q[e] == own && j + e < i;
        }
    }
    sums[warp][0][lane] = less;
    sums[warp][1][lane] = upto;
    sums[warp][2][lane] = before;
    __syncthreads();
    zero_wait();
    if (warp > 0 || i >= a.n)
        return;
    for (int w = 1; w < RANK_W; ++w) {
        less += sums[w][0][lane];
        upto += sums[w][1][lane];
        before += sums[w][2][lane];
    }
    const int at = less + before, length = upto - less;
    int what = NOTHING;
    if (own < (unsigned)a.V) {
        what = MIDDLE;
        if ((before & 63) == 0)
            what = length > 64 ? 2 * (at >> 6) + (before == 0 ? 1 : 0) : WHOLE;
    }
    a.order[at] = make_int4(i, (int)own, what, length);
}

// ---------------------------------------------------------------- chunk sums

constexpr int ES_G = 2;             // 4-element groups per lane
constexpr int ES_U = 8;             // rows in flight
constexpr int ES_COLS = 32 * 4 * ES_G;
constexpr int ES_CTAS = 2;          // per SM

// A row's piece in a lane: ES_G groups of four columns.  Group g begins
// at column c0 + 4 (lane + 32 g); where rows are not on 4-element boundaries its elements
// are c0 + lane + 32 (4 g + e) instead.
template <bool VEC> __device__ __forceinline__ int64_t sum_col(int64_t c0, int lane, int g, int e)
{
    return c0 + (VEC ? 4 * (lane + 32 * g) + e : lane + 32 * (4 * g + e));
}

// left as single floats until they are added: packing them here would wait for the load
template <typename TD, bool VEC>
__device__ __forceinline__ void sum_load(const TD* s, int64_t c0, int64_t D, int lane, float (&x)[ES_G][4])
{
#pragma unroll
    for (int g = 0; g < ES_G; ++g) {
        if (VEC) {
            if (sum_col<VEC>(c0, lane, g, 0) < D) {
                const float4 v = stream4(s + sum_col<VEC>(c0, lane, g, 0));
                x[g][0] = v.x, x[g][1] = v.y, x[g][2] = v.z, x[g][3] = v.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (sum_col<VEC>(c0, lane, g, e) < D)
                    x[g][e] = to_f32<TD>(s[sum_col<VEC>(c0, lane, g, e)]);
        }
    }
}

// table (+) v where this is the only addition the element gets: the memory's own binary32
// addition rounds to nearest and flushes subnormals like fadd_ftz, and the warp does not
// wait for the old value (reading it first made the accumulating call 1.3 times as long)
__device__ __forceinline__ void add_once(float* p, float4 v)
{
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};"
                 :: "l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// a finished chunk: a partial row as it is, a token's only chunk scaled into the table
template <bool VEC>
__device__ __forceinline__ void sum_store(float* dst, bool part, bool wide, bool accumulate, float sc, int64_t c0,
                                          int64_t D, int lane, const u64 (&acc)[ES_G][2])
{
#pragma unroll
    for (int g = 0; g < ES_G; ++g) {
        float v[4];
        unpack2(acc[g][0], v[0], v[1]);
        unpack2(acc[g][1], v[2], v[3]);
        if (!part) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = fmul_flush(v[e], sc);
        }
        const int64_t c = sum_col<VEC>(c0, lane, g, 0);
        if (VEC && wide) {
            if (c >= D)
                continue;
            if (!part && accumulate)
                add_once(dst + c, make_float4(v[0], v[1], v[2], v[3]));
            else
                store4(dst + c, make_float4(v[0], v[1], v[2], v[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t ce = sum_col<VEC>(c0, lane, g, e);
                if (ce < D) {
                    if (!part && accumulate)
                        atomicAdd(dst + ce, v[e]);
                    else
                        dst[ce] = v[e];
                }
            }
        }
    }
}

// A warp takes the chunks that begin among `span` sorted indexes, for one piece of the
// columns, as one stream of rows: 8 rows are on their way at any time, across the chunks'
// ends (most tokens occur once or twice; chunk by chunk every one cost a trip to
// memory).  `span` leaves one stream to a warp.  What a row needs of the order is its
// position and one bit; the rest is looked up where a chunk begins.
template <typename TD, bool VEC>
__global__ void __launch_bounds__(256, ES_CTAS)
k_embed_sum(const TD* __restrict__ dout, int64_t dout_ld, const int4* __restrict__ order, int n, int span,
            int64_t D, float scale, float* __restrict__ table, int64_t table_ld, bool accumulate,
            float* __restrict__ parts, int pieces, bool vec_out, int4* __restrict__ joins, int* njoins)
{
    pdl_wait();
    pdl_trigger();
    constexpr unsigned ALL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const float sc = flush(scale);
    const int64_t pitch = (D + 3) & ~3LL;
    const u64 zero = pack2(-0.0f, -0.0f);
    const int64_t items = (int64_t)((n + span - 1) / span) * pieces;
    for (int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); item < items; item += (int64_t)gridDim.x * 8) {
        const int range = (int)(item / pieces);
        const int64_t c0 = (item - (int64_t)range * pieces) * ES_COLS;
        const int lo = range * span, hi = min(n, lo + span);
        // the first index of the range at which a chunk begins
        int at = hi;
        for (int i = lo; i < hi && at == hi; i += 32) {
            const unsigned m = __ballot_sync(ALL, i + lane < hi && order[i + lane].z >= WHOLE);
            if (m)
                at = i + __ffs(m) - 1;
        }
        if (at >= hi)
            continue;
        // 32 entries of the order at a time, the next 32 fetched ahead; the stream ends at
        // `end`: the first chunk past the range, the first index without a token, or n
        const int4 none = make_int4(0, 0, NOTHING, 0);
        int end = n;
        auto window = [&](int from, int4& v, unsigned& starts) {
            v = from + lane < n ? order[from + lane] : none;
            starts = __ballot_sync(ALL, v.z != MIDDLE);
            const unsigned stop = __ballot_sync(ALL, v.z == NOTHING || (v.z != MIDDLE && from + lane >= hi));
            if (stop)
                end = min(end, from + __ffs(stop) - 1);
        };
        int4 cur, ahead;
        unsigned starts, starts_ahead;
        window(at, cur, starts);
        window(at + 32, ahead, starts_ahead);
        float x[ES_U][ES_G][4] = {};
        u64 acc[ES_G][2] = {};
        auto fetch = [&](int k, float (&v)[ES_G][4]) {   // row k < 64 of the window
            const int pos = __shfl_sync(ALL, k < 32 ? cur.x : ahead.x, k & 31);
            if (at + k < end)
                sum_load<TD, VEC>(dout + (int64_t)pos * dout_ld, c0, D, lane, v);
        };
#pragma unroll
        for (int u = 0; u < ES_U; ++u)
            fetch(u, x[u]);
        int slot = 0, row = -1;   // the open chunk: partial row or WHOLE, token
        int k = 0;                // window index of the row in x[0]
        for (bool done = false; !done;) {
#pragma unroll
            for (int u = 0; u < ES_U; ++u) {
                // (one place for both ends of a chunk: the loop is unrolled and has to stay in
                // the instruction cache; two took the call from 86 to 133 us)
                const bool over = at + k + u >= end;
                if (over || (starts >> (k + u) & 1u)) {
                    if (row >= 0)
                        sum_store<VEC>(slot >= 0 ? parts + (int64_t)slot * pitch : table + (int64_t)row * table_ld,
                                       slot >= 0, slot >= 0 || vec_out, accumulate, sc, c0, D, lane, acc);
                    slot = __shfl_sync(ALL, cur.z, k + u);
                    row = __shfl_sync(ALL, cur.y, k + u);
                    row = over ? -1 : row;
                    done = over;
                    if (c0 == 0 && !over && slot >= 0 && (slot & 1) && lane == k + u)   // a token's first of several
                        joins[atomicAdd(njoins, 1)] = make_int4(at + k + u, (cur.w + 63) / 64, row, 0);
#pragma unroll
                    for (int g = 0; g < ES_G; ++g)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            acc[g][e] = fadd2_ftz(pack2(x[u][g][2 * e], x[u][g][2 * e + 1]), zero);
                } else {
#pragma unroll
                    for (int g = 0; g < ES_G; ++g)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            acc[g][e] = fadd2_ftz(acc[g][e], pack2(x[u][g][2 * e], x[u][g][2 * e + 1]));
                }
                fetch(k + ES_U + u, x[u]);
            }
            k += ES_U;
            if (k == 32) {
                at += 32;
                k = 0;
                cur = ahead;
                starts = starts_ahead;
                window(at + 32, ahead, starts_ahead);
            }
        }
    }
}

// workspace: sorted pairs twice, chunk and join lists, counters, partial rows
struct EmbedWs {
    size_t a, b, seg, order, joins, counts, parts, total;
};

EmbedWs embed_ws(int64_t n, int64_t V, int64_t D)
{
    EmbedWs w;
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    const int64_t blocks = (n + 63) / 64;
    w.a = 0;
    w.b = w.a + up((size_t)n * 8);
    w.seg = w.b + up((size_t)n * 8);
    w.order = w.seg + up((size_t)V * 8);
    w.joins = w.order + up((size_t)n * 16);
    w.counts = w.joins + up((size_t)blocks * 16);
    w.parts = w.counts + 256;
    // a token with several chunks has more than 64 positions
    w.total = w.parts + (n > 64 ? (size_t)(2 * blocks) * (size_t)((D + 3) & ~3LL) * 4 : 0);
    return w;
}

// Shared memory that the first launch may ask for: a bitmap of REPRO_EMBED_MAX_V / 56 rows and
// the zeros (a constant: what one call sets is every host thread's limit)
constexpr int FIRST_SMEM = 54 * 1024;
static_assert((16777215 / 56 + 32) / 32 * 4 + 128 + ZERO_BYTES <= FIRST_SMEM, "fill_ctas() is 56 at least");

// CTAs that may zero rows beside the sorting cluster: a cluster's CTAs share a GPC,
// so fewer clusters than SMs / 8 run at a time, and one more would start when the
// others are done (all 18 of them: 57 us for 268 MB instead of 43)
int fill_ctas()
{
    static std::atomic<int> known{0};
    int v = known.load(std::memory_order_relaxed);
    if (v == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(SORT_CTAS);
        cfg.blockDim = dim3(SORT_NT);
        cfg.dynamicSmemBytes = sizeof(SortSmem);
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, k_embed_sort, &cfg) != cudaSuccess)
            cudaGetLastError();
        v = (clusters < 8 ? 7 : clusters - 1) * SORT_CTAS;
        known.store(v, std::memory_order_relaxed);
    }
    return v;
}

template <typename TT, typename TO>
cudaError_t fwd_typed(const EmbedFwdArgs& a, cudaStream_t st)
{
    const int segs = (int)((a.D + EF_COLS - 1) / EF_COLS);
    const int64_t ctas = (a.n * segs + 7) / 8;
    const bool vec = a.D % 4 == 0 && rows4<TT>(a.table, a.table_ld) && rows4<TO>(a.out, a.out_ld);
    const TT* table = static_cast<const TT*>(a.table);
    TO* out = static_cast<TO*>(a.out);
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)ctas, 256, 0, st>>>(table, a.table_ld, a.s_w, a.tokens, a.index_bytes, a.n, a.V,
                                               a.D, a.scale, a.pad, out, a.out_ld, segs, a.err);
    };
    if (vec)
        go(k_embed_fwd<TT, TO, true>);
    else
        go(k_embed_fwd<TT, TO, false>);
    count_launches(1);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, cudaStream_t st)
{
    const bool of = a.out_type == 0;
    switch (a.table_type) {
    case 0: return of ? fwd_typed<float, float>(a, st) : fwd_typed<float, __nv_bfloat16>(a, st);
    case 1: return of ? fwd_typed<__nv_bfloat16, float>(a, st) : fwd_typed<__nv_bfloat16, __nv_bfloat16>(a, st);
    default: return of ? fwd_typed<int8_t, float>(a, st) : fwd_typed<int8_t, __nv_bfloat16>(a, st);
    }
}

size_t embed_bwd_ws_bytes(int64_t n, int64_t V, int64_t D) { return embed_ws(n, V, D).total; }

cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, void* ws, cudaStream_t st)
{
    const EmbedWs w = embed_ws(a.n, a.V, a.D);
    char* p = static_cast<char*>(ws);
    SortArgs s;
    s.tokens = a.tokens;
    s.index_bytes = a.index_bytes;
    s.n = (int)a.n;
    s.V = (int)a.V;
    s.pad = a.pad;
    s.a = reinterpret_cast<uint2*>(p + w.a);
    s.b = reinterpret_cast<uint2*>(p + w.b);
    s.seg = reinterpret_cast<int2*>(p + w.seg);
    s.order = reinterpret_cast<int4*>(p + w.order);
    int4* joins = reinterpret_cast<int4*>(p + w.joins);   // {first sorted index, chunks, token, 0}
    s.counts = reinterpret_cast<int*>(p + w.counts);
    s.table = a.table;
    s.table_ld = a.table_ld;
    s.D = a.D;
    s.vec = a.D % 4 == 0 && rows4<float>(a.table, a.table_ld);
    s.err = a.err;
    s.passes = 1;
    while (((int64_t)1 << (8 * s.passes)) <= a.V)   // keys 0 .. V
        ++s.passes;
    const bool ranked = a.n <= (a.accumulate ? RANKED : RANKED_NEW);
    // zeroing: beside the cluster, or a share for every CTA, two per SM
    const int ranks = (int)((a.n + 31) / 32);
    const int fill = a.accumulate ? 0 : ranked ? 2 * num_sms() : fill_ctas();
    const int per = fill > 0 ? (int)((a.V + fill - 1) / fill) : 0;
    const size_t fill_smem = fill > 0 ? (size_t)(per + 31) / 32 * 4 + 128 + ZERO_BYTES : 0;   // a bitmap and the zeros
    const size_t smem = ranked ? (size_t)((a.n + 127) & ~127LL) * 4 + fill_smem
                               : fill_smem > sizeof(SortSmem) ? fill_smem : sizeof(SortSmem);
    const int ctas = ranks > fill ? ranks : fill;
    auto first = [&](auto kernel, auto launch) {
        if (smem > 40 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FIRST_SMEM);
            if (e != cudaSuccess)
                return e;
        }
        launch();
        count_launches(1);
        return cudaGetLastError();
    };
    cudaError_t e = cudaSuccess;
    if (!ranked)
        e = first(k_embed_sort, [&] { k_embed_sort<<<SORT_CTAS + fill, SORT_NT, smem, st>>>(s); });
    else if (ctas > 0)
        e = first(k_embed_rank, [&] { k_embed_rank<<<ctas, RANK_NT, smem, st>>>(s, ranks, per); });
    if (e != cudaSuccess || a.n == 0)
        return e;
    float* parts = reinterpret_cast<float*>(p + w.parts);
    const int pieces = (int)((a.D + ES_COLS - 1) / ES_COLS);
    const int64_t warps = (int64_t)num_sms() * ES_CTAS * 8;
    const int span = (int)((a.n * pieces + warps - 1) / warps);
    const int64_t most = ((a.n + span - 1) / span * pieces + 7) / 8, cap = warps / 8;
    const unsigned grid = (unsigned)(most < cap ? most : cap);
    const bool vec_out = s.vec;
    auto sum = [&](auto type) {
        using T = decltype(type);
        auto go = [&](auto kernel) {
            return launch_pdl(kernel, dim3(grid), dim3(256), 0, st, static_cast<const T*>(a.dout), a.dout_ld,
                              (const int4*)s.order, (int)a.n, span, a.D, a.scale, a.table, a.table_ld,
                              a.accumulate, parts, pieces, vec_out, joins, s.counts);
        };
        return a.D % 4 == 0 && rows4<T>(a.dout, a.dout_ld) ? go(k_embed_sum<T, true>) : go(k_embed_sum<T, false>);
    };
    e = a.dout_type == 0 ? sum(float()) : sum(__nv_bfloat16());
    count_launches(1);
    if (e != cudaSuccess || a.n <= 64)
        return e;
    RowTree t = {};
    t.parts[0] = parts;
    t.pitch = (a.D + 3) & ~3LL;
    t.joins = joins;
    t.njoins = s.counts;
    t.D = a.D;
    t.out[0] = a.table;
    t.out_ld = a.table_ld;
    t.scale = a.scale;
    t.accumulate = a.accumulate;
    return launch_row_tree(t, num_sms() * 8, st);
}

} // namespace repro
