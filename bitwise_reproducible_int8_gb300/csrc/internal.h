// internal.h -- launchers shared between the C-ABI layer (api.cu) and the
// kernel translation units.  Arguments are already validated by the caller.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#define REPRO_MAX_PARTS_INTERNAL 64
#define REPRO_MAX_TENSORS_INTERNAL 64

namespace repro {

struct LaunchCfg {
    int bwd_segment_log2;   // chunks per backward reduction segment = 2^k (0..8)
    int reduce_block_log2;  // chunk partials per block in the scale reduction (0..10)
    int fwd_path;           // 0: CUDA-core exact path, 1: tensor cores 128 x 256 tiles, 2: 128 x 128
    int elementwise_blocks; // 0: default grid for streaming kernels
    int bwd_kernel;         // 8: tensor-copy-fed kernel (default), 1: register-prefetch kernel
    int fwd_selftest;       // -1: gate the tensor-core forward on its self-test; 1: treat it as failed
};

const LaunchCfg& launch_cfg();
// debug mode (repro_set_debug): the scans of a call's float inputs, enqueued
// before its kernels; REPRO_OK, or REPRO_ERR_LAUNCH if one could not be enqueued
struct FloatSpan {
    const float* p;
    int64_t n;
};
int scan_inputs(void* stream, std::initializer_list<FloatSpan> spans);
int num_sms();
int* device_error_word();   // device address of the error word: bit 0 a bounded wait gave up,
                            // bit 1 the debug scan found a non-finite input,
                            // bit 2 a token, position, index or label out of range
constexpr int kErrTimeoutBit = 1, kErrNonfiniteBit = 2, kErrIndexBit = 4;
int arch_status();          // REPRO_OK when the current device is a GB300
void count_launches(int k); // adds k to the process-wide launch counter
// status code of a CUDA runtime result, the same for every entry point
inline int status_of(cudaError_t e) { return e == cudaSuccess ? 0 : -5; }   // REPRO_OK / REPRO_ERR_LAUNCH

// ---- scale (k_scale.cu)
size_t wscale_ws_bytes(int64_t n, int block_log2);
cudaError_t launch_wscale_meanabs(const float* x, int64_t n, int qmax, float* scale_out,
                                  void* ws, int block_log2, cudaStream_t st);
cudaError_t launch_wscale_amax(const float* x, int64_t n, int qmax, float* scale_out,
                               void* ws, int grid, cudaStream_t st);
int amax_grid(int64_t n);
// several tensors in one pass: scales[t] of xs[t] (mode 0 weight, 1 activation)
size_t wscale_multi_ws_bytes(const int64_t* ns, int count);
cudaError_t launch_wscale_multi(const float* const* xs, const int64_t* ns, int count, int mode,
                                int qmax, float* scales, void* ws, int block_log2,
                                cudaStream_t st);

cudaError_t launch_sumsq(const float* x, int64_t n, float* out, void* ws, int block_log2,
                         cudaStream_t st);

// ---- optimiser (k_optim.cu)
struct AdamWArgs {
    float lr, beta1, beta2, eps, weight_decay, max_norm;
};
cudaError_t launch_adamw(float* p, float* m, float* v, const float* g, int64_t n,
                         const float* sumsq, const AdamWArgs& h, int64_t t, int grid,
                         cudaStream_t st);

// ---- quantiser (k_quant.cu)
cudaError_t launch_quant(const float* x, int64_t n, const float* scale, int qmax, int8_t* q,
                         int grid, cudaStream_t st);
cudaError_t launch_quant_multi(const float* const* xs, const int64_t* ns, int count,
                               const float* scales, int qmax, int8_t* const* qs, int grid,
                               cudaStream_t st);

// ---- forward (k_fwd.cu)
cudaError_t launch_fwd_cuda_core(const int8_t* xq, const int8_t* wq, const float* s_x,
                                 const float* s_w, float* y, int64_t M, int64_t N, int64_t K,
                                 cudaStream_t st);

// ---- forward on tensor cores (k_fwd_tc.cu)
bool fwd_tc_supported(int64_t M, int64_t N, int64_t K);
size_t fwd_tc_ws_bytes(int64_t M, int64_t N, int64_t K);
cudaError_t launch_fwd_tc(const int8_t* xq, const int8_t* wq, const float* s_x, const float* s_w,
                          float* y, int64_t M, int64_t N, int64_t K, void* ws, bool wide,
                          cudaStream_t st);

// ---- backward (k_bwd.cu)
size_t bwd_ws_bytes(int64_t M, int64_t N, int64_t K, int seg_log2);
cudaError_t launch_bwd_dx(const float* dy, const int8_t* wq, const float* s_w, float* dx,
                          int64_t M, int64_t N, int64_t K, int seg_log2, float* ws,
                          cudaStream_t st);
cudaError_t launch_bwd_dw(const float* dy, const int8_t* xq, const float* s_x, float* dw,
                          int64_t M, int64_t N, int64_t K, int seg_log2, bool accumulate,
                          float* ws, cudaStream_t st);

// ---- reductions (k_reduce.cu)
cudaError_t launch_grad_accum(float* acc, const float* g, int64_t n, int grid, cudaStream_t st);
cudaError_t launch_running_sum(const float* const* parts, int S, int64_t n, float* out, int grid,
                               cudaStream_t st);
cudaError_t launch_treefold(const float* const* parts, int R, int64_t n, float* out, int grid,
                            cudaStream_t st);

// ---- attention with int8 P.V (k_attn_fwd.cu, k_attn_bwd.cu)
size_t attn_fwd_ws_bytes(int64_t B, int64_t T, int64_t Hq, int64_t W);
cudaError_t launch_attn_fwd(const float* q, const float* k, const int8_t* vq, const float* s_v,
                            float* o, float* m, float* l, int64_t B, int64_t T, int64_t Hq,
                            int64_t Hkv, int64_t W, void* cache, bool tc, cudaStream_t st);

size_t attn_bwd_ws_bytes(int64_t B, int64_t T, int64_t Hq, int64_t W);   // W = -1: without the cache
cudaError_t launch_attn_bwd(const float* q, const float* k, const int8_t* vq, const float* s_v,
                            const float* o, const float* dout, const float* m, const float* l,
                            float* dq, float* dk, float* dv, int64_t B, int64_t T, int64_t Hq,
                            int64_t Hkv, int64_t W, void* ws, const void* lcache,
                            cudaStream_t st);

// ---- bounded-wait probe (k_bwd_tma.cu)
cudaError_t launch_wait_probe(int arrive, cudaStream_t st);
// debug mode: ORs kErrNonfiniteBit into *err if any of the n floats at p is a
// NaN or an infinity
cudaError_t launch_check_finite(const float* p, int64_t n, int* err, cudaStream_t st);

// ---- forward exactness self-test (k_selftest.cu)
size_t selftest_ws_bytes();
int run_selftest(void* ws, cudaStream_t st);

// ---- embedding (k_embed.cu); types as REPRO_F32, REPRO_BF16, REPRO_I8
struct EmbedFwdArgs {
    const void* table;
    int table_type;
    int64_t table_ld;
    const float* s_w;
    const void* tokens;
    int index_bytes;
    int64_t n, V, D;
    float scale;
    int64_t pad;
    void* out;
    int out_type;
    int64_t out_ld;
    int* err;
};
cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, cudaStream_t st);
struct EmbedBwdArgs {
    const void* dout;
    int dout_type;
    int64_t dout_ld;
    const void* tokens;
    int index_bytes;
    int64_t n, V, D;
    float scale;
    int64_t pad;
    float* table;
    int64_t table_ld;
    bool accumulate;
    int* err;
};
size_t embed_bwd_ws_bytes(int64_t n, int64_t V, int64_t D);
cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, void* ws, cudaStream_t st);

// ---- pairwise tree over partial rows (k_rowtree.cu), shared by the table's and the gains' gradients
struct RowTree {
    float* parts[2];     // partial rows, `pitch` floats apart (used as scratch)
    int64_t pitch;
    const int4* joins;   // {first sorted index, chunks, output row, 0}, or NULL: `jobs` joins, job i
                         // over the count[i] consecutive partial rows of parts[i], into out[i]
    const int* njoins;   // device count of joins
    int jobs;
    int64_t count[2];
    int64_t D;
    float* out[2];
    int64_t out_ld;
    float scale;         // applied to the sum (1: leaves it)
    bool accumulate;     // out (+) the scaled sum
};
cudaError_t launch_row_tree(const RowTree& t, int max_ctas, cudaStream_t st);

// ---- norm of query and key heads with the rotation (k_qknorm.cu)
struct QkTensor {        // one of q, k
    const void* x;
    int64_t ld, hs;      // token and head strides
    int64_t H;
    const float* gain;
    float* out;          // forward: [n][H][D]
    const float* dout;   // backward: [n][H][D]
    void* dx;
    int64_t dx_ld, dx_hs;
    float* dgain;
};
struct QkArgs {
    QkTensor t[2];
    int type;
    const float* rope;
    int64_t P;
    const int32_t* positions;
    int64_t T;
    float eps;
    int64_t n, D, R;
    bool interleaved, accumulate;
    float inv;           // 1 / D where D is a power of two, else 0
    int w;               // elements loaded at a time (set by the launchers)
    int* err;
};
cudaError_t launch_qk_fwd(const QkArgs& a, cudaStream_t st);
size_t qk_bwd_ws_bytes(int64_t n, int64_t Hq, int64_t Hkv, int64_t D);
cudaError_t launch_qk_bwd(const QkArgs& a, void* ws, cudaStream_t st);

// ---- loss against a teacher's top logits (k_distill.cu)
struct DistillArgs {
    const void* z;
    int z_type;
    int64_t z_ld;
    const void* t_idx;
    const void* t_val;
    int t_type;
    const void* labels;
    int index_bytes;
    int64_t n, V, K;
    float tau, w_kd, w_ce, w_z;
    bool logprobs;
    float* loss;
    float* stats;
    const float* g;
    int64_t g_stride;
    void* dz;
    int64_t dz_ld;
    int* err;
};
size_t distill_ws_bytes(int64_t n, int64_t V);
cudaError_t launch_distill_fwd(const DistillArgs& a, void* ws, cudaStream_t st);
cudaError_t launch_distill_bwd(const DistillArgs& a, cudaStream_t st);

// ---- debug scan of strided rows (k_rowtree.cu): n rows of D elements of `type`, ld apart
cudaError_t launch_check_finite_rows(const void* p, int type, int64_t n, int64_t D, int64_t ld, int* err,
                                     cudaStream_t st);

// ---- state hash (k_hash.cu)
int64_t hash_leaf_count(const int64_t* nbytes, int nbuf, int64_t leaf_bytes);
size_t hash_ws_bytes(int64_t nleaves);
cudaError_t launch_state_hash(const void* const* bufs, const int64_t* nbytes, int nbuf,
                              int64_t leaf_bytes, uint8_t* digest, void* ws, cudaStream_t st);

} // namespace repro
