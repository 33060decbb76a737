// Internal launchers, one per kernel family.  Arguments are validated by the
// C-ABI layer (api.cu) before these are called.
#pragma once

#include <cstdint>
#include <mutex>
#include <cuda_runtime.h>

namespace w4 {

// A kernel's dynamic shared-memory limit, raised once per device to the
// largest size launched so far.  Host threads may launch concurrently, so the
// record is kept under a mutex.  `check` (optional) runs once per device
// before the first raise and may refuse the kernel.
struct SmemLimit {
    std::mutex mu;
    int bytes[64] = {};
    template <typename Check>
    cudaError_t ensure(const void *kern, int device, int need, Check check) {
        std::lock_guard<std::mutex> lk(mu);
        const int d = device & 63;
        if (bytes[d] >= need) return cudaSuccess;
        if (bytes[d] == 0) {
            const cudaError_t e = check();
            if (e != cudaSuccess) return e;
        }
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, need);
        if (e == cudaSuccess) bytes[d] = need;
        return e;
    }
    cudaError_t ensure(const void *kern, int device, int need) {
        return ensure(kern, device, need, [] { return cudaSuccess; });
    }
};

struct DeviceInfo {
    int device;
    int num_sms;
    int max_smem_optin;
    unsigned int inject;  // test-only injection flags (w4a16_debug_inject), normally 0
};

cudaError_t launch_dequant(int fmt, const uint8_t *qw, const uint16_t *s,
                           const uint16_t *z, void *out, int out_dtype,
                           int64_t rows, int64_t K, int group,
                           cudaStream_t st, const DeviceInfo &dev);

cudaError_t launch_gemv_int4(const uint16_t *x, const uint8_t *qw,
                             const uint16_t *s, const uint16_t *z, uint16_t *y,
                             int64_t N, int64_t K, cudaStream_t st,
                             unsigned int *status, const DeviceInfo &dev);

// Activation rows one INT4 streaming pass can share at this K (2 or more).
int gemv_int4_max_mv(int64_t K);

// M = 2..4 rows through the streaming GEMV (one pass over the weights).
cudaError_t launch_gemv_int4_batched(const uint16_t *X, const uint8_t *qw,
                                     const uint16_t *s, const uint16_t *z, uint16_t *Y,
                                     int64_t M, int64_t N, int64_t K, cudaStream_t st,
                                     unsigned int *status, const DeviceInfo &dev);

// One INT4 linear of a chain (M = 1), as the chain kernel reads it.
struct ChainOp {
    const uint16_t *x;
    const uint8_t *qw;
    const uint16_t *s;
    const uint16_t *z;  // null: symmetric INT4
    uint16_t *y;
    int N, K;
    int dep;                // op of the same launch that must be finished everywhere first (-1: none)
    unsigned char tt_log2;  // log2 of the threads per row (one thread per 128-code group)
    unsigned char rpt;      // rows per thread per stage (1 or 2)
    unsigned char report;   // a later op of the launch depends on this one: count its completion
    unsigned char pad;
};
constexpr int kChainMaxOps = 192;  // ops per launch (kernel parameter space)
// The team shape of an op with K columns: threads per row (log2) and rows
// per thread, as the single GEMV chooses them.
void gemv_chain_shape(int64_t K, unsigned char &tt_log2, unsigned char &rpt);
// A chain of count <= kChainMaxOps ops in one persistent launch; `done`:
// count + 1 zeroed counters in device memory (left zeroed).  ops[i].dep and
// ops[i].report index ops of this launch.
cudaError_t launch_gemv_chain(const ChainOp *ops, int count, unsigned int *done, cudaStream_t st,
                              unsigned int *status, const DeviceInfo &dev);

// Batched-expert FP4 GEMM (M tokens x topk experts): scratch bytes needed
// for P = M * topk pairs, and the three launches (route, gather, GEMM).
int64_t moe_fp4_gemm_scratch(int64_t P, int64_t E, int64_t K);
cudaError_t launch_moe_fp4_gemm(const uint16_t *X, const uint8_t *qw, const uint16_t *s, const int32_t *ids, int M,
                                int topk, uint16_t *Y, int64_t E, int64_t N, int64_t K, void *scratch,
                                cudaStream_t st, unsigned int *status, const DeviceInfo &dev);

cudaError_t launch_moe_fp4(const uint16_t *x, const uint8_t *qw,
                           const uint16_t *s, const int32_t *ids, int topk,
                           uint16_t *y, int64_t E, int64_t N, int64_t K,
                           cudaStream_t st, unsigned int *status,
                           const DeviceInfo &dev);

// INT4 prefill GEMM with binary16 operands (pre-pass of X into
// stream-ordered scratch, then one accumulator over all of K).
int gemm_int4_f16_smem(int64_t M, int64_t K, bool sym);
cudaError_t launch_gemm_int4_f16(const uint16_t *X, const uint8_t *qw, const uint16_t *s, const uint16_t *z,
                                 uint16_t *Y, int64_t M, int64_t N, int64_t K, cudaStream_t st, unsigned int *status,
                                 const DeviceInfo &dev);

cudaError_t launch_gemm_int4(const uint16_t *X, const uint8_t *qw,
                             const uint16_t *s, const uint16_t *z, uint16_t *Y,
                             int64_t M, int64_t N, int64_t K, cudaStream_t st,
                             unsigned int *status, const DeviceInfo &dev);

// Dense BF16 GEMM Y = X W^T (the second pass of the unfused path).
cudaError_t launch_bf16_gemm(const uint16_t *X, const uint16_t *W, uint16_t *Y,
                             int64_t M, int64_t N, int64_t K, cudaStream_t st,
                             unsigned int *status, const DeviceInfo &dev);

// dst[0, bytes) = src[0, bytes) by a kernel (addresses the device can
// dereference, already translated and checked by the caller).
cudaError_t launch_copy(void *dst, const void *src, int64_t bytes, cudaStream_t st, const DeviceInfo &dev);

// ------------------------------------------- operators around the 4-bit cache
// Sizes and layouts as the C header states them; block_size = 1 << bs_log2.

struct Kv4PlanArgs {
    const int32_t *ctx_lens, *new_lens;
    int32_t *block_table;
    const int32_t *free_blocks;
    int32_t *seq_lens, *cu_new, *positions;
    int64_t *slots;
    int32_t *taken;
    unsigned int *status;
    int64_t max_blocks, num_free, num_tokens;
    int requests, bs_log2;
};
cudaError_t launch_kv4_plan(const Kv4PlanArgs &a, cudaStream_t st, const DeviceInfo &dev);

// Heads of q, k and v of every token in one pass; cache == nullptr: k goes to
// k_out (and there is no v), else k and v go to the cache.
struct Kv4RopeArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const uint16_t *q_weight, *k_weight;
    const float *cos_sin;
    const int32_t *positions;
    const int64_t *slots;
    uint16_t *q_out, *k_out;
    unsigned char *cache;
    unsigned int *status;
    int64_t T, num_slots, num_positions;
    int Hq, Hk, Hv, rot, bs_log2, interleaved;
    float eps, weight_offset;
};
cudaError_t launch_kv4_rope(const Kv4RopeArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);

struct Kv4GatherArgs {
    const unsigned char *cache;
    const int64_t *slots;
    uint16_t *k, *v;
    unsigned int *status;
    int64_t T, num_slots;
    int Hkv, bs_log2;
};
cudaError_t launch_kv4_gather(const Kv4GatherArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);

struct Kv4AttnArgs {
    const uint16_t *q;
    const unsigned char *cache;
    const int32_t *block_table, *seq_lens, *cu_new;
    uint16_t *out;
    unsigned char *scratch;
    unsigned int *status;
    int64_t q_stride, num_blocks, max_blocks, T, window, sinks, max_new;
    int requests, Hq, Hkv, bs_log2;
    float scale;
    // set by launch_kv4_attention: the streaming kernel takes requests of
    // rows_least to rows_most rows (new tokens x query heads per key head), the
    // prompt kernel those of more than rows_above; the first launch of a call
    // zeroes the rows of no request and looks for lengths out of range
    int rows_least, rows_most, rows_above, first_launch;
    unsigned int inject;  // test-only injection flags (0 normally)
};
constexpr int PROMPT_COUNTERS = 13056;  // byte offset in the scratch of the prompt kernel's two counters
cudaError_t launch_kv4_prompt(const Kv4AttnArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);
int64_t kv4_attention_scratch(int Hq, int Hkv, int D);
cudaError_t launch_kv4_attention(const Kv4AttnArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);

struct SampleArgs {
    const void *logits;
    const float *u, *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
    int32_t *tokens;
    int64_t row_stride, rows;
    int vocab;
    bool bf16;
};
cudaError_t launch_sample(const SampleArgs &a, cudaStream_t st, const DeviceInfo &dev);

}  // namespace w4
