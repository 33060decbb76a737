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
    static constexpr bool kShared = false;  // keys of a row in several stretches
    static constexpr bool kTail = true;     // rows that belong to no request are zeroed
    static constexpr bool kUnits = false;   // a share of few segments ends with its segment
};
constexpr int PROMPT_COUNTERS = 13056;  // byte offset in the scratch of the prompt kernel's two counters
constexpr int PLAN_READY = 13184;       // of a word that is 1 from the end of kv4_prefix_attention's plan to that of its join
cudaError_t launch_kv4_prompt(const Kv4AttnArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);
int64_t kv4_attention_scratch(int Hq, int Hkv, int D);
cudaError_t launch_kv4_attention(const Kv4AttnArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);
// The same attention with rows split otherwise: of kv4_prefix_attention over small caches.
struct Kv4UnitArgs : Kv4AttnArgs {
    static constexpr bool kUnits = true;
};
cudaError_t launch_kv4_attention(const Kv4UnitArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);

// kv4_sparse_attention: "requests" are tokens, block_table is their tables
// [T, Hkv, max_blocks] and seq_lens the tokens in them.
struct Kv4TableArgs : Kv4AttnArgs {
    static constexpr bool kTail = false, kUnits = true;
};
cudaError_t launch_kv4_sparse(const Kv4TableArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);

// A stretch of keys [from, end) of the block table's row `row`, from a multiple
// of 16, and the new tokens that see it: all of it where base = end, else token i
// those up to position base + i.  Its results go to places `place` and on (tokens x
// Hq), or to the output where that is negative.
struct alignas(16) Kv4Stretch {
    int token, tokens, from, end, base, row;
    int64_t place;
};
// kv4_prefix_attention: the groups' stretches, then the requests'; `requests`
// counts them all.
struct Kv4SharedArgs : Kv4AttnArgs {
    static constexpr bool kShared = true, kTail = false;
    const Kv4Stretch *stretches;  // those that are streamed,
    const Kv4Stretch *pieces;     // those of many rows, in pieces: counts[0] of them,
    const int32_t *items_before, *counts;  // [pieces + 1] items before each
    float *partials;  // the parts of a launch's split rows; the launch's number, 0 or 1
    int launch;
    bool early;       // begins beside the kernel before it
    float2 *weights;  // [places] maximum (of base-2 exponents) and sum of the weights
    float *values;    // [places, D] weighted values
};
cudaError_t launch_kv4_prompt(const Kv4SharedArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);
// Rows to be joined: of the new tokens from `token` on, with `before` tokens of
// other such stretches before them; beside each one's own part `parts` of a shared
// stretch, `step` places apart.
struct alignas(16) Kv4Share {
    int64_t before, place, step;
    int token, parts;
};
// The arguments of a call besides.
struct Kv4PrefixArgs : Kv4SharedArgs {
    const int32_t *prefix_lens, *cu_groups;
    // the plan, to be written: of `stretches`, `pieces`, `items_before`, `counts`,
    Kv4Stretch *plan, *cut;
    int32_t *before, *count;
    Kv4Share *shares;     // [groups + members]: count[1] of them, with joined[0] tokens
    int64_t *joined;
    float *both_partials[2];
    int32_t *piece_of;    // [members]
    int groups, members;  // members: the call's requests
    int most_pieces;      // there is room for
    int64_t max_group;
    // rows from which a shared stretch, a request goes to the tensor cores; rows of an
    // item there; items that run at once; cost of 16 streamed rows in eighths of an item's
    int least_shared, least_own, item_rows, workers, stream_cost;
};
int64_t kv4_prefix_scratch(int64_t T, int requests, int groups, int Hq, int Hkv, int D, Kv4PrefixArgs *a);
cudaError_t launch_kv4_prefix(const Kv4PrefixArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);

// Bounds of pages: uint8 [num_blocks, Hkv, 2 D + 16].
struct Kv4BoundsArgs {
    const unsigned char *cache;
    const int64_t *slots;
    unsigned char *bounds;
    unsigned int *status;
    int64_t T, num_slots;
    int Hkv, bs_log2;
};
cudaError_t launch_kv4_bounds(const Kv4BoundsArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);

struct Kv4SelectArgs {
    const uint16_t *q;
    const unsigned char *bounds;
    const int32_t *block_table, *seq_lens, *cu_new;
    int32_t *tables, *lens;
    unsigned int *status;
    int64_t q_stride, num_blocks, max_blocks, T;
    int requests, Hq, Hkv, bs_log2, top, first, recent;
};
constexpr int64_t KV4_SELECT_PAGES = 32768;  // of a request: their scores lie in one SM's shared memory
cudaError_t launch_kv4_select(const Kv4SelectArgs &a, int D, cudaStream_t st, const DeviceInfo &dev);

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
