// C ABI of the operators around the 4-bit key/value cache (include/w4a16.h):
// argument checks on the host, then one launch.
#include "w4a16.h"
#include "api_common.h"
#include "kv4.cuh"

using namespace w4api;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// An array of a call, for the check of overlap.
struct Span {
    const char *name;
    const void *p;
    int64_t bytes;
};

// None of the arrays from number `inputs` on, which are written, may share
// bytes with another one.
template <int N>
int check_apart(const char *fn, int inputs, const Span (&x)[N]) {
    for (int i = inputs; i < N; ++i)
        for (int j = 0; j < i; ++j) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(x[i].p), b = reinterpret_cast<uintptr_t>(x[j].p);
            if (a < b + x[j].bytes && b < a + x[i].bytes && x[i].bytes > 0 && x[j].bytes > 0)
                return fail(W4A16_ERR_INVALID_ARG, "%s: %s and %s overlap", fn, x[i].name, x[j].name);
        }
    return W4A16_OK;
}

// log2 of a page size, or -1.
int page_log2(int block_size) {
    for (int l = 4; l <= 8; ++l)
        if (block_size == 1 << l) return l;
    return -1;
}

int check_head_dim(const char *fn, int D) {
    if (D != 64 && D != 128 && D != 256)
        return fail(W4A16_ERR_UNSUPPORTED, "%s: head dimension %d (64, 128 or 256)", fn, D);
    return W4A16_OK;
}

int check_page(const char *fn, int block_size, int64_t num_blocks) {
    if (page_log2(block_size) < 0)
        return fail(W4A16_ERR_UNSUPPORTED, "%s: block size %d (16, 32, 64, 128 or 256)", fn, block_size);
    if (num_blocks < 1 || num_blocks > 0x7fffffff)
        return fail(W4A16_ERR_INVALID_ARG, "%s: num_blocks=%lld outside 1 .. 2^31 - 1", fn, (long long)num_blocks);
    return W4A16_OK;
}

// The rows of one of q, k, v: `heads` heads of D elements in each of T rows.
int check_rows(const char *fn, const char *name, const void *p, int64_t stride, int heads, int D) {
    if (!p) return fail(W4A16_ERR_INVALID_ARG, "%s: null %s", fn, name);
    if (!aligned16(p)) return fail(W4A16_ERR_MISALIGNED, "%s: %s must be 16-byte aligned", fn, name);
    if (stride < static_cast<int64_t>(heads) * D || stride % 8 != 0 || stride > (int64_t(1) << 30))
        return fail(W4A16_ERR_INVALID_ARG,
                    "%s: the token stride of %s is %lld elements (at least heads * D, a multiple of 8, at most 2^30)", fn,
                    name, (long long)stride);
    return W4A16_OK;
}

// What norm and rotation share.
int check_rope(const char *fn, int64_t T, int Hq, int Hkv, int D, const void *q_weight, const void *k_weight,
               const void *cos_sin, int64_t num_positions, int rot, const void *positions, float eps) {
    if (T < 0 || Hq < 0 || Hkv < 0)
        return fail(W4A16_ERR_INVALID_ARG, "%s: T=%lld Hq=%d Hkv=%d must not be negative", fn, (long long)T, Hq, Hkv);
    if (int r = check_head_dim(fn, D)) return r;
    if (T > kMaxTokens || Hq > 1024 || Hkv > 1024 || T * (Hq + 2 * int64_t(Hkv)) > (int64_t(1) << 30))
        return fail(W4A16_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(cos_sin))
        return fail(W4A16_ERR_MISALIGNED, "%s: weights and cos_sin must be 16-byte aligned", fn);
    if (cos_sin) {
        if (!positions) return fail(W4A16_ERR_INVALID_ARG, "%s: null positions", fn);
        if (!aligned(positions, 4)) return fail(W4A16_ERR_MISALIGNED, "%s: positions must be 4-byte aligned", fn);
        if (rot < 16 || rot > D || rot % 16 != 0)
            return fail(W4A16_ERR_UNSUPPORTED, "%s: rot=%d (a multiple of 16 up to D=%d)", fn, rot, D);
        if (num_positions < 1 || num_positions > 0x7fffffff)
            return fail(W4A16_ERR_INVALID_ARG, "%s: num_positions=%lld outside 1 .. 2^31 - 1", fn,
                        (long long)num_positions);
    }
    if ((q_weight || k_weight) && !(eps >= 0.f && eps < 1e30f))
        return fail(W4A16_ERR_INVALID_ARG, "%s: eps=%g must be finite and not negative", fn, static_cast<double>(eps));
    return W4A16_OK;
}

}  // namespace

extern "C" {

int kv4_plan(const int32_t *ctx_lens, const int32_t *new_lens, int requests, int32_t *block_table,
             int64_t max_blocks, const int32_t *free_blocks, int64_t num_free, int block_size, int64_t num_tokens,
             int32_t *seq_lens, int32_t *cu_new, int32_t *positions, int64_t *slots, int32_t *taken, void *stream) {
    const char *fn = "kv4_plan";
    if (requests < 1 || num_tokens < 0 || max_blocks < 1 || num_free < 0)
        return fail(W4A16_ERR_INVALID_ARG, "%s: requests=%d num_tokens=%lld max_blocks=%lld num_free=%lld", fn, requests,
                    (long long)num_tokens, (long long)max_blocks, (long long)num_free);
    if (!ctx_lens || !new_lens || !block_table || !seq_lens || !cu_new || !taken || (num_free > 0 && !free_blocks) ||
        (num_tokens > 0 && (!positions || !slots)))
        return fail(W4A16_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (page_log2(block_size) < 0)
        return fail(W4A16_ERR_UNSUPPORTED, "%s: block size %d (16, 32, 64, 128 or 256)", fn, block_size);
    if (requests > 8192 || num_tokens > kMaxTokens || max_blocks > 0x7fffffff / block_size || num_free > 0x7fffffff)
        return fail(W4A16_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(free_blocks, 4) ||
        !aligned(seq_lens, 4) || !aligned(cu_new, 4) || !aligned(positions, 4) || !aligned(slots, 8) ||
        !aligned(taken, 4))
        return fail(W4A16_ERR_MISALIGNED, "%s: arrays must be aligned to their elements", fn);
    // every CTA reads the lengths again while the first one writes its results
    const Span arrays[] = {{"ctx_lens", ctx_lens, 4 * int64_t(requests)}, {"new_lens", new_lens, 4 * int64_t(requests)},
                           {"free_blocks", free_blocks, 4 * num_free}, {"block_table", block_table, 4 * requests * max_blocks},
                           {"seq_lens", seq_lens, 4 * int64_t(requests)}, {"cu_new", cu_new, 4 * int64_t(requests) + 4},
                           {"positions", positions, 4 * num_tokens}, {"slots", slots, 8 * num_tokens}, {"taken", taken, 4}};
    if (int r = check_apart(fn, 3, arrays)) return r;
    w4::DeviceInfo dev;
    w4::Kv4PlanArgs a;
    if (int r = device_state(dev, a.status)) return r;
    if (int r = check_device_ptrs(fn, dev.device, {ctx_lens, new_lens, block_table, num_free ? free_blocks : nullptr,
                                                   seq_lens, cu_new, num_tokens ? positions : nullptr,
                                                   num_tokens ? slots : nullptr, taken}))
        return r;
    a.ctx_lens = ctx_lens;
    a.new_lens = new_lens;
    a.block_table = block_table;
    a.free_blocks = free_blocks;
    a.seq_lens = seq_lens;
    a.cu_new = cu_new;
    a.positions = positions;
    a.slots = slots;
    a.taken = taken;
    a.max_blocks = max_blocks;
    a.num_free = num_free;
    a.num_tokens = num_tokens;
    a.requests = requests;
    a.bs_log2 = page_log2(block_size);
    return launched(w4::launch_kv4_plan(a, static_cast<cudaStream_t>(stream), dev), fn);
}

int w4a16_qk_norm_rope(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride,
                       const uint16_t *q_weight, const uint16_t *k_weight, const float *cos_sin,
                       int64_t num_positions, int rot, const int32_t *positions, uint16_t *q_out, uint16_t *k_out,
                       int64_t T, int Hq, int Hkv, int D, float eps, float weight_offset, int interleaved,
                       void *stream) {
    const char *fn = "w4a16_qk_norm_rope";
    if (int r = check_rope(fn, T, Hq, Hkv, D, q_weight, k_weight, cos_sin, num_positions, rot, positions, eps)) return r;
    if (T == 0 || Hq + Hkv == 0) return ok();
    if (Hq > 0) {
        if (int r = check_rows(fn, "q", q, q_stride, Hq, D)) return r;
        if (int r = check_rows(fn, "q_out", q_out, static_cast<int64_t>(Hq) * D, Hq, D)) return r;
    }
    if (Hkv > 0) {
        if (int r = check_rows(fn, "k", k, k_stride, Hkv, D)) return r;
        if (int r = check_rows(fn, "k_out", k_out, static_cast<int64_t>(Hkv) * D, Hkv, D)) return r;
    }
    w4::DeviceInfo dev;
    w4::Kv4RopeArgs a = {};
    if (int r = device_state(dev, a.status)) return r;
    if (int r = check_device_ptrs(fn, dev.device,
                                  {Hq ? q : nullptr, Hkv ? k : nullptr, q_weight, k_weight, cos_sin,
                                   cos_sin ? positions : nullptr, Hq ? q_out : nullptr, Hkv ? k_out : nullptr}))
        return r;
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.cos_sin = cos_sin;
    a.positions = positions;
    a.q_out = q_out;
    a.k_out = k_out;
    a.T = T;
    a.num_positions = num_positions;
    a.Hq = Hq;
    a.Hk = Hkv;
    a.rot = rot;
    a.interleaved = interleaved;
    a.eps = eps;
    a.weight_offset = weight_offset;
    return launched(w4::launch_kv4_rope(a, D, static_cast<cudaStream_t>(stream), dev), fn);
}

int kv4_append(const uint16_t *q, int64_t q_stride, const uint16_t *k, int64_t k_stride, const uint16_t *v,
               int64_t v_stride, const uint16_t *q_weight, const uint16_t *k_weight, const float *cos_sin,
               int64_t num_positions, int rot, const int32_t *positions, const int64_t *slots, uint16_t *q_out,
               uint8_t *cache, int64_t num_blocks, int block_size, int64_t T, int Hq, int Hkv, int D, float eps,
               float weight_offset, int interleaved, void *stream) {
    const char *fn = "kv4_append";
    if (int r = check_rope(fn, T, Hq, Hkv, D, q_weight, k_weight, cos_sin, num_positions, rot, positions, eps)) return r;
    if (Hkv < 1) return fail(W4A16_ERR_INVALID_ARG, "%s: Hkv=%d must be >= 1", fn, Hkv);
    if (int r = check_page(fn, block_size, num_blocks)) return r;
    if (T == 0) return ok();
    if (Hq > 0) {
        if (int r = check_rows(fn, "q", q, q_stride, Hq, D)) return r;
        if (int r = check_rows(fn, "q_out", q_out, static_cast<int64_t>(Hq) * D, Hq, D)) return r;
    }
    if (int r = check_rows(fn, "k", k, k_stride, Hkv, D)) return r;
    if (int r = check_rows(fn, "v", v, v_stride, Hkv, D)) return r;
    if (!slots || !cache) return fail(W4A16_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(slots, 8) || !aligned16(cache))
        return fail(W4A16_ERR_MISALIGNED, "%s: slots must be 8-byte, the cache 16-byte aligned", fn);
    w4::DeviceInfo dev;
    w4::Kv4RopeArgs a = {};
    if (int r = device_state(dev, a.status)) return r;
    if (int r = check_device_ptrs(fn, dev.device,
                                  {Hq ? q : nullptr, k, v, q_weight, k_weight, cos_sin, cos_sin ? positions : nullptr,
                                   slots, Hq ? q_out : nullptr, cache}))
        return r;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.cos_sin = cos_sin;
    a.positions = positions;
    a.slots = slots;
    a.q_out = q_out;
    a.cache = cache;
    a.T = T;
    a.num_slots = num_blocks * block_size;
    a.num_positions = num_positions;
    a.Hq = Hq;
    a.Hk = a.Hv = Hkv;
    a.rot = rot;
    a.bs_log2 = page_log2(block_size);
    a.interleaved = interleaved;
    a.eps = eps;
    a.weight_offset = weight_offset;
    return launched(w4::launch_kv4_rope(a, D, static_cast<cudaStream_t>(stream), dev), fn);
}

int kv4_gather(const uint8_t *cache, int64_t num_blocks, int block_size, const int64_t *slots, uint16_t *k,
               uint16_t *v, int64_t T, int Hkv, int D, void *stream) {
    const char *fn = "kv4_gather";
    if (T < 0 || Hkv < 1)
        return fail(W4A16_ERR_INVALID_ARG, "%s: T=%lld must not be negative, Hkv=%d >= 1", fn, (long long)T, Hkv);
    if (int r = check_head_dim(fn, D)) return r;
    if (int r = check_page(fn, block_size, num_blocks)) return r;
    if (T > kMaxTokens || Hkv > 1024 || T * 2 * Hkv > (int64_t(1) << 30))
        return fail(W4A16_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    if (T == 0) return ok();
    if (!cache || !slots || !k || !v) return fail(W4A16_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(cache) || !aligned16(k) || !aligned16(v) || !aligned(slots, 8))
        return fail(W4A16_ERR_MISALIGNED, "%s: slots must be 8-byte, the other arrays 16-byte aligned", fn);
    w4::DeviceInfo dev;
    w4::Kv4GatherArgs a;
    if (int r = device_state(dev, a.status)) return r;
    if (int r = check_device_ptrs(fn, dev.device, {cache, slots, k, v})) return r;
    a.cache = cache;
    a.slots = slots;
    a.k = k;
    a.v = v;
    a.T = T;
    a.num_slots = num_blocks * block_size;
    a.Hkv = Hkv;
    a.bs_log2 = page_log2(block_size);
    return launched(w4::launch_kv4_gather(a, D, static_cast<cudaStream_t>(stream), dev), fn);
}

int64_t kv4_attention_scratch_bytes(int Hq, int Hkv, int D) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (D != 64 && D != 128 && D != 256)) return 0;
    return w4::kv4_attention_scratch(Hq, Hkv, D);
}

int kv4_attention(const uint16_t *q, int64_t q_stride, const uint8_t *cache, int64_t num_blocks, int block_size,
                  const int32_t *block_table, int64_t max_blocks, const int32_t *seq_lens, const int32_t *cu_new,
                  int requests, uint16_t *out, int64_t T, int Hq, int Hkv, int D, float scale, int64_t window,
                  int64_t sinks, int64_t max_new, void *scratch, int64_t scratch_bytes, void *stream) {
    const char *fn = "kv4_attention";
    if (requests < 1 || T < 0 || Hq < 1 || Hkv < 1 || max_blocks < 1)
        return fail(W4A16_ERR_INVALID_ARG, "%s: requests=%d T=%lld Hq=%d Hkv=%d max_blocks=%lld", fn, requests,
                    (long long)T, Hq, Hkv, (long long)max_blocks);
    if (Hq % Hkv != 0) return fail(W4A16_ERR_INVALID_ARG, "%s: Hq=%d not a multiple of Hkv=%d", fn, Hq, Hkv);
    if (window < 0 || sinks < 0 || max_new < 1)
        return fail(W4A16_ERR_INVALID_ARG, "%s: window=%lld sinks=%lld must not be negative, max_new=%lld >= 1", fn,
                    (long long)window, (long long)sinks, (long long)max_new);
    if (!(scale > -1e30f && scale < 1e30f))
        return fail(W4A16_ERR_INVALID_ARG, "%s: scale=%g must be finite", fn, static_cast<double>(scale));
    if (int r = check_head_dim(fn, D)) return r;
    if (int r = check_page(fn, block_size, num_blocks)) return r;
    if (requests > 4096 || T > kMaxTokens || Hq > 1024 || max_blocks > 0x7fffffff / block_size)
        return fail(W4A16_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    if (T == 0) return ok();
    if (int r = check_rows(fn, "q", q, q_stride, Hq, D)) return r;
    if (int r = check_rows(fn, "out", out, static_cast<int64_t>(Hq) * D, Hq, D)) return r;
    if (!cache || !block_table || !seq_lens || !cu_new || !scratch)
        return fail(W4A16_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned16(cache) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_new, 4) ||
        !aligned(scratch, 256))
        return fail(W4A16_ERR_MISALIGNED, "%s: the cache must be 16-byte, the scratch 256-byte, the arrays 4-byte aligned",
                    fn);
    const int64_t need = w4::kv4_attention_scratch(Hq, Hkv, D);
    if (scratch_bytes < need)
        return fail(W4A16_ERR_INVALID_ARG, "%s: scratch of %lld bytes, %lld needed", fn, (long long)scratch_bytes,
                    (long long)need);
    w4::DeviceInfo dev;
    w4::Kv4AttnArgs a = {};
    if (int r = device_state(dev, a.status)) return r;
    if (int r = check_device_ptrs(fn, dev.device, {q, cache, block_table, seq_lens, cu_new, out, scratch})) return r;
    a.q = q;
    a.cache = cache;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.cu_new = cu_new;
    a.out = out;
    a.scratch = static_cast<unsigned char *>(scratch);
    a.q_stride = q_stride;
    a.num_blocks = num_blocks;
    a.max_blocks = max_blocks;
    a.T = T;
    a.window = window;
    a.sinks = sinks;
    a.max_new = max_new;
    a.requests = requests;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.bs_log2 = page_log2(block_size);
    a.scale = scale;
    return launched(w4::launch_kv4_attention(a, D, static_cast<cudaStream_t>(stream), dev), fn);
}

int w4a16_sample(const void *logits, int dtype, int64_t row_stride, int64_t rows, int64_t vocab, const float *u,
                 const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                 int32_t *tokens, void *stream) {
    const char *fn = "w4a16_sample";
    if (dtype != W4_OUT_F32 && dtype != W4_OUT_BF16)
        return fail(W4A16_ERR_INVALID_ARG, "%s: unknown logits dtype %d", fn, dtype);
    if (rows < 0 || vocab < 1)
        return fail(W4A16_ERR_INVALID_ARG, "%s: rows=%lld must not be negative, vocab=%lld >= 1", fn, (long long)rows,
                    (long long)vocab);
    if (row_stride < vocab)
        return fail(W4A16_ERR_INVALID_ARG, "%s: row stride %lld < vocab %lld", fn, (long long)row_stride,
                    (long long)vocab);
    if (rows > (1 << 20) || vocab > (1 << 18))
        return fail(W4A16_ERR_UNSUPPORTED, "%s: rows=%lld vocab=%lld (at most 2^20 rows of 2^18)", fn, (long long)rows,
                    (long long)vocab);
    if (rows == 0) return ok();
    if (!logits || !u || !tokens) return fail(W4A16_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(logits, dtype == W4_OUT_F32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) ||
        !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4))
        return fail(W4A16_ERR_MISALIGNED, "%s: arrays must be aligned to their elements", fn);
    w4::DeviceInfo dev;
    unsigned int *status;
    if (int r = device_state(dev, status)) return r;
    if (int r = check_device_ptrs(fn, dev.device, {logits, u, temperature, top_k, top_p, min_p, tokens})) return r;
    (void)status;
    w4::SampleArgs a;
    a.logits = logits;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.tokens = tokens;
    a.row_stride = row_stride;
    a.rows = rows;
    a.vocab = static_cast<int>(vocab);
    a.bf16 = dtype == W4_OUT_BF16;
    return launched(w4::launch_sample(a, static_cast<cudaStream_t>(stream), dev), fn);
}

}  // extern "C"
