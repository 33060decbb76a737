// kv4_attention (C header): which of a call's requests the streaming kernel
// (kv4_stream.cuh) takes and which the one for long pieces (kv4_prompt.cu).
#include "kv4_stream.cuh"

namespace w4 {

int64_t kv4_attention_scratch(int, int, int D) {
    return (COUNTER_BYTES + int64_t(MAX_CTAS) * 2 * warp_rows(D) * (D + 4) * 4 + 255) / 256 * 256;
}

namespace {

template <class A>
cudaError_t attend(const A &args, int D, cudaStream_t st, const DeviceInfo &dev) {
    A a = args;
    const int G = a.Hq / a.Hkv;
    int64_t rows = (a.max_new < a.T ? a.max_new : a.T) * G;  // the most a request has
    const int64_t few = stream_rows(a.requests * a.Hkv, D, dev);
    a.rows_least = 1;
    a.rows_most = 0x7fffffff;
    a.first_launch = 1;
    a.inject = dev.inject;
    if (rows > few) {
        // requests of many rows to the tensor cores; the others of a mixed step to
        // the streaming kernel, those of a token or so (most, as a rule) by the
        // form for them: 64 requests, one of them a prompt, would take 201 us
        // instead of 124 in the form for 16 rows
        a.rows_above = a.requests > 1 ? static_cast<int>(few) : 0;
        if (cudaError_t e = launch_kv4_prompt(static_cast<const Kv4AttnArgs &>(a), D, st, dev)) return e;
        if (a.requests == 1) return cudaSuccess;
        a.first_launch = 0;
        a.rows_most = D == 256 ? 2 : D == 128 ? 4 : 8;
        if (G <= a.rows_most)
            if (cudaError_t e = stream(a, D, a.rows_most, st, dev)) return e;
        a.rows_least = a.rows_most + 1;
        a.rows_most = static_cast<int>(few);
        rows = few;
    }
    return stream(a, D, rows, st, dev);
}

}  // namespace

cudaError_t launch_kv4_attention(const Kv4AttnArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) { return attend(a, D, st, dev); }
cudaError_t launch_kv4_attention(const Kv4UnitArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) { return attend(a, D, st, dev); }

}  // namespace w4
