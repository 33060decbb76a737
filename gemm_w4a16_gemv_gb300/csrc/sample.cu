// Sampling of a token from each row of logits with temperature, top-k, top-p
// and min-p, from given uniform numbers (w4a16_sample in the C header).
//
// The probabilities are whole numbers: token i has the mass
//   m_i = rint(2^40 exp(l_i / T - max))
// so that every sum of them is exact in 64 bits and neither the order of
// summation nor the batch changes a result.  Order: top-k by logit (ties to
// the lower index), top-p on what is left (the shortest prefix in that order
// whose mass reaches p of it), min-p (m_i >= min_p 2^40), then the first
// token, by index, at which the running mass of the kept ones exceeds u of
// their sum.
//
// Simple form: one CTA per row; the k-th key and the top-p boundary are found
// by radix selection, 8 bits of the order-preserving key per pass, reading the
// row again each time.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {
namespace {

constexpr int SAMPLE_THREADS = 1024;
constexpr float UNIT = 1099511627776.f;  // 2^40

// Unsigned key with the order of the logits; +0 and -0 alike, NaN below all.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (v != v) return 0u;
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

struct Row {
    const void *p;
    bool bf16;
    __device__ float at(int64_t i) const {
        return bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
    }
};

template <typename T>
__device__ T block_sum(T v, T *buf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    T s = 0;
    for (int w = 0; w < SAMPLE_THREADS / 32; ++w) s += buf[w];
    return s;
}

__global__ void __launch_bounds__(SAMPLE_THREADS) sample_kernel(const SampleArgs a) {
    __shared__ unsigned long long hist[256], buf[32], pick[3];
    __shared__ uint32_t best_key[32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Row r{static_cast<const char *>(a.logits) + row * a.row_stride * (a.bf16 ? 2 : 4), a.bf16};
    const int V = a.vocab;
    // largest logit
    uint32_t mx = 0;
    for (int i = tid; i < V; i += SAMPLE_THREADS) mx = max(mx, key_of(r.at(i)));
    for (int o = 16; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) best_key[warp] = mx;
    __syncthreads();
    for (int w = 0; w < 32; ++w) mx = max(mx, best_key[w]);
    const uint32_t none = key_of(-INFINITY);
    if (mx <= none) {
        if (tid == 0) a.tokens[row] = -1;
        return;
    }
    const float T = a.temperature ? a.temperature[row] : 1.f;
    const float top = __fdiv_rn(logit_of(mx), T);
    // chunks of consecutive indices, so that sums by thread are sums by index
    const int per = (V + SAMPLE_THREADS - 1) / SAMPLE_THREADS;
    const int i0 = min(tid * per, V), i1 = min(i0 + per, V);
    if (!(T > 0.f) || !(fabsf(top) < INFINITY)) {
        int at = 0x7fffffff;
        for (int i = i0; i < i1 && at == 0x7fffffff; ++i)
            if (key_of(r.at(i)) == mx) at = i;
        if (tid == 0) pick[0] = 0x7fffffff;
        __syncthreads();
        if (at != 0x7fffffff) atomicMin(&pick[0], static_cast<unsigned long long>(at));
        __syncthreads();
        if (tid == 0) a.tokens[row] = static_cast<int>(pick[0]);
        return;
    }
    auto mass = [&](uint32_t key) -> unsigned long long {
        if (key <= none) return 0ull;
        return static_cast<unsigned long long>(__float2ll_rn(expf(__fdiv_rn(logit_of(key), T) - top) * UNIT));
    };
    // finds the key of the element at which the running sum (in falling order
    // of key) of count or mass reaches `goal`, and what of the goal is left there
    auto select = [&](uint32_t floor_key, bool by_mass, unsigned long long goal, uint32_t &found,
                      unsigned long long &left) {
        uint32_t prefix = 0, mask = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            __syncthreads();
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int i = tid; i < V; i += SAMPLE_THREADS) {
                const uint32_t k = key_of(r.at(i));
                if ((k & mask) == prefix && k >= floor_key)
                    atomicAdd(&hist[(k >> shift) & 255u], by_mass ? mass(k) : 1ull);
            }
            __syncthreads();
            if (tid == 0) {
                unsigned long long s = 0;
                int bin = 255;
                for (; bin > 0 && s + hist[bin] < goal; --bin) s += hist[bin];
                pick[0] = static_cast<unsigned long long>(bin);
                pick[1] = goal - s;
            }
            __syncthreads();
            prefix |= static_cast<uint32_t>(pick[0]) << shift;
            mask |= 255u << shift;
            goal = pick[1];
        }
        found = prefix;
        left = goal;
    };
    // kept: keys above `edge`, and the first `ties` tokens (by index) at it
    uint32_t edge = 0;
    unsigned long long ties = ~0ull;
    const int k = a.top_k ? a.top_k[row] : 0;
    if (k > 0 && k < V) select(0u, false, static_cast<unsigned long long>(k), edge, ties);
    const float p = a.top_p ? a.top_p[row] : 1.f;
    if (p < 1.f) {
        unsigned long long s = 0, eq = 0;
        for (int i = tid; i < V; i += SAMPLE_THREADS) {
            const uint32_t key = key_of(r.at(i));
            if (key > edge) s += mass(key);
            eq += key == edge;
        }
        s = block_sum(s, buf);
        eq = block_sum(eq, buf);
        const unsigned long long me = mass(edge);
        s += (ties < eq ? ties : eq) * me;
        const float pc = p > 0.f ? p : 0.f;
        unsigned long long goal = static_cast<unsigned long long>(__double2ll_rz(static_cast<double>(s) * static_cast<double>(pc)));
        if (goal < 1) goal = 1;
        uint32_t e2;
        unsigned long long left;
        select(edge, true, goal, e2, left);
        const unsigned long long m2 = mass(e2);
        const unsigned long long n2 = m2 ? (left + m2 - 1) / m2 : 1ull;
        ties = e2 == edge ? (n2 < ties ? n2 : ties) : n2;
        edge = e2;
    }
    const double least = static_cast<double>(a.min_p ? a.min_p[row] : 0.f) * static_cast<double>(UNIT);
    // ties before this thread's chunk
    unsigned long long eq = 0;
    for (int i = i0; i < i1; ++i) eq += key_of(r.at(i)) == edge;
    unsigned long long before = eq;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = before;
    __syncthreads();
    before -= eq;
    for (int w = 0; w < warp; ++w) before += buf[w];
    auto kept = [&](int i, unsigned long long &seen) -> unsigned long long {
        const uint32_t key = key_of(r.at(i));
        if (key < edge) return 0ull;
        if (key == edge && seen++ >= ties) return 0ull;
        const unsigned long long m = mass(key);
        return static_cast<double>(m) >= least ? m : 0ull;
    };
    unsigned long long mine = 0, seen = before;
    for (int i = i0; i < i1; ++i) mine += kept(i, seen);
    unsigned long long upto = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    __syncthreads();
    if (lane == 31) buf[warp] = upto;
    __syncthreads();
    unsigned long long total = 0, base = 0;
    for (int w = 0; w < 32; ++w) {
        if (w < warp) base += buf[w];
        total += buf[w];
    }
    upto += base;
    const float u = a.u[row];
    unsigned long long goal = u > 0.f ? static_cast<unsigned long long>(__double2ll_rz(static_cast<double>(total) * static_cast<double>(fminf(u, 1.f)))) : 0ull;
    if (goal > total - 1) goal = total - 1;
    if (upto > goal && upto - mine <= goal) {
        unsigned long long s = upto - mine;
        seen = before;
        for (int i = i0; i < i1; ++i) {
            s += kept(i, seen);
            if (s > goal) {
                a.tokens[row] = i;
                break;
            }
        }
    }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t st, const DeviceInfo &) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows));
    cfg.blockDim = dim3(SAMPLE_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel, a);
}

}  // namespace w4
