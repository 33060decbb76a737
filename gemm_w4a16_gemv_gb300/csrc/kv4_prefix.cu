// kv4_prefix_attention (C header): attention of requests that share the first
// tokens of their contexts, which are attended to once for all rows of a group.
//
// A row's softmax over all keys is joined from its parts over stretches of them:
//   m = max_i m_i,  l = sum_i 2^(m_i - m) l_i,  o = sum_i 2^(m_i - m) o_i / l
// with m_i, l_i, o_i the reference, the sum of weights and the weighted values
// of stretch i (all binary32).  The stretches of a call are those that the
// groups share, each seen whole by all rows of the group, and what is left of
// each request.  Launches:
//   plan   the stretches, from the lengths (one CTA);
//   parts  of all stretches, by the kernel of kv4_stream.cuh;
//   join   of each row's parts.
#include "kv4_stream.cuh"

namespace w4 {
namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int JOIN_THREADS = 256;

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const Kv4PrefixArgs a) {
    extern __shared__ int plan_smem[];
    int *const shared = plan_smem;                // [groups] keys that the group shares
    int *const owner = plan_smem + a.groups;      // [members]
    __shared__ long long sums[PLAN_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const long long cap = static_cast<long long>(a.max_blocks) << a.bs_log2;
    for (int b = tid; b < a.members; b += PLAN_THREADS) owner[b] = -1;
    __syncthreads();
    bool bad = false;
    // a warp per group: the tokens before all of its members' new ones
    for (int g = warp; g < a.groups; g += PLAN_THREADS / 32) {
        const int from = a.cu_groups[g], to = a.cu_groups[g + 1], len = a.prefix_lens[g];
        bad |= from < 0 || to < from || to > a.members || len < 0;
        const int first = min(max(from, 0), a.members), last = min(max(to, first), a.members);
        long long least = len;
        int rows = 0, row = a.members;
        for (int b = first + lane; b < last; b += 32) {
            const int n = rows_before(a, b + 1) - rows_before(a, b);
            if (n <= 0) continue;
            least = min(least, static_cast<long long>(a.seq_lens[b]) - n);
            row = min(row, b);
            ++rows;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        rows = __reduce_add_sync(0xffffffffu, rows);
        row = __reduce_min_sync(0xffffffffu, row);
        least = rows < 2 ? 0 : min(max(least, 0ll), cap) & ~15ll;  // (one request shares nothing)
        for (int b = first + lane; b < last; b += 32) owner[b] = g;
        if (lane == 0) {
            shared[g] = static_cast<int>(least);
            const int token = rows_before(a, first);
            Kv4Stretch s = {};
            s.token = token;
            s.tokens = least > 0 ? max(rows_before(a, last) - token, 0) : 0;
            s.end = s.base = static_cast<int>(least);
            s.row = min(row, a.members - 1);
            a.plan[g] = s;
        }
    }
    __syncthreads();
    // places of the groups' parts, behind those of the requests
    long long next = a.T * a.Hq;
    for (int g0 = 0; g0 < a.groups; g0 += PLAN_THREADS) {
        const int g = g0 + tid;
        const long long n = g < a.groups ? static_cast<long long>(a.plan[g].tokens) * a.Hq : 0;
        long long in = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += v;
        }
        if (lane == 31) sums[warp] = in;
        __syncthreads();
        long long all = 0;
        for (int w = 0; w < PLAN_THREADS / 32; ++w) {
            if (w < warp) in += sums[w];
            all += sums[w];
        }
        if (g < a.groups) {
            const long long place = next + in - n;
            if (place + n <= a.places) a.plan[g].place = place;
            else {  // (lengths that fall somewhere)
                a.plan[g].tokens = 0;
                shared[g] = 0;
                bad = true;
            }
        }
        next += all;
        __syncthreads();
    }
    for (int b = tid; b < a.members; b += PLAN_THREADS) {
        check_lengths(a, b);
        const int g = owner[b];
        Kv4Stretch s;
        s.token = rows_before(a, b);
        s.tokens = max(rows_before(a, b + 1) - s.token, 0);
        s.from = g >= 0 ? shared[g] : 0;
        s.end = static_cast<int>(min(cap, 0x7fffffffll));
        s.base = a.seq_lens[b] - s.tokens;
        s.row = b;
        s.place = s.from > 0 ? static_cast<int64_t>(s.token) * a.Hq : -1;
        a.plan[a.groups + b] = s;
        a.group_of[b] = s.from > 0 ? g : -1;
    }
    if (bad) atomicOr(a.status, kDevBadIndex);
}

// Four dimensions of a row a thread, JOIN_THREADS of a token's Hq D / 4 a CTA.
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const Kv4PrefixArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    const int at = blockIdx.y * JOIN_THREADS + threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const int b = request_of(a.cu_new, a.members, t, lane);
    if (at >= a.Hq * (D / 4)) return;
    const int head = at / (D / 4), d = at % (D / 4) * 4;
    uint16_t *const to = a.out + (t * a.Hq + head) * D + d;
    if (b < 0) {  // of no request
        *reinterpret_cast<uint2 *>(to) = make_uint2(0, 0);
        return;
    }
    const int g = a.group_of[b];
    if (g < 0) return;  // written by the kernel of its only stretch
    const Kv4Stretch s = a.stretches[g];
    const int64_t place[2] = {t * a.Hq + head, s.place + (t - s.token) * a.Hq + head};
    float2 w[2];
    float4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = __ldcg(a.weights + place[i]);
        v[i] = __ldcg(reinterpret_cast<const float4 *>(a.values + place[i] * D + d));
    }
    const float m = fmaxf(w[0].x, w[1].x), f0 = ex2(w[0].x - m), f1 = ex2(w[1].x - m);
    const float l = fmaf(f0, w[0].y, f1 * w[1].y), inv = l == 0.f ? 0.f : 1.f / l;
    const float o[4] = {fmaf(f0, v[0].x, f1 * v[1].x) * inv, fmaf(f0, v[0].y, f1 * v[1].y) * inv,
                        fmaf(f0, v[0].z, f1 * v[1].z) * inv, fmaf(f0, v[0].w, f1 * v[1].w) * inv};
    *reinterpret_cast<uint2 *>(to) =
        make_uint2(static_cast<uint32_t>(f32_to_bf16_bits(o[0])) | static_cast<uint32_t>(f32_to_bf16_bits(o[1])) << 16,
                   static_cast<uint32_t>(f32_to_bf16_bits(o[2])) | static_cast<uint32_t>(f32_to_bf16_bits(o[3])) << 16);
}

cudaError_t launch(const void *kernel, Kv4PrefixArgs &a, dim3 grid, int threads, int smem, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    void *args[] = {&a};
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace

// Scratch: kv4_attention's, the plan, the parts.
int64_t kv4_prefix_scratch(int64_t T, int requests, int groups, int Hq, int, int D, Kv4PrefixArgs *a) {
    int64_t at = kv4_attention_scratch(Hq, 1, D);
    const int64_t places = 2 * T * Hq;  // a row's own stretch and its group's
    auto take = [&](int64_t bytes) {
        const int64_t from = at;
        at += (bytes + 255) / 256 * 256;
        return from;
    };
    const int64_t plan = take((static_cast<int64_t>(groups) + requests) * sizeof(Kv4Stretch)), group = take(4 * static_cast<int64_t>(requests));
    const int64_t weights = take(places * sizeof(float2)), values = take(places * D * 4);
    if (a) {
        a->plan = reinterpret_cast<Kv4Stretch *>(a->scratch + plan);
        a->stretches = a->plan;
        a->group_of = reinterpret_cast<int32_t *>(a->scratch + group);
        a->weights = reinterpret_cast<float2 *>(a->scratch + weights);
        a->values = reinterpret_cast<float *>(a->scratch + values);
        a->places = places;
    }
    return at;
}

cudaError_t launch_kv4_prefix(const Kv4PrefixArgs &args, int D, cudaStream_t st, const DeviceInfo &dev) {
    Kv4PrefixArgs a = args;
    const int G = a.Hq / a.Hkv;
    a.members = a.requests;
    a.requests = a.groups + a.members;
    a.rows_least = 1;
    a.rows_most = 0x7fffffff;
    a.inject = dev.inject;
    const int smem = (a.groups + a.members) * 4;
    if (cudaError_t e = launch(reinterpret_cast<const void *>(plan_kernel), a, dim3(1), PLAN_THREADS, smem, st)) return e;
    const int64_t most = a.max_group > a.max_new ? a.max_group : a.max_new;
    if (cudaError_t e = stream(static_cast<const Kv4SharedArgs &>(a), D, (most < a.T ? most : a.T) * G, st, dev)) return e;
    const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>((a.Hq * (D / 4) + JOIN_THREADS - 1) / JOIN_THREADS));
    const void *const join = D == 64    ? reinterpret_cast<const void *>(join_kernel<64>)
                             : D == 128 ? reinterpret_cast<const void *>(join_kernel<128>)
                                        : reinterpret_cast<const void *>(join_kernel<256>);
    return launch(join, a, grid, JOIN_THREADS, 0, st);
}

}  // namespace w4
