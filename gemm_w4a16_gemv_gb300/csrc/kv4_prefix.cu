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
//   parts  of those with many rows by the tensor cores (kv4_prompt.cu), the shared
//          ones cut along the keys to fill the GPU; of the others by the kernel of
//          kv4_stream.cuh;
//   join   of each row's parts.
#include "kv4_stream.cuh"

namespace w4 {
namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int JOIN_THREADS = 256;
constexpr int AHEAD = 4;       // parts that a thread of the join asks for together
constexpr int KEYS = 128;      // of a key tile of the tensor cores' kernel
constexpr int ROUNDS = 4;      // items to a worker at most, where stretches are cut
constexpr int OVERHEAD = 4;    // cost of an item beside its key tiles, in key tiles

// Exclusive sum over the CTA's threads; `all` is the sum of all.
__device__ __forceinline__ long long sum_before(long long v, long long &all, long long *sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) in += u;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = in;
    __syncthreads();
    long long before = in - v;
    all = 0;
    for (int w = 0; w < PLAN_THREADS / 32; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    return before;
}

// The stretches of a call, by one CTA.  A shared stretch of many rows is cut into
// pieces of `cut` key tiles, so that its items (a block of rows and a key head
// each) fill the workers: of the smallest cuts that give at most one, two, ... items
// to a worker the one with the shortest time, an item's cost beside its key tiles
// being about OVERHEAD of them.
__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const Kv4PrefixArgs a) {
    extern __shared__ int plan_smem[];
    int *const shared = plan_smem;           // [groups] keys that the group shares
    int *const weight = shared + a.groups;   // [groups] items of it for each piece, or 0
    int *const owner = weight + a.groups;    // [members] the group
    __shared__ long long sums[PLAN_THREADS / 32];
    __shared__ unsigned long long own_items;  // of requests of many rows
    __shared__ int longest, cuts[ROUNDS], costs[ROUNDS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.Hq / a.Hkv;
    pdl_launch_dependents();
    pdl_wait();
    const long long cap = min(static_cast<long long>(a.max_blocks) << a.bs_log2, 0x7fffff00ll);
    if (tid == 0) longest = 0, own_items = 0;
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
        const int token = rows_before(a, first), tokens = max(rows_before(a, last) - token, 0);
        least = rows < 2 || tokens == 0 ? 0 : min(max(least, 0ll), cap) & ~15ll;  // (one request shares nothing)
        for (int b = first + lane; b < last; b += 32) owner[b] = g;
        if (lane == 0) {
            shared[g] = static_cast<int>(least);
            const bool many = least > 0 && static_cast<long long>(tokens) * G >= a.least_shared;
            weight[g] = many ? (tokens * G + a.item_rows - 1) / a.item_rows * a.Hkv : 0;
            if (many) atomicMax(&longest, static_cast<int>((least + KEYS - 1) / KEYS));
            Kv4Stretch s;
            s.token = token;
            s.tokens = least > 0 && !many ? tokens : 0;
            s.from = 0;
            s.end = s.base = static_cast<int>(least);
            s.row = min(row, a.members - 1);
            s.place = tokens;  // (until it has one)
            a.plan[g] = s;
        }
    }
    // requests of many rows
    for (int b = tid; b < a.members; b += PLAN_THREADS) {
        const int rows = max(rows_before(a, b + 1) - rows_before(a, b), 0) * G;
        if (rows >= a.least_own) atomicAdd(&own_items, static_cast<unsigned long long>((rows + a.item_rows - 1) / a.item_rows * a.Hkv));
    }
    __syncthreads();
    // (more than that only where cu_new falls somewhere)
    const int least_own = own_items > 0 && own_items < (1ull << 30) ? a.least_own : 0x7fffffff;
    // ---- the cut, a warp for each number of rounds
    if (warp < ROUNDS && longest > 0) {
        const int k = warp + 1;
        auto items = [&](int c) -> long long {
            long long n = 0;
            for (int g = lane; g < a.groups; g += 32)
                if (weight[g]) n += static_cast<long long>(weight[g]) * (((shared[g] + KEYS - 1) / KEYS + c - 1) / c);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
            return n + static_cast<long long>(own_items);
        };
        int lo = 0, hi = longest;  // more items than that with lo; hi is tried last
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (items(mid) <= static_cast<long long>(k) * a.workers) hi = mid;
            else lo = mid;
        }
        const bool fits = items(hi) <= static_cast<long long>(k) * a.workers;
        if (lane == 0) {
            cuts[warp] = hi;
            costs[warp] = fits ? k * (hi + OVERHEAD) : 0x7fffffff;
        }
    }
    __syncthreads();
    int cut = longest;
    if (longest > 0) {
        int best = 0x7fffffff;
        for (int k = 0; k < ROUNDS; ++k)
            if (costs[k] < best) {
                best = costs[k];
                cut = cuts[k];
            }
    }
    // ---- pieces: the requests' first (they differ in length), then the groups'.
    // (pieces << 40 | items) before each
    constexpr long long ITEMS = (1ll << 40) - 1;
    long long at = 0, all;
    auto put = [&](long long n, const Kv4Stretch &s) {
        a.cut[n >> 40] = s;
        a.before[n >> 40] = static_cast<int>(n & ITEMS);
    };
    if (least_own != 0x7fffffff)  // (the same for all threads)
        for (int b0 = 0; b0 < a.members; b0 += PLAN_THREADS) {
            const int b = b0 + tid;
            const int rows = b < a.members ? max(rows_before(a, b + 1) - rows_before(a, b), 0) * G : 0;
            const bool many = rows >= least_own;
            const long long n = many ? 1ll << 40 | static_cast<long long>((rows + a.item_rows - 1) / a.item_rows * a.Hkv) : 0;
            const long long mine = at + sum_before(n, all, sums);
            if (many) put(mine, {rows_before(a, b), rows / G, 0, 0, 0, b, -1});  // (its keys follow below)
            if (b < a.members) a.group_of[b] = many ? static_cast<int>(mine >> 40) : -1;
            at += all;
        }
    long long place = a.T * a.Hq;  // behind the requests' own
    for (int g0 = 0; g0 < a.groups; g0 += PLAN_THREADS) {
        const int g = g0 + tid;
        const bool on = g < a.groups && shared[g] > 0;
        const int tokens = on ? static_cast<int>(a.plan[g].place) : 0, tiles = on ? (shared[g] + KEYS - 1) / KEYS : 0;
        const int parts = !on ? 0 : weight[g] ? (tiles + cut - 1) / cut : 1;
        const long long step = static_cast<long long>(tokens) * a.Hq;
        const long long from = place + sum_before(parts * step, all, sums);
        place += all;
        const bool fits = from + parts * step <= a.places;  // (not if lengths fall somewhere)
        const long long n = on && fits && weight[g] ? static_cast<long long>(parts) << 40 | static_cast<long long>(parts) * weight[g] : 0;
        const long long mine = at + sum_before(n, all, sums);
        at += all;
        const bool room = (at >> 40) <= a.most_pieces;
        if (on) {
            Kv4Stretch s = a.plan[g];
            if (!fits || !room) {
                bad = true;
                shared[g] = 0;
                a.plan[g].tokens = 0;
            } else {
                a.shares[g] = {s.token, parts, from, step};
                s.place = from;
                if (weight[g] == 0) a.plan[g] = s;
                s.tokens = tokens;
                s.base = s.end;
                const int end = s.end;
                for (int i = 0; weight[g] && i < parts; ++i) {
                    s.from = i * cut * KEYS;
                    s.end = min((i + 1) * cut * KEYS, end);
                    s.place = from + i * step;
                    put(mine + (static_cast<long long>(i) << 40 | static_cast<long long>(i) * weight[g]), s);
                }
            }
        }
        if (!room) at -= all;
    }
    __syncthreads();
    if (tid == 0) {
        a.count[0] = static_cast<int>(at >> 40);
        a.before[at >> 40] = static_cast<int>(at & ITEMS);
    }
    // ---- what is left of each request
    for (int b = tid; b < a.members; b += PLAN_THREADS) {
        check_lengths(a, b);
        const int g = owner[b];
        Kv4Stretch s;
        s.token = rows_before(a, b);
        s.tokens = max(rows_before(a, b + 1) - s.token, 0);
        s.from = g >= 0 ? shared[g] : 0;
        s.end = static_cast<int>(cap);
        s.base = a.seq_lens[b] - s.tokens;
        s.row = b;
        s.place = s.from > 0 ? static_cast<int64_t>(s.token) * a.Hq : -1;
        if (s.tokens * G >= least_own) {
            a.cut[a.group_of[b]] = s;
            s.tokens = 0;
        }
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
    const Kv4Share s = a.shares[g];
    const int64_t own = t * a.Hq + head, first = s.place + (t - s.token) * a.Hq + head;
    float2 w = __ldcg(a.weights + own);
    float4 v = __ldcg(reinterpret_cast<const float4 *>(a.values + own * D + d));
    float m = w.x, l = w.y;
    // AHEAD parts at a time, all on their way together
    for (int i0 = 0; i0 < s.parts; i0 += AHEAD) {
        float2 wi[AHEAD];
        float4 vi[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t at = first + min(i0 + i, s.parts - 1) * s.step;
            wi[i] = __ldcg(a.weights + at);
            vi[i] = __ldcg(reinterpret_cast<const float4 *>(a.values + at * D + d));
        }
        float up = m;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) up = fmaxf(up, wi[i].x);
        const float old = ex2(m - up);
        m = up;
        l *= old;
        v.x *= old, v.y *= old, v.z *= old, v.w *= old;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const float f = i0 + i < s.parts ? ex2(wi[i].x - m) : 0.f;
            l = fmaf(f, wi[i].y, l);
            v.x = fmaf(f, vi[i].x, v.x);
            v.y = fmaf(f, vi[i].y, v.y);
            v.z = fmaf(f, vi[i].z, v.z);
            v.w = fmaf(f, vi[i].w, v.w);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float o[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
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
int64_t kv4_prefix_scratch(int64_t T, int requests, int groups, int Hq, int Hkv, int D, Kv4PrefixArgs *a) {
    // a row's own stretch and its group's; cut ones: ROUNDS items of 128 rows at most
    // for each SM (of 256 for each two), and no more than as many pieces of every row
    const int64_t items = ROUNDS * MAX_CTAS, rows = T * Hq;
    const int64_t more = rows * (items / Hkv), places = 2 * rows + (more < items * 128 ? more : items * 128);
    const int most_pieces = requests + (groups < requests / 2 ? groups : requests / 2) + static_cast<int>(items);
    int64_t at = kv4_attention_scratch(Hq, Hkv, D);
    auto take = [&](int64_t bytes) {
        const int64_t from = at;
        at += (bytes + 255) / 256 * 256;
        return from;
    };
    const int64_t plan = take((static_cast<int64_t>(groups) + requests) * sizeof(Kv4Stretch));
    const int64_t cut = take(most_pieces * static_cast<int64_t>(sizeof(Kv4Stretch)));
    const int64_t before = take(4 * (static_cast<int64_t>(most_pieces) + 1)), count = take(4);
    const int64_t shares = take(groups * static_cast<int64_t>(sizeof(Kv4Share))), group_of = take(4 * static_cast<int64_t>(requests));
    const int64_t weights = take(places * sizeof(float2)), values = take(places * D * 4);
    if (a) {
        unsigned char *const p = a->scratch;
        a->stretches = a->plan = reinterpret_cast<Kv4Stretch *>(p + plan);
        a->pieces = a->cut = reinterpret_cast<Kv4Stretch *>(p + cut);
        a->items_before = a->before = reinterpret_cast<int32_t *>(p + before);
        a->counts = a->count = reinterpret_cast<int32_t *>(p + count);
        a->shares = reinterpret_cast<Kv4Share *>(p + shares);
        a->group_of = reinterpret_cast<int32_t *>(p + group_of);
        a->weights = reinterpret_cast<float2 *>(p + weights);
        a->values = reinterpret_cast<float *>(p + values);
        a->places = places;
        a->most_pieces = most_pieces;
    }
    return at;
}

cudaError_t launch_kv4_prefix(const Kv4PrefixArgs &args, int D, cudaStream_t st, const DeviceInfo &dev) {
    Kv4PrefixArgs a = args;
    const int G = a.Hq / a.Hkv;
    a.members = a.requests;
    a.inject = dev.inject;
    a.item_rows = D == 64 ? 128 : 256;
    a.workers = D == 64 ? dev.num_sms : dev.num_sms / 2;
    // Rows that are streamed at most.  An item of the tensor cores' kernel takes as
    // long as ROWS / 16 streamed blocks; pieces fill the workers, so it is that of
    // one block or two.  (One group alone goes there whole, without a look at it.)
    constexpr int NONE_OF = 0x7fffffff;
    const int64_t own = (a.max_new < a.T ? a.max_new : a.T) * G, group = (a.max_group < a.T ? a.max_group : a.T) * G;
    const int64_t few_own = stream_rows(static_cast<int64_t>(a.members) * a.Hkv, D, dev), few_shared = D == 128 ? 32 : 16;
    const bool tensor = group > few_shared || own > few_own;
    a.least_shared = !tensor ? NONE_OF : a.groups == 1 ? 1 : static_cast<int>(few_shared) + 1;
    a.least_own = tensor && own > few_own ? static_cast<int>(few_own) + 1 : NONE_OF;
    const int smem = (2 * a.groups + a.members) * 4;
    static SmemLimit limit;
    if (smem > 40 * 1024)
        if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(plan_kernel), dev.device, smem)) return e;
    if (cudaError_t e = launch(reinterpret_cast<const void *>(plan_kernel), a, dim3(1), PLAN_THREADS, smem, st)) return e;
    Kv4SharedArgs s = a;
    if (tensor) {
        s.requests = a.most_pieces;
        if (cudaError_t e = launch_kv4_prompt(s, D, st, dev)) return e;
    }
    // the others by the form for few rows, and those with more of them by another
    s.requests = a.groups + a.members;
    const int64_t small = D == 256 ? 2 : D == 128 ? 4 : 8;
    int64_t most = own < few_own || !tensor ? own : few_own;
    const int64_t most_shared = !tensor ? group : a.groups == 1 ? 0 : group < few_shared ? group : few_shared;
    if (most_shared > most) most = most_shared;
    s.rows_least = 1;
    s.rows_most = NONE_OF;
    if (most > small && G <= small) {
        s.rows_most = static_cast<int>(small);
        if (cudaError_t e = stream(s, D, small, st, dev)) return e;
        s.rows_least = s.rows_most + 1;
        s.rows_most = NONE_OF;
    }
    if (cudaError_t e = stream(s, D, most, st, dev)) return e;
    const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>((a.Hq * (D / 4) + JOIN_THREADS - 1) / JOIN_THREADS));
    const void *const join = D == 64    ? reinterpret_cast<const void *>(join_kernel<64>)
                             : D == 128 ? reinterpret_cast<const void *>(join_kernel<128>)
                                        : reinterpret_cast<const void *>(join_kernel<256>);
    return launch(join, a, grid, JOIN_THREADS, 0, st);
}

}  // namespace w4
