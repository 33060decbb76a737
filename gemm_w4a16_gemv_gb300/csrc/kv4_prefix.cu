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
//
// Bound: operations of the tensor cores' kernel where a group has many rows, latency
// where it has few.  16 heads of 256 on 8: 128 requests behind 32768 tokens, 1 to 2000
// of their own, 117 us (each for itself: 790): the plan 8; the shared part 62, of which
// 11 until the first scores are there, 1.55 a key tile (the tensor pipe 1.0), 4 its end; the
// rest 22; the join 5.5; the rest between the launches.  With one token of their own, 16384
// more shared tokens are 30 us from 16384 to 32768 and 23 beyond (1500 TFLOP/s, 79% of the
// tensor cores' rate).  12 prompts of 101 to 700 tokens behind 6016: 362 us, 1080 TFLOP/s
// (nothing shared: their rows fill the items by themselves); 4 samples behind 2048, which lie
// in L2, 15.3 us without sharing, 34 with it (SMALL goes by the table's width).  32 heads of
// 128 on 8, 7 groups of up to 30 requests of 1 to 4 new tokens: 125 us: the plan 8, the
// shared parts 60 to 70, the rest 22, the join 5.
#include "kv4_stream.cuh"

namespace w4 {
namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int JOIN_THREADS = 128;
constexpr int64_t SMALL = 64 << 20;  // bytes of the cache that all requests can name
constexpr int AHEAD = 5;       // parts that a thread of the join asks for together
constexpr int KEYS = 128;      // of a key tile of the tensor cores' kernel
constexpr int ROUNDS = 4;      // items to a worker at most, where stretches are cut
constexpr int OVERHEAD = 4;    // cost of an item beside its key tiles, in key tiles,
constexpr int PARTS = 8;       // and of the parts that it writes
constexpr int SORTED = 256;    // requests that are compared with one another
constexpr int WHOLE = 1 << 24; // key tiles: more than any stretch has

// The stretches of a call, by one CTA.
//
// Sharing costs the writing and joining of parts, so a group shares only where
// that is less than its requests' own reading: in units of an item's key tile (a
// block of item_rows rows), a request costs an item for each such block, or
// stream_cost / 8 for each block of 16 where it is streamed; the shared stretch the
// same for all rows together, PARTS more for each item (its parts written and read
// back) and OVERHEAD for each item that begins anew.
//
// A shared stretch of many rows is cut into pieces, so that its items (a block of
// rows and a key head each) fill the workers: with w items a piece and t key
// tiles, cuts of c tiles give sum w ceil(t / c) items, at least sum w t / c and less
// than sum w more.  Between what these two say lies the least c that gives at most k
// items to a worker; of k = 1 .. ROUNDS the one is taken that ends first, after
// k (c + OVERHEAD) or all items' cost over the workers, those of the requests' own
// rows included, which fill what the others leave.  So items begin in the order of
// their length: those of requests with as many key tiles as a piece has, the pieces,
// the other requests', these by length too.  (The requests' first and as they come, and
// as if each took as long as a piece: prompts of 101 to 700 tokens, 4 groups of 3 behind
// 500 to 9000 tokens 255 us, now 184; 12 after 1000 to 9000 of their own behind 6016 627,
// now 559.)
//
// Every array is read once, all elements on their way together: the kernel is a
// chain of latencies (before the others can begin).
struct PlanSmem {
    int *cu, *ctx, *owner;              // [members + 1] rows before, [members] tokens before the step, the group
    int *border, *shared, *weight;      // [groups + 1], [groups] keys that are shared, items of a piece or 0
    int *tiles, *order;                 // [members] key tiles of those with many rows or 0; the longest first
    long long *place, *piece;           // [groups] first place; first piece << 40 | first item
    __device__ PlanSmem(unsigned char *p, int groups, int members) {
        place = reinterpret_cast<long long *>(p);
        piece = place + groups;
        cu = reinterpret_cast<int *>(piece + groups);
        ctx = cu + members + 1;
        owner = ctx + members;
        border = owner + members;
        shared = border + groups + 1;
        weight = shared + groups;
        tiles = weight + groups;
        order = tiles + members;
    }
    static int bytes(int groups, int members) { return 28 * groups + 20 * members + 8; }
};

__global__ void __launch_bounds__(PLAN_THREADS) plan_kernel(const Kv4PrefixArgs a) {
    extern __shared__ __align__(16) unsigned char plan_smem[];
    const PlanSmem x(plan_smem, a.groups, a.members);
    __shared__ long long all_weight, all_tiles, all_own;  // sums of w, of w t, of the requests' own items' cost
    __shared__ int longest, cut_tiles, cuts[ROUNDS], counts[ROUNDS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.Hq / a.Hkv;
    pdl_launch_dependents();
    pdl_wait();
    const long long table = a.max_blocks << a.bs_log2, cap = min(table, 0x7fffff00ll);
    const long long most = min(cap, 0x7fffff00ll - a.T);  // keys of a shared stretch (key and row number together: 31 bits)
    if (tid == 0) all_weight = all_tiles = all_own = 0, longest = 0;
    // ---- lengths and borders; if some are out of range, nothing is shared
    bool bad = false;
    for (int i = tid; i <= a.members; i += PLAN_THREADS) {
        const int v = a.cu_new[i];
        bad |= v < 0 || v > a.T;
        x.cu[i] = static_cast<int>(min(max(static_cast<long long>(v), 0ll), static_cast<long long>(a.T)));
    }
    for (int i = tid; i < a.members; i += PLAN_THREADS) {
        x.ctx[i] = a.seq_lens[i];
        x.owner[i] = -1;
    }
    for (int i = tid; i <= a.groups; i += PLAN_THREADS) {
        const int v = a.cu_groups[i];
        bad |= v < 0 || v > a.members;
        x.border[i] = min(max(v, 0), a.members);
    }
    for (int i = tid; i < a.groups; i += PLAN_THREADS) x.shared[i] = a.prefix_lens[i];
    __syncthreads();
    bool wrong = bad;  // (a length that is too long does not speak against sharing)
    for (int i = tid; i < a.members; i += PLAN_THREADS) {
        const int n = x.cu[i + 1] - x.cu[i], len = x.ctx[i];
        wrong |= n < 0;
        bad |= n < 0 || (n > 0 && (len < 0 || len > table));
        x.ctx[i] = max(len, -(1 << 30)) - max(n, 0);
    }
    for (int i = tid; i < a.groups; i += PLAN_THREADS) {
        wrong |= x.border[i + 1] < x.border[i];
        bad |= x.shared[i] < 0;
    }
    const bool sane = !__syncthreads_or(wrong);
    if (bad || wrong) atomicOr(a.status, kDevBadIndex);
    const int least_own = sane ? a.least_own : 0x7fffffff;
    auto blocks = [&](int rows, int of) { return (rows + of - 1) / of; };
    // ---- a warp per group: the tokens before all of its members' new ones
    for (int g = warp; g < a.groups; g += PLAN_THREADS / 32) {
        const int first = x.border[g], last = sane ? x.border[g + 1] : first;
        int least = x.shared[g], count = 0, apart = 0, begun = 0;
        for (int b = first + lane; b < last; b += 32) {
            x.owner[b] = g;
            const int rows = (x.cu[b + 1] - x.cu[b]) * G;
            if (rows <= 0) continue;
            least = min(least, x.ctx[b]);
            ++count;
            if (rows >= least_own) {
                apart += 8 * blocks(rows, a.item_rows);
                begun += blocks(rows, a.item_rows);
            } else apart += a.stream_cost * blocks(rows, 16);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        count = __reduce_add_sync(0xffffffffu, count);
        apart = __reduce_add_sync(0xffffffffu, apart);
        begun = __reduce_add_sync(0xffffffffu, begun);
        const int rows = (x.cu[last] - x.cu[first]) * G;
        int keys = count < 2 ? 0 : static_cast<int>(min(static_cast<long long>(max(least, 0)), most)) & ~15;
        const int tiles = (keys + KEYS - 1) / KEYS, items = blocks(rows, a.item_rows);
        const bool many = rows >= a.least_shared;
        const long long together = many ? 8ll * items * (tiles + PARTS + OVERHEAD) + 8ll * begun * OVERHEAD
                                        : static_cast<long long>(a.stream_cost) * blocks(rows, 16) * (tiles + 1);
        if (together >= static_cast<long long>(apart) * tiles) keys = 0;
        if (lane == 0) {
            x.shared[g] = keys;
            x.weight[g] = keys > 0 && many ? items * a.Hkv : 0;
            if (keys > 0 && many) {
                atomicAdd(reinterpret_cast<unsigned long long *>(&all_weight), static_cast<unsigned long long>(x.weight[g]));
                atomicAdd(reinterpret_cast<unsigned long long *>(&all_tiles), static_cast<unsigned long long>(x.weight[g]) * tiles);
                atomicMax(&longest, tiles);
            }
        }
    }
    // key tiles of a request's own
    auto own_tiles = [&](int b) {
        const int g = x.owner[b];
        const long long keys = min(static_cast<long long>(x.ctx[b]) + (x.cu[b + 1] - x.cu[b]), cap) - (g >= 0 ? x.shared[g] : 0);
        return static_cast<int>((max(keys, 1ll) + KEYS - 1) / KEYS);
    };
    if (least_own != 0x7fffffff) {
        __syncthreads();
        for (int b = tid; b < a.members; b += PLAN_THREADS) {
            const int rows = (x.cu[b + 1] - x.cu[b]) * G;
            const int tiles = rows >= least_own ? own_tiles(b) : 0;
            x.tiles[b] = tiles;
            if (tiles)
                atomicAdd(reinterpret_cast<unsigned long long *>(&all_own),
                          static_cast<unsigned long long>(blocks(rows, a.item_rows)) * a.Hkv * (tiles + OVERHEAD));
        }
    }
    __syncthreads();
    if (all_own > 0)
        for (int b = tid; b < a.members; b += PLAN_THREADS) {
            int at = b;
            if (a.members <= SORTED) {
                const int mine = x.tiles[b];
                at = 0;
                for (int o = 0; o < a.members; ++o) at += x.tiles[o] > mine || (x.tiles[o] == mine && o < b);
            }
            x.order[at] = b;
        }
    // ---- the cut, a warp for each number of rounds
    if (warp < ROUNDS && all_weight > 0) {
        const long long workers = static_cast<long long>(warp + 1) * a.workers;
        int hi = 0, count = static_cast<int>(workers);  // (0: more than so many at best)
        if (workers > all_weight) {
            hi = static_cast<int>(min((all_tiles + workers - all_weight - 1) / (workers - all_weight), static_cast<long long>(WHOLE)));
            int lo = static_cast<int>((all_tiles + workers - 1) / workers);
            while (lo < hi && a.groups <= 256) {  // the least that gives so few
                const int mid = (lo + hi) >> 1;
                int items = 0;  // (2^31 are not possible: mid is at least their mean)
                for (int g = lane; g < a.groups; g += 32)
                    if (x.shared[g] > 0) items += x.weight[g] * (((x.shared[g] + KEYS - 1) / KEYS + mid - 1) / mid);
                items = __reduce_add_sync(0xffffffffu, items);
                if (items <= workers) hi = mid, count = items;
                else lo = mid + 1;
            }
        }
        if (lane == 0) cuts[warp] = hi, counts[warp] = count;
    }
    bool loose = false;  // requests that share nothing and are streamed: some of their rows may be split
    auto is_loose = [&](int b) {
        const int n = x.cu[b + 1] - x.cu[b];
        return n > 0 && n * G < least_own && (x.owner[b] < 0 || x.shared[x.owner[b]] == 0);
    };
    for (int b = tid; b < a.members; b += PLAN_THREADS) loose |= is_loose(b);
    loose = __syncthreads_or(loose);
    // ---- pieces and places in their order
    if (warp == 0) {
        long long cost = 0x7fffffffffffffffll;
        int cut = WHOLE;
        for (int k = 0; k < ROUNDS && all_weight > 0; ++k) {
            const long long its = max((k + 1) * (static_cast<long long>(cuts[k]) + OVERHEAD),
                                      (all_tiles + static_cast<long long>(counts[k]) * OVERHEAD + all_own) / a.workers);
            if (cuts[k] > 0 && its < cost) cost = its, cut = cuts[k];
        }
        if (lane == 0) cut_tiles = cut;
        long long at = 0, place = a.T * a.Hq;  // (places of the requests' own come first)
        long long joined = 0;
        int shares = 0;
        auto before = [&](long long v, long long &total) {
            long long in = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, in, o);
                if (lane >= o) in += u;
            }
            const long long mine = total + in - v;
            total += __shfl_sync(0xffffffffu, in, 31);
            return mine;
        };
        const int most_tiles = min(cut, longest);  // of a piece
        auto own = [&](bool those_long) {
            for (int b0 = 0; all_own > 0 && b0 < a.members; b0 += 32) {
                const int b = b0 + lane < a.members ? x.order[b0 + lane] : 0, tiles = b0 + lane < a.members ? x.tiles[b] : 0;
                const int rows = (x.cu[b + 1] - x.cu[b]) * G;
                const bool many = tiles > 0 && (tiles >= most_tiles) == those_long;
                const long long mine = before(many ? 1ll << 40 | static_cast<long long>(blocks(rows, a.item_rows)) * a.Hkv : 0, at);
                if (many) {
                    a.before[mine >> 40] = static_cast<int>(mine & ((1ll << 40) - 1));
                    a.piece_of[b] = static_cast<int>(mine >> 40);
                }
            }
        };
        own(true);
        for (int g0 = 0; g0 < a.groups; g0 += 32) {
            const int g = g0 + lane;
            const bool on = g < a.groups && x.shared[g] > 0;
            const int tiles = on ? (x.shared[g] + KEYS - 1) / KEYS : 0, weight = on ? x.weight[g] : 0;
            int parts = on;
            if (weight) {
                parts = (tiles + cut - 1) / cut;
                const int even = (tiles + parts - 1) / parts;  // pieces of a length
                parts = (tiles + even - 1) / even;
            }
            const long long step = on ? static_cast<long long>(x.cu[x.border[g + 1]] - x.cu[x.border[g]]) * a.Hq : 0;
            const long long p = before(parts * step, place), tokens_before = before(step, joined) / a.Hq;
            const long long n = before(weight ? static_cast<long long>(parts) << 40 | static_cast<long long>(parts) * weight : 0, at);
            const unsigned some = __ballot_sync(0xffffffffu, on);
            if (on) {
                x.place[g] = p;
                x.piece[g] = n;
                a.shares[shares + __popc(some & ((1u << lane) - 1))] = {tokens_before, p, step, x.cu[x.border[g]], parts};
            }
            shares += __popc(some);
        }
        own(false);
        for (int b0 = 0; loose && b0 < a.members; b0 += 32) {
            const int b = b0 + lane;
            const bool on = b < a.members && is_loose(b);
            const unsigned some = __ballot_sync(0xffffffffu, on);
            const long long tokens_before = before(on ? static_cast<long long>(x.cu[b + 1] - x.cu[b]) * a.Hq : 0, joined) / a.Hq;
            if (on) a.shares[shares + __popc(some & ((1u << lane) - 1))] = {tokens_before, 0, 0, x.cu[b], 0};
            shares += __popc(some);
        }
        if (lane == 0) {
            a.count[0] = static_cast<int>(at >> 40);
            a.count[1] = shares;
            a.joined[0] = joined / a.Hq;
            a.before[at >> 40] = static_cast<int>(at & ((1ll << 40) - 1));
        }
    }
    __syncthreads();
    // ---- the groups' stretches, a warp each
    for (int g = warp; g < a.groups; g += PLAN_THREADS / 32) {
        Kv4Stretch s = {};
        const int keys = x.shared[g], weight = x.weight[g];
        if (keys > 0) {
            int row = a.members;  // a member with new tokens: the others' rows of the table may be old
            for (int b = x.border[g] + lane; b < x.border[g + 1]; b += 32)
                if (x.cu[b + 1] > x.cu[b]) row = min(row, b);
            row = __reduce_min_sync(0xffffffffu, row);
            s.token = x.cu[x.border[g]];
            s.tokens = x.cu[x.border[g + 1]] - s.token;
            s.end = s.base = keys;
            s.row = row;
            s.place = x.place[g];
            if (weight) {
                const int tiles = (keys + KEYS - 1) / KEYS, n = (tiles + cut_tiles - 1) / cut_tiles, even = (tiles + n - 1) / n;
                const int parts = (tiles + even - 1) / even;
                Kv4Stretch p = s;
                for (int i = lane; i < parts; i += 32) {
                    const int at = static_cast<int>(x.piece[g] >> 40) + i;
                    p.from = i * even * KEYS;
                    p.end = min((i + 1) * even * KEYS, keys);
                    p.place = s.place + static_cast<int64_t>(i) * s.tokens * a.Hq;
                    a.cut[at] = p;
                    a.before[at] = static_cast<int>(x.piece[g] & ((1ll << 40) - 1)) + i * weight;
                }
                s.tokens = 0;
            }
        }
        if (lane == 0) a.plan[g] = s;
    }
    // ---- what is left of each request
    for (int b = tid; b < a.members; b += PLAN_THREADS) {
        const int g = x.owner[b];
        Kv4Stretch s;
        s.token = x.cu[b];
        s.tokens = max(x.cu[b + 1] - s.token, 0);
        s.from = g >= 0 ? x.shared[g] : 0;
        s.end = static_cast<int>(cap);
        s.base = x.ctx[b];
        s.row = b;
        s.place = s.from > 0 ? static_cast<int64_t>(s.token) * a.Hq : -1;
        if (s.tokens * G >= least_own) {
            a.cut[a.piece_of[b]] = s;
            s.tokens = 0;
        }
        a.plan[a.groups + b] = s;
    }
    // for kernels that read it without waiting for this one's end
    __syncthreads();
    if (tid == 0) store_release(reinterpret_cast<unsigned int *>(a.scratch + PLAN_READY), 1);
}

// Four dimensions of a row a thread, JOIN_THREADS of a token's Hq D / 4 a CTA, which
// goes from one token of the shared stretches to the next; and the rows of no request.
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS, 8) join_kernel(const Kv4PrefixArgs a) {
    const int lane = threadIdx.x & 31;
    const int at = blockIdx.y * JOIN_THREADS + threadIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0 && at == 0) *reinterpret_cast<unsigned int *>(a.scratch + PLAN_READY) = 0;  // no kernel looks at it any more
    const int shares = a.counts[1];
    const int64_t tokens = *a.joined;
    const Kv4Share front = a.shares[0];  // (asked for beside their number)
    const int head = at / (D / 4), d = at % (D / 4) * 4;
    const bool on = at < a.Hq * (D / 4);
    for (int64_t t = rows_before(a, a.members) + blockIdx.x; on && t < a.T; t += gridDim.x)
        *reinterpret_cast<uint2 *>(a.out + (t * a.Hq + head) * D + d) = make_uint2(0, 0);
    for (int64_t i = blockIdx.x; i < tokens; i += gridDim.x) {
        int lo = 0, hi = shares;  // the last with `before` <= i
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, k = lo + lane * step;
            const unsigned below = __ballot_sync(0xffffffffu, k < hi && a.shares[k < hi ? k : lo].before <= i);
            lo += max(__popc(below) - 1, 0) * step;
            hi = min(hi, lo + step);
        }
        if (!on) continue;
        Kv4Share s = front;
        if (lo > 0) s = a.shares[lo];
        const int64_t row = static_cast<int64_t>(s.token + (i - s.before)) * a.Hq + head;  // of the output, and place of its own part
        const int64_t first = s.place + (i - s.before) * a.Hq + head;
        float m = NONE, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        // n parts, given their weights and values: AHEAD at a time, all on their way together
        auto add = [&](int n, auto weights_of, auto values_of) {
            for (int k0 = 0; k0 < n; k0 += AHEAD) {
                float2 w[AHEAD];
                float4 x[AHEAD];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    w[k] = __ldcg(weights_of(min(k0 + k, n - 1)));
                    x[k] = __ldcg(reinterpret_cast<const float4 *>(values_of(min(k0 + k, n - 1))));
                }
                float up = m;
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) up = fmaxf(up, w[k].x);
                const float old = ex2(m - up);
                m = up;
                l *= old;
                v.x *= old, v.y *= old, v.z *= old, v.w *= old;
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    const float f = k0 + k < n ? ex2(w[k].x - m) : 0.f;
                    l = fmaf(f, w[k].y, l);
                    v.x = fmaf(f, x[k].x, v.x);
                    v.y = fmaf(f, x[k].y, v.y);
                    v.z = fmaf(f, x[k].z, v.z);
                    v.w = fmaf(f, x[k].w, v.w);
                }
            }
        };
        // n of the arrays' parts from `at` on, or what teams left of the first one (w: what its place
        // holds; a sum that is NaN is a part like any other)
        auto add_at = [&](float2 w, int64_t at, int n, int64_t step) {
            if (!(w.y < 0.f)) {
                add(n, [&](int k) { return a.weights + at + k * step; }, [&](int k) { return a.values + (at + k * step) * D + d; });
                return;
            }
            // (kv4_stream.cuh: of a team two places for a row block, the second where it
            // begins; what a launch that timed out left there is no such place)
            const int what = __float_as_int(w.x), rows = what & 31, r = what >> 5 & 31, team = what >> 10 & 4095;
            const int count = static_cast<int>(fminf(-w.y, 4096.f));
            if (what >> 23 != 0 || r >= rows || count < 2 || (team + count) * rows > MAX_CTAS * warp_rows(D)) return;
            const float *const from = a.both_partials[what >> 22] + r * (D + 4);
            auto part = [&](int k) { return from + static_cast<int64_t>(2 * (team + k) + (k == 0)) * rows * (D + 4); };
            add(count, [&](int k) { return reinterpret_cast<const float2 *>(part(k)); }, [&](int k) { return part(k) + 4 + d; });
        };
        const float2 w_own = __ldcg(a.weights + row), w_first = s.parts ? __ldcg(a.weights + first) : w_own;
        if (w_own.y == PART_DONE) continue;
        if (s.parts) add_at(w_first, first, s.parts, s.step);
        add_at(w_own, row, 1, 0);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float o[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
        *reinterpret_cast<uint2 *>(a.out + row * D + d) =
            make_uint2(static_cast<uint32_t>(f32_to_bf16_bits(o[0])) | static_cast<uint32_t>(f32_to_bf16_bits(o[1])) << 16,
                       static_cast<uint32_t>(f32_to_bf16_bits(o[2])) | static_cast<uint32_t>(f32_to_bf16_bits(o[3])) << 16);
    }
}

// Borders and prefixes out of range, where nothing else looks at them.
__global__ void __launch_bounds__(JOIN_THREADS) check_kernel(const Kv4PrefixArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    bool bad = false;
    for (int g = threadIdx.x; g < a.groups; g += JOIN_THREADS) {
        const int from = a.cu_groups[g], to = a.cu_groups[g + 1];
        bad |= from < 0 || to < from || to > a.requests || a.prefix_lens[g] < 0;
    }
    if (bad) atomicOr(a.status, kDevBadIndex);
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
    const int64_t before = take(4 * (static_cast<int64_t>(most_pieces) + 1)), count = take(8);
    const int64_t shares = take((static_cast<int64_t>(groups) + requests) * sizeof(Kv4Share)), joined = take(8), piece_of = take(4 * static_cast<int64_t>(requests));
    const int64_t weights = take(places * sizeof(float2)), values = take(places * D * 4);
    const int64_t partials = take(kv4_attention_scratch(Hq, Hkv, D));
    if (a) {
        unsigned char *const p = a->scratch;
        a->stretches = a->plan = reinterpret_cast<Kv4Stretch *>(p + plan);
        a->pieces = a->cut = reinterpret_cast<Kv4Stretch *>(p + cut);
        a->items_before = a->before = reinterpret_cast<int32_t *>(p + before);
        a->counts = a->count = reinterpret_cast<int32_t *>(p + count);
        a->shares = reinterpret_cast<Kv4Share *>(p + shares);
        a->piece_of = reinterpret_cast<int32_t *>(p + piece_of);
        a->weights = reinterpret_cast<float2 *>(p + weights);
        a->values = reinterpret_cast<float *>(p + values);
        a->joined = reinterpret_cast<int64_t *>(p + joined);
        a->both_partials[0] = reinterpret_cast<float *>(p + COUNTER_BYTES);
        a->both_partials[1] = reinterpret_cast<float *>(p + partials);
        a->most_pieces = most_pieces;
    }
    return at;
}

cudaError_t launch_kv4_prefix(const Kv4PrefixArgs &args, int D, cudaStream_t st, const DeviceInfo &dev) {
    Kv4PrefixArgs a = args;
    const int G = a.Hq / a.Hkv;
    // what lies in L2 after its first reading is not worth sharing
    if ((static_cast<int64_t>(a.requests) * a.max_blocks << a.bs_log2) * a.Hkv * kv4_tile_bytes(D) / KV4_TILE <= SMALL) {
        if (cudaError_t e = launch_kv4_attention(Kv4UnitArgs{a}, D, st, dev)) return e;
        return launch(reinterpret_cast<const void *>(check_kernel), a, dim3(1), JOIN_THREADS, 0, st);
    }
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
    a.stream_cost = D == 128 ? 4 : 6;
    const int smem = PlanSmem::bytes(a.groups, a.members);
    static SmemLimit limit;
    if (smem > 40 * 1024)
        if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(plan_kernel), dev.device, smem)) return e;
    if (cudaError_t e = launch(reinterpret_cast<const void *>(plan_kernel), a, dim3(1), PLAN_THREADS, smem, st)) return e;
    Kv4SharedArgs s = a;
    if (tensor) {
        s.requests = a.most_pieces;
        if (cudaError_t e = launch_kv4_prompt(s, D, st, dev)) return e;
    }
    // the others; by two forms where most requests have few rows (most are decoded)
    s.requests = a.groups + a.members;
    const int64_t small = D == 256 ? 2 : D == 128 ? 4 : 8;
    int64_t most = own < few_own || !tensor ? own : few_own;
    const int64_t most_shared = !tensor ? group : a.groups == 1 ? 0 : group < few_shared ? group : few_shared;
    if (most_shared > most) most = most_shared;
    s.rows_least = 1;
    s.rows_most = NONE_OF;
    s.launch = 0;
    s.partials = a.both_partials[0];
    s.early = tensor;
    if (most > small && G <= small && (own <= small || own > few_own)) {
        s.rows_most = static_cast<int>(small);
        if (cudaError_t e = stream(s, D, small, st, dev)) return e;
        s.rows_least = s.rows_most + 1;
        s.rows_most = NONE_OF;
        s.launch = 1;
        s.partials = a.both_partials[1];
        s.early = true;
    }
    if (cudaError_t e = stream(s, D, most, st, dev)) return e;
    const unsigned wide = static_cast<unsigned>((a.Hq * (D / 4) + JOIN_THREADS - 1) / JOIN_THREADS);
    const unsigned rows = 8u * static_cast<unsigned>(dev.num_sms) / wide + 1;
    const dim3 grid(a.T < rows ? static_cast<unsigned>(a.T) : rows, wide);
    const void *const join = D == 64    ? reinterpret_cast<const void *>(join_kernel<64>)
                             : D == 128 ? reinterpret_cast<const void *>(join_kernel<128>)
                                        : reinterpret_cast<const void *>(join_kernel<256>);
    return launch(join, a, grid, JOIN_THREADS, 0, st);
}

}  // namespace w4
