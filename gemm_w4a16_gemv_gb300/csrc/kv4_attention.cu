// Attention over the paged 4-bit cache, streaming form (kv4_attention in the
// C header): decode steps and short pieces.
//
//   o = sum_j softmax_j(scale q . k_j) v_j  over the keys j that query p sees:
//   j <= p, and with a window w also p - j < w or j < sinks.
//
// Bound: memory.  A token's K and V of one head are 18 D / 16 bytes and every
// byte is read once; a row block of up to 8 NT rows (the G query heads of a
// key head times the request's new tokens) shares the read.  Measured, 16 query
// heads of 256 on 8: 64 requests of 255 to 32767 tokens 190 us, 5.3 TB/s or 78%
// of the copy bandwidth (the ALU pipe 58% busy, issue slots 64%: the codes'
// logic and parameters, then the memory); 128 requests with a window of 1024 and
// 4 sinks 69 us, 4.2 TB/s; one request of 8200 tokens 13 us (the memory would take
// 2.8: lengths, shares and pages 4, the copies 3.5, two tiles a warp that arrive
// together 3, the join in the CTA 1.3, the one across CTAs the rest).  The parts
// of a split row are read eight at a time: 14.9 -> 13.1 us, 200 -> 190, 71 -> 69;
// spread over more threads of the CTA besides it was 13.1 still.
//
// Work.  The unit is a cache tile (16 tokens of one head, one contiguous run
// fetched by one bulk copy).  The visible tiles of all (request, row block,
// head) segments are numbered in a row and split evenly over teams, so lengths
// of any raggedness, windows and one long request alike fill the GPU.  A team
// is one warp where there are many segments (it joins nothing with its
// neighbours but the segments at the ends of its share), a CTA's warps
// together where there are few (joined in shared memory first, or one long
// row would leave two thousand partial results).  Every team finds its share
// itself from the lengths (a prefix sum in shared memory).  A segment inside
// one share is finished there; of one that several share, each team writes its
// partial result (maximum, sum, weighted values) to scratch and the last to
// arrive joins them in the order of the teams, so results do not depend on
// timing.  No team waits for another.
//
// Each warp has its own ring of stages and barriers: no producer warp and no
// barrier between warps inside a segment.
//
// Arithmetic per tile, all products on mma.m16n8k16 (binary16 in, binary32
// out) with the CODES as the A operand: the low and high nibble pairs of a
// word masked in place are binary16 subnormals c 2^-24 and 16 c 2^-24, exact,
// so 8 codes cost 5 logic operations and no conversion.
//   S^T = K Q^T (16 keys x 8 columns), a sum per group of 64 dimensions:
//     x += s (acc - z sum(q))                        binary32, exact products
//     (q enters as binary16 after a power-of-two scale of its row)
//   O^T += (V - z)^T P^T (16 dimensions x 8 columns), per group with P' = p s
//     rounded to binary16.  Here code and zero are subtracted first (exact, a
//     pair operation per two codes): summed apart, p c - p z would leave
//     2^-24 of p z where a value is zero.
// The 8 columns are rows of the segment, with accumulators for each group of
// dimensions; or, where 8 / groups rows are enough (SPLIT), groups x rows: Q
// and P' are zero outside their group, one set of accumulators serves all
// groups (16 registers instead of 64 at D = 256), and each lane handles the
// parameters of one group instead of all.
// The reference of the exponentials follows the running maximum of x + log2(s),
// so that the largest P' lies in [2^7, 2^15] whatever the magnitude of V (binary16
// then keeps 11 bits of weights down to 2^-21 of it); it moves (and the
// accumulators are scaled) only when P' would pass 2^15.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {
namespace {

constexpr int MAX_CTAS = 160;         // scratch is sized for this many
constexpr int MAX_WARPS = 20;         // of a CTA
constexpr int MAX_TEAMS = MAX_CTAS * MAX_WARPS;
constexpr int COUNTER_BYTES = 13312;  // arrival counters and the prompt kernel's two
static_assert(MAX_TEAMS * 4 <= PROMPT_COUNTERS && PROMPT_COUNTERS + 8 <= COUNTER_BYTES, "counters");
// Partial results that two slots per team can need: warps x rows of an instance.
constexpr int warp_rows(int D) { return D == 256 ? 128 : D == 128 ? 192 : 256; }
constexpr int TEAM_RATIO = 5;         // warps to a segment up to which a warp is a team of its own
constexpr float NONE = -1e30f;        // reference of a row that has seen no key

// 2^x by the hardware's approximation (2 ulp): a weight is rounded to 11 bits
// after it.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// Binary16 pairs, subnormals included.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// The larger magnitude of each half, with some sign.
__device__ __forceinline__ uint32_t maxabs_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Keys of the MMA's rows 0..7 within a half tile.  Any order is right (both
// products sum over keys); this one makes the 8-byte reads of K (lanes of
// four consecutive rows) and the 4-byte reads of V (keys of rows 2 t, and of
// rows 2 t + 1) fall into different banks.
__device__ __forceinline__ int key_of_row(int r) { return (0x57463120u >> (4 * r)) & 15; }

// Rows of request b that this kernel answers: new tokens x query heads of a
// key head, or none when the prompt kernel takes them.
__device__ __forceinline__ int rows_of(const Kv4AttnArgs &a, int b, int G) {
    const int rows = (rows_before(a, b + 1) - rows_before(a, b)) * G;
    return rows >= a.rows_least && rows <= a.rows_most ? rows : 0;
}

// A segment: the rows [r0, r0 + rows) of (request b, key head h) and the cache
// tiles they see: the first ns, then from `low` on; nt in all.
struct Segment {
    int b, h, r0, rows;
    int nt, ns, low;
    int end;        // keys at or past this are seen by no row
    int base;       // position of row r is base + r / G
};

template <int R>
__device__ __forceinline__ void shape_segment(const Kv4AttnArgs &a, int b, int r0, int G, Segment &s) {
    const int n = rows_before(a, b + 1) - rows_before(a, b);
    const int total = n * G;
    s.b = b;
    s.r0 = r0;
    s.rows = min(R, total - r0);
    const long long seq = a.seq_lens[b];
    const long long cap = static_cast<long long>(a.max_blocks) << a.bs_log2;
    s.base = static_cast<int>(seq - n);
    const long long p_lo = seq - n + r0 / G, p_hi = seq - n + (r0 + s.rows - 1) / G;
    long long end = p_hi + 1 < cap ? p_hi + 1 : cap;
    if (end < 0) end = 0;
    long long low = 0, ns = 0;
    if (a.window > 0) {
        low = p_lo - a.window + 1;
        low = low > 0 ? low >> 4 : 0;
        const long long sk = a.sinks < end ? a.sinks : end;
        ns = (sk + 15) >> 4;
        if (low < ns) low = ns;
    }
    const long long hi = (end + 15) >> 4;
    long long nt = ns + (hi > low ? hi - low : 0);
    if (nt < 1) nt = 1;  // a segment that sees nothing still writes its zeros
    s.end = static_cast<int>(end);
    s.ns = static_cast<int>(ns);
    s.low = static_cast<int>(low);
    s.nt = static_cast<int>(nt);
}

// Walks the segments in order: key heads of a row block, row blocks of a
// request, requests.  `first` is the segment's first tile relative to the
// start of this CTA's share (negative when it began in an earlier CTA).
template <int R>
struct Cursor {
    Segment s;
    int first;
    __device__ __forceinline__ void next(const Kv4AttnArgs &a, int G) {
        first += s.nt;
        if (++s.h < a.Hkv) return;
        s.h = 0;
        int b = s.b, r0 = s.r0 + R;
        if (r0 >= rows_of(a, b, G)) {
            r0 = 0;
            do ++b;
            while (b < a.requests && rows_of(a, b, G) == 0);
            if (b >= a.requests) return;  // past the last segment: not used
        }
        shape_segment<R>(a, b, r0, G, s);
    }
    __device__ __forceinline__ int tile(int u) const {
        const int k = u - first;
        return k < s.ns ? k : k - s.ns + s.low;
    }
};

// Shapes of an instance: D, columns' sets of 8, warps, warps of a team, and
// whether the columns are split between groups and rows.
template <int D, int NT, int W, int TEAM, bool SPLIT>
struct Stream {
    static constexpr int G64 = D / 64;
    static constexpr int SETS = SPLIT ? 1 : G64;              // sets of accumulators
    static constexpr int RPT = SPLIT ? 8 / G64 : 8;           // rows of 8 columns
    static constexpr int R = RPT * NT;                        // rows of a segment
    static constexpr int TEAMS = W / TEAM;                    // of a CTA
    static constexpr int QBUF = TEAM == 1 ? 1 : 2;            // buffers of Q
    static constexpr int QFRAG = NT * SETS * 2 * 32 * 16;     // bytes: [NT][set][mma pair][lane] 4 words
    static constexpr int REGION = 2 * 64 + 4;                 // floats: two rows of 64 dimensions
    static constexpr int MERGE_WARP = NT * SETS * 4 * REGION;
    // per team, offsets in bytes
    static constexpr int q = 0;                               // [QBUF][QFRAG]
    static constexpr int qs = q + QBUF * QFRAG;               // [QBUF][SETS][8 NT] scaled row sums
    static constexpr int fr = qs + QBUF * SETS * NT * 32;     // [QBUF][8 NT] factor of the scores
    static constexpr int bars = fr + QBUF * NT * 32;          // [TEAM][8] barriers
    static constexpr int team_bytes = (bars + TEAM * 64 + 15) / 16 * 16;
    // of the CTA
    static constexpr int teams = 128;                         // after 16 zero bytes and a word for the CTA
    static constexpr int mx = teams + TEAMS * team_bytes;     // [2][W][R], or the prefix sum's W sums
    static constexpr int sm = mx + (TEAM == 1 ? W * 8 : 2 * W * R * 4);
    static constexpr int merge = (sm + (TEAM == 1 ? 0 : 2 * W * R * 4) + 127) / 128 * 128;  // [W / 2][MERGE_WARP] floats
    static constexpr int ring = (merge + (TEAM == 1 ? 0 : W / 2 * MERGE_WARP * 4) + 127) / 128 * 128;
};

// Q of 8 columns of a segment as the MMA's B operand, by one warp: lane (g, t)
// takes column g, 16 dimensions from 64 i + 16 t on of its group(s).
template <typename L, int D, bool SPLIT>
__device__ __forceinline__ void build_q(const Kv4AttnArgs &a, const Segment &s, int G, int nt, int nts, unsigned char *team,
                                        int par, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int r = L::RPT * nt + g % L::RPT;
    const bool on = r < s.rows;
    const int row = s.r0 + (on ? r : 0);
    const int tok = rows_before(a, s.b) + row / G;
    const int own = SPLIT ? g / L::RPT : 0;  // group of the column
    const uint16_t *src = a.q + static_cast<int64_t>(tok) * a.q_stride + static_cast<int64_t>(s.h * G + row % G) * D +
                          64 * own + 16 * t;
    uint4 raw[L::SETS][2];
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < L::SETS; ++i) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            raw[i][k] = on ? *reinterpret_cast<const uint4 *>(src + 64 * i + 8 * k) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {raw[i][k].x, raw[i][k].y, raw[i][k].z, raw[i][k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u))));
        }
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    if (SPLIT) {  // the row's other groups are other columns
        if (L::G64 == 4) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 8));
        if (L::G64 >= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 16));
    }
    // the row's largest magnitude to [2^13, 2^14): the sums of the odd
    // dimensions' 1/16 stay exact down to 2^-33 of it
    int kappa = big > 0.f ? 13 - (static_cast<int>(__float_as_uint(big) >> 23) - 127) : 0;
    kappa = min(max(kappa, -110), 110);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + kappa) << 23);
#pragma unroll
    for (int i = 0; i < L::SETS; ++i) {
        float v[16], sum = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {raw[i][k].x, raw[i][k].y, raw[i][k].z, raw[i][k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * k + 2 * j] = __uint_as_float(w[j] << 16) * up;
                v[8 * k + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u) * up;
                sum += v[8 * k + 2 * j] + v[8 * k + 2 * j + 1];
            }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (t == 0)
            reinterpret_cast<float *>(team + L::qs)[(par * L::SETS + i) * 8 * nts + 8 * nt + g] =
                sum * 5.9604644775390625e-8f;  // 2^-24
        uint4 *dst = reinterpret_cast<uint4 *>(team + L::q + par * L::QFRAG) + (nt * L::SETS + i) * 2 * 32 + lane;
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // word k of the lane's two: dimensions 8 k .. 8 k + 7
            const float *x = v + 8 * k;
            dst[k * 32] = make_uint4(pack_f16(x[0], x[4]), pack_f16(x[1] * 0.0625f, x[5] * 0.0625f),
                                     pack_f16(x[2], x[6]), pack_f16(x[3] * 0.0625f, x[7] * 0.0625f));
        }
    }
    if (t == 0)
        reinterpret_cast<float *>(team + L::fr)[par * 8 * nts + 8 * nt + g] =
            on ? a.scale * 1.4426950408889634f * (16777216.f * __uint_as_float(static_cast<uint32_t>(127 - kappa) << 23))
               : 0.f;
}

template <int D, int NT, int W, int TEAM, bool SPLIT>
__global__ void __launch_bounds__(W * 32, 1) attn_stream_kernel(const Kv4AttnArgs a, const int depth) {
    using L = Stream<D, NT, W, TEAM, SPLIT>;
    constexpr int R = L::R, RPT = L::RPT, G64 = L::G64, SETS = L::SETS, TB = kv4_tile_bytes(D);
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int G = a.Hq / a.Hkv;
    const int tw = warp % TEAM;  // the warp's number in its team
    unsigned char *const team = smem + L::teams + (warp / TEAM) * L::team_bytes;
    uint64_t *const bars = reinterpret_cast<uint64_t *>(team + L::bars) + tw * 8;
    unsigned char *const ring = smem + L::ring + static_cast<size_t>(warp) * depth * TB;
    long long *const cum = reinterpret_cast<long long *>(smem + L::ring + static_cast<size_t>(W) * depth * TB);
    volatile int *const misc = reinterpret_cast<volatile int *>(smem + 16);
    auto team_sync = [&]() {
        if (TEAM == 1) __syncwarp();
        else __syncthreads();
    };

    if (tid < 4) reinterpret_cast<uint32_t *>(smem)[tid] = 0;
    if (lane == 0)
        for (int i = 0; i < depth; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
    pdl_launch_dependents();
    pdl_wait();

    // ---- tiles of the requests, their running sum
    {
        const int per = (a.requests + W * 32 - 1) / (W * 32);
        const int b0 = min(tid * per, a.requests), b1 = min(b0 + per, a.requests);
        long long sum = 0;
        for (int b = b0; b < b1; ++b) {
            asm volatile("prefetch.global.L1 [%0];" ::"l"(a.seq_lens + b));  // asked for beside cu_new
            if (a.first_launch && blockIdx.x == 0) check_lengths(a, b);
            const int rows = rows_of(a, b, G);
            long long n = 0;
            for (int r0 = 0; r0 < rows; r0 += R) {
                Segment s;
                shape_segment<R>(a, b, r0, G, s);
                n += s.nt;
            }
            cum[b + 1] = n * a.Hkv;
            sum += n * a.Hkv;
        }
        long long in = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, in, o);
            if (lane >= o) in += v;
        }
        long long *const tot = reinterpret_cast<long long *>(smem + L::mx);  // W sums, before its first use
        if (lane == 31) tot[warp] = in;
        __syncthreads();
        long long at = in - sum;
        for (int w = 0; w < warp; ++w) at += tot[w];
        if (tid == 0) cum[0] = 0;
        for (int b = b0; b < b1; ++b) {
            at += cum[b + 1];
            cum[b + 1] = at;
        }
        __syncthreads();
    }
    if (a.first_launch) {  // rows that belong to no request
        const int64_t from = static_cast<int64_t>(rows_before(a, a.requests)) * a.Hq * D / 8;
        const int64_t to = a.T * a.Hq * D / 8;
        for (int64_t i = from + static_cast<int64_t>(blockIdx.x) * W * 32 + tid; i < to;
             i += static_cast<int64_t>(gridDim.x) * W * 32)
            reinterpret_cast<uint4 *>(a.out)[i] = make_uint4(0, 0, 0, 0);
    }
    // teams that take part: no more than there are tiles, so that none between
    // the first and the last of a shared segment is without a part of it
    const long long U = cum[a.requests];
    const long long all_teams = static_cast<long long>(gridDim.x) * L::TEAMS, C = U < all_teams ? U : all_teams;
    // (neighbouring teams on different SMs: a small U fills them evenly)
    const int me = static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) * (warp / TEAM);
    if (me >= C) return;
    const long long u0 = U * me / C;
    const int mine = static_cast<int>(U * (me + 1) / C - u0);

    // ---- the segment of the first tile
    Cursor<R> cur;
    {
        int lo = 0, hi = a.requests;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cum[mid] <= u0) lo = mid;
            else hi = mid;
        }
        long long rest = u0 - cum[lo];
        int r0 = 0;
        while (true) {
            shape_segment<R>(a, lo, r0, G, cur.s);
            if (rest < static_cast<long long>(cur.s.nt) * a.Hkv) break;
            rest -= static_cast<long long>(cur.s.nt) * a.Hkv;
            r0 += R;
        }
        cur.s.h = static_cast<int>(rest / cur.s.nt);
        cur.first = -static_cast<int>(rest - static_cast<long long>(cur.s.h) * cur.s.nt);
    }
    Cursor<R> pre = cur;     // of the next tile to fetch
    int pre_u = tw;          // its number in the team's share
    bool bad = false;
    const int sub_log2 = a.bs_log2 - 4;
    const size_t page_bytes = (static_cast<size_t>(a.Hkv) << sub_log2) * TB;
    const int32_t *pages = a.block_table + static_cast<int64_t>(pre.s.b) * a.max_blocks;
    // the next tile's page and place in it (-1: nothing to fetch); asked for a
    // step before the copy is issued, so that the latency is not waited for
    int page = -1, place = -1;
    auto ask = [&]() {
        page = place = -1;
        if (pre_u >= mine) return;
        if (pre_u >= pre.first + pre.s.nt) {
            do pre.next(a, G);
            while (pre_u >= pre.first + pre.s.nt);
            pages = a.block_table + static_cast<int64_t>(pre.s.b) * a.max_blocks;
        }
        const int tile = pre.tile(pre_u);
        if (tile * 16 >= pre.s.end) return;
        page = pages[tile >> sub_log2];
        place = ((pre.s.h << sub_log2) + (tile & ((1 << sub_log2) - 1))) * TB;
    };
    uint32_t live = 0;       // bit of a stage: it holds a tile
    // lane 0 issues the copies (test-only injection: none) until one of its waits
    // runs out: a stage whose copy has not arrived must not be handed out again
    bool issues = lane == 0 && !(a.inject & kInjectStallPipeline);
    auto fetch = [&](int stage) {
        const bool in = place >= 0 && page >= 0 && page < a.num_blocks;
        bad |= place >= 0 && !in;
        if (in && issues) {
            mbar_arrive_expect_tx(&bars[stage], TB);
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem_u32(ring + static_cast<size_t>(stage) * TB)),
                         "l"(a.cache + static_cast<size_t>(page) * page_bytes + place), "r"(TB), "r"(smem_u32(&bars[stage]))
                         : "memory");
        }
        live = in ? live | (1u << stage) : live & ~(1u << stage);
        pre_u += TEAM;
        ask();
    };
    ask();
    for (int i = 0; i < depth; ++i) fetch(i);

    uint32_t parity = 0;  // bit per stage
    int stage = 0;
    int u = tw;
    int par = 0;          // of the per-segment buffers
    bool ok = true;
    const int kA = key_of_row(g), vA = key_of_row(2 * t), vB = key_of_row(2 * t + 1);
    // SPLIT: group of this lane's two accumulator columns, and of its column of B
    const int col_group = SPLIT ? 2 * t / RPT : 0, b_group = SPLIT ? g / RPT : 0;

    if (tw >= TEAM - NT || TEAM == 1) {
        if (TEAM == 1) {
            for (int n = 0; n < NT; ++n) build_q<L, D, SPLIT>(a, cur.s, G, n, NT, team, 0, lane);
        } else build_q<L, D, SPLIT>(a, cur.s, G, TEAM - 1 - tw, NT, team, 0, lane);
    }
    team_sync();

    while (true) {
        const Segment s = cur.s;
        const int seg_end = min(cur.first + s.nt, mine);
        float O[NT][SETS][4][4], M[NT][2], Ls[NT][2], QS[NT][SETS][2], F[NT][2];
        int P[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < SETS; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[n][i][k][e] = 0.f;
                const float2 v = *reinterpret_cast<const float2 *>(team + L::qs + ((par * SETS + i) * 8 * NT + 8 * n + 2 * t) * 4);
                QS[n][i][0] = v.x;
                QS[n][i][1] = v.y;
            }
            const float2 f = *reinterpret_cast<const float2 *>(team + L::fr + (par * 8 * NT + 8 * n + 2 * t) * 4);
            F[n][0] = f.x;
            F[n][1] = f.y;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                M[n][e] = NONE;
                Ls[n][e] = 0.f;
                P[n][e] = s.base + (s.r0 + min(RPT * n + (2 * t + e) % RPT, s.rows - 1)) / G;
            }
        }
        const int p_lo = s.base + s.r0 / G, p_hi = s.base + (s.r0 + s.rows - 1) / G;

        for (; u < seg_end; u += TEAM) {
            if (live >> stage & 1u) {
                if (!mbar_try_wait(smem_u32(&bars[stage]), parity >> stage & 1u) && ok) {
                    ok = mbar_wait(&bars[stage], parity >> stage & 1u, a.status);
                    if (!ok && issues) {
                        // no copy may be under way when the CTA ends: wait (bounded)
                        // for those issued and not waited for
#pragma unroll 1
                        for (int i = 0; live >> i; ++i)
                            if (live >> i & 1u) mbar_wait(&bars[i], parity >> i & 1u, nullptr);
                        issues = false;
                    }
                }
                parity ^= 1u << stage;
                const unsigned char *tile = ring + static_cast<size_t>(stage) * TB;
                const int j0 = cur.tile(u) * 16;
                const uint4 *qf = reinterpret_cast<const uint4 *>(team + L::q + par * L::QFRAG) + lane;
                // ---- scores
                float acc[NT][SETS][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < SETS; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[n][i][e] = 0.f;
#pragma unroll
                for (int i = 0; i < G64; ++i) {
                    const uint2 k0 = *reinterpret_cast<const uint2 *>(tile + (i * 16 + kA) * 32 + t * 8);
                    const uint2 k1 = *reinterpret_cast<const uint2 *>(tile + (i * 16 + kA + 8) * 32 + t * 8);
                    // SPLIT: columns of other groups read the zeros at the start
                    const bool zero = SPLIT && b_group != i;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t w0 = k ? k0.y : k0.x, w1 = k ? k1.y : k1.x;
                        const uint32_t w0h = w0 >> 8, w1h = w1 >> 8;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 b = *(zero ? reinterpret_cast<const uint4 *>(smem)
                                                   : qf + ((n * SETS + (SPLIT ? 0 : i)) * 2 + k) * 32);
                            float(&c)[4] = acc[n][SPLIT ? 0 : i];
                            mma_f16(c, w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, b.x, b.y);
                            mma_f16(c, w0h & 0x000f000fu, w1h & 0x000f000fu, w0h & 0x00f000f0u, w1h & 0x00f000f0u, b.z, b.w);
                        }
                    }
                }
                float x[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
#pragma unroll
                for (int i = 0; i < SETS; ++i) {
                    const int at = SPLIT ? col_group : i;
                    const uint32_t sz0 = *reinterpret_cast<const uint32_t *>(tile + 16 * D + (at * 16 + kA) * 4);
                    const uint32_t sz1 = *reinterpret_cast<const uint32_t *>(tile + 16 * D + (at * 16 + kA + 8) * 4);
                    const float s0 = f16_lo(sz0), z0 = f16_hi(sz0), s1 = f16_lo(sz1), z1 = f16_hi(sz1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        x[n][0] = fmaf(s0, fmaf(-z0, QS[n][i][0], acc[n][i][0]), x[n][0]);
                        x[n][1] = fmaf(s0, fmaf(-z0, QS[n][i][1], acc[n][i][1]), x[n][1]);
                        x[n][2] = fmaf(s1, fmaf(-z1, QS[n][i][0], acc[n][i][2]), x[n][2]);
                        x[n][3] = fmaf(s1, fmaf(-z1, QS[n][i][1], acc[n][i][3]), x[n][3]);
                    }
                }
                if (SPLIT && G64 > 1) {  // the groups are on neighbouring lanes
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[n][e] += __shfl_xor_sync(0xffffffffu, x[n][e], 2);
                            if (G64 == 4) x[n][e] += __shfl_xor_sync(0xffffffffu, x[n][e], 1);
                        }
                }
                // ---- V's parameters; what lies past the last key of the
                // cache may hold anything and counts as zeros
                const int ja = j0 + kA, jb = ja + 8;
                const bool whole = j0 + 16 <= s.end;
                uint32_t vz0[SETS], vz1[SETS];  // (scale, zero) of keys kA, kA + 8
                uint32_t top0 = 0, top1 = 0;
#pragma unroll
                for (int i = 0; i < SETS; ++i) {
                    const int at = SPLIT ? col_group : i;
                    vz0[i] = *reinterpret_cast<const uint32_t *>(tile + 17 * D + (at * 16 + kA) * 4);
                    vz1[i] = *reinterpret_cast<const uint32_t *>(tile + 17 * D + (at * 16 + kA + 8) * 4);
                    if (!whole) {
                        vz0[i] = ja < s.end ? vz0[i] : 0u;
                        vz1[i] = jb < s.end ? vz1[i] : 0u;
                    }
                    top0 = maxabs_f16x2(top0, vz0[i]);
                    top1 = maxabs_f16x2(top1, vz1[i]);
                }
                // (SPLIT: each lane its own group's; the reference below takes the largest of the lanes)
                const float l0 = lg2(fmaxf(fabsf(f16_lo(top0)), 5.9604644775390625e-8f));
                const float l1 = lg2(fmaxf(fabsf(f16_lo(top1)), 5.9604644775390625e-8f));
                // ---- mask and running reference
                const bool free = j0 + 16 <= p_lo + 1 && (a.window <= 0 || p_hi - j0 < a.window || j0 + 16 <= a.sinks);
                bool grow = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] *= F[n][e & 1];
                    if (!free) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = e < 2 ? ja : jb, p = P[n][e & 1];
                            const bool see = j <= p && j < s.end && (a.window <= 0 || p - j < a.window || j < a.sinks);
                            x[n][e] = see ? x[n][e] : -INFINITY;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        grow |= fmaxf(x[n][e] + l0, x[n][e + 2] + l1) > M[n][e] + 15.f;
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = fmaxf(x[n][e] + l0, x[n][e + 2] + l1);
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            if (SPLIT && G64 > 1) {
                                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                                if (G64 == 4) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                            }
                            m = fmaxf(m - 7.f, M[n][e]);
                            const float f = ex2(M[n][e] - m);
                            M[n][e] = m;
                            Ls[n][e] *= f;
#pragma unroll
                            for (int i = 0; i < SETS; ++i)
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    O[n][i][k][e] *= f;
                                    O[n][i][k][e + 2] *= f;
                                }
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[n][e] = ex2(x[n][e] - M[n][e & 1]);
                        Ls[n][e & 1] += x[n][e];
                    }
                // ---- weights times scales as the B operand; zeros of this
                // lane's four keys (SPLIT: of group b_group)
                uint32_t b[SETS][NT][2], zab[SETS], zcd[SETS];
#pragma unroll
                for (int i = 0; i < SETS; ++i) {
                    const float v0 = f16_lo(vz0[i]), v1 = f16_lo(vz1[i]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        b[i][n][0] = transpose8x8(pack_f16(x[n][0] * v0, x[n][1] * v0));
                        b[i][n][1] = transpose8x8(pack_f16(x[n][2] * v1, x[n][3] * v1));
                    }
                    zab[i] = transpose8x8(__byte_perm(vz0[i], 0, 0x3232));
                    zcd[i] = transpose8x8(__byte_perm(vz1[i], 0, 0x3232));
                }
                // ---- weighted values
#pragma unroll
                for (int i = 0; i < G64; ++i) {
                    const unsigned char *vt = tile + 8 * D + i * 512 + g * 4;
                    const uint32_t wA = *reinterpret_cast<const uint32_t *>(vt + vA * 32);
                    const uint32_t wB = *reinterpret_cast<const uint32_t *>(vt + vB * 32);
                    const uint32_t wC = *reinterpret_cast<const uint32_t *>(vt + (vA + 8) * 32);
                    const uint32_t wD = *reinterpret_cast<const uint32_t *>(vt + (vB + 8) * 32);
                    uint32_t za = zab[SPLIT ? 0 : i], zc = zcd[SPLIT ? 0 : i];
                    if (SPLIT && G64 > 1) {  // from a lane whose column is of group i
                        za = __shfl_sync(0xffffffffu, za, i * RPT * 4 + t);
                        zc = __shfl_sync(0xffffffffu, zc, i * RPT * 4 + t);
                    }
                    // in the codes' units, 2^-24 and 2^-20
                    const uint32_t za1 = mul_f16x2(za, 0x00010001u), za16 = mul_f16x2(za, 0x00100010u);
                    const uint32_t zc1 = mul_f16x2(zc, 0x00010001u), zc16 = mul_f16x2(zc, 0x00100010u);
                    uint32_t bi[NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        bi[n][0] = SPLIT ? (b_group == i ? b[0][n][0] : 0u) : b[SPLIT ? 0 : i][n][0];
                        bi[n][1] = SPLIT ? (b_group == i ? b[0][n][1] : 0u) : b[SPLIT ? 0 : i][n][1];
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // dimensions 8 g + 2 k and 8 g + 2 k + 1 of keys A, B and C, D
                        const uint32_t sel = k < 2 ? 0x5410u : 0x7632u;
                        uint32_t ab = __byte_perm(wA, wB, sel), cd = __byte_perm(wC, wD, sel);
                        if (k & 1) ab >>= 8, cd >>= 8;
                        const uint32_t a0 = sub_f16x2(ab & 0x000f000fu, za1), a1 = sub_f16x2(ab & 0x00f000f0u, za16);
                        const uint32_t a2 = sub_f16x2(cd & 0x000f000fu, zc1), a3 = sub_f16x2(cd & 0x00f000f0u, zc16);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(O[n][SPLIT ? 0 : i][k], a0, a1, a2, a3, bi[n][0], bi[n][1]);
                    }
                }
                __syncwarp();
            }
            fetch(stage);
            stage = stage + 1 == depth ? 0 : stage + 1;
        }

        // ---- the segment's end
        const int seg_first = cur.first, seg_nt = s.nt;
        const bool last = seg_first + seg_nt >= mine;  // no further segment in this share
        const bool split = seg_first < 0 || seg_first + seg_nt > mine;
        int c_first = 0, c_last = 0;
        if (split) {
            const long long seg_u0 = u0 + seg_first;
            c_first = static_cast<int>(((seg_u0 + 1) * C - 1) / U);
            c_last = static_cast<int>(((seg_u0 + seg_nt) * C - 1) / U);
        }
        // partial results: [team][2][R][D + 4], slot 1 where the segment begins in
        // the share; of a row: maximum, sum, two unused, weighted values
        constexpr int PART = R * (D + 4);
        float *const parts = reinterpret_cast<float *>(a.scratch + COUNTER_BYTES);
        float *const part = parts + (static_cast<size_t>(me) * 2 + (seg_first >= 0 ? 1 : 0)) * PART;
        unsigned int *const count = reinterpret_cast<unsigned int *>(a.scratch) + c_first;
        auto row_of = [&](int r) -> uint16_t * {  // out of row r
            const int row = s.r0 + r, tok = rows_before(a, s.b) + row / G;
            return a.out + (static_cast<int64_t>(tok) * a.Hq + s.h * G + row % G) * D;
        };
        // accumulators to their units (2^-24 for even dimensions, 2^-20 for odd
        // ones), and the sums over the keys
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = Ls[n][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                Ls[n][e] = l;
            }
        if constexpr (TEAM == 1) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = RPT * n + (2 * t + e) % RPT;
                    if (r < s.rows) {
                        const float inv = Ls[n][e] == 0.f ? 0.f : 1.f / Ls[n][e];
#pragma unroll
                        for (int i = 0; i < SETS; ++i) {
                            const int d = 64 * (SPLIT ? col_group : i) + 8 * g;
                            float v[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                v[2 * k] = O[n][i][k][e] * 16777216.f;
                                v[2 * k + 1] = O[n][i][k][e + 2] * 1048576.f;
                            }
                            if (!split) {
                                uint32_t w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    w[k] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * k] * inv)) |
                                           static_cast<uint32_t>(f32_to_bf16_bits(v[2 * k + 1] * inv)) << 16;
                                *reinterpret_cast<uint4 *>(row_of(r) + d) = make_uint4(w[0], w[1], w[2], w[3]);
                            } else {
                                float *const to = part + r * (D + 4);
                                __stcg(reinterpret_cast<float4 *>(to + 4 + d), make_float4(v[0], v[1], v[2], v[3]));
                                __stcg(reinterpret_cast<float4 *>(to + 8 + d), make_float4(v[4], v[5], v[6], v[7]));
                                if (d == 0) __stcg(reinterpret_cast<float2 *>(to), make_float2(M[n][e], Ls[n][e]));
                            }
                        }
                    }
                }
        } else {
            float *const sM = reinterpret_cast<float *>(smem + L::mx) + par * W * R;
            float *const sL = reinterpret_cast<float *>(smem + L::sm) + par * W * R;
            if (g == 0 && col_group == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        sM[warp * R + RPT * n + (2 * t + e) % RPT] = M[n][e];
                        sL[warp * R + RPT * n + (2 * t + e) % RPT] = Ls[n][e];
                    }
            }
            __syncthreads();
            float *const buf = reinterpret_cast<float *>(smem + L::merge) + (warp >= W / 2 ? warp - W / 2 : warp) * L::MERGE_WARP;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float f[2];
                const int r = RPT * n + 2 * t % RPT;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = NONE;
                    for (int w = 0; w < W; ++w) m = fmaxf(m, sM[w * R + r + e]);
                    f[e] = ex2(M[n][e] - m);
                }
                const float e0 = f[0] * 16777216.f, e1 = f[1] * 16777216.f, d0 = f[0] * 1048576.f, d1 = f[1] * 1048576.f;
#pragma unroll
                for (int i = 0; i < SETS; ++i)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        O[n][i][k][0] *= e0;
                        O[n][i][k][1] *= e1;
                        O[n][i][k][2] *= d0;
                        O[n][i][k][3] *= d1;
                        if (warp >= W / 2 && r < s.rows)
                            *reinterpret_cast<float4 *>(buf + ((n * SETS + i) * 4 + t) * L::REGION + (8 * g + 2 * k) * 2) =
                                make_float4(O[n][i][k][0], O[n][i][k][1], O[n][i][k][2], O[n][i][k][3]);
                    }
            }
            __syncthreads();
            if (warp < W / 2) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (RPT * n + 2 * t % RPT < s.rows)
#pragma unroll
                        for (int i = 0; i < SETS; ++i)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float4 *const at =
                                    reinterpret_cast<float4 *>(buf + ((n * SETS + i) * 4 + t) * L::REGION + (8 * g + 2 * k) * 2);
                                const float4 o = *at;
                                *at = make_float4(O[n][i][k][0] + o.x, O[n][i][k][1] + o.y, O[n][i][k][2] + o.z, O[n][i][k][3] + o.w);
                            }
            }
            if (!last) {
                Cursor<R> after = cur;
                after.next(a, G);
                if (tw >= TEAM - NT) build_q<L, D, SPLIT>(a, after.s, G, TEAM - 1 - tw, NT, team, par ^ 1, lane);
            }
            __syncthreads();
            // each thread two rows of a dimension
            const float *const all = reinterpret_cast<const float *>(smem + L::merge);
            for (int i = tid; i < (s.rows + 1) / 2 * D; i += W * 32) {
                const int pr = i / D, d = i % D;
                constexpr int PPT = RPT / 2;  // row pairs of 8 columns
                const int n = pr / PPT, set = SPLIT ? 0 : d >> 6, tt = SPLIT ? (d >> 6) * PPT + pr % PPT : pr % PPT;
                float o[2] = {0.f, 0.f};
#pragma unroll
                for (int w = 0; w < W / 2; ++w) {
                    const float2 v = *reinterpret_cast<const float2 *>(all + w * L::MERGE_WARP +
                                                                       ((n * SETS + set) * 4 + tt) * L::REGION + (d & 63) * 2);
                    o[0] += v.x;
                    o[1] += v.y;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * pr + e;
                    if (r >= s.rows) break;
                    float m = NONE, l = 0.f;
                    for (int w = 0; w < W; ++w) m = fmaxf(m, sM[w * R + r]);
                    for (int w = 0; w < W; ++w) l += sL[w * R + r] * ex2(sM[w * R + r] - m);
                    if (!split) row_of(r)[d] = f32_to_bf16_bits(l == 0.f ? 0.f : o[e] / l);
                    else {
                        __stcg(part + r * (D + 4) + 4 + d, o[e]);
                        if (d == 0) __stcg(reinterpret_cast<float2 *>(part + r * (D + 4)), make_float2(m, l));
                    }
                }
            }
        }
        if (split) {
            // the last team to arrive joins the parts, in the order of the teams
            __threadfence();
            team_sync();
            bool done = false;
            if (TEAM == 1 ? lane == 0 : tid == 0) {
                done = atomicAdd(count, 1u) == static_cast<unsigned int>(c_last - c_first);
                if (done) *count = 0;  // for the next call
                if (TEAM > 1) misc[0] = done;
                __threadfence();
            }
            if (TEAM == 1) done = __shfl_sync(0xffffffffu, done, 0);
            else {
                __syncthreads();
                done = misc[0];
            }
            if (done) {
                if (TEAM == 1) __threadfence();  // (otherwise the first thread's, and the barrier)
                const int step = TEAM == 1 ? 32 : W * 32;
                for (int i = TEAM == 1 ? lane : tid; i < s.rows * (D / 4); i += step) {
                    const int r = i / (D / 4), d = i % (D / 4) * 4;
                    const float *const base = parts + r * (D + 4);
                    auto slot = [&](int c) { return (static_cast<size_t>(c) * 2 + (c == c_first)) * PART; };
                    // JOIN parts at a time, all on their way together: their
                    // latency is most of the join's time
                    constexpr int JOIN = 8;
                    float m = NONE, l = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c0 = c_first; c0 <= c_last; c0 += JOIN) {
                        float2 ml[JOIN];
                        float4 v[JOIN];
#pragma unroll
                        for (int j = 0; j < JOIN; ++j) {
                            const float *const from = base + slot(min(c0 + j, c_last));
                            ml[j] = __ldcg(reinterpret_cast<const float2 *>(from));
                            v[j] = __ldcg(reinterpret_cast<const float4 *>(from + 4 + d));
                        }
                        float up = m;
#pragma unroll
                        for (int j = 0; j < JOIN; ++j) up = fmaxf(up, ml[j].x);
                        const float old = ex2(m - up);
                        m = up;
                        l *= old;
                        o.x *= old, o.y *= old, o.z *= old, o.w *= old;
#pragma unroll
                        for (int j = 0; j < JOIN; ++j) {
                            const float f = c0 + j <= c_last ? ex2(ml[j].x - m) : 0.f;
                            l = fmaf(f, ml[j].y, l);
                            o.x = fmaf(f, v[j].x, o.x);
                            o.y = fmaf(f, v[j].y, o.y);
                            o.z = fmaf(f, v[j].z, o.z);
                            o.w = fmaf(f, v[j].w, o.w);
                        }
                    }
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    *reinterpret_cast<uint2 *>(row_of(r) + d) =
                        make_uint2(static_cast<uint32_t>(f32_to_bf16_bits(o.x * inv)) |
                                       static_cast<uint32_t>(f32_to_bf16_bits(o.y * inv)) << 16,
                                   static_cast<uint32_t>(f32_to_bf16_bits(o.z * inv)) |
                                       static_cast<uint32_t>(f32_to_bf16_bits(o.w * inv)) << 16);
                }
            }
        }
        if (last) break;
        cur.next(a, G);
        if (TEAM == 1) {
            __syncwarp();
            for (int n = 0; n < NT; ++n) build_q<L, D, SPLIT>(a, cur.s, G, n, NT, team, 0, lane);
            __syncwarp();
        } else par ^= 1;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kDevBadIndex);
}

template <int D, int NT, int W, int TEAM, bool SPLIT>
cudaError_t launch_stream(const Kv4AttnArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    using L = Stream<D, NT, W, TEAM, SPLIT>;
    static_assert(L::TEAMS * L::R <= warp_rows(D) && W <= MAX_WARPS, "scratch size");
    const int table = (a.requests + 1) * 8;
    int depth = (dev.max_smem_optin - L::ring - table) / (W * kv4_tile_bytes(D));
    if (depth > 8) depth = 8;
    if (depth < 1) return cudaErrorNotSupported;
    const int smem = L::ring + W * depth * kv4_tile_bytes(D) + table;
    static SmemLimit limit;
    const void *kern = reinterpret_cast<const void *>(attn_stream_kernel<D, NT, W, TEAM, SPLIT>);
    if (cudaError_t e = limit.ensure(kern, dev.device, smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms < MAX_CTAS ? dev.num_sms : MAX_CTAS));
    cfg.blockDim = dim3(W * 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_stream_kernel<D, NT, W, TEAM, SPLIT>, a, depth);
}

// One warp to a team when there are segments enough for that (rows is the
// most a request has).  Warps alone against a CTA's warps together, one new
// token after 4000, 16 heads of 256 on 8 (32 of 128 on 8):
//     requests   1         16       32       48        64       128
//     alone     144 (149)  55 (50)  78 (64)  101 (79)  124 (95) 219 (159) us
//     together   13 (13)   44 (35)  72 (56)  100 (75)  127 (95) 235 (171) us
template <int D, int NT, int W, bool SPLIT>
cudaError_t launch_teams(const Kv4AttnArgs &a, int64_t rows, cudaStream_t st, const DeviceInfo &dev) {
    constexpr int R = Stream<D, NT, W, 1, SPLIT>::R;
    const int64_t segments = a.requests * a.Hkv * ((rows + R - 1) / R);
    if (segments * TEAM_RATIO >= static_cast<int64_t>(dev.num_sms) * W) return launch_stream<D, NT, W, 1, SPLIT>(a, st, dev);
    return launch_stream<D, NT, W, W, SPLIT>(a, st, dev);
}

// Groups as columns (SPLIT) where the rows leave room for them, two blocks of
// columns where one is too few.  64 requests, one token after 4000, 8 key
// heads; us with SPLIT, one block, two blocks (- : not possible):
//     D = 256   1 row  119 140 197   2 rows 124 143 201   4 - 151 208   8 - 167 222
//     D = 128   1 row   86  89 116   2 rows  89  92 117   4 95 98 122   8 - 111 131
//     D = 64                                              4 - 70  83    8 -  77  90
cudaError_t stream(const Kv4AttnArgs &a, int D, int64_t rows, cudaStream_t st, const DeviceInfo &dev) {
    if (D == 64) return rows <= 8 ? launch_teams<64, 1, 16, false>(a, rows, st, dev) : launch_teams<64, 2, 16, false>(a, rows, st, dev);
    if (D == 128)
        return rows <= 4   ? launch_teams<128, 1, 16, true>(a, rows, st, dev)
               : rows <= 8 ? launch_teams<128, 1, 16, false>(a, rows, st, dev)
                           : launch_teams<128, 2, 12, false>(a, rows, st, dev);
    return rows <= 2   ? launch_teams<256, 1, 16, true>(a, rows, st, dev)
           : rows <= 8 ? launch_teams<256, 1, 12, false>(a, rows, st, dev)
                       : launch_teams<256, 2, 8, false>(a, rows, st, dev);
}

// Requests of up to this many rows are streamed.  A streamed block of 16 rows
// costs its share of the GPU, an item of the prompt kernel (up to 256 rows, 128
// at D = 64) a whole worker, and a round of items as long as one of them; in
// units of a round, per key, a streamed block of one segment costs 1 / (ratio x
// workers) with the measured ratio below.  So few segments stream more rows:
//     8 segments, 8000 keys, rows     16   32   64  128     (us: streamed / prompt)
//       D = 256                       33   41   51   70  / 113 for all
//     128 segments, 4000 keys         16   24   32   64
//       D = 256                       74  184  185  249  / 135
//       D = 128                       49    -   97  147  / 108
//     512 segments, 1000 keys         16   24   32   48   64
//       D = 256                      118  163  163  214  260  / 143
//       D = 128                       75    -   96  122  147  / 114
//       D = 64                        57   65   66   83   99  / 58
int64_t stream_rows(int64_t segments, int D, const DeviceInfo &dev) {
    const int64_t workers = D == 64 ? dev.num_sms : dev.num_sms / 2, rounds = (segments + workers - 1) / workers;
    const int64_t blocks = (D == 128 ? 8 : 5) * workers * rounds / (4 * segments);
    return 16 * (blocks > 1 ? blocks : 1);
}

}  // namespace

int64_t kv4_attention_scratch(int, int, int D) {
    return (COUNTER_BYTES + int64_t(MAX_CTAS) * 2 * warp_rows(D) * (D + 4) * 4 + 255) / 256 * 256;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs &args, int D, cudaStream_t st, const DeviceInfo &dev) {
    Kv4AttnArgs a = args;
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
        if (cudaError_t e = launch_kv4_prompt(a, D, st, dev)) return e;
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

}  // namespace w4
