// Attention over the paged 4-bit cache, streaming form (kv4_attention in the
// C header): decode steps and short pieces.
//
//   o = sum_j softmax_j(scale q . k_j) v_j  over the keys j that query p sees:
//   j <= p, and with a window w also p - j < w or j < sinks.
//
// Bound: memory.  A token's K and V of one head are 18 D / 16 bytes and every
// byte is read once; a row block of up to 8 NT rows (the G query heads of a
// key head times the request's new tokens) shares the read.
//
// Work.  The unit is a cache tile (16 tokens of one head, one contiguous run
// fetched by one bulk copy).  The visible tiles of all (request, row block,
// head) segments are numbered in a row and split evenly over one CTA per SM,
// so lengths of any raggedness, windows and one long request alike fill the
// GPU.  Every CTA finds its share itself from the lengths (a prefix sum in
// shared memory).  A segment that lies in one CTA is finished there; of one
// that several CTAs share, each writes its partial result (maximum, sum,
// weighted values) to scratch and the last to arrive joins them in the order
// of the CTAs, so results do not depend on timing.  No CTA waits for another.
//
// A CTA's warps take its tiles in turn, each with its own ring of stages and
// barriers: no producer warp and no barrier between warps inside a segment.
//
// Arithmetic per tile, all products on mma.m16n8k16 (binary16 in, binary32
// out) with the CODES as the A operand: the low and high nibble pairs of a
// word masked in place are binary16 subnormals c 2^-24 and 16 c 2^-24, exact,
// so 8 codes cost 5 logic operations and no conversion.
//   S^T = K Q^T (16 keys x 8 rows), a sum per group of 64 dimensions:
//     x += s (acc - z sum(q))                        binary32, exact products
//     (q enters as binary16 after a power-of-two scale of its row)
//   O^T += (V - z)^T P^T (16 dimensions x 8 rows), per group with P' = p s
//     rounded to binary16.  Here code and zero are subtracted first (exact, a
//     pair operation per two codes): summed apart, p c - p z would leave
//     2^-24 of p z where a value is zero.
// The reference of the exponentials is a running maximum of x + log2(s), so
// that the largest P' is near 1 whatever the magnitude of V; it moves (and
// the accumulators are scaled) only when it would grow by more than 2^8.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {
namespace {

constexpr int MAX_CTAS = 160;         // scratch is sized for this many
constexpr int MAX_ROWS = 16;          // rows of a segment
constexpr int COUNTER_BYTES = 1024;   // arrival counters at the head of the scratch
constexpr int PROMPT_ROWS = 48;       // requests with more rows go to the tensor cores
constexpr float NEG_INF = -INFINITY;

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
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Keys of the MMA's rows 0..7 within a half tile.  Any order is right (both
// products sum over keys); this one makes the 8-byte reads of K (lanes of
// four consecutive rows) and the 4-byte reads of V (keys of rows 2 t, and of
// rows 2 t + 1) fall into different banks.
__device__ __forceinline__ int key_of_row(int r) { return (0x57463120u >> (4 * r)) & 15; }

// Rows before request b; whatever the array holds, inside the tensors.
__device__ __forceinline__ int rows_before(const Kv4AttnArgs &a, int b) {
    return static_cast<int>(min(max(static_cast<int64_t>(a.cu_new[b]), int64_t(0)), a.T));
}

// Rows of request b that this kernel answers: new tokens x query heads of a
// key head, or none when the prompt kernel takes them.
__device__ __forceinline__ int rows_of(const Kv4AttnArgs &a, int b, int G) {
    const int rows = (rows_before(a, b + 1) - rows_before(a, b)) * G;
    return rows > 0 && rows <= a.rows_most ? rows : 0;
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

template <int D, int NT, int W>
struct StreamSmem {
    static constexpr int R = 8 * NT;
    static constexpr int G64 = D / 64;
    static constexpr int MERGE_T = 2 * D + 4;                 // floats of a row pair
    static constexpr int MERGE_WARP = NT * 4 * MERGE_T;       // floats of a warp
    static constexpr int QFRAG = NT * G64 * 2 * 32 * 16;      // bytes: [NT][group][mma pair][lane] 4 words
    // offsets in bytes
    static constexpr int q = 0;                               // [2][QFRAG]
    static constexpr int qs = q + 2 * QFRAG;                  // [2][G64][R] scaled row sums
    static constexpr int fr = qs + 2 * G64 * R * 4;           // [2][R] factor of the scores
    static constexpr int mx = fr + 2 * R * 4;                 // [2][W][R]
    static constexpr int sm = mx + 2 * W * R * 4;             // [2][W][R]
    static constexpr int misc = sm + 2 * W * R * 4;           // 64 bytes
    static constexpr int bars = misc + 64;                    // [W][8] barriers
    static constexpr int merge = (bars + W * 8 * 8 + 127) / 128 * 128;  // [W / 2][MERGE_WARP] floats
    static constexpr int ring = (merge + W / 2 * MERGE_WARP * 4 + 127) / 128 * 128;
};

// Q of a segment as the MMA's B operand, by one warp per 8 rows: lane (g, t)
// takes row g, 16 dimensions from 64 gi + 16 t on of each group.
template <int D, int NT, int W>
__device__ __forceinline__ void build_q(const Kv4AttnArgs &a, const Segment &s, int G, int nt, unsigned char *smem,
                                        int par, int lane) {
    using L = StreamSmem<D, NT, W>;
    const int g = lane >> 2, t = lane & 3;
    const int r = 8 * nt + g;
    const bool on = r < s.rows;
    const int row = s.r0 + (on ? r : 0);
    const int tok = rows_before(a, s.b) + row / G;
    const uint16_t *src = a.q + static_cast<int64_t>(tok) * a.q_stride + static_cast<int64_t>(s.h * G + row % G) * D + 16 * t;
    uint4 raw[L::G64][2];
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < L::G64; ++i) {
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
    // the row's largest magnitude to [2^13, 2^14): the sums of the odd
    // dimensions' 1/16 stay exact down to 2^-33 of it
    int kappa = big > 0.f ? 13 - (static_cast<int>(__float_as_uint(big) >> 23) - 127) : 0;
    kappa = min(max(kappa, -110), 110);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + kappa) << 23);
#pragma unroll
    for (int i = 0; i < L::G64; ++i) {
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
            reinterpret_cast<float *>(smem + L::qs)[(par * L::G64 + i) * L::R + r] = sum * 5.9604644775390625e-8f;  // 2^-24
        uint4 *dst = reinterpret_cast<uint4 *>(smem + L::q + par * L::QFRAG) + (nt * L::G64 + i) * 2 * 32 + lane;
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // word k of the lane's two: dimensions 8 k .. 8 k + 7
            const float *x = v + 8 * k;
            dst[k * 32] = make_uint4(pack_f16(x[0], x[4]), pack_f16(x[1] * 0.0625f, x[5] * 0.0625f),
                                     pack_f16(x[2], x[6]), pack_f16(x[3] * 0.0625f, x[7] * 0.0625f));
        }
    }
    if (t == 0)
        reinterpret_cast<float *>(smem + L::fr)[par * L::R + r] =
            on ? a.scale * 1.4426950408889634f * (16777216.f * __uint_as_float(static_cast<uint32_t>(127 - kappa) << 23))
               : 0.f;
}

template <int D, int NT, int W>
__global__ void __launch_bounds__(W * 32, 1) attn_stream_kernel(const Kv4AttnArgs a, const int depth) {
    using L = StreamSmem<D, NT, W>;
    constexpr int R = L::R, G64 = L::G64, TB = kv4_tile_bytes(D);
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int G = a.Hq / a.Hkv;
    uint64_t *const bars = reinterpret_cast<uint64_t *>(smem + L::bars) + warp * 8;
    unsigned char *const ring = smem + L::ring + static_cast<size_t>(warp) * depth * TB;
    long long *const cum = reinterpret_cast<long long *>(smem + L::ring + static_cast<size_t>(W) * depth * TB);
    volatile int *const misc = reinterpret_cast<volatile int *>(smem + L::misc);

    if (lane == 0)
        for (int i = 0; i < depth; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
    pdl_launch_dependents();
    pdl_wait();

    // ---- this CTA's share: tiles of the requests, their running sum
    {
        const int per = (a.requests + W * 32 - 1) / (W * 32);
        const int b0 = min(tid * per, a.requests), b1 = min(b0 + per, a.requests);
        long long sum = 0;
        for (int b = b0; b < b1; ++b) {
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
    if (a.zero_rest) {  // rows that belong to no request
        const int64_t from = static_cast<int64_t>(rows_before(a, a.requests)) * a.Hq * D / 8;
        const int64_t to = a.T * a.Hq * D / 8;
        for (int64_t i = from + static_cast<int64_t>(blockIdx.x) * W * 32 + tid; i < to;
             i += static_cast<int64_t>(gridDim.x) * W * 32)
            reinterpret_cast<uint4 *>(a.out)[i] = make_uint4(0, 0, 0, 0);
    }
    // CTAs that take part: no more than there are tiles, so that none between
    // the first and the last of a shared segment is without a part of it
    const long long U = cum[a.requests], C = U < gridDim.x ? U : gridDim.x;
    if (blockIdx.x >= C) return;
    const long long u0 = U * blockIdx.x / C;
    const int mine = static_cast<int>(U * (blockIdx.x + 1) / C - u0);

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
    int pre_u = warp;        // its number in the CTA's share
    bool bad = false;
    // the page of a tile, or -1 where there is nothing to fetch; asked for one
    // step before the copy is issued, so that its latency is not waited for
    auto page_of = [&]() -> int {
        if (pre_u >= mine) return -1;
        while (pre_u >= pre.first + pre.s.nt) pre.next(a, G);
        const int tile = pre.tile(pre_u);
        if (tile * 16 >= pre.s.end) return -1;
        const int id = a.block_table[static_cast<int64_t>(pre.s.b) * a.max_blocks + (tile >> (a.bs_log2 - 4))];
        return id;
    };
    uint32_t live = 0;       // bit of a stage: it holds a tile
    int page = page_of();
    auto fetch = [&](int stage) {
        const bool in = page >= 0 && page < a.num_blocks;
        if (pre_u < mine) {
            const int tile = pre.tile(pre_u);
            if (!in && tile * 16 < pre.s.end) bad = true;
            if (in) {
                if (lane == 0) {
                    const int sub = tile & ((1 << (a.bs_log2 - 4)) - 1);
                    const size_t at =
                        (((static_cast<size_t>(page) * a.Hkv + pre.s.h) << (a.bs_log2 - 4)) + sub) * static_cast<size_t>(TB);
                    mbar_arrive_expect_tx(&bars[stage], TB);
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                            smem_u32(ring + static_cast<size_t>(stage) * TB)),
                        "l"(a.cache + at), "r"(TB), "r"(smem_u32(&bars[stage]))
                        : "memory");
                }
            }
        }
        live = in && pre_u < mine ? live | (1u << stage) : live & ~(1u << stage);
        pre_u += W;
        page = page_of();
    };
    for (int i = 0; i < depth; ++i) fetch(i);

    uint32_t parity = 0;  // bit per stage
    int stage = 0;
    int u = warp;
    int par = 0;          // of the per-segment buffers
    bool ok = true;
    const int kA = key_of_row(g), vA = key_of_row(2 * t), vB = key_of_row(2 * t + 1);

    if (warp >= W - NT) build_q<D, NT, W>(a, cur.s, G, W - 1 - warp, smem, 0, lane);
    __syncthreads();

    while (true) {
        const Segment s = cur.s;
        const int seg_end = min(cur.first + s.nt, mine);
        float O[NT][G64][4][4], M[NT][2], Ls[NT][2], QS[NT][G64][2], F[NT][2];
        int P[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < G64; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[n][i][k][e] = 0.f;
                const float2 v = *reinterpret_cast<const float2 *>(smem + L::qs + ((par * G64 + i) * R + 8 * n + 2 * t) * 4);
                QS[n][i][0] = v.x;
                QS[n][i][1] = v.y;
            }
            const float2 f = *reinterpret_cast<const float2 *>(smem + L::fr + (par * R + 8 * n + 2 * t) * 4);
            F[n][0] = f.x;
            F[n][1] = f.y;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                M[n][e] = NEG_INF;
                Ls[n][e] = 0.f;
                P[n][e] = s.base + (s.r0 + min(8 * n + 2 * t + e, s.rows - 1)) / G;
            }
        }
        const int p_lo = s.base + s.r0 / G, p_hi = s.base + (s.r0 + s.rows - 1) / G;

        for (; u < seg_end; u += W) {
            if (live >> stage & 1u) {
                ok = mbar_wait(&bars[stage], parity >> stage & 1u, a.status) && ok;
                parity ^= 1u << stage;
                const unsigned char *tile = ring + static_cast<size_t>(stage) * TB;
                const int j0 = cur.tile(u) * 16;
                const uint4 *qf = reinterpret_cast<const uint4 *>(smem + L::q + par * L::QFRAG) + lane;
                float x[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
                // ---- scores
#pragma unroll
                for (int i = 0; i < G64; ++i) {
                    const uint2 k0 = *reinterpret_cast<const uint2 *>(tile + (i * 16 + kA) * 32 + t * 8);
                    const uint2 k1 = *reinterpret_cast<const uint2 *>(tile + (i * 16 + kA + 8) * 32 + t * 8);
                    const uint32_t sz0 = *reinterpret_cast<const uint32_t *>(tile + 16 * D + (i * 16 + kA) * 4);
                    const uint32_t sz1 = *reinterpret_cast<const uint32_t *>(tile + 16 * D + (i * 16 + kA + 8) * 4);
                    float acc[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t w0 = k ? k0.y : k0.x, w1 = k ? k1.y : k1.x;
                        const uint32_t w0h = w0 >> 8, w1h = w1 >> 8;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint4 b = qf[((n * G64 + i) * 2 + k) * 32];
                            mma_f16(acc[n], w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, b.x, b.y);
                            mma_f16(acc[n], w0h & 0x000f000fu, w1h & 0x000f000fu, w0h & 0x00f000f0u, w1h & 0x00f000f0u, b.z,
                                    b.w);
                        }
                    }
                    const float s0 = f16_lo(sz0), z0 = f16_hi(sz0), s1 = f16_lo(sz1), z1 = f16_hi(sz1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        x[n][0] = fmaf(s0, fmaf(-z0, QS[n][i][0], acc[n][0]), x[n][0]);
                        x[n][1] = fmaf(s0, fmaf(-z0, QS[n][i][1], acc[n][1]), x[n][1]);
                        x[n][2] = fmaf(s1, fmaf(-z1, QS[n][i][0], acc[n][2]), x[n][2]);
                        x[n][3] = fmaf(s1, fmaf(-z1, QS[n][i][1], acc[n][3]), x[n][3]);
                    }
                }
                // ---- V's parameters; what lies past the last key of the
                // cache may hold anything and counts as zeros
                const int ja = j0 + kA, jb = ja + 8;
                const bool whole = j0 + 16 <= s.end;
                uint32_t vz0[G64], vz1[G64];  // (scale, zero) of keys kA, kA + 8
                float top0 = 0.f, top1 = 0.f;
#pragma unroll
                for (int i = 0; i < G64; ++i) {
                    vz0[i] = *reinterpret_cast<const uint32_t *>(tile + 17 * D + (i * 16 + kA) * 4);
                    vz1[i] = *reinterpret_cast<const uint32_t *>(tile + 17 * D + (i * 16 + kA + 8) * 4);
                    if (!whole) {
                        vz0[i] = ja < s.end ? vz0[i] : 0u;
                        vz1[i] = jb < s.end ? vz1[i] : 0u;
                    }
                    top0 = fmaxf(top0, fabsf(f16_lo(vz0[i])));
                    top1 = fmaxf(top1, fabsf(f16_lo(vz1[i])));
                }
                const float l0 = lg2(fmaxf(top0, 5.9604644775390625e-8f)), l1 = lg2(fmaxf(top1, 5.9604644775390625e-8f));
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
                            x[n][e] = see ? x[n][e] : NEG_INF;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        grow |= fmaxf(x[n][e] + l0, x[n][e + 2] + l1) > M[n][e] + 8.f;
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
                            m = fmaxf(m, M[n][e]);
                            const float f = m == NEG_INF ? 1.f : ex2(M[n][e] - m);
                            M[n][e] = m;
                            Ls[n][e] *= f;
#pragma unroll
                            for (int i = 0; i < G64; ++i)
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    O[n][i][k][e] *= f;
                                    O[n][i][k][e + 2] *= f;
                                }
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float m = M[n][e & 1];
                        x[n][e] = ex2(x[n][e] - (m == NEG_INF ? 0.f : m));
                        Ls[n][e & 1] += x[n][e];
                    }
                }
                // ---- weighted values
#pragma unroll
                for (int i = 0; i < G64; ++i) {
                    const unsigned char *vt = tile + 8 * D + i * 512 + g * 4;
                    const uint32_t wA = *reinterpret_cast<const uint32_t *>(vt + vA * 32);
                    const uint32_t wB = *reinterpret_cast<const uint32_t *>(vt + vB * 32);
                    const uint32_t wC = *reinterpret_cast<const uint32_t *>(vt + (vA + 8) * 32);
                    const uint32_t wD = *reinterpret_cast<const uint32_t *>(vt + (vB + 8) * 32);
                    uint32_t b[NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float v0 = f16_lo(vz0[i]), v1 = f16_lo(vz1[i]);
                        b[n][0] = transpose8x8(pack_f16(x[n][0] * v0, x[n][1] * v0));
                        b[n][1] = transpose8x8(pack_f16(x[n][2] * v1, x[n][3] * v1));
                    }
                    // zeros of this lane's four keys in the codes' units, 2^-24 and 2^-20
                    const uint32_t zab = transpose8x8(__byte_perm(vz0[i], 0, 0x3232)), zcd = transpose8x8(__byte_perm(vz1[i], 0, 0x3232));
                    const uint32_t zab1 = mul_f16x2(zab, 0x00010001u), zab16 = mul_f16x2(zab, 0x00100010u);
                    const uint32_t zcd1 = mul_f16x2(zcd, 0x00010001u), zcd16 = mul_f16x2(zcd, 0x00100010u);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // dimensions 8 g + 2 k and 8 g + 2 k + 1 of keys A, B and C, D
                        const uint32_t sel = k < 2 ? 0x5410u : 0x7632u;
                        uint32_t ab = __byte_perm(wA, wB, sel), cd = __byte_perm(wC, wD, sel);
                        if (k & 1) ab >>= 8, cd >>= 8;
                        const uint32_t a0 = sub_f16x2(ab & 0x000f000fu, zab1), a1 = sub_f16x2(ab & 0x00f000f0u, zab16);
                        const uint32_t a2 = sub_f16x2(cd & 0x000f000fu, zcd1), a3 = sub_f16x2(cd & 0x00f000f0u, zcd16);
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma_f16(O[n][i][k], a0, a1, a2, a3, b[n][0], b[n][1]);
                    }
                }
                __syncwarp();
            }
            fetch(stage);
            stage = stage + 1 == depth ? 0 : stage + 1;
        }

        // ---- the segment's end: join the warps
        float *const sM = reinterpret_cast<float *>(smem + L::mx) + par * W * R;
        float *const sL = reinterpret_cast<float *>(smem + L::sm) + par * W * R;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = Ls[n][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                if (g == 0) {
                    sM[warp * R + 8 * n + 2 * t + e] = M[n][e];
                    sL[warp * R + 8 * n + 2 * t + e] = l;
                }
            }
        __syncthreads();
        float *const buf = reinterpret_cast<float *>(smem + L::merge) + (warp >= W / 2 ? warp - W / 2 : warp) * L::MERGE_WARP;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float m = NEG_INF;
                for (int w = 0; w < W; ++w) m = fmaxf(m, sM[w * R + 8 * n + 2 * t + e]);
                f[e] = M[n][e] == NEG_INF ? 0.f : ex2(M[n][e] - m);
            }
            // the codes' units: 2^-24 for even dimensions, 2^-20 for odd ones
            const float e0 = f[0] * 16777216.f, e1 = f[1] * 16777216.f, d0 = f[0] * 1048576.f, d1 = f[1] * 1048576.f;
#pragma unroll
            for (int i = 0; i < G64; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    O[n][i][k][0] *= e0;
                    O[n][i][k][1] *= e1;
                    O[n][i][k][2] *= d0;
                    O[n][i][k][3] *= d1;
                    if (warp >= W / 2 && 8 * n + 2 * t < s.rows)
                        *reinterpret_cast<float4 *>(buf + (n * 4 + t) * L::MERGE_T + (64 * i + 8 * g + 2 * k) * 2) =
                            make_float4(O[n][i][k][0], O[n][i][k][1], O[n][i][k][2], O[n][i][k][3]);
                }
        }
        __syncthreads();
        const bool last = cur.first + s.nt >= mine;  // no further segment in this CTA
        const int seg_first = cur.first, seg_nt = s.nt;
        if (warp < W / 2) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (8 * n + 2 * t < s.rows)
#pragma unroll
                    for (int i = 0; i < G64; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float4 *const at =
                                reinterpret_cast<float4 *>(buf + (n * 4 + t) * L::MERGE_T + (64 * i + 8 * g + 2 * k) * 2);
                            const float4 o = *at;
                            *at = make_float4(O[n][i][k][0] + o.x, O[n][i][k][1] + o.y, O[n][i][k][2] + o.z, O[n][i][k][3] + o.w);
                        }
        }
        if (!last) {
            cur.next(a, G);
            if (warp >= W - NT) build_q<D, NT, W>(a, cur.s, G, W - 1 - warp, smem, par ^ 1, lane);
        }
        __syncthreads();
        // ---- each thread two rows of a dimension
        const bool split = seg_first < 0 || seg_first + seg_nt > mine;
        const float *const all = reinterpret_cast<const float *>(smem + L::merge);
        const long long seg_u0 = u0 + seg_first;
        int c_first = 0, c_last = 0;
        if (split) {
            c_first = static_cast<int>(((seg_u0 + 1) * C - 1) / U);
            c_last = static_cast<int>(((seg_u0 + seg_nt) * C - 1) / U);
        }
        // partial results: [CTA][2][MAX_ROWS][D + 2], slot 1 where the segment begins in the CTA
        float *const parts = reinterpret_cast<float *>(a.scratch + COUNTER_BYTES);
        constexpr int PART = MAX_ROWS * (D + 2);
        float *const part = parts + (static_cast<size_t>(blockIdx.x) * 2 + (seg_first >= 0 ? 1 : 0)) * PART;
        for (int i = tid; i < (s.rows + 1) / 2 * D; i += W * 32) {
            const int pr = i / D, d = i % D;
            float o0 = 0.f, o1 = 0.f;
#pragma unroll
            for (int w = 0; w < W / 2; ++w) {
                const float2 v = *reinterpret_cast<const float2 *>(all + w * L::MERGE_WARP + pr * L::MERGE_T + d * 2);
                o0 += v.x;
                o1 += v.y;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 2 * pr + e;
                if (r >= s.rows) break;
                float m = NEG_INF, l = 0.f;
                for (int w = 0; w < W; ++w) m = fmaxf(m, sM[w * R + r]);
                for (int w = 0; w < W; ++w) {
                    const float mw = sM[w * R + r];
                    l += mw == NEG_INF ? 0.f : sL[w * R + r] * ex2(mw - m);
                }
                const float o = e ? o1 : o0;
                if (!split) {
                    const int row = s.r0 + r, tok = rows_before(a, s.b) + row / G;
                    a.out[(static_cast<int64_t>(tok) * a.Hq + s.h * G + row % G) * D + d] =
                        f32_to_bf16_bits(l == 0.f ? 0.f : o / l);
                } else {
                    __stcg(part + r * (D + 2) + 2 + d, o);
                    if (d == 0) {
                        __stcg(part + r * (D + 2), m);
                        __stcg(part + r * (D + 2) + 1, l);
                    }
                }
            }
        }
        if (split) {
            unsigned int *const count = reinterpret_cast<unsigned int *>(a.scratch) + c_first;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const bool done = atomicAdd(count, 1u) == static_cast<unsigned int>(c_last - c_first);
                if (done) *count = 0;  // for the next call
                misc[0] = done;
                __threadfence();
            }
            __syncthreads();
            if (misc[0]) {
                for (int i = tid; i < s.rows * D; i += W * 32) {
                    const int r = i / D, d = i % D;
                    float m = NEG_INF;
                    for (int c = c_first; c <= c_last; ++c)
                        m = fmaxf(m, __ldcg(parts + (static_cast<size_t>(c) * 2 + (c == c_first)) * PART + r * (D + 2)));
                    float l = 0.f, o = 0.f;
                    for (int c = c_first; c <= c_last; ++c) {
                        const float *const q = parts + (static_cast<size_t>(c) * 2 + (c == c_first)) * PART + r * (D + 2);
                        const float mc = __ldcg(q);
                        const float f = mc == NEG_INF ? 0.f : ex2(mc - m);
                        l += f * __ldcg(q + 1);
                        o += f * __ldcg(q + 2 + d);
                    }
                    const int row = s.r0 + r, tok = rows_before(a, s.b) + row / G;
                    a.out[(static_cast<int64_t>(tok) * a.Hq + s.h * G + row % G) * D + d] =
                        f32_to_bf16_bits(l == 0.f ? 0.f : o / l);
                }
            }
        }
        if (last) break;
        par ^= 1;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kDevBadIndex);
    // every copy of this warp has been waited for, unless a wait gave up: then
    // wait (bounded) for what may still be under way before the CTA ends
    if (!__all_sync(0xffffffffu, ok))
        for (int i = 0; i < depth; ++i)
            if (live >> i & 1u) mbar_wait(&bars[i], parity >> i & 1u, nullptr);
}

template <int D, int NT, int W>
cudaError_t launch_stream(const Kv4AttnArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    using L = StreamSmem<D, NT, W>;
    const int table = (a.requests + 1) * 8;
    int depth = (dev.max_smem_optin - L::ring - table) / (W * kv4_tile_bytes(D));
    if (depth > 8) depth = 8;
    if (depth < 1) return cudaErrorNotSupported;
    const int smem = L::ring + W * depth * kv4_tile_bytes(D) + table;
    static SmemLimit limit;
    const void *kern = reinterpret_cast<const void *>(attn_stream_kernel<D, NT, W>);
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
    return cudaLaunchKernelEx(&cfg, attn_stream_kernel<D, NT, W>, a, depth);
}

}  // namespace

int64_t kv4_attention_scratch(int, int, int D) {
    return (COUNTER_BYTES + int64_t(MAX_CTAS) * 2 * MAX_ROWS * (D + 2) * 4 + 255) / 256 * 256;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs &args, int D, cudaStream_t st, const DeviceInfo &dev) {
    Kv4AttnArgs a = args;
    const int G = a.Hq / a.Hkv;
    a.rows_most = 0x7fffffff;
    a.zero_rest = 1;
    if (a.max_new * G > PROMPT_ROWS) {
        // requests of many rows to the tensor cores, the others of a mixed step
        // to the streaming kernel
        a.rows_above = a.requests > 1 ? PROMPT_ROWS : 0;
        if (cudaError_t e = launch_kv4_prompt(a, D, st, dev)) return e;
        if (a.requests == 1) return cudaSuccess;
        a.rows_most = PROMPT_ROWS;
        a.zero_rest = 0;
    }
    // rows that share a read of the cache: 8 or 16 to a segment
    const bool few = a.max_new * G <= 8;
    if (D == 64) return few ? launch_stream<64, 1, 16>(a, st, dev) : launch_stream<64, 2, 16>(a, st, dev);
    if (D == 128) return few ? launch_stream<128, 1, 16>(a, st, dev) : launch_stream<128, 2, 12>(a, st, dev);
    return few ? launch_stream<256, 1, 12>(a, st, dev) : launch_stream<256, 2, 8>(a, st, dev);
}

}  // namespace w4
