// Pages of the 4-bit cache by a cheap score: their bounds (kv4_bounds) and the
// choice of the highest for each new token and key head (kv4_select).
//
// The bounds of a page and key head are, for each of the D elements, the largest
// and the smallest key in it, in 8 bits as whole numbers of a step for 64
// elements.  No key of the page gives a query head more than
//   sum_d max(q_d high_d, q_d low_d),
// the page's score, with the query in 8 bits too: a sum of products of whole
// numbers, exact in any order, times the steps (binary32, in one order), so that
// the choice does not depend on how the work is split.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {
namespace {

constexpr float STEP = 65.f / 8192.f;  // of the largest magnitude: whole numbers to 127 at most

__host__ __device__ constexpr int bounds_bytes(int D) { return 2 * D + 16; }

// ---------------------------------------------------------------- bounds

constexpr int BOUNDS_WARPS = 4;  // (8: 31 us below, 2: 33)

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// v = x s + k of both halves of a pair x, s binary16.
__device__ __forceinline__ void fma_f16(uint32_t x, uint32_t s, float k, float &lo, float &hi) {
    asm("{\n\t.reg .b16 x0, x1, s0, s1;\n\tmov.b32 {x0, x1}, %2;\n\tmov.b32 {s0, s1}, %3;\n\t"
        "fma.rn.f32.f16 %0, x0, s0, %4;\n\tfma.rn.f32.f16 %1, x1, s0, %4;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(x), "r"(s), "f"(k));
}

// A warp takes `slots` slots and one key head.  A lane holds 8 elements: D / 8
// lanes a token, 256 / D tokens side by side.
//
// A code c masked in place under the exponent of 1024 is the binary16 number 1024 +
// c, or in the next four bits under that of 64 the number 64 + c, so that a key is
// one fused multiply-add, exact:
//   (1024 + c) s - (1024 + z) s   or   (64 + c) s - (64 + z) s,
// and two tokens enter the extremes with one comparison each way.
// Bound: instructions (five a code) and the loads' latency, about half of the time each.
// 65519 tokens of 8 heads of 256, pages of 64: 29.7 us, 2.7 TB/s; the ALU pipe 64% and the
// issue slots 67% busy, 38% of the warps that an SM holds active.  (16 elements a lane, so
// that half as many instructions go to the scales: 32 us, for its registers.)
template <int D>
__global__ void __launch_bounds__(BOUNDS_WARPS * 32) bounds_kernel(const Kv4BoundsArgs a, const int slots) {
    constexpr int LANES = D / 8, SIDE = 32 / LANES, HALF = 8 / SIDE, TB = kv4_tile_bytes(D);
    const int lane = threadIdx.x & 31, h = blockIdx.y * BOUNDS_WARPS + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    if (h >= a.Hkv) return;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * slots + lane;
    const int64_t slot = lane < slots && t < a.T ? a.slots[t] : -1;
    if (slot >= a.num_slots && h == 0) atomicOr(a.status, kDevBadIndex);
    const int64_t size = int64_t(1) << a.bs_log2;
    unsigned full = __ballot_sync(0xffffffffu, slot >= 0 && slot < a.num_slots && (slot & (size - 1)) == size - 1);
    const int i = lane % LANES, group = i / 8, side = lane / LANES;
    while (full) {
        const int64_t block = __shfl_sync(0xffffffffu, slot, __ffs(full) - 1) >> a.bs_log2;
        full &= full - 1;
        const unsigned char *tile = a.cache + ((block * a.Hkv + h) << (a.bs_log2 - 4)) * TB;
        float high[8], low[8];  // of elements 0 4 1 5 2 6 3 7
#pragma unroll
        for (int e = 0; e < 8; ++e) high[e] = -INFINITY, low[e] = INFINITY;
        // half a tile's rows at a time, the next ones on their way meanwhile
        const int steps = 2 << (a.bs_log2 - 4);
        uint32_t codes[HALF], para[HALF];
        auto load = [&](int n) {
#pragma unroll
            for (int j = 0; j < HALF; ++j) {
                const unsigned char *const from = tile + (n >> 1) * TB;
                const int row = group * 16 + ((n & 1) * HALF + j) * SIDE + side;
                codes[j] = *reinterpret_cast<const uint32_t *>(from + row * 32 + i % 8 * 4);
                para[j] = *reinterpret_cast<const uint32_t *>(from + 16 * D + row * 4);
            }
        };
        load(0);
#pragma unroll 1
        for (int n = 0; n < steps; ++n) {
            uint32_t w[HALF], p[HALF];
#pragma unroll
            for (int j = 0; j < HALF; ++j) w[j] = codes[j], p[j] = para[j];
            load(min(n + 1, steps - 1));
#pragma unroll
            for (int j = 0; j < HALF; j += 2) {
                float v[2][8];
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const uint32_t u = w[j + o] >> 8;
                    const float s = f16_lo(p[j + o]), z = f16_hi(p[j + o]);
                    const float k1024 = -(1024.f + z) * s, k64 = fmaf(960.f, s, k1024);
                    fma_f16((w[j + o] & 0x000f000fu) | 0x64006400u, p[j + o], k1024, v[o][0], v[o][1]);
                    fma_f16((w[j + o] & 0x00f000f0u) | 0x54005400u, p[j + o], k64, v[o][2], v[o][3]);
                    fma_f16((u & 0x000f000fu) | 0x64006400u, p[j + o], k1024, v[o][4], v[o][5]);
                    fma_f16((u & 0x00f000f0u) | 0x54005400u, p[j + o], k64, v[o][6], v[o][7]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    high[e] = max3(high[e], v[0][e], v[1][e]);
                    low[e] = min3(low[e], v[0][e], v[1][e]);
                }
            }
        }
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
            for (int o = LANES; o < 32; o <<= 1) {
                high[e] = fmaxf(high[e], __shfl_xor_sync(0xffffffffu, high[e], o));
                low[e] = fminf(low[e], __shfl_xor_sync(0xffffffffu, low[e], o));
            }
            most = fmaxf(most, fmaxf(fabsf(high[e]), fabsf(low[e])));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const float step = most * STEP, by = step > 0.f ? step : 1.f;
        uint32_t up[2] = {0, 0}, down[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = e / 2 + 4 * (e & 1);
            up[d / 4] |= (static_cast<uint32_t>(__float2int_ru(__fdiv_rn(high[e], by))) & 255u) << 8 * (d % 4);
            down[d / 4] |= (static_cast<uint32_t>(__float2int_rd(__fdiv_rn(low[e], by))) & 255u) << 8 * (d % 4);
        }
        unsigned char *const row = a.bounds + (block * a.Hkv + h) * bounds_bytes(D);
        if (side == 0) {
            *reinterpret_cast<uint2 *>(row + 8 * i) = make_uint2(up[0], up[1]);
            *reinterpret_cast<uint2 *>(row + D + 8 * i) = make_uint2(down[0], down[1]);
            if (i % 8 == 0) *reinterpret_cast<float *>(row + 2 * D + 4 * group) = step;
        }
    }
}

template <int D>
cudaError_t launch_bounds(const Kv4BoundsArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    // few slots: few to a warp, since each may fill a page
    const int slots = a.T <= 1024 ? 4 : 32;
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + slots - 1) / slots),
                       static_cast<unsigned>((a.Hkv + BOUNDS_WARPS - 1) / BOUNDS_WARPS));
    cfg.blockDim = dim3(BOUNDS_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bounds_kernel<D>, a, slots);
}

// ---------------------------------------------------------------- select

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int NO_PAGE = -0x7fffffff - 1;

// Scores in the order of whole numbers.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);  // (-0 as 0)
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A query head's elements, four of them in each of a warp's lanes (or two times four).
template <int D>
struct Query {
    static constexpr int WORDS = D / 4, PER = (WORDS + 31) / 32;
    uint2 raw[PER];
};
template <int D>
__device__ __forceinline__ Query<D> load_query(const uint16_t *q, int lane) {
    Query<D> r;
#pragma unroll
    for (int k = 0; k < Query<D>::PER; ++k) r.raw[k] = *reinterpret_cast<const uint2 *>(q + 4 * ((lane + 32 * k) % Query<D>::WORDS));
    return r;
}
// In whole numbers of 8 bits (NaN as 0, infinities as the largest finite number);
// their unit.  By a whole warp.
template <int D>
__device__ __forceinline__ float whole_numbers(const Query<D> &r, float (&x)[Query<D>::PER][4]) {
    float most = 0.f;
#pragma unroll
    for (int k = 0; k < Query<D>::PER; ++k) {
        const uint2 raw = r.raw[k];
        const uint32_t bits[4] = {raw.x << 16, raw.x & 0xffff0000u, raw.y << 16, raw.y & 0xffff0000u};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float v = __uint_as_float(bits[e]);
            x[k][e] = v != v ? 0.f : fminf(fmaxf(v, -3.3895314e38f), 3.3895314e38f);
            most = fmaxf(most, fabsf(x[k][e]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float unit = most * STEP, by = unit > 0.f ? unit : 1.f;
#pragma unroll
    for (int k = 0; k < Query<D>::PER; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[k][e] = rintf(__fdiv_rn(x[k][e], by));
    return unit;
}
// As bytes, and which of them are negative.
template <int D>
__device__ __forceinline__ void quantise(const uint16_t *q, uint32_t *out, float &unit, int lane) {
    float x[Query<D>::PER][4];
    const float step = whole_numbers<D>(load_query<D>(q, lane), x);
#pragma unroll
    for (int k = 0; k < Query<D>::PER; ++k) {
        const int w = lane + 32 * k;
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) word |= (static_cast<uint32_t>(static_cast<int>(x[k][e])) & 255u) << 8 * e;
        if (w < Query<D>::WORDS) {
            out[w] = word;
            out[Query<D>::WORDS + w] = __vcmplts4(word, 0);
        }
    }
    if (lane == 0) unit = step;
}
__device__ __forceinline__ uint32_t pair(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Lengths and running sums of the step out of range; by the first CTA.
__device__ __forceinline__ void check_step(const Kv4SelectArgs &a) {
    if (blockIdx.x != 0) return;
    for (int b = threadIdx.x; b < a.requests; b += blockDim.x) {
        const int64_t from = a.cu_new[b], to = a.cu_new[b + 1], len = a.seq_lens[b];
        if (from < 0 || to < from || to > a.T || (to > from && (len < 0 || len > a.max_blocks << a.bs_log2)))
            atomicOr(a.status, kDevBadIndex);
    }
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Stores to the shared memory of the cluster's first CTA.
__device__ __forceinline__ void store_first(uint32_t *p, uint32_t v) {
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\tst.shared::cluster.u32 [a], %1;\n\t}" ::"r"(smem_u32(p)),
                 "r"(v)
                 : "memory");
}

// A team chooses for one token and key head: a CTA, or a warp.
template <bool WARP>
struct Team {
    static constexpr int COUNT = WARP ? 32 : THREADS;       // threads
    __device__ static int thread() { return WARP ? threadIdx.x & 31 : threadIdx.x; }
    __device__ static int warp() { return WARP ? 0 : threadIdx.x >> 5; }
    __device__ static void sync() {
        if (WARP) __syncwarp();
        else __syncthreads();
    }
};

// Key at which the `need` largest of keys[0 .. n) end, and how many of those
// equal to it are among them.  Between the smallest and the largest key a count for
// each of 256 steps shows the one in which they end; its keys, a few as a rule, are
// compared with one another, and otherwise counted again in 256 steps of it.
struct Cut {
    uint32_t key;
    int equal;
};
template <class T>
__device__ __forceinline__ Cut find_cut(const uint32_t *keys, int n, int need, int *scratch) {
    int *const count = scratch, *const ends = scratch + 256, *const pick = ends + 2 * WARPS;
    const int tid = T::thread(), lane = tid & 31;
    uint32_t low = 0xffffffffu, high = 0;
    for (int i = tid; i < n; i += T::COUNT) low = min(low, keys[i]), high = max(high, keys[i]);
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (T::COUNT > 32) {
        if (lane == 0) ends[T::warp()] = static_cast<int>(low), ends[WARPS + T::warp()] = static_cast<int>(high);
        T::sync();
        low = static_cast<uint32_t>(ends[lane % WARPS]), high = static_cast<uint32_t>(ends[WARPS + lane % WARPS]);
        low = __reduce_min_sync(0xffffffffu, low);
        high = __reduce_max_sync(0xffffffffu, high);
    }
    while (true) {
        const uint32_t span = high - low;
        const int shift = span > 255 ? 24 - __clz(span) : 0;  // (span >> shift is 8 bits)
        for (int i = tid; i < 256; i += T::COUNT) count[i] = 0;
        if (tid == 0) pick[0] = 0;
        T::sync();
        for (int i = tid; i < n; i += T::COUNT)
            if (keys[i] - low <= span) atomicAdd(&count[(keys[i] - low) >> shift], 1);
        T::sync();
        if (T::warp() == 0) {  // lane l: the steps 255 - 8 l and the seven below
            int c[8], sum = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += c[e] = count[255 - 8 * lane - e];
            int at = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += v;
            }
            if (at - sum < need && need <= at) {
                at -= sum;
                int e = 0;
#pragma unroll
                for (int k = 0; k < 7; ++k)
                    if (at + c[k] < need && e == k) at += c[k], e = k + 1;
                pick[1] = 255 - 8 * lane - e;
                pick[2] = need - at;
                pick[3] = count[255 - 8 * lane - e];
            }
        }
        T::sync();
        const int held = pick[3];
        need = pick[2];
        low += static_cast<uint32_t>(pick[1]) << shift;
        if (shift == 0) return {low, need};
        high = low + ((1u << shift) - 1u);
        if (held > 256) {
            T::sync();
            continue;
        }
        // ---- the candidates against one another
        uint32_t *const list = reinterpret_cast<uint32_t *>(count);
        for (int i = tid; i < n; i += T::COUNT)
            if (keys[i] - low <= high - low) list[atomicAdd(&pick[0], 1)] = keys[i];
        T::sync();
        for (int j = tid; j < held; j += T::COUNT) {
            const uint32_t key = list[j];
            int above = 0, equal = 0;
            for (int k = 0; k < held; ++k) above += list[k] > key, equal += list[k] == key;
            if (above < need && need <= above + equal) pick[4] = static_cast<int>(key), pick[5] = need - above;  // (the same of equal ones)
        }
        T::sync();
        return {static_cast<uint32_t>(pick[4]), pick[5]};
    }
}

// What token t sees: its position, the pages, how many of these are taken; of them
// the first `few` and those from number `late` on in any case, and `need` of the n
// pages between.
struct View {
    const int32_t *pages;
    int64_t p;
    int b, seen, taken, few, late, need, n;
};
__device__ __forceinline__ View view_of(const Kv4SelectArgs &a, int64_t t, int lane) {
    View v;
    v.b = request_of(a.cu_new, a.requests, t, lane);
    const int64_t cap = a.max_blocks << a.bs_log2;
    v.p = v.b < 0 ? -1 : min(static_cast<int64_t>(a.seq_lens[v.b]) - a.cu_new[v.b + 1] + t, cap - 1);
    v.seen = v.p < 0 ? 0 : static_cast<int>(v.p >> a.bs_log2) + 1;
    v.taken = min(a.top, v.seen);
    v.pages = a.block_table + (v.b < 0 ? 0 : v.b) * a.max_blocks;
    v.few = v.seen > a.top ? a.first : v.taken;
    v.late = v.taken - (v.seen > a.top ? a.recent : 0);
    v.need = v.late - v.few;
    v.n = v.seen - (v.taken - v.need);
    return v;
}

// The table and the length of a token, from the keys of the pages between.
template <class T>
__device__ __forceinline__ void choose(const Kv4SelectArgs &a, int64_t t, int h, const View &v, const uint32_t *keys, int *scratch,
                                       bool &bad) {
    const int tid = T::thread(), lane = tid & 31, warp = T::warp();
    int32_t *const out = a.tables + (t * a.Hkv + h) * a.top;
    auto id_of = [&](int page) -> int {
        const int id = v.pages[page];
        if (id >= 0 && id < a.num_blocks) return id;
        bad = true;
        return -1;
    };
    if (h == 0 && tid == 0)
        a.lens[t] = v.p < 0 ? 0 : static_cast<int>(((v.taken - 1) << a.bs_log2) + (v.p & ((1 << a.bs_log2) - 1)) + 1);
    for (int i = v.taken + tid; i < a.top; i += T::COUNT) out[i] = -1;
    for (int i = tid; i < v.taken; i += T::COUNT)
        if (i < v.few || i >= v.late) out[i] = id_of(i < v.few ? i : v.seen - v.taken + i);
    if (v.need <= 0) return;
    const Cut cut = find_cut<T>(keys, v.n, v.need, scratch);
    // in the order of the pages: a warp's share in a row, counted first where there
    // are several
    const int share = (v.n + T::COUNT - 1) / T::COUNT * 32, from = warp * share, upto = min(from + share, v.n);
    int above = 0, equal = 0;
    if (T::COUNT > 32) {
        int *const sums = scratch;
        for (int i = from + lane; i - lane < upto; i += 32) {
            const uint32_t key = i < upto ? keys[i] : 0u;
            above += __popc(__ballot_sync(0xffffffffu, i < upto && key > cut.key));
            equal += __popc(__ballot_sync(0xffffffffu, i < upto && key == cut.key));
        }
        T::sync();
        if (lane == 0) sums[warp] = above, sums[WARPS + warp] = equal;
        T::sync();
        above = equal = 0;
        for (int w = 0; w < warp; ++w) above += sums[w], equal += sums[WARPS + w];
    }
    const unsigned under = (1u << lane) - 1;
    for (int i = from + lane; i - lane < upto; i += 32) {
        const uint32_t key = i < upto ? keys[i] : 0u;
        const unsigned more = __ballot_sync(0xffffffffu, i < upto && key > cut.key);
        const unsigned same = __ballot_sync(0xffffffffu, i < upto && key == cut.key);
        const int ties = equal + __popc(same & under);
        if (i < upto && (key > cut.key || (key == cut.key && ties < cut.equal)))
            out[v.few + above + __popc(more & under) + min(ties, cut.equal)] = id_of(v.few + i);
        above += __popc(more);
        equal += __popc(same);
    }
}

// Words of shared memory of select_kernel: keys, queries, units, scratch.
__host__ __device__ constexpr int select_words(int width, int G, int D) {
    return width + G * (D / 2) + (G + 3) / 4 * 4 + (256 + 2 * WARPS + 8);
}

// ---- a cluster for a token and key head: its CTAs have a share of the pages each,
// the first one then chooses.
//
// Score.  A lane holds 16 elements of a page's bounds: D / 16 lanes a page, PPI
// pages side by side and four (SLOTS) times as many at a time.  Each four lanes
// have a group of 64 elements: of its sums for four pages every lane adds up one.
// One pass over the bounds for any number of query heads.  Bound: memory, where
// there are pages and tokens enough (64 requests of 63 to 3750 pages 57 us, 4.4 TB/s);
// about 45 instructions a query head for 4 PPI pages.  16 bytes of high and of low a
// lane and slot are on their way at once, 4 KB a warp.  (A ring of further rows in
// shared memory, 72 us, or in registers, 59 us, left fewer CTAs on an SM.)
template <int D>
__global__ void __launch_bounds__(THREADS, 3) select_kernel(const Kv4SelectArgs a) {
    using Us = Team<false>;
    constexpr int LPP = D / 16, PPI = 32 / LPP, SLOTS = 4, BATCH = SLOTS * PPI;
    extern __shared__ __align__(16) uint32_t select_smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = static_cast<int>(cluster_ctas()), rank = static_cast<int>(cluster_rank());
    int64_t t = blockIdx.x / ctas / a.Hkv;
    const int h = static_cast<int>(blockIdx.x / ctas % a.Hkv), G = a.Hq / a.Hkv;
    // of the pages between the first and the recent ones; [G][2][D / 4] the queries, 8
    // bits an element, and which are negative; [G] their units; scratch
    const int width = static_cast<int>((a.max_blocks + 3) / 4 * 4);
    uint32_t *const keys = select_smem, *const query = keys + width;
    float *const unit = reinterpret_cast<float *>(query + G * (D / 2));
    int *const scratch = reinterpret_cast<int *>(unit + (G + 3) / 4 * 4);
    cluster_arrive();  // (there, for the other CTAs' stores)
    pdl_launch_dependents();
    pdl_wait();
    check_step(a);
    if (a.requests == a.T && a.requests > 1 && a.requests <= THREADS) {
        // a token each: those of the longest contexts first (62 -> 56 us for 64 ragged ones)
        int *const lens = scratch;
        if (tid < a.requests) lens[tid] = a.seq_lens[tid];
        __syncthreads();
        if (tid < a.requests) {
            const int mine = lens[tid];
            int before = 0;
            for (int i = 0; i < a.requests; ++i) before += lens[i] > mine || (lens[i] == mine && i < tid);
            if (before == t) lens[THREADS] = tid;
        }
        __syncthreads();
        t = lens[THREADS];
        __syncthreads();
    }
    for (int g = warp; g < G; g += WARPS)
        quantise<D>(a.q + t * a.q_stride + static_cast<int64_t>(h * G + g) * D, query + g * (D / 2), unit[g], lane);
    const View v = view_of(a, t, lane);
    const int n = v.n;
    bool bad = false;
    __syncthreads();
    cluster_wait();
    if (v.need > 0) {
        const int s = lane % LPP, side = lane / LPP;
        const int step = ctas * WARPS * BATCH;
        // the page whose sums this lane has in the end
        const int mine = (2 * (lane & 1) + (lane >> 1 & 1)) * PPI + side;
        const unsigned char *const bounds = a.bounds + static_cast<int64_t>(h) * bounds_bytes(D);
        const int64_t page_bytes = static_cast<int64_t>(a.Hkv) * bounds_bytes(D);
        // (looked at when they are used: a test here would wait for them)
        auto ids = [&](int p0) { return lane < BATCH && p0 + lane < n ? v.pages[v.few + p0 + lane] : NO_PAGE; };
        auto known = [&](int id) {
            const bool in = id >= 0 && id < a.num_blocks;
            bad |= !in && id != NO_PAGE;
            return in ? id : -1;
        };
        const int first = (rank * WARPS + warp) * BATCH;
        int raw = ids(first);
        for (int p0 = first; p0 < n; p0 += step) {
            const int id = known(raw);
            raw = ids(p0 + step);  // on its way meanwhile
            const int whose = __shfl_sync(0xffffffffu, id, mine);
            const float unit_of = *reinterpret_cast<const float *>(bounds + max(whose, 0) * page_bytes + 2 * D + s / 4 * 4);
            uint32_t high[SLOTS][4], low[SLOTS][4];
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const int page = __shfl_sync(0xffffffffu, id, j * PPI + side);
                const unsigned char *const row = bounds + max(page, 0) * page_bytes;
                const uint4 up = *reinterpret_cast<const uint4 *>(row + 16 * s), down = *reinterpret_cast<const uint4 *>(row + D + 16 * s);
                high[j][0] = up.x, high[j][1] = up.y, high[j][2] = up.z, high[j][3] = up.w;
                low[j][0] = down.x, low[j][1] = down.y, low[j][2] = down.z, low[j][3] = down.w;
            }
            float best = -INFINITY;
#pragma unroll 2
            for (int g = 0; g < G; ++g) {
                const uint4 c = *reinterpret_cast<const uint4 *>(query + g * (D / 2) + 4 * s);
                const uint4 m = *reinterpret_cast<const uint4 *>(query + g * (D / 2) + D / 4 + 4 * s);
                const uint32_t qw[4] = {c.x, c.y, c.z, c.w}, below[4] = {m.x, m.y, m.z, m.w};
                int dot[SLOTS];
#pragma unroll
                for (int j = 0; j < SLOTS; ++j) {
                    dot[j] = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        dot[j] = __dp4a(static_cast<int>((high[j][k] & ~below[k]) | (low[j][k] & below[k])), static_cast<int>(qw[k]), dot[j]);
                }
                // (of slot 2 (lane & 1) + (lane >> 1 & 1), over the four lanes of a group)
                const bool odd = lane & 1, upper = lane & 2;
                const int a0 = (odd ? dot[2] : dot[0]) + __shfl_xor_sync(0xffffffffu, odd ? dot[0] : dot[2], 1);
                const int a1 = (odd ? dot[3] : dot[1]) + __shfl_xor_sync(0xffffffffu, odd ? dot[1] : dot[3], 1);
                const int sum = (upper ? a1 : a0) + __shfl_xor_sync(0xffffffffu, upper ? a0 : a1, 2);
                float x = __fmul_rn(static_cast<float>(sum), unit_of);
                if (LPP >= 8) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, 4));
                if (LPP >= 16) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, 8));
                best = fmaxf(best, __fmul_rn(x, unit[g]));
            }
            if (s < 4 && p0 + mine < n) store_first(keys + p0 + mine, ordered(whose < 0 ? -INFINITY : best));
        }
    }
    __syncwarp();
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else __syncthreads();
    if (rank == 0) choose<Us>(a, t, h, v, keys, scratch, bad);
    if (bad) atomicOr(a.status, kDevBadIndex);
}

// ---- tokens of one request: a CTA for as many as fill the eight columns of a
// product, with the 2^lg query heads of a key head (some twice where that is more than
// there are).  Its warps take the pages in turn, 16 at a time, and then a token each to
// choose for.
//
// Score.  16 pages x 8 columns by the 16-bit MMA, both operands whole numbers as
// binary16: a byte under the exponent of 1024, minus 1152.  Sums of 64 products below
// 2^14 are exact in binary32.  The queries' parts above 0 meet `high`, those below 0
// `low`.  A lane's 16 bytes of a row are the operands of four products, in any order
// of the 64 elements that is the queries' too.  Two groups of 64 of the rows are on
// their way meanwhile.  Bound: the conversions and products beside them, and the choice
// (301 tokens x 470 pages, 32 heads of 128 on 8, 30 us; with 8-bit products by dp4a, a
// warp each, 45; the 8-bit MMA takes 64 cycles for what the 16-bit one does in 16).
constexpr int COLUMNS = 8;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four whole numbers of 8 bits as binary16 pairs.
__device__ __forceinline__ void halves(uint32_t w, uint32_t &lo, uint32_t &hi) {
    w ^= 0x80808080u;
    lo = __byte_perm(w, 0x64646464u, 0x4140);
    hi = __byte_perm(w, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
}

// Words of shared memory, for NB times 8 columns and W warps: keys of the tokens,
// queries, units, what the tokens see, and of each warp scratch.
__host__ __device__ constexpr int piece_words(int width, int lg, int D, int NB, int W) {
    return NB * ((width << (3 - lg)) + D * 8 + 3 * COLUMNS) + W * (256 + 2 * WARPS + 8);
}

template <int D, int NB, int W>
__global__ void __launch_bounds__(W * 32, (NB == 1 ? 16 : 12) / W) piece_kernel(const Kv4SelectArgs a, const int lg) {
    using Us = Team<true>;
    constexpr int G64 = D / 64, NEXT = G64 > 1 ? 2 : 1;  // groups on their way
    extern __shared__ __align__(16) uint32_t select_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int tokens = NB * (COLUMNS >> lg), G = a.Hq / a.Hkv, h = static_cast<int>(blockIdx.x % a.Hkv);
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / a.Hkv) * tokens;
    const int here = static_cast<int>(min(static_cast<int64_t>(tokens), a.T - t0));
    const int width = static_cast<int>((a.max_blocks + 3) / 4 * 4);
    uint32_t *const keys = select_smem;
    uint2 *const query = reinterpret_cast<uint2 *>(keys + NB * (width << (3 - lg)));  // [NB][G64][4 products][high, low][32 lanes]
    float *const unit = reinterpret_cast<float *>(query + NB * D * 4);
    int *const request = reinterpret_cast<int *>(unit + NB * COLUMNS), *const count = request + NB * COLUMNS;  // of each token: pages between
    int *const scratch = count + NB * COLUMNS + warp * (256 + 2 * WARPS + 8);
    pdl_launch_dependents();
    pdl_wait();
    check_step(a);
    for (int c = warp; c < NB * COLUMNS; c += W) {
        const int64_t t = t0 + min(c >> lg, here - 1);
        const Query<D> raw = load_query<D>(a.q + t * a.q_stride + static_cast<int64_t>(h * G + (c & ((1 << lg) - 1)) % G) * D, lane);
        float x[Query<D>::PER][4];
        const float step = whole_numbers<D>(raw, x);
#pragma unroll
        for (int k = 0; k < Query<D>::PER; ++k) {
            const int w = lane + 32 * k;  // elements 4 w and on: group w / 16, lane w / 4 % 4, product w % 4
            if (w >= Query<D>::WORDS) continue;
            uint2 *const to = query + c / COLUMNS * D * 4 + ((w >> 4) * 4 + (w & 3)) * 64 + c % COLUMNS * 4 + (w >> 2 & 3);
            to[0] = make_uint2(pair(fmaxf(x[k][0], 0.f), fmaxf(x[k][1], 0.f)), pair(fmaxf(x[k][2], 0.f), fmaxf(x[k][3], 0.f)));
            to[32] = make_uint2(pair(fminf(x[k][0], 0.f), fminf(x[k][1], 0.f)), pair(fminf(x[k][2], 0.f), fminf(x[k][3], 0.f)));
        }
        if (lane == 0) unit[c] = step;
    }
    View own;  // of this warp's first token
    for (int i = warp; i < here; i += W) {
        const View v = view_of(a, t0 + i, lane);
        if (lane == 0) request[i] = v.b, count[i] = v.need > 0 ? v.n : 0;
        if (i == warp) own = v;
    }
    __syncthreads();
    bool bad = false;
    const unsigned char *const bounds = a.bounds + static_cast<int64_t>(h) * bounds_bytes(D);
    const int64_t page_bytes = static_cast<int64_t>(a.Hkv) * bounds_bytes(D);
    // the token (of 8 columns) whose keys this lane writes: 2 q and the next, or one (or none)
    const int mine = lg == 0 ? 2 * q : lg == 1 ? q : lg == 2 ? q >> 1 : 0;
    const bool writes = lg <= 1 || (lg == 2 ? (q & 1) == 0 : q == 0);
    for (int from = 0, upto; from < here; from = upto) {
        // tokens of one request
        int n = count[from];
        for (upto = from + 1; upto < here && request[upto] == request[from]; ++upto) n = max(n, count[upto]);
        if (n == 0) continue;
        auto keys_of = [&](int token) { return writes && token >= from && token < upto ? count[token] : 0; };
        int n0[NB], n1[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            n0[b] = keys_of(b * (COLUMNS >> lg) + mine);
            n1[b] = lg == 0 ? keys_of(b * COLUMNS + mine + 1) : 0;
        }
        const int32_t *const pages = a.block_table + static_cast<int64_t>(request[from]) * a.max_blocks + a.first;
        constexpr int STEP = 16 * W;
        auto ids = [&](int p0) { return lane < 16 && p0 + lane < n ? pages[p0 + lane] : NO_PAGE; };
        struct Pages {
            const unsigned char *row[2];  // of pages g and g + 8
            int id[2];
        };
        auto find = [&](int raw) {
            const bool in = raw >= 0 && raw < a.num_blocks;
            bad |= !in && raw != NO_PAGE;
            Pages r;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                r.id[k] = __shfl_sync(0xffffffffu, in ? raw : -1, g + 8 * k);
                r.row[k] = bounds + max(r.id[k], 0) * page_bytes;
            }
            return r;
        };
        struct Rows {
            uint4 high[2], low[2];
        };
        auto load = [&](const Pages &r, int i) {
            Rows x;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                x.high[k] = *reinterpret_cast<const uint4 *>(r.row[k] + 64 * i + 16 * q);
                x.low[k] = *reinterpret_cast<const uint4 *>(r.row[k] + D + 64 * i + 16 * q);
            }
            return x;
        };
        Pages now = find(ids(16 * warp));
        int raw = ids(16 * warp + STEP);
        Rows ahead[NEXT];
#pragma unroll
        for (int k = 0; k < NEXT; ++k) ahead[k] = load(now, k);
        for (int p0 = 16 * warp; p0 < n; p0 += STEP) {
            const Pages next = find(raw);
            raw = ids(p0 + 2 * STEP);
            float steps[2][G64];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < G64; ++i) steps[k][i] = *reinterpret_cast<const float *>(now.row[k] + 2 * D + 4 * i);
            float sum[NB][2][4];  // of each half of the groups
#pragma unroll
            for (int i = 0; i < G64; ++i) {
                const Rows x = ahead[i % NEXT];
                ahead[i % NEXT] = i + NEXT < G64 ? load(now, i + NEXT) : load(next, i + NEXT - G64);
                float up[NB][4] = {}, down[NB][4] = {};
                const uint32_t high[2][4] = {{x.high[0].x, x.high[0].y, x.high[0].z, x.high[0].w}, {x.high[1].x, x.high[1].y, x.high[1].z, x.high[1].w}};
                const uint32_t low[2][4] = {{x.low[0].x, x.low[0].y, x.low[0].z, x.low[0].w}, {x.low[1].x, x.low[1].y, x.low[1].z, x.low[1].w}};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
                    halves(high[0][s], a0, a2);
                    halves(high[1][s], a1, a3);
                    halves(low[0][s], b0, b2);
                    halves(low[1][s], b1, b3);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint2 above = query[b * D * 4 + (i * 4 + s) * 64 + lane], below = query[b * D * 4 + (i * 4 + s) * 64 + 32 + lane];
                        mma_f16(up[b], a0, a1, a2, a3, above.x, above.y);
                        mma_f16(down[b], b0, b1, b2, b3, below.x, below.y);
                    }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = __fmul_rn(up[b][e] + down[b][e], steps[e >> 1][i]);
                        sum[b][i >> 1][e] = i & 1 ? __fadd_rn(sum[b][i >> 1][e], y) : y;
                    }
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int page = p0 + g + 8 * k;
                    float x0 = G64 == 4 ? __fadd_rn(sum[b][0][2 * k], sum[b][1][2 * k]) : sum[b][0][2 * k];
                    float x1 = G64 == 4 ? __fadd_rn(sum[b][0][2 * k + 1], sum[b][1][2 * k + 1]) : sum[b][0][2 * k + 1];
                    x0 = now.id[k] < 0 ? -INFINITY : __fmul_rn(x0, unit[b * COLUMNS + 2 * q]);
                    x1 = now.id[k] < 0 ? -INFINITY : __fmul_rn(x1, unit[b * COLUMNS + 2 * q + 1]);
                    if (lg >= 1) x0 = fmaxf(x0, x1);
                    x0 = fmaxf(x0, -INFINITY), x1 = fmaxf(x1, -INFINITY);  // (NaN, of all heads where these are several: the lowest)
                    if (lg >= 2) x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                    if (lg >= 3) x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                    uint32_t *const to = keys + (b * (COLUMNS >> lg) + mine) * width + page;
                    if (page < n0[b]) *to = ordered(x0);
                    if (page < n1[b]) to[width] = ordered(x1);
                }
            now = next;
        }
    }
    __syncthreads();
    for (int i = warp; i < here; i += W)
        choose<Us>(a, t0 + i, h, i == warp ? own : view_of(a, t0 + i, lane), keys + i * width, scratch, bad);
    if (bad) atomicOr(a.status, kDevBadIndex);
}

// CTAs of a cluster: so many that the GPU has four or more for each SM, none with
// less than a batch of pages for each warp.  16 query heads of 256 on 8, with 1 / 2 /
// 4 / 8 CTAs: one request of 2048 pages 27 / 17 / 12 / 10 us, 64 of 63 to 3750 pages
// 83 / 56 / 63 / 79 us.
int select_ctas(const Kv4SelectArgs &a, int D, const DeviceInfo &dev) {
    const int64_t tasks = a.T * a.Hkv, pages = WARPS * 4 * 32 / (D / 16);
    int ctas = 1;
    while (ctas < 8 && tasks * ctas < 4 * dev.num_sms && a.max_blocks > pages * ctas) ctas *= 2;
    return ctas;
}

template <int D>
cudaError_t launch_clusters(const Kv4SelectArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    const int ctas = select_ctas(a, D, dev);
    const int smem = select_words(static_cast<int>((a.max_blocks + 3) / 4 * 4), a.Hq / a.Hkv, D) * 4;
    static SmemLimit limit;
    if (smem > 40 * 1024)
        if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(select_kernel<D>), dev.device, smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.T * a.Hkv * ctas));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, select_kernel<D>, a);
}

template <int D, int NB, int W>
cudaError_t launch_piece(const Kv4SelectArgs &a, int lg, int smem, cudaStream_t st, const DeviceInfo &dev) {
    static SmemLimit limit;
    if (smem > 40 * 1024)
        if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(piece_kernel<D, NB, W>), dev.device, smem)) return e;
    const int64_t tokens = NB * (COLUMNS >> lg);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + tokens - 1) / tokens * a.Hkv));
    cfg.blockDim = dim3(W * 32);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, piece_kernel<D, NB, W>, a, lg);
}

// Tokens of a request together where there are four or more (on average), not too many
// query heads and room for the scores.
//
// Warps of a CTA: 8, or 4 or 2 where one wave of such CTAs takes them and one of larger
// ones does not (so many warps score a token's pages, and one chooses); with more than that
// 16 columns, whose conversions serve twice as many, and 4 warps, or 2 in two waves or more
// for the few tokens of a CTA with four query heads (600 tokens: 59 | 71).  470 pages, us: a cluster for each token | 8
// columns with 8, 4, 2 warps | 16 columns with 4, 2:
//     new tokens                16                 96                 301                 1200
//     32 heads of 128 on 8   11 | 12 12 16 | -   24 | 25 19 26 | -   63 | 51 37 31 | 40 38   230 | 194 142 116 | 116 109
//     16 heads of 256 on 8   15 | 14 16 28 | -   28 | 19 26 32 | -   77 | 36 29 35 | 34 42   280 | 140 113 109 |  99 131
//     16 heads of 64 on 16        9 15 26 | -         12 19 28 | -         22 20 29 | 28 48          85  75  72 |  67 104
template <int D>
cudaError_t launch_select(const Kv4SelectArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    const int width = static_cast<int>((a.max_blocks + 3) / 4 * 4), G = a.Hq / a.Hkv;
    const int lg = G <= 1 ? 0 : G <= 2 ? 1 : G <= 4 ? 2 : 3;
    if (G <= COLUMNS && a.T >= 4 * static_cast<int64_t>(a.requests)) {
        const int64_t ctas = (a.T + (COLUMNS >> lg) - 1) / (COLUMNS >> lg) * a.Hkv, sms = dev.num_sms;
        auto bytes = [&](int NB, int W) { return piece_words(width, lg, D, NB, W) * 4; };
        // (so many CTAs that the registers allow find room)
        auto room = [&](int NB, int W) { return bytes(NB, W) <= 220 * 1024 / ((NB == 1 ? 16 : 12) / W); };
        if (ctas > 24 * sms && lg >= 2 && room(2, 2)) return launch_piece<D, 2, 2>(a, lg, bytes(2, 2), st, dev);
        if (ctas > 8 * sms && room(2, 4)) return launch_piece<D, 2, 4>(a, lg, bytes(2, 4), st, dev);
        if (ctas > 4 * sms && room(1, 2)) return launch_piece<D, 1, 2>(a, lg, bytes(1, 2), st, dev);
        if (ctas > 2 * sms && room(1, 4)) return launch_piece<D, 1, 4>(a, lg, bytes(1, 4), st, dev);
        if (room(1, 8)) return launch_piece<D, 1, 8>(a, lg, bytes(1, 8), st, dev);
    }
    return launch_clusters<D>(a, st, dev);
}

}  // namespace

cudaError_t launch_kv4_bounds(const Kv4BoundsArgs &a, int D, cudaStream_t st, const DeviceInfo &) {
    return D == 64 ? launch_bounds<64>(a, st) : D == 128 ? launch_bounds<128>(a, st) : launch_bounds<256>(a, st);
}

cudaError_t launch_kv4_select(const Kv4SelectArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    return D == 64 ? launch_select<64>(a, st, dev) : D == 128 ? launch_select<128>(a, st, dev) : launch_select<256>(a, st, dev);
}

}  // namespace w4
