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

constexpr int BOUNDS_WARPS = 8;

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

// A query head in whole numbers of 8 bits (NaN as 0, infinities as the largest
// finite number), which bytes of them are negative, and their unit.  By a whole
// warp.
template <int D>
__device__ __forceinline__ void quantise(const uint16_t *q, uint32_t *out, float &unit, int lane) {
    constexpr int WORDS = D / 4, PER = (WORDS + 31) / 32;
    float x[PER][4], most = 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int w = lane + 32 * k;
        const uint2 raw = w < WORDS ? *reinterpret_cast<const uint2 *>(q + 4 * w) : make_uint2(0, 0);
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
    const float step = most * STEP, by = step > 0.f ? step : 1.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) word |= (static_cast<uint32_t>(__float2int_rn(__fdiv_rn(x[k][e], by))) & 255u) << 8 * e;
        if (lane + 32 * k < WORDS) {
            out[lane + 32 * k] = word;
            out[WORDS + lane + 32 * k] = __vcmplts4(word, 0);
        }
    }
    if (lane == 0) unit = step;
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

// Words of shared memory of a team: keys, queries, units, scratch.
__host__ __device__ constexpr int select_words(int width, int G, int D) {
    return width + G * (D / 2) + (G + 3) / 4 * 4 + (256 + 2 * WARPS + 8);
}

// A team works on one token and key head: a CTA (with others of its cluster), or a
// warp where there are tokens enough for that.
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

// The CTAs of a cluster have a share of a token's pages each; the first one then
// chooses.  A warp alone does both; the warps of a CTA have neighbouring tokens
// then, which share most of their pages in L1.
//
// Score.  A lane holds 16 elements of a page's bounds: D / 16 lanes a page, PPI
// pages side by side and four (SLOTS) times as many at a time.  Each four lanes
// have a group of 64 elements: of its sums for four pages every lane adds up one.
// One pass over the bounds for any number of query heads.  Bound: memory, where
// there are pages and tokens enough; about 45 instructions a query head for 4 PPI
// pages.  16 bytes of high and of low a lane and slot are on their way at once,
// 4 KB a warp.
template <int D, bool WARP>
__global__ void __launch_bounds__(THREADS, WARP ? 2 : 3) select_kernel(const Kv4SelectArgs a) {
    using Us = Team<WARP>;
    constexpr int LPP = D / 16, PPI = 32 / LPP, SLOTS = 4, BATCH = SLOTS * PPI;
    extern __shared__ __align__(16) uint32_t select_smem[];
    const int tid = Us::thread(), lane = tid & 31, warp = Us::warp();
    const int ctas = WARP ? 1 : static_cast<int>(cluster_ctas()), rank = WARP ? 0 : static_cast<int>(cluster_rank());
    const int64_t task = blockIdx.x / ctas;
    int64_t t = WARP ? task / a.Hkv * WARPS + (threadIdx.x >> 5) : task / a.Hkv;
    const int h = static_cast<int>(task % a.Hkv), G = a.Hq / a.Hkv;
    // of the pages between the first and the recent ones; [G][2][D / 4] the queries, 8
    // bits an element, and which are negative; [G] their units; scratch
    const int width = static_cast<int>((a.max_blocks + 3) / 4 * 4);
    uint32_t *const keys = select_smem + (WARP ? (threadIdx.x >> 5) * select_words(width, G, D) : 0);
    uint32_t *const query = keys + width;
    float *const unit = reinterpret_cast<float *>(query + G * (D / 2));
    int *const scratch = reinterpret_cast<int *>(unit + (G + 3) / 4 * 4);
    if (!WARP) cluster_arrive();  // (there, for the other CTAs' stores)
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.requests; b += THREADS) {
            const int64_t from = a.cu_new[b], to = a.cu_new[b + 1], len = a.seq_lens[b];
            if (from < 0 || to < from || to > a.T || (to > from && (len < 0 || len > a.max_blocks << a.bs_log2)))
                atomicOr(a.status, kDevBadIndex);
        }
    if (WARP && t >= a.T) return;
    if (!WARP && a.requests == a.T && a.requests > 1 && a.requests <= THREADS) {
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
    for (int g = warp; g < G; g += Us::COUNT / 32)
        quantise<D>(a.q + t * a.q_stride + static_cast<int64_t>(h * G + g) * D, query + g * (D / 2), unit[g], lane);
    const int b = request_of(a.cu_new, a.requests, t, lane);
    const int64_t cap = a.max_blocks << a.bs_log2;
    const int64_t p = b < 0 ? -1 : min(static_cast<int64_t>(a.seq_lens[b]) - a.cu_new[b + 1] + t, cap - 1);
    const int seen = p < 0 ? 0 : static_cast<int>(p >> a.bs_log2) + 1;
    const int taken = min(a.top, seen);
    int32_t *const out = a.tables + (t * a.Hkv + h) * a.top;
    const int32_t *const pages = a.block_table + (b < 0 ? 0 : b) * a.max_blocks;
    bool bad = false;
    auto id_of = [&](int page) -> int {
        const int id = pages[page];
        if (id >= 0 && id < a.num_blocks) return id;
        bad = true;
        return -1;
    };
    const int few = seen > a.top ? a.first : taken, late = taken - (seen > a.top ? a.recent : 0);
    // need of n pages, from number `few` on
    const int need = late - few, n = seen - (taken - need);
    Us::sync();
    if (!WARP) cluster_wait();
    if (need > 0) {
        const int s = lane % LPP, side = lane / LPP;
        const int step = ctas * (Us::COUNT / 32) * BATCH;
        // the page whose sums this lane has in the end
        const int mine = (2 * (lane & 1) + (lane >> 1 & 1)) * PPI + side;
        const unsigned char *const bounds = a.bounds + static_cast<int64_t>(h) * bounds_bytes(D);
        const int64_t page_bytes = static_cast<int64_t>(a.Hkv) * bounds_bytes(D);
        // (looked at when they are used: a test here would wait for them)
        auto ids = [&](int p0) { return lane < BATCH && p0 + lane < n ? pages[few + p0 + lane] : NO_PAGE; };
        auto known = [&](int id) {
            const bool in = id >= 0 && id < a.num_blocks;
            bad |= !in && id != NO_PAGE;
            return in ? id : -1;
        };
        const int first = (rank * (Us::COUNT / 32) + warp) * BATCH;
        struct Rows {
            uint4 high[SLOTS], low[SLOTS];
            float step;  // of this lane's page and group
            int whose;
        };
        auto load = [&](int id) -> Rows {
            Rows r;
            r.whose = __shfl_sync(0xffffffffu, id, mine);
            r.step = *reinterpret_cast<const float *>(bounds + max(r.whose, 0) * page_bytes + 2 * D + s / 4 * 4);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const int page = __shfl_sync(0xffffffffu, id, j * PPI + side);
                const unsigned char *const row = bounds + max(page, 0) * page_bytes;
                r.high[j] = *reinterpret_cast<const uint4 *>(row + 16 * s);
                r.low[j] = *reinterpret_cast<const uint4 *>(row + D + 16 * s);
            }
            return r;
        };
        // the ids of the next pages are on their way meanwhile; to a warp alone, which
        // has fewer others beside it on the SM, their rows too
        int raw = ids(first);
        Rows rows;
        if (WARP) {
            rows = load(known(raw));
            raw = ids(first + step);
        }
        for (int p0 = first; p0 < n; p0 += step) {
            Rows next;
            if (WARP) {
                next = load(known(raw));
                raw = ids(p0 + 2 * step);
            } else {
                rows = load(known(raw));
                raw = ids(p0 + step);
            }
            uint32_t high[SLOTS][4], low[SLOTS][4];
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                high[j][0] = rows.high[j].x, high[j][1] = rows.high[j].y, high[j][2] = rows.high[j].z, high[j][3] = rows.high[j].w;
                low[j][0] = rows.low[j].x, low[j][1] = rows.low[j].y, low[j][2] = rows.low[j].z, low[j][3] = rows.low[j].w;
            }
            const float unit_of = rows.step;
            const int whose = rows.whose;
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
            if (s < 4 && p0 + mine < n) {
                const uint32_t key = ordered(whose < 0 ? -INFINITY : best);
                if (WARP) keys[p0 + mine] = key;
                else store_first(keys + p0 + mine, key);
            }
            if (WARP) rows = next;
        }
    }
    __syncwarp();
    if (ctas > 1) {
        cluster_arrive();
        cluster_wait();
    } else Us::sync();
    if (rank == 0) {
        if (h == 0 && tid == 0)
            a.lens[t] = p < 0 ? 0 : static_cast<int>(((taken - 1) << a.bs_log2) + (p & ((1 << a.bs_log2) - 1)) + 1);
        for (int i = taken + tid; i < a.top; i += Us::COUNT) out[i] = -1;
        for (int i = tid; i < taken; i += Us::COUNT)
            if (i < few || i >= late) out[i] = id_of(i < few ? i : seen - taken + i);
        if (need > 0) {
            const Cut cut = find_cut<Us>(keys, n, need, scratch);
            // in the order of the pages: a warp's share in a row, counted first where
            // there are several
            const int share = (n + Us::COUNT - 1) / Us::COUNT * 32, from = warp * share, upto = min(from + share, n);
            int above = 0, equal = 0;
            if (!WARP) {
                int *const sums = scratch;
                for (int i = from + lane; i - lane < upto; i += 32) {
                    const uint32_t key = i < upto ? keys[i] : 0u;
                    above += __popc(__ballot_sync(0xffffffffu, i < upto && key > cut.key));
                    equal += __popc(__ballot_sync(0xffffffffu, i < upto && key == cut.key));
                }
                Us::sync();
                if (lane == 0) sums[warp] = above, sums[WARPS + warp] = equal;
                Us::sync();
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
                    out[few + above + __popc(more & under) + min(ties, cut.equal)] = id_of(few + i);
                above += __popc(more);
                equal += __popc(same);
            }
        }
    }
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

template <int D, bool WARP>
cudaError_t launch_select(const Kv4SelectArgs &a, int ctas, cudaStream_t st, const DeviceInfo &dev) {
    const int words = select_words(static_cast<int>((a.max_blocks + 3) / 4 * 4), a.Hq / a.Hkv, D), smem = (WARP ? WARPS : 1) * words * 4;
    static SmemLimit limit;
    if (smem > 40 * 1024)
        if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(select_kernel<D, WARP>), dev.device, smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((WARP ? (a.T + WARPS - 1) / WARPS : a.T) * a.Hkv * ctas));
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
    cfg.numAttrs = WARP ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, select_kernel<D, WARP>, a);
}

// A warp for a token and key head where that gives each SM eight warps or more, and
// their scores leave room for two CTAs: 301 tokens with 470 pages, 32 heads of 128 on
// 8, 45 us, with CTAs 62.
template <int D>
cudaError_t launch_select(const Kv4SelectArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    const int words = select_words(static_cast<int>((a.max_blocks + 3) / 4 * 4), a.Hq / a.Hkv, D);
    if (a.T * a.Hkv >= 8 * static_cast<int64_t>(dev.num_sms) && WARPS * words * 4 <= 100 * 1024) return launch_select<D, true>(a, 1, st, dev);
    return launch_select<D, false>(a, select_ctas(a, D, dev), st, dev);
}

}  // namespace

cudaError_t launch_kv4_bounds(const Kv4BoundsArgs &a, int D, cudaStream_t st, const DeviceInfo &) {
    return D == 64 ? launch_bounds<64>(a, st) : D == 128 ? launch_bounds<128>(a, st) : launch_bounds<256>(a, st);
}

cudaError_t launch_kv4_select(const Kv4SelectArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    return D == 64 ? launch_select<64>(a, st, dev) : D == 128 ? launch_select<128>(a, st, dev) : launch_select<256>(a, st, dev);
}

}  // namespace w4
