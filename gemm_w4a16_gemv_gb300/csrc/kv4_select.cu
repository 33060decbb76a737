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

// A warp takes 32 slots and one key head.  A lane holds 8 elements: D / 8 lanes
// a token, 256 / D tokens side by side.
template <int D>
__global__ void __launch_bounds__(BOUNDS_WARPS * 32) bounds_kernel(const Kv4BoundsArgs a) {
    constexpr int LANES = D / 8, SIDE = 32 / LANES, TB = kv4_tile_bytes(D);
    const int lane = threadIdx.x & 31, h = blockIdx.y * BOUNDS_WARPS + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    if (h >= a.Hkv) return;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const int64_t slot = t < a.T ? a.slots[t] : -1;
    if (slot >= a.num_slots && h == 0) atomicOr(a.status, kDevBadIndex);
    const int64_t size = int64_t(1) << a.bs_log2;
    unsigned full = __ballot_sync(0xffffffffu, slot >= 0 && slot < a.num_slots && (slot & (size - 1)) == size - 1);
    const int i = lane % LANES, group = i / 8, side = lane / LANES;
    while (full) {
        const int64_t block = __shfl_sync(0xffffffffu, slot, __ffs(full) - 1) >> a.bs_log2;
        full &= full - 1;
        const unsigned char *tile = a.cache + ((block * a.Hkv + h) << (a.bs_log2 - 4)) * TB;
        float high[8], low[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) high[e] = -INFINITY, low[e] = INFINITY;
#pragma unroll 1
        for (int n = 0; n < 1 << (a.bs_log2 - 4); ++n, tile += TB) {
            uint32_t codes[16 / SIDE], para[16 / SIDE];
#pragma unroll
            for (int j = 0; j < 16 / SIDE; ++j) {
                const int row = group * 16 + j * SIDE + side;
                codes[j] = *reinterpret_cast<const uint32_t *>(tile + row * 32 + i % 8 * 4);
                para[j] = *reinterpret_cast<const uint32_t *>(tile + 16 * D + row * 4);
            }
#pragma unroll
            for (int j = 0; j < 16 / SIDE; ++j) {
                const float s = f16_lo(para[j]), z = f16_hi(para[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = (static_cast<float>(codes[j] >> 4 * e & 15u) - z) * s;  // exact
                    high[e] = fmaxf(high[e], v);
                    low[e] = fminf(low[e], v);
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
            up[e / 4] |= (static_cast<uint32_t>(__float2int_ru(__fdiv_rn(high[e], by))) & 255u) << 8 * (e % 4);
            down[e / 4] |= (static_cast<uint32_t>(__float2int_rd(__fdiv_rn(low[e], by))) & 255u) << 8 * (e % 4);
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
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + 31) / 32), static_cast<unsigned>((a.Hkv + BOUNDS_WARPS - 1) / BOUNDS_WARPS));
    cfg.blockDim = dim3(BOUNDS_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, bounds_kernel<D>, a);
}

// ---------------------------------------------------------------- select

constexpr int THREADS = 256, WARPS = THREADS / 32;

// Scores in the order of whole numbers.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);  // (-0 as 0)
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// A query head in whole numbers of 8 bits (NaN as 0, infinities as the largest
// finite number) and their unit.  By a whole warp.
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
        if (lane + 32 * k < WORDS) out[lane + 32 * k] = word;
    }
    if (lane == 0) unit = step;
}

// Half of N sums for each of two lanes, lane ^ o the other one: those of the
// first half where bit o of `lane` is 0.
template <int N, class T, int M>
__device__ __forceinline__ void fold(T (&v)[M], int o, int lane) {
    const bool second = lane & o;
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        const T keep = second ? v[k + N / 2] : v[k], give = second ? v[k] : v[k + N / 2];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
}

// One CTA for a token and key head.
//
// Score.  A warp takes 32 pages; a lane holds 16 elements, so LPP = D / 16 lanes
// a page and PPI pages side by side, LPP times.  The sums over a page's lanes
// are formed for all its 32 pages together: with every lane that is added, half
// of the pages go to either side, until each lane has one page.
template <int D, int HC>
__global__ void __launch_bounds__(THREADS) select_kernel(const Kv4SelectArgs a) {
    constexpr int LPP = D / 16, PPI = 32 / LPP;
    extern __shared__ uint32_t keys[];      // of the pages between the first and the recent ones
    __shared__ uint32_t query[HC][D / 4];   // 8 bits an element
    __shared__ float unit[HC];
    __shared__ int histogram[256], sums[2 * WARPS], pick[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x / a.Hkv;
    const int h = static_cast<int>(blockIdx.x % a.Hkv), G = a.Hq / a.Hkv;
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0)
        for (int b = tid; b < a.requests; b += THREADS) {
            const int64_t from = a.cu_new[b], to = a.cu_new[b + 1], len = a.seq_lens[b];
            if (from < 0 || to < from || to > a.T || (to > from && (len < 0 || len > a.max_blocks << a.bs_log2)))
                atomicOr(a.status, kDevBadIndex);
        }
    const int b = request_of(a.cu_new, a.requests, t, lane);
    const int64_t cap = a.max_blocks << a.bs_log2;
    const int64_t p = b < 0 ? -1 : min(static_cast<int64_t>(a.seq_lens[b]) - a.cu_new[b + 1] + t, cap - 1);
    const int seen = p < 0 ? 0 : static_cast<int>(p >> a.bs_log2) + 1;
    const int taken = min(a.top, seen);
    int32_t *const out = a.tables + (t * a.Hkv + h) * a.top;
    if (h == 0 && tid == 0)
        a.lens[t] = p < 0 ? 0 : static_cast<int>(((taken - 1) << a.bs_log2) + (p & ((1 << a.bs_log2) - 1)) + 1);
    for (int i = taken + tid; i < a.top; i += THREADS) out[i] = -1;
    const int32_t *const pages = a.block_table + (b < 0 ? 0 : b) * a.max_blocks;
    bool bad = false;
    auto id_of = [&](int page) -> int {
        const int id = pages[page];
        if (id >= 0 && id < a.num_blocks) return id;
        bad = true;
        return -1;
    };
    const int few = seen > a.top ? a.first : taken, late = taken - (seen > a.top ? a.recent : 0);
    for (int i = tid; i < taken; i += THREADS)
        if (i < few || i >= late) out[i] = id_of(i < few ? i : seen - taken + i);
    // need of n pages, from number `few` on
    const int need = late - few, n = seen - (taken - need);
    if (need > 0) {
        const int s = lane % LPP, side = lane / LPP;
        for (int g0 = 0; g0 < G; g0 += HC) {
            __syncthreads();
            for (int g = warp; g < HC; g += WARPS) quantise<D>(a.q + t * a.q_stride + static_cast<int64_t>(h * G + min(g0 + g, G - 1)) * D, query[g], unit[g], lane);
            __syncthreads();
            uint32_t qw[HC][4], below[HC][4];
#pragma unroll
            for (int g = 0; g < HC; ++g)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    qw[g][k] = query[g][4 * s + k];
                    below[g][k] = __vcmplts4(qw[g][k], 0);
                }
            for (int p0 = warp * 32; p0 < n; p0 += THREADS) {
                const int id = p0 + lane < n ? id_of(few + p0 + lane) : -1;
                auto row_of = [&](int slot) -> const unsigned char * {  // of the page of `slot` beside this lane, or null
                    const int page = __shfl_sync(0xffffffffu, id, slot * PPI + side);
                    return page < 0 ? nullptr : a.bounds + (static_cast<int64_t>(page) * a.Hkv + h) * bounds_bytes(D);
                };
                int dot[HC][LPP];
#pragma unroll
                for (int j = 0; j < LPP; ++j) {
                    const unsigned char *const row = row_of(j);
                    uint4 up = make_uint4(0, 0, 0, 0), down = up;
                    if (row) {
                        up = *reinterpret_cast<const uint4 *>(row + 16 * s);
                        down = *reinterpret_cast<const uint4 *>(row + D + 16 * s);
                    }
                    const uint32_t high[4] = {up.x, up.y, up.z, up.w}, low[4] = {down.x, down.y, down.z, down.w};
#pragma unroll
                    for (int g = 0; g < HC; ++g) {
                        dot[g][j] = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            dot[g][j] = __dp4a(static_cast<int>((high[k] & ~below[g][k]) | (low[k] & below[g][k])),
                                               static_cast<int>(qw[g][k]), dot[g][j]);
                    }
                }
                // over the 4 lanes of a group of 64: LPP / 4 pages left, slots `slot` and on
                const int slot = (lane & 1 ? LPP / 2 : 0) + (lane & 2 ? LPP / 4 : 0);
                float x[HC][LPP / 4];
#pragma unroll
                for (int g = 0; g < HC; ++g) {
                    fold<LPP>(dot[g], 1, lane);
                    fold<LPP / 2>(dot[g], 2, lane);
                }
#pragma unroll
                for (int j = 0; j < LPP / 4; ++j) {
                    const unsigned char *const row = row_of(slot + j);
                    const float step = row ? *reinterpret_cast<const float *>(row + 2 * D + s / 4 * 4) : 0.f;
#pragma unroll
                    for (int g = 0; g < HC; ++g) x[g][j] = __fmul_rn(static_cast<float>(dot[g][j]), step);
                }
                // over the groups
                float best = -INFINITY;
#pragma unroll
                for (int g = 0; g < HC; ++g) {
                    if (LPP >= 8) fold<LPP / 4>(x[g], 4, lane);
                    if (LPP >= 16) fold<LPP / 8>(x[g], 8, lane);
                    best = fmaxf(best, __fmul_rn(x[g][0], unit[g]));
                }
                const int last = slot + (LPP >= 8 && (lane & 4) ? LPP / 8 : 0) + (LPP >= 16 && (lane & 8) ? LPP / 16 : 0);
                const int mine = last * PPI + side;
                if (__shfl_sync(0xffffffffu, id, mine) < 0) best = -INFINITY;
                if (p0 + mine < n) {
                    const uint32_t key = ordered(best);
                    keys[p0 + mine] = g0 == 0 ? key : max(key, keys[p0 + mine]);
                }
            }
        }
        // the `need` largest keys: their smallest by 8 bits at a time, and how many
        // of those equal to it (the first ones)
        uint32_t cut = 0, known = 0;
        int rest = need;
#pragma unroll 1
        for (int shift = 24; shift >= 0; shift -= 8) {
            histogram[tid] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += THREADS)
                if ((keys[i] & known) == cut) atomicAdd(&histogram[keys[i] >> shift & 255u], 1);
            __syncthreads();
            if (warp == 0) {  // lane l: the digits 255 - 8 l and the seven below
                int c[8], sum = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += c[e] = histogram[255 - 8 * lane - e];
                int at = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, at, o);
                    if (lane >= o) at += v;
                }
                at -= sum;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (at < rest && rest <= at + c[e]) {
                        pick[0] = 255 - 8 * lane - e;
                        pick[1] = rest - at;
                    }
                    at += c[e];
                }
            }
            __syncthreads();
            cut |= static_cast<uint32_t>(pick[0]) << shift;
            known |= 255u << shift;
            rest = pick[1];
        }
        // in the order of the pages: thread i looks at `per` in a row
        const int per = (n + THREADS - 1) / THREADS, from = min(tid * per, n), upto = min(from + per, n);
        int above = 0, equal = 0;
        for (int i = from; i < upto; ++i) {
            above += keys[i] > cut;
            equal += keys[i] == cut;
        }
        int above_in = above, equal_in = equal;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, above_in, o), w = __shfl_up_sync(0xffffffffu, equal_in, o);
            if (lane >= o) above_in += v, equal_in += w;
        }
        if (lane == 31) sums[warp] = above_in, sums[WARPS + warp] = equal_in;
        __syncthreads();
        int before = above_in - above, ties = equal_in - equal;
        for (int w = 0; w < warp; ++w) before += sums[w], ties += sums[WARPS + w];
        for (int i = from; i < upto; ++i) {
            const uint32_t key = keys[i];
            if (key > cut || (key == cut && ties < rest)) out[few + before + min(ties, rest)] = id_of(few + i);
            before += key > cut;
            ties += key == cut;
        }
    }
    if (bad) atomicOr(a.status, kDevBadIndex);
}

template <int D, int HC>
cudaError_t launch_select(const Kv4SelectArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    const int smem = static_cast<int>((a.max_blocks + 1) * 4);
    static SmemLimit limit;
    if (smem > 40 * 1024)
        if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(select_kernel<D, HC>), dev.device, smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.T * a.Hkv));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel<D, HC>, a);
}

template <int D>
cudaError_t launch_select(const Kv4SelectArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    const int G = a.Hq / a.Hkv;
    return G == 1 ? launch_select<D, 1>(a, st, dev) : G == 2 ? launch_select<D, 2>(a, st, dev) : launch_select<D, 4>(a, st, dev);
}

}  // namespace

cudaError_t launch_kv4_bounds(const Kv4BoundsArgs &a, int D, cudaStream_t st, const DeviceInfo &) {
    return D == 64 ? launch_bounds<64>(a, st) : D == 128 ? launch_bounds<128>(a, st) : launch_bounds<256>(a, st);
}

cudaError_t launch_kv4_select(const Kv4SelectArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    return D == 64 ? launch_select<64>(a, st, dev) : D == 128 ? launch_select<128>(a, st, dev) : launch_select<256>(a, st, dev);
}

}  // namespace w4
