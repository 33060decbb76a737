// Attention over the paged 4-bit cache for pieces of many new tokens, on the
// tcgen05 tensor cores (kv4_attention in the C header; the streaming form for
// few rows is kv4_attention.cu).
//
// An item is 128 rows (new tokens x the G query heads of one key head) of a
// request; its keys are taken 128 at a time:
//   S = Q K^T          M 128, N 128, K D      -> tensor memory (two buffers)
//   P = exp2(S' - M)   128 threads, one row each, back into tensor memory
//   O += P V           M 128, N D, K 128      P from tensor memory
// Bound: at D = 256 the two products take 2 x 1024 cycles of the tensor pipe
// per 128 x 128 tile.  The same tile costs 2 x 32768 codes to be formed as
// binary16 operands (14 instructions per 8 codes and lane: 1300 cycles of the
// SM's issue slots) and 16384 exponentials with 3 other instructions each (500
// cycles; 1024 of the special-function units), all at the same time.
//
// Items are handed out by a counter in scratch, the longest first (requests
// sorted by length, the last rows of a request first), and announced to the
// roles through a small ring in shared memory.
//
// Roles: warps 0-3 softmax and epilogue (warp w owns the tensor memory lanes
// 32 w ..), warps 4-11 form the operands (a warp per 16-token cache tile,
// 16-byte loads of the codes one step ahead in registers), warp 12 issues the
// products in the order Q K(i+1), P(i) V(i), so that the operands of one are
// formed while the other runs.
//
// Operands.  (code - zero) is exact in binary16; times the scale it is rounded
// once.  The scales of a tile are multiplied by a power of two that brings the
// largest to [2^10, 2^11), so that scales 2^25 apart keep all their bits; the
// power of K's goes into the factor of the scores, that of V's into the
// exponent: P = exp2(x + e - M), and the sum of weights takes P 2^-e.  A row
// of Q enters after a power-of-two scale of its own.  K and V lie in shared
// memory as they come from the cache, a row of 64 dimensions per token and
// group with the 128-byte swizzle: K-major for the first product, MN-major
// (dimensions contiguous) for the second.  A word's codes leave in the order
// 0 4 1 5 2 6 3 7; Q is stored in the same order and the epilogue undoes it.
//
// The running reference M of a row moves only when it would grow by more than
// 2^8; then the softmax warps scale O in tensor memory themselves, between
// two products.  Every wait is bounded; on a timeout the roles still go
// through all their arrivals.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "tc_common.cuh"

namespace w4 {
namespace {

constexpr int ROWS = 128;
constexpr int KEYS = 128;
constexpr int SOFT_THREADS = 128;
constexpr int FORM_WARPS = 8;
constexpr int FORM_THREADS = FORM_WARPS * 32;
constexpr int THREADS = SOFT_THREADS + FORM_THREADS + 32;
constexpr float NONE = -1e30f;       // reference of a row that has seen no key
constexpr int METAS = 3;             // buffers of what the softmax needs to know of a key tile
constexpr int QUEUE = 4;             // items announced ahead
constexpr int SORT_MOST = 512;       // requests that are put in order of length
constexpr int SUB = KEYS * 128;      // bytes of 128 rows x 64 binary16

struct Bars {
    uint64_t qfull, kfull, kfree, vfull, vfree, sfull[2], pfull[2], ifull[QUEUE];
    uint32_t tmem;
    int item[QUEUE];
};
// Of a key tile, from the warps that form it: the exponents of its scales and
// which of its cache tiles there are.
struct alignas(8) Meta {
    unsigned char there[8];
    float k_factor, v_exponent, v_factor;
};

// MN-major operand with the 128-byte swizzle: 64 contiguous elements x 8 rows
// of K per 1024 bytes; the next 64 elements `lead` bytes on, the next 8 rows
// of K 1024 bytes on.
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t saddr, uint32_t lead) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two binary32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\t"
        "mov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ int rows_before(const Kv4AttnArgs &a, int b) {
    return static_cast<int>(min(max(static_cast<int64_t>(a.cu_new[b]), int64_t(0)), a.T));
}

struct Item {
    int b, h, tok0, r0, rows;   // rows [r0, r0 + rows) of the request; its first token
    int base;                   // position of row r is base + r / G
    int end;                    // keys at or past this are seen by no row
    int n, ns, low;             // key tiles: the first ns, then from `low` on
    __device__ __forceinline__ int key0(int i) const { return (i < ns ? i : i - ns + low) * KEYS; }
};

__device__ __forceinline__ bool taken(const Kv4AttnArgs &a, int rows) { return rows > a.rows_above; }

__device__ __forceinline__ Item item_of(const Kv4AttnArgs &a, const int *cum, const int *order, int index, int G) {
    Item it;
    int lo = 0, hi = a.requests;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= index) lo = mid;
        else hi = mid;
    }
    const int local = index - cum[lo];
    lo = order[lo];
    it.b = lo;
    it.tok0 = rows_before(a, lo);
    const int n = rows_before(a, lo + 1) - it.tok0;
    const int total = n * G, blocks = (total + ROWS - 1) / ROWS;
    it.h = local % a.Hkv;
    it.r0 = (blocks - 1 - local / a.Hkv) * ROWS;  // the rows that see most first
    it.rows = min(ROWS, total - it.r0);
    const long long first = static_cast<long long>(a.seq_lens[lo]) - n;
    it.base = static_cast<int>(first);
    const long long cap = static_cast<long long>(a.max_blocks) << a.bs_log2;
    const long long p_lo = first + it.r0 / G, p_hi = first + (it.r0 + it.rows - 1) / G;
    long long end = p_hi + 1 < cap ? p_hi + 1 : cap;
    if (end < 0) end = 0;
    long long low = 0, ns = 0;
    if (a.window > 0) {
        low = p_lo - a.window + 1;
        low = low > 0 ? low / KEYS : 0;
        ns = ((a.sinks < end ? a.sinks : end) + KEYS - 1) / KEYS;
        if (low < ns) low = ns;
    }
    const long long last = (end + KEYS - 1) / KEYS;
    it.end = static_cast<int>(end);
    it.ns = static_cast<int>(ns);
    it.low = static_cast<int>(low);
    // (rows that see nothing take one empty tile and come out as zeros)
    it.n = static_cast<int>(max(ns + (last > low ? last - low : 0), 1ll));
    return it;
}

template <int D>
struct PromptSmem {
    static constexpr int G64 = D / 64;
    static constexpr int q = 0, k = G64 * SUB, v = 2 * G64 * SUB;
    static constexpr int meta = 3 * G64 * SUB;            // [METAS] Meta
    static constexpr int peak = meta + 128;               // [2][FORM_WARPS][2] largest scales of K and V
    static constexpr int bars = peak + 128;
    static constexpr int cum = bars + 256;                // [requests + 1] ints, then [requests] order
};

// 16 bytes of codes of one token (32 dimensions of a group) to 64 bytes of
// binary16 (code - zero) * scale in the swizzled row.
__device__ __forceinline__ void form(const uint4 raw, uint32_t s2, uint32_t z1024, uint32_t z64, unsigned char *row, int x7,
                                     int half) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t lo = w[c], hi = w[c] >> 8;
        uint4 o;
        o.x = mul_f16x2(add_f16x2((lo & 0x000f000fu) | 0x64006400u, z1024), s2);
        o.y = mul_f16x2(fma_f16x2((lo & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, z64), s2);
        o.z = mul_f16x2(add_f16x2((hi & 0x000f000fu) | 0x64006400u, z1024), s2);
        o.w = mul_f16x2(fma_f16x2((hi & 0x00f000f0u) | 0x64006400u, 0x2c002c00u, z64), s2);
        *reinterpret_cast<uint4 *>(row + (((half * 4 + c) ^ x7) << 4)) = o;
    }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1) attn_prompt_kernel(const Kv4AttnArgs a) {
    using L = PromptSmem<D>;
    constexpr int G64 = L::G64;
    constexpr uint32_t COL_S = D, IDESC_QK = idesc_kind_f16(ROWS, KEYS, 0u),
                       IDESC_PV = idesc_kind_f16(ROWS, D, 0u) | (1u << 16);
    extern __shared__ unsigned char smem_raw[];
    unsigned char *const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars &bar = *reinterpret_cast<Bars *>(smem + L::bars);
    int *const cum = reinterpret_cast<int *>(smem + L::cum);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.Hq / a.Hkv;

    if (tid == 0) {
        mbar_init(&bar.qfull, SOFT_THREADS);
        mbar_init(&bar.kfull, FORM_THREADS);
        mbar_init(&bar.vfull, FORM_THREADS);
        mbar_init(&bar.kfree, 1);
        mbar_init(&bar.vfree, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.sfull[i], 1);
            mbar_init(&bar.pfull[i], SOFT_THREADS);
        }
        for (int i = 0; i < QUEUE; ++i) mbar_init(&bar.ifull[i], 1);
        fence_barrier_init();
    }
    if (warp == 12) {
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    pdl_wait();
    int *const order = cum + a.requests + 1;
    // requests by falling length (few enough to compare all pairs), then the
    // items before each
    for (int b = tid; b < a.requests; b += THREADS) {
        int at = b;
        if (a.requests <= SORT_MOST) {
            const int mine = a.seq_lens[b];
            at = 0;
            for (int o = 0; o < a.requests; ++o) {
                const int len = a.seq_lens[o];
                at += len > mine || (len == mine && o < b);
            }
        }
        order[at] = b;
    }
    __syncthreads();
    if (warp == 0) {
        int at = 0;
        for (int b0 = 0; b0 < a.requests; b0 += 32) {
            const int i = b0 + lane;
            int n = 0;
            if (i < a.requests) {
                const int b = order[i];
                const int rows = (rows_before(a, b + 1) - rows_before(a, b)) * G;
                n = taken(a, rows) ? (rows + ROWS - 1) / ROWS * a.Hkv : 0;
            }
            int in = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, in, o);
                if (lane >= o) in += v;
            }
            if (i < a.requests) cum[i + 1] = at + in;
            at += __shfl_sync(0xffffffffu, in, 31);
        }
        if (lane == 0) cum[0] = 0;
    }
    if (a.zero_rest) {  // rows that belong to no request
        const int64_t from = static_cast<int64_t>(rows_before(a, a.requests)) * a.Hq * D / 8, to = a.T * a.Hq * D / 8;
        for (int64_t i = from + static_cast<int64_t>(blockIdx.x) * THREADS + tid; i < to;
             i += static_cast<int64_t>(gridDim.x) * THREADS)
            reinterpret_cast<uint4 *>(a.out)[i] = make_uint4(0, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    const int items = cum[a.requests];
    unsigned int *const counter = reinterpret_cast<unsigned int *>(a.scratch + PROMPT_COUNTERS);
    // the k-th item of this CTA (items or more: there is none)
    auto item_at = [&](int k) -> int {
        mbar_wait(&bar.ifull[k % QUEUE], (k / QUEUE) & 1, a.status);
        return bar.item[k % QUEUE];
    };

    if (warp < 4) {
        // ------------------------------------------------ softmax, epilogue
        const int r = tid;
        const uint32_t t_row = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        unsigned char *const qrow = smem + L::q + r * 128;
        int g = 0;  // key tiles so far, over all items
        const int window = static_cast<int>(min(a.window, int64_t(0x7fffffff)));
        const int sinks = a.window > 0 ? static_cast<int>(min(a.sinks, int64_t(0x7fffffff))) : 0;
        // Q of an item: this thread's row; returns the factor of its scores
        auto build = [&](const Item &it) -> float {
            const bool on = r < it.rows;
            const int row = it.r0 + (on ? r : 0);
            const uint16_t *src = a.q + static_cast<int64_t>(it.tok0 + row / G) * a.q_stride +
                                  static_cast<int64_t>(it.h * G + row % G) * D;
            float big = 0.f;
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src + 8 * c);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u))));
            }
            int kappa = big > 0.f ? 13 - (static_cast<int>(__float_as_uint(big) >> 23) - 127) : 0;
            kappa = min(max(kappa, -110), 110);
            const float up = on ? (a.scale < 0.f ? -pow2(kappa) : pow2(kappa)) : 0.f;
#pragma unroll 8
            for (int c = 0; c < D / 8; ++c) {
                const uint4 v = *reinterpret_cast<const uint4 *>(src + 8 * c);
                const float x0 = __uint_as_float(v.x << 16) * up, x1 = __uint_as_float(v.x & 0xffff0000u) * up;
                const float x2 = __uint_as_float(v.y << 16) * up, x3 = __uint_as_float(v.y & 0xffff0000u) * up;
                const float x4 = __uint_as_float(v.z << 16) * up, x5 = __uint_as_float(v.z & 0xffff0000u) * up;
                const float x6 = __uint_as_float(v.w << 16) * up, x7 = __uint_as_float(v.w & 0xffff0000u) * up;
                *reinterpret_cast<uint4 *>(qrow + (c >> 3) * SUB + (((c & 7) ^ (r & 7)) << 4)) =
                    make_uint4(pack_f16(x0, x4), pack_f16(x1, x5), pack_f16(x2, x6), pack_f16(x3, x7));
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar.qfull);
            return fmaxf(fabsf(a.scale) * 1.4426950408889634f * pow2(-kappa), 1e-37f);
        };
        int k_item = 0;
        Item it;
        float F = 0.f;
        bool have = false;
        auto next_item = [&]() {
            const int index = item_at(k_item++);
            have = index < items;
            if (!have) return;
            it = item_of(a, cum, order, index, G);
            F = build(it);
        };
        next_item();
        while (have) {
            const Item cur = it;
            const float Fr = F;
            float M = NONE, l = 0.f;
            const int p = cur.base + (cur.r0 + min(r, cur.rows - 1)) / G;
            const int p_lo = cur.base + cur.r0 / G, p_hi = cur.base + (cur.r0 + cur.rows - 1) / G;
            for (int i = 0; i < cur.n; ++i, ++g) {
                const int j0 = cur.key0(i);
                const Meta &meta = reinterpret_cast<const Meta *>(smem + L::meta)[g % METAS];
                const uint32_t t_s = t_row + COL_S + (g & 1) * KEYS;
                mbar_wait(&bar.sfull[g & 1], (g >> 1) & 1, a.status);
                tc_fence_after();
                const uint2 there = *reinterpret_cast<const uint2 *>(meta.there);
                const bool free = (there.x & there.y) == 0x01010101u && j0 + KEYS <= p_lo + 1 &&
                                  (window == 0 || p_hi - j0 < window || j0 + KEYS <= sinks);
                const float A = Fr * meta.k_factor, B = meta.v_exponent;
                // 64 keys at a time: scores in, weights out into the columns of
                // scores already read (half as wide)
                float m = M, scaled = 1.f;
                float2 sum = make_float2(0.f, 0.f), sum1 = sum;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[2][32];
                    tmem_ld_32x32b_x32(t_s + 64 * c, x[0]);
                    tmem_ld_32x32b_x32(t_s + 64 * c + 32, x[1]);
                    tmem_ld_wait();
                    if (!free) {
                        // keys from .. upto of these 64 are seen, and those before `first`
                        const int at = j0 + 64 * c;
                        const int upto = min(p + 1, cur.end) - at, from = window == 0 ? 0 : p - window + 1 - at, first = sinks - at;
                        const uint32_t pages = c ? there.y : there.x;
#pragma unroll
                        for (int e = 0; e < 64; ++e) {
                            const bool see = e < upto && (e >= from || e < first) && (pages >> (8 * (e / 16)) & 1u);
                            x[e >> 5][e & 31] = see ? x[e >> 5][e & 31] : 0xff800000u;  // -infinity
                        }
                    }
                    float top[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t *const y = &x[q >> 1][(q & 1) * 16];
                        top[q] = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
#pragma unroll
                        for (int e = 2; e < 16; e += 2) top[q] = max3(top[q], __uint_as_float(y[e]), __uint_as_float(y[e + 1]));
                    }
                    const float mx = fmaf(max3(fmaxf(top[0], top[1]), top[2], top[3]), A, B);
                    if (__any_sync(0xffffffffu, mx > m + 8.f)) {
                        // the reference moves: what this tile has written so far, its
                        // sum, and (below) what earlier tiles left shrink with it
                        const float up = fmaxf(m, ceilf(mx)), f = ex2(m - up);  // whole numbers: f is a power of two
                        m = up;
                        sum.x *= f;
                        sum.y *= f;
                        sum1.x *= f;
                        sum1.y *= f;
                        scaled *= f;
                        if (c > 0) {
                            const uint32_t f2 = pack_f16(f, f);
                            tmem_st_wait();
#pragma unroll 1
                            for (int q = 0; q < 2; ++q) {
                                uint32_t w[16];
                                tmem_ld_32x32b_x16(t_s + 16 * q, w);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) w[e] = mul_f16x2(w[e], f2);
                                tmem_st_32x32b_x16(t_s + 16 * q, w);
                            }
                        }
                    }
                    const float2 A2 = make_float2(A, A), B2 = make_float2(B - m, B - m);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float2 v = fma2(make_float2(__uint_as_float(x[q][e]), __uint_as_float(x[q][e + 1])), A2, B2);
                            v.x = ex2(v.x);
                            v.y = ex2(v.y);
                            if (e & 2) sum1 = add2(sum1, v);
                            else sum = add2(sum, v);
                            w[e / 2] = pack_f16(v.x, v.y);
                        }
                        tmem_st_32x32b_x16(t_s + 32 * c + 16 * q, w);
                    }
                }
                if (__any_sync(0xffffffffu, m != M)) {
                    l *= scaled;
                    if (i > 0) {  // O holds the earlier tiles once their product is done
                        mbar_wait(&bar.vfree, (g - 1) & 1, a.status);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(t_row + 32 * c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scaled);
                            tmem_st_32x32b_x32(t_row + 32 * c, o);
                        }
                    }
                    M = m;
                }
                l = fmaf((sum.x + sum.y) + (sum1.x + sum1.y), meta.v_factor, l);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bar.pfull[g & 1]);
            }
            // every product Q K of this item is done: the next item's Q may be written
            next_item();
            mbar_wait(&bar.vfree, (g - 1) & 1, a.status);
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int row = cur.r0 + r;
            uint16_t *const dst = a.out + (static_cast<int64_t>(cur.tok0 + row / G) * a.Hq + cur.h * G + row % G) * D;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(t_row + 32 * c, o);
                tmem_ld_wait();
                if (r < cur.rows) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
                        const uint32_t *x = o + 8 * e;  // dimensions 0 4 1 5 2 6 3 7
                        const int at[8] = {0, 2, 4, 6, 1, 3, 5, 7};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = static_cast<uint32_t>(f32_to_bf16_bits(__uint_as_float(x[at[2 * k]]) * inv)) |
                                   static_cast<uint32_t>(f32_to_bf16_bits(__uint_as_float(x[at[2 * k + 1]]) * inv)) << 16;
                        *reinterpret_cast<uint4 *>(dst + 32 * c + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc_fence_before();
        }
    } else if (warp < 4 + FORM_WARPS) {
        // ------------------------------------------- operands from the cache
        const int w = warp - 4, token = lane >> 1, half = lane & 1;
        const int row = w * 16 + token;         // key row within the tile
        unsigned char *const krow = smem + L::k + row * 128, *const vrow = smem + L::v + row * 128;
        const int x7 = row & 7;
        const size_t page_bytes = (static_cast<size_t>(a.Hkv) << (a.bs_log2 - 4)) * kv4_tile_bytes(D);
        int g = 0;
        bool bad = false;
        for (int k_item = 0;; ++k_item) {
            const int index = item_at(k_item);
            if (index >= items) break;
            const Item it = item_of(a, cum, order, index, G);
            // this warp's cache tile of key tile i: the page is asked for a step
            // before it is looked at (-1: nothing there)
            const int32_t *const pages = a.block_table + static_cast<int64_t>(it.b) * a.max_blocks;
            auto page_of = [&](int i) -> int {
                if (i >= it.n) return -1;
                const int j = it.key0(i) + w * 16;
                return j < it.end ? pages[j >> a.bs_log2] : -1;
            };
            auto tile_of = [&](int i, int id) -> const unsigned char * {
                if (i >= it.n) return nullptr;
                const int j = it.key0(i) + w * 16;
                if (j >= it.end) return nullptr;
                if (id < 0 || id >= a.num_blocks) {
                    bad = true;
                    return nullptr;
                }
                const int off = ((it.h << (a.bs_log2 - 4)) + ((j & ((1 << a.bs_log2) - 1)) >> 4)) * kv4_tile_bytes(D);
                return a.cache + static_cast<size_t>(id) * page_bytes + off;
            };
            uint4 kraw[G64], vraw[G64];
            uint32_t kpar[G64], vpar[G64];
            auto load_k = [&](const unsigned char *t, bool on) {
#pragma unroll
                for (int i = 0; i < G64; ++i) {
                    kraw[i] = t ? *reinterpret_cast<const uint4 *>(t + (i * 16 + token) * 32 + half * 16) : make_uint4(0, 0, 0, 0);
                    kpar[i] = on ? *reinterpret_cast<const uint32_t *>(t + 16 * D + (i * 16 + token) * 4) : 0u;
                }
            };
            uint32_t vnext[G64];  // V's parameters of the tile whose K is in hand
            auto load_vpar = [&](const unsigned char *t, bool on) {
#pragma unroll
                for (int i = 0; i < G64; ++i)
                    vnext[i] = on ? *reinterpret_cast<const uint32_t *>(t + 17 * D + (i * 16 + token) * 4) : 0u;
            };
            auto load_v = [&](const unsigned char *t, bool on) {
#pragma unroll
                for (int i = 0; i < G64; ++i) {
                    vraw[i] = t ? *reinterpret_cast<const uint4 *>(t + 8 * D + (i * 16 + token) * 32 + half * 16)
                                : make_uint4(0, 0, 0, 0);
                    vpar[i] = on ? *reinterpret_cast<const uint32_t *>(t + 17 * D + (i * 16 + token) * 4) : 0u;
                }
            };
            auto valid = [&](int i, const unsigned char *t) { return t != nullptr && it.key0(i) + row < it.end; };
            // largest scale of this lane's groups, as its bits
            auto peak = [](const uint32_t (&par)[G64]) -> unsigned {
                unsigned top = 0;
#pragma unroll
                for (int i = 0; i < G64; ++i) top = max(top, par[i] & 0x7fffu);
                return top;
            };
            // e with scale < 2^e
            auto exponent = [](unsigned bits) -> int {
                return bits ? static_cast<int>(__float_as_uint(f16_lo(bits)) >> 23) - 126 : 0;
            };
            auto put = [&](const uint4 (&raw)[G64], const uint32_t (&par)[G64], float up, unsigned char *rowp) {
#pragma unroll
                for (int i = 0; i < G64; ++i) {
                    const float s = f16_lo(par[i]) * up, z = f16_hi(par[i]);
                    form(raw[i], pack_f16(s, s), pack_f16(-1024.f - z, -1024.f - z), pack_f16(-64.f - z, -64.f - z),
                         rowp + i * SUB, x7, half);
                }
            };
            float v_up = 0.f, v_up_next = 0.f;
            // K of tile number i (g + i over all items), with what the softmax
            // has to know of the tile
            auto put_k = [&](int i, bool there) {
                const int gi = g + i;
                unsigned *const peaks = reinterpret_cast<unsigned *>(smem + L::peak) + (gi & 1) * 2 * FORM_WARPS;
                const unsigned pk = __reduce_max_sync(0xffffffffu, peak(kpar)), pv = __reduce_max_sync(0xffffffffu, peak(vnext));
                if (lane == 0) {
                    peaks[w] = pk;
                    peaks[FORM_WARPS + w] = pv;
                }
                named_bar_sync(1, FORM_THREADS);
                unsigned tk = 0, tv = 0;
#pragma unroll
                for (int o = 0; o < FORM_WARPS; ++o) {
                    tk = max(tk, peaks[o]);
                    tv = max(tv, peaks[FORM_WARPS + o]);
                }
                const int ek = exponent(tk) - 11, ev = exponent(tv) - 11;
                v_up = v_up_next;
                v_up_next = pow2(-ev);
                if (gi > 0) mbar_wait(&bar.kfree, (gi - 1) & 1, a.status);
                put(kraw, kpar, pow2(-ek), krow);
                if (lane == 0) {
                    Meta &meta = reinterpret_cast<Meta *>(smem + L::meta)[gi % METAS];
                    meta.there[w] = there;
                    if (w == 0) {
                        meta.k_factor = pow2(ek);
                        meta.v_exponent = static_cast<float>(ev);
                        meta.v_factor = pow2(-ev);
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&bar.kfull);
            };
            auto put_v = [&](int i, float up) {
                const int gi = g + i;
                if (gi > 0) mbar_wait(&bar.vfree, (gi - 1) & 1, a.status);
                put(vraw, vpar, up, vrow);
                fence_proxy_async_smem();
                mbar_arrive(&bar.vfull);
            };
            // K(i), then V(i - 1); the loads run one tile ahead
            int id1 = page_of(1);
            const unsigned char *t0 = tile_of(0, page_of(0)), *t1 = nullptr;
            load_k(t0, valid(0, t0));
            load_vpar(t0, valid(0, t0));
            load_v(t0, valid(0, t0));
#pragma unroll 1
            for (int i = 0; i <= it.n; ++i) {
                const int id2 = page_of(i + 2);
                if (i < it.n) {
                    put_k(i, t0 != nullptr);
                    t1 = tile_of(i + 1, id1);
                    load_k(t1, valid(i + 1, t1));
                    load_vpar(t1, valid(i + 1, t1));
                }
                if (i > 0) {
                    put_v(i - 1, i < it.n ? v_up : v_up_next);
                    load_v(t0, valid(i, t0));
                }
                t0 = t1;
                t1 = nullptr;
                id1 = id2;
            }
            g += it.n;
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kDevBadIndex);
    } else {
        // ------------------------------------------------------- products
        const uint32_t qa = smem_u32(smem + L::q), ka = smem_u32(smem + L::k), va = smem_u32(smem + L::v);
        int g = 0;
        auto qk = [&](int gi) {
            mbar_wait(&bar.kfull, gi & 1, a.status);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * SUB + (k & 3) * 32;
                umma_f16_w(tmem + COL_S + (gi & 1) * KEYS, smem_desc_sw128_kmajor(qa + off), smem_desc_sw128_kmajor(ka + off),
                           IDESC_QK, k != 0);
            }
            umma_commit_w(&bar.sfull[gi & 1]);
            umma_commit_w(&bar.kfree);
        };
        auto pv = [&](int gi, bool first) {
            mbar_wait(&bar.pfull[gi & 1], (gi >> 1) & 1, a.status);
            mbar_wait(&bar.vfull, gi & 1, a.status);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < KEYS / 16; ++k)
                umma_f16_tmem_a_w(tmem, tmem + COL_S + (gi & 1) * KEYS + 8 * k, desc_sw128_mn(va + k * 2048, SUB), IDESC_PV,
                                  !(first && k == 0));
            umma_commit_w(&bar.vfree);
        };
        auto announce = [&](int k, int index) {
            if (lane == 0) {
                bar.item[k % QUEUE] = index;
                mbar_arrive(&bar.ifull[k % QUEUE]);
            }
            __syncwarp();
        };
        // the first item is the CTA's number, the others come from the counter;
        // one is fetched ahead.  A slot of the ring is written again four items
        // later, when every role has left it: the softmax is at most an item
        // behind, and the forming warps are ahead.
        int index = static_cast<int>(blockIdx.x);
        announce(0, index);
        for (int k = 0; index < items; ++k) {
            int next = 0;
            if (lane == 0) next = static_cast<int>(gridDim.x + atomicAdd(counter, 1u));
            next = __shfl_sync(0xffffffffu, next, 0);
            announce(k + 1, next);
            const Item it = item_of(a, cum, order, index, G);
            index = next;
            mbar_wait(&bar.qfull, k & 1, a.status);
#pragma unroll 1
            for (int i = 0; i <= it.n; ++i) {
                if (i < it.n) qk(g + i);
                if (i > 0) pv(g + i - 1, i == 1);
            }
            g += it.n;
        }
        // the last CTA to run out of items leaves the counters at zero
        if (lane == 0) {
            __threadfence();
            if (atomicAdd(counter + 1, 1u) == gridDim.x - 1) {
                counter[0] = 0;
                counter[1] = 0;
            }
        }
        // tensor memory is released only when every product has completed
        if (g > 0) mbar_wait(&bar.vfree, (g - 1) & 1, nullptr);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch(const Kv4AttnArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    const int smem = 1024 + PromptSmem<D>::cum + (2 * a.requests + 1) * 4;
    if (smem > dev.max_smem_optin) return cudaErrorNotSupported;
    static SmemLimit limit;
    if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(attn_prompt_kernel<D>), dev.device, smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_prompt_kernel<D>, a);
}

}  // namespace

cudaError_t launch_kv4_prompt(const Kv4AttnArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    if (D == 64) return launch<64>(a, st, dev);
    if (D == 128) return launch<128>(a, st, dev);
    return launch<256>(a, st, dev);
}

}  // namespace w4
