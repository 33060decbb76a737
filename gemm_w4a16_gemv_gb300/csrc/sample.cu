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
// Bound: latency.  A row is read once, by a cluster of up to 8 CTAs that keep
// it in shared memory; what they need of one another (maxima, sums,
// histograms) goes through distributed shared memory, a cluster barrier per
// exchange.  Nothing is sorted but short lists.  Rows past what is resident (at most
// 38 clusters of 8 CTAs, two to an SM by registers and by shared memory) follow in
// waves.  us for 262144 BF16 logits (a bell and 40 that stand out), one row and
// 128 rows: greedy 5.3 and 30, top-k 40 10.2 and 48 (with top-p 0.92 10.7 and
// 50), top-k 300 22.5 and 122, min-p 0.02 6.9 and 35, none of them 10.7 and 58,
// top-p alone 39 and 217 at 0.92, 31 and 166 at 0.5 (the masses and the cut), a
// mixture of settings 11.4 and 102; of binary32 logits the mixture 12.8 and 174.
//
// Small top-k (up to 256): a histogram of the threads' largest logits gives a
// bin that at least k of them reach, so everything kept lies in the bins up
// to it; those few candidates go to one CTA, which sorts them and does the
// rest alone.  Exponentials are taken of the candidates only.  Against the
// general way below: top-k 40 9.7 / 19.0 us (with top-p 10.2 / 34), 256 18.4 /
// 19.8 (18.5 / 35) for one row of 262144; 128 rows 48 / 100 (50 / 193) and 67 /
// 108 (67 / 200); 64 rows of 32000, 256 21.0 / 17.9 (20.6 / 30.6): beyond 256 the
// sort of the candidates costs what is saved.
//
// Otherwise one pass forms all masses, their sum and a histogram over
// (max - l) / T in 1024 bins, 36 to a unit (masses shortened to 15 bits with
// a shift per bin).  The element at which the running mass (or, for a large
// top-k, count) in falling order reaches its goal is then found by exact sums
// above and inside the bin (moved by a bin where the shortening misled), by
// halving the bin's range of keys while more than 128 elements with different
// keys are left, and by comparing all pairs of the rest.  Ties at the cut are
// told apart by index, by the same search that picks the token: sums per
// thread, each owning neighbouring indices.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

#include <cooperative_groups.h>
#include <type_traits>

namespace cg = cooperative_groups;

namespace w4 {
namespace {

typedef unsigned long long u64;

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 1024;
constexpr int LIST = 128;            // candidates at a cut, compared in pairs
constexpr int SMALL_K = 256;         // top-k that goes by candidates
constexpr int CANDIDATES = 1024;
constexpr float UNIT = 1099511627776.f;  // 2^40
constexpr float BINS_PER_UNIT = 36.f;    // 28.4 units: beyond that a mass is 0
constexpr float NO_MASS = 40.f * BINS_PER_UNIT;  // certainly (2^40 exp(-40) < 1 / 2), whatever was rounded

// Unsigned key with the order of the logits (which hold no NaN and no -0).
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

struct Exchange {            // what a CTA's peers write into its shared memory
    u64 sums[2][8][3];
    uint32_t lo[2][8], hi[2][8];
    uint32_t found_key;
    int found_index;
    u64 found_left, found_equal;
};
struct Shared {
    alignas(16) uint32_t hist[BINS];
    Exchange ex;
    u64 part[WARPS][3];
    uint32_t plo[WARPS], phi[WARPS];
    u64 scan[WARPS];
    u64 list_mass[LIST];
    uint32_t list_key[LIST];
    u64 cand[CANDIDATES];    // key << 32 | ~index
    u64 cand_mass[SMALL_K];
    int list_n, cand_n, bin;
};

// Pairs of BF16: the larger of each (a NaN gives way), and -0 as +0.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t plus_zero_bf16x2(uint32_t a) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(0u));
    return d;
}

// A row's masses.  The quotient l / T is the correctly rounded one: for T = 1
// the logit itself; for T well inside the exponent range by Markstein's
// correction (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990): with y the rounded reciprocal and q = l y
// rounded, the remainder l - q T is exact in a fused multiply-add and q + r y
// rounds to the quotient; else, and for a largest quotient of 10^6 or more, whose
// neighbours are no longer close on the scale of the exponential, by division.
enum { MODE_ONE, MODE_FUSED, MODE_DIVIDE };
struct Masses {
    float T, inv, top, half_top, per_half;
    int mode;
    __device__ __forceinline__ Masses(float temperature, float top_l) : T(temperature), half_top(0.5f * top_l) {
        inv = __frcp_rn(T);
        top = __fdiv_rn(top_l, T);
        per_half = fminf(2.f * BINS_PER_UNIT * inv, 2e30f);
        mode = T == 1.f ? MODE_ONE
               : T > 1e-15f && T < 1e15f && fabsf(top_l) < 1e15f && fabsf(top) < 1e6f ? MODE_FUSED : MODE_DIVIDE;
    }
    // (max - l) / T in bins, not rounded to one; rises as l falls.  From half the
    // difference, which no two finite logits take past binary32's range.
    __device__ __forceinline__ float depth(float l) const { return fmaf(-0.5f, l, half_top) * per_half; }
    // max itself, but for the last bit of a subnormal
    __device__ __forceinline__ float largest() const { return 2.f * half_top; }
    // mass before rounding
    template <int MODE>
    __device__ __forceinline__ float scaled(float l) const {
        float x = l;
        if (MODE == MODE_FUSED) {
            if (!(depth(l) < NO_MASS)) return 0.f;  // (-infinity, or a quotient out of range)
            const float q = l * inv;
            x = fmaf(fmaf(-q, T, l), inv, q);
        } else if (MODE == MODE_DIVIDE) {
            // (quotients may lie so far apart that ones of different depth are equal)
            const float below = __fsub_rn(__fdiv_rn(l, T), top);
            return below > -40.f ? expf(below) * UNIT : 0.f;
        }
        return expf(__fsub_rn(x, top)) * UNIT;
    }
    // The whole number nearest to t <= 2^40 (ties to even) as hi 2^20 + lo: the
    // part above 2^20 cut off by adding 2^23 rounded down, the rest (exact)
    // rounded by adding 2^23.  Sums of 64 of either part fit 32 bits.
    static __device__ __forceinline__ void whole(float t, uint32_t &hi, uint32_t &lo) {
        const float h = __fadd_rd(t * 9.5367431640625e-7f, 8388608.f);  // 2^-20
        hi = __float_as_uint(h) - 0x4b000000u;
        lo = __float_as_uint(__fadd_rn(fmaf(__fsub_rn(h, 8388608.f), -1048576.f, t), 8388608.f)) - 0x4b000000u;
    }
    static __device__ __forceinline__ u64 whole(float t) {
        uint32_t hi, lo;
        whole(t, hi, lo);
        return (static_cast<u64>(hi) << 20) + lo;
    }
    template <int MODE>
    __device__ __forceinline__ u64 mass(float l) const {
        return whole(scaled<MODE>(l));
    }
    __device__ __forceinline__ u64 of(float l) const {
        return mode == MODE_ONE ? mass<MODE_ONE>(l) : mode == MODE_FUSED ? mass<MODE_FUSED>(l) : mass<MODE_DIVIDE>(l);
    }
};

// EPT neighbouring logits per thread: element e of the CTA's slice belongs to
// thread e / EPT.  They are read in units of 16 bytes (8 BF16 or 4 binary32),
// the threads of a warp rotated against each other so that they fall into
// different banks, and a unit's exponentials are formed together, without
// branches between them.
template <bool BF16, int EPT>
__global__ void __launch_bounds__(THREADS) sample_kernel(const SampleArgs a) {
    constexpr int N = BF16 ? 8 : 4, UNITS = EPT / N;  // logits of a unit, units of a thread
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    uint32_t *const row = reinterpret_cast<uint32_t *>(smem + (sizeof(Shared) + 127) / 128 * 128);
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int64_t r = blockIdx.x / CS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int V = a.vocab;
    const int slice = rank * EPT * THREADS;           // first index of the CTA
    const int rot = UNITS >= 8 ? lane : (lane * UNITS) >> 3;
    const uint4 *const own = reinterpret_cast<const uint4 *>(row) + tid * UNITS;
    if (tid == 0) sh.list_n = sh.cand_n = 0;
    for (int i = tid; i < BINS; i += THREADS) sh.hist[i] = 0;
    // every CTA of the cluster has started (waited for before the first write
    // into another's shared memory)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_launch_dependents();
    pdl_wait();
    // the row's settings, on their way beside the row
    const float T = a.temperature ? a.temperature[r] : 1.f, p = a.top_p ? a.top_p[r] : 1.f, u = a.u[r];
    const float wanted = a.min_p ? a.min_p[r] : 0.f, min_p = wanted > 0.f ? fminf(wanted, 1.f) : 0.f;
    const int k = a.top_k ? a.top_k[r] : 0;

    // ---- the row into shared memory, once; NaN as -infinity, -0 as +0
    float best = -INFINITY;
    {
        uint32_t best2 = 0xff80ff80u;  // of a pair
        auto clean = [&](uint32_t w) -> uint32_t {
            if (BF16) {
                w = plus_zero_bf16x2(max_bf16x2(w, 0xff80ff80u));
                best2 = max_bf16x2(best2, w);
                return w;
            }
            float v = __uint_as_float(w);
            v = v != v ? -INFINITY : v + 0.f;
            best = fmaxf(best, v);
            return __float_as_uint(v);
        };
        constexpr int PER = BF16 ? 8 : 4;  // logits of 16 bytes
        const unsigned char *from = static_cast<const unsigned char *>(a.logits) +
                                    (r * a.row_stride + slice) * (BF16 ? 2 : 4);
        const bool vec = (reinterpret_cast<uintptr_t>(from) & 15u) == 0;
        constexpr int COUNT = EPT / PER, BATCH = COUNT < 8 ? COUNT : 8;  // vectors a thread, and at a time
        const bool inside = vec && V - slice >= EPT * THREADS;
#pragma unroll 1
        for (int i0 = 0; i0 < COUNT; i0 += BATCH) {
            uint4 w[BATCH];
            if (inside) {
#pragma unroll
                for (int q = 0; q < BATCH; ++q)
                    w[q] = *reinterpret_cast<const uint4 *>(from + 16 * static_cast<int64_t>((i0 + q) * THREADS + tid));
            } else {
#pragma unroll
                for (int q = 0; q < BATCH; ++q) {
                    const int first = ((i0 + q) * THREADS + tid) * PER, left = V - slice - first;  // logits from here on
                    uint32_t x[4];
                    if (vec && left >= PER) {
                        w[q] = *reinterpret_cast<const uint4 *>(from + 16 * static_cast<int64_t>((i0 + q) * THREADS + tid));
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < PER; ++e) {
                        if (BF16) {
                            const uint32_t h = e < left ? reinterpret_cast<const uint16_t *>(from)[first + e] : 0xff80u;
                            x[e / 2] = e & 1 ? x[e / 2] | h << 16 : h;
                        } else x[e & 3] = e < left ? reinterpret_cast<const uint32_t *>(from)[first + e] : 0xff800000u;
                    }
                    w[q] = make_uint4(x[0], x[1], x[2], x[3]);
                }
            }
#pragma unroll
            for (int q = 0; q < BATCH; ++q) {
                reinterpret_cast<uint4 *>(row)[(i0 + q) * THREADS + tid] =
                    make_uint4(clean(w[q].x), clean(w[q].y), clean(w[q].z), clean(w[q].w));
            }
        }
        if (BF16) best = fmaxf(__uint_as_float(best2 << 16), __uint_as_float(best2 & 0xffff0000u));
    }

    // f(N logits, element of the first) of every own unit, in no particular order
    auto each = [&](auto f) {
#pragma unroll 1
        for (int j = 0; j < UNITS; ++j) {
            const int q = (j + rot) & (UNITS - 1);
            const uint4 w = own[q];
            float l[N];
            if constexpr (BF16) {
                l[0] = __uint_as_float(w.x << 16), l[1] = __uint_as_float(w.x & 0xffff0000u);
                l[2] = __uint_as_float(w.y << 16), l[3] = __uint_as_float(w.y & 0xffff0000u);
                l[4] = __uint_as_float(w.z << 16), l[5] = __uint_as_float(w.z & 0xffff0000u);
                l[6] = __uint_as_float(w.w << 16), l[7] = __uint_as_float(w.w & 0xffff0000u);
            } else {
                l[0] = __uint_as_float(w.x), l[1] = __uint_as_float(w.y);
                l[2] = __uint_as_float(w.z), l[3] = __uint_as_float(w.w);
            }
            f(l, tid * EPT + q * N);
        }
    };
    auto logit = [&](int e) -> float {  // element e of the slice
        if (BF16) return __uint_as_float(e & 1 ? row[e >> 1] & 0xffff0000u : row[e >> 1] << 16);
        return __uint_as_float(row[e]);
    };

    // ---- COUNT sums, and with KEYS a least and a largest key, over the cluster
    int turn = 0;
    auto reduce = [&](auto count, auto keys, u64 *sum, uint32_t &lo, uint32_t &hi) {
        constexpr int COUNT = count.value;
        constexpr bool KEYS = keys.value;
        auto warps = [&](u64 *x, uint32_t &l, uint32_t &h) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < COUNT; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
            if (KEYS) {
                l = __reduce_min_sync(0xffffffffu, l);
                h = __reduce_max_sync(0xffffffffu, h);
            }
        };
        warps(sum, lo, hi);
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < COUNT; ++i) sh.part[warp][i] = sum[i];
            if (KEYS) {
                sh.plo[warp] = lo;
                sh.phi[warp] = hi;
            }
        }
        __syncthreads();
        if (warp == 0) {
            const int from = lane & (WARPS - 1);
#pragma unroll
            for (int i = 0; i < COUNT; ++i) sum[i] = lane < WARPS ? sh.part[from][i] : 0;
            if (KEYS) {
                lo = sh.plo[from];
                hi = sh.phi[from];
            }
            warps(sum, lo, hi);
            if (lane < CS) {
                Exchange &to = cluster.map_shared_rank(&sh, lane)->ex;
#pragma unroll
                for (int i = 0; i < COUNT; ++i) to.sums[turn][rank][i] = sum[i];
                if (KEYS) {
                    to.lo[turn][rank] = lo;
                    to.hi[turn][rank] = hi;
                }
            }
        }
        cluster.sync();
#pragma unroll
        for (int i = 0; i < COUNT; ++i) sum[i] = 0;
        if (KEYS) {
            lo = 0xffffffffu;
            hi = 0;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < CS) {
#pragma unroll
                for (int i = 0; i < COUNT; ++i) sum[i] += sh.ex.sums[turn][c][i];
                if (KEYS) {
                    lo = min(lo, sh.ex.lo[turn][c]);
                    hi = max(hi, sh.ex.hi[turn][c]);
                }
            }
        turn ^= 1;
    };
    typedef std::integral_constant<int, 0> none;
    typedef std::integral_constant<int, 1> one;
    typedef std::integral_constant<int, 2> two;
    typedef std::integral_constant<int, 3> three;
    auto reduce_sum = [&](u64 &v) {
        uint32_t lo = 0, hi = 0;
        reduce(one(), none(), &v, lo, hi);
    };
    // Inclusive sum over the CTA's threads.
    auto block_scan = [&](u64 v) -> u64 {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        __syncthreads();
        if (lane == 31) sh.scan[warp] = v;
        __syncthreads();
        for (int k = 0; k < warp; ++k) v += sh.scan[k];
        return v;
    };
    // The first index at which the running sum of the threads' `mine` exceeds
    // goal(total); inside the thread that holds it the warp looks at its
    // elements, value(element of the slice), together.
    auto locate = [&](u64 mine, auto value, auto goal_of, auto hit) {
        u64 all = mine;
        const int t = turn;
        reduce_sum(all);
        const u64 goal = goal_of(all);
        u64 before = 0;
        for (int c = 0; c < rank; ++c) before += sh.ex.sums[t][c][0];
        if (goal < before || goal >= before + sh.ex.sums[t][rank][0]) return;
        const u64 upto = before + block_scan(mine);
        const unsigned holds = __ballot_sync(0xffffffffu, goal < upto && goal >= upto - mine);
        if (holds == 0) return;
        const int src = __ffs(holds) - 1;
        constexpr int PER = EPT >= 32 ? EPT / 32 : 1;
        const int e0 = (warp * 32 + src) * EPT + lane * PER;
        u64 v[PER], sum = 0;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            v[q] = lane * PER < EPT ? value(e0 + q) : 0ull;
            sum += v[q];
        }
        u64 at = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 x = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += x;
        }
        at += __shfl_sync(0xffffffffu, upto - mine, src) - sum;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            if (goal >= at && goal < at + v[q]) hit(slice + e0 + q);
            at += v[q];
        }
    };

    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

    // ---- the largest logit
    float top_l;
    {
        uint32_t lo = 0, hi = key_of(best);
        reduce(none(), one(), nullptr, lo, hi);
        top_l = logit_of(hi);
    }
    if (top_l == -INFINITY) {  // nothing to choose from
        if (rank == 0 && tid == 0) a.tokens[r] = -1;
        return;                // every CTA of the cluster is past its last access to the others
    }
    const Masses mass(T, top_l);
    if (!(T > 0.f) || !(fabsf(mass.top) < INFINITY)) {
        // the largest logit: the first index that holds it
        u64 n = 0;
        each([&](const float(&l)[N], int) {
#pragma unroll
            for (int e = 0; e < N; ++e) n += l[e] == top_l;
        });
        locate(n, [&](int e) -> u64 { return logit(e) == top_l; }, [](u64) -> u64 { return 0; },
               [&](int index) { a.tokens[r] = index; });
        return;
    }
    auto bin_of = [&](float v) -> int { return static_cast<int>(fminf(mass.depth(v), static_cast<float>(BINS - 1))); };
    // f(MODE) for the row's mode
    auto in_mode = [&](auto f) {
        if (mass.mode == MODE_ONE) f(std::integral_constant<int, MODE_ONE>());
        else if (mass.mode == MODE_FUSED) f(std::integral_constant<int, MODE_FUSED>());
        else f(std::integral_constant<int, MODE_DIVIDE>());
    };
    // masses of bin b are below 2^(40 - 0.04 b): shortened to 15 bits
    auto shift_of = [](int b) -> int { return max(0, 26 - static_cast<int>(static_cast<float>(b) * 0.0400748f)); };
    // min_p 2^40, rounded up to a whole mass (NaN: off)
    const double min_mass = static_cast<double>(min_p) * static_cast<double>(UNIT);
    const u64 least = min_mass > 0. ? static_cast<u64>(__double2ll_ru(min_mass)) : 0ull;
    auto share_of = [](u64 total, float x) -> u64 {  // trunc(x of total), x in [0, 1]
        return static_cast<u64>(__double2ll_rz(static_cast<double>(total) * static_cast<double>(x)));
    };
    auto draw = [&](u64 total) -> u64 {
        const u64 g = u > 0.f ? share_of(total, fminf(u, 1.f)) : 0ull;
        return g < total ? g : total - 1;
    };
    // The bin at which the running sum of the cluster's histograms reaches
    // goal: the same in every CTA.  If none does: the last bin, or where sums
    // are shortened the last one with anything.
    auto goal_bin = [&](u64 goal, bool shortened) -> int {
        // four bins a thread (16 bytes of each CTA's histogram), half the threads
        constexpr int PER = 4;
        u64 part[PER] = {}, sum = 0;
        if (tid < BINS / PER) {
            uint4 v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[c] = c < CS ? reinterpret_cast<const uint4 *>(cluster.map_shared_rank(&sh, c)->hist)[tid] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                part[0] += v[c].x;
                part[1] += v[c].y;
                part[2] += v[c].z;
                part[3] += v[c].w;
            }
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                if (shortened) part[q] <<= shift_of(tid * PER + q);
                sum += part[q];
            }
        }
        if (tid == 0) sh.bin = -1;
        u64 upto = block_scan(sum);   // (its barriers order the line above)
        u64 at = upto - sum;
        int last = shortened ? -1 : BINS - 1;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            if (at < goal && at + part[q] >= goal) sh.bin = tid * PER + q;
            at += part[q];
            if (shortened && part[q]) last = tid * PER + q;
        }
        __syncthreads();
        if (sh.bin < 0) {
            __syncthreads();
            if (last >= 0) atomicMax(&sh.bin, last);
            __syncthreads();
        }
        const int bin = max(sh.bin, 0);
        __syncthreads();
        return bin;
    };

    // ---- small top-k: the candidates to the first CTA
    if (k > 0 && k <= SMALL_K && k < V) {
        if (best > -INFINITY) atomicAdd(&sh.hist[bin_of(best)], 1u);
        cluster.sync();
        const float deepest = static_cast<float>(goal_bin(static_cast<u64>(k), false) + 1);
        const bool all = deepest >= static_cast<float>(BINS);
        Shared *const head = cluster.map_shared_rank(&sh, 0);
        // (a bound that no logit as deep as that lies below, whatever was rounded:
        // most units have none above it)
        const float reach = mass.largest() - 2.f * deepest / mass.per_half * 1.0001f;
        const float bound = all ? -INFINITY : reach - 1e-5f * (fabsf(reach) + fabsf(mass.largest()));
        each([&](const float(&l)[N], int e0) {
            float most = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
            if (N == 8) most = fmaxf(most, fmaxf(fmaxf(l[N - 4], l[N - 3]), fmaxf(l[N - 2], l[N - 1])));
            if (most < bound) return;
            unsigned in = 0;
#pragma unroll
            for (int e = 0; e < N; ++e)
                in |= static_cast<unsigned>((mass.depth(l[e]) < deepest || all) && l[e] > -INFINITY) << e;
            if (in == 0) return;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (in >> e & 1u) {
                    const int at = atomicAdd(&head->cand_n, 1);
                    if (at < CANDIDATES)
                        head->cand[at] = static_cast<u64>(key_of(l[e])) << 32 | (0xffffffffu - static_cast<uint32_t>(slice + e0 + e));
                }
        });
        cluster.sync();
        const int n = *static_cast<volatile int *>(&head->cand_n);
        // (nobody may leave, or clear the count, while another still reads it)
        cluster.sync();
        if (n <= CANDIDATES) {
            if (rank != 0) return;
            // falling order of key, rising order of index
            if (n <= THREADS / 2) {  // every candidate counts those ahead of it
                const u64 own_cand = tid < n ? sh.cand[tid] : 0;
                int ahead = 0;
#pragma unroll 4
                for (int j = 0; j < n; ++j) ahead += sh.cand[j] > own_cand;
                __syncthreads();
                if (tid < n) sh.cand[ahead] = own_cand;
                __syncthreads();
            } else {
                int size = 2;
                while (size < n) size <<= 1;
                for (int i = n + tid; i < size; i += THREADS) sh.cand[i] = 0;
                __syncthreads();
                for (int s = 2; s <= size; s <<= 1)
                    for (int d = s >> 1; d; d >>= 1) {
                        for (int i = tid; i < size / 2; i += THREADS) {
                            const int x = 2 * i - (i & (d - 1)), y = x + d;
                            const u64 A = sh.cand[x], B = sh.cand[y];
                            if ((A < B) == ((x & s) == 0)) {
                                sh.cand[x] = B;
                                sh.cand[y] = A;
                            }
                        }
                        __syncthreads();
                    }
            }
            const int top = min(k, n);
            u64 m = 0;
            if (tid < top) m = mass.of(logit_of(static_cast<uint32_t>(sh.cand[tid] >> 32)));
            const u64 upto = block_scan(m);
            if (tid == THREADS - 1) sh.ex.found_left = upto;
            __syncthreads();
            if (p < 1.f) {
                const u64 goal = max(share_of(sh.ex.found_left, p > 0.f ? p : 0.f), 1ull);
                if (upto - m >= goal) m = 0;
            }
            if (m < least) m = 0;
            if (tid < top) sh.cand_mass[tid] = m;
            const u64 kept = block_scan(m);
            if (tid == THREADS - 1) sh.ex.found_equal = kept;
            __syncthreads();
            if (m) {
                const u64 goal = draw(sh.ex.found_equal);
                const uint32_t me = static_cast<uint32_t>(sh.cand[tid]);  // falls as the index rises
                u64 before = 0;
#pragma unroll 4
                for (int j = 0; j < top; ++j)
                    if (static_cast<uint32_t>(sh.cand[j]) > me) before += sh.cand_mass[j];
                if (goal >= before && goal < before + m) a.tokens[r] = static_cast<int>(0xffffffffu - me);
            }
            return;
        }
        for (int i = tid; i < BINS; i += THREADS) sh.hist[i] = 0;  // too many: the general way
        __syncthreads();
    }

    // The logit at which the running count or mass of the logits not below
    // floor_l, in falling order, reaches `goal`; what of the goal is left there
    // and how many elements are equal to it.  The histogram is in place.
    auto select = [&](float floor_l, bool by_mass, u64 goal, float &cut, u64 &left, u64 &equal) {
        int bin = goal_bin(goal, by_mass);
        auto measure = [&](float l) -> u64 { return by_mass ? mass.of(l) : 1ull; };
        u64 found[3], &above = found[0], &inside = found[1], &count = found[2];
        uint32_t klo, khi;
        while (true) {
            above = inside = count = 0;
            klo = 0xffffffffu, khi = 0;
            // the last bin has no lower end: a finite logit may lie infinitely deep
            // (no comparison with NaN holds)
            const float upper = static_cast<float>(bin), lower = bin == BINS - 1 ? NAN : static_cast<float>(bin + 1);
            in_mode([&](auto mode) {
                uint32_t his = 0, los = 0;
                each([&](const float(&l)[N], int) {
                    unsigned in = 0;
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float d = mass.depth(l[e]);
                        const bool here = !(d >= lower) && l[e] >= floor_l;
                        in |= static_cast<unsigned>(here && d >= upper) << e;
                        if (by_mass) {
                            uint32_t hi, lo;
                            Masses::whole(here && d < upper ? mass.template scaled<mode.value>(l[e]) : 0.f, hi, lo);
                            his += hi;
                            los += lo;
                        } else los += here && d < upper;
                    }
                    if (in) {
#pragma unroll
                        for (int e = 0; e < N; ++e)
                            if ((in >> e & 1u) && l[e] > -INFINITY) {
                                inside += by_mass ? mass.template mass<mode.value>(l[e]) : 1ull;
                                ++count;
                                klo = min(klo, key_of(l[e]));
                                khi = max(khi, key_of(l[e]));
                            }
                    }
                });
                above += (static_cast<u64>(his) << 20) + los;
            });
            reduce(three(), one(), found, klo, khi);
            if (above >= goal && bin > 0) --bin;
            else if (above + inside < goal && bin < BINS - 1) ++bin;
            else break;
        }
        // BF16: a count per distinct key of the bin says everything (equal keys
        // have equal masses)
        if (BF16 && count > LIST && klo < khi && (khi - klo) >> 16 < static_cast<uint32_t>(BINS) &&
            (khi ^ klo) >> 31 == 0) {  // (of one sign: the keys are 2^16 apart)
            // (every CTA has read the first histogram: the sums above were exchanged since)
            for (int i = tid; i < BINS; i += THREADS) sh.hist[i] = 0;
            __syncthreads();
            const float flo = fmaxf(logit_of(klo), floor_l), fhi = logit_of(khi);
            each([&](const float(&l)[N], int) {
                unsigned in = 0;
#pragma unroll
                for (int e = 0; e < N; ++e) in |= static_cast<unsigned>(l[e] >= flo && l[e] <= fhi) << e;
                if (in) {
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (in >> e & 1u) atomicAdd(&sh.hist[(khi - key_of(l[e])) >> 16], 1u);
                }
            });
            cluster.sync();
            u64 sum = 0, part[4] = {};
            uint32_t counts[4] = {};
            if (tid < BINS / 4) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c < CS) {
                        const uint4 v = reinterpret_cast<const uint4 *>(cluster.map_shared_rank(&sh, c)->hist)[tid];
                        counts[0] += v.x;
                        counts[1] += v.y;
                        counts[2] += v.z;
                        counts[3] += v.w;
                    }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (counts[q]) part[q] = counts[q] * measure(logit_of(khi - (static_cast<uint32_t>(tid * 4 + q) << 16)));
                    sum += part[q];
                }
            }
            u64 at = above + block_scan(sum) - sum;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (at < goal && at + part[q] >= goal) {
                    sh.ex.found_key = khi - (static_cast<uint32_t>(tid * 4 + q) << 16);
                    sh.ex.found_left = goal - at;
                    sh.ex.found_equal = counts[q];
                }
                at += part[q];
            }
            cluster.sync();  // (the histogram may be written again, and nobody is still reading)
            cut = logit_of(sh.ex.found_key);
            left = sh.ex.found_left;
            equal = sh.ex.found_equal;
            return;
        }
        while (count > LIST && klo < khi) {
            const uint32_t mid = klo + (khi - klo) / 2;
            u64 part[2] = {0, 0}, &sum = part[0], &n = part[1];
            uint32_t up = 0xffffffffu, down = 0;
            const float flo = fmaxf(logit_of(klo), floor_l), fhi = logit_of(khi);
            each([&](const float(&l)[N], int) {
                unsigned in = 0;
#pragma unroll
                for (int e = 0; e < N; ++e) in |= static_cast<unsigned>(l[e] >= flo && l[e] <= fhi) << e;
                if (in) {
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (in >> e & 1u) {
                            const uint32_t key = key_of(l[e]);
                            if (key > mid) {
                                sum += measure(l[e]);
                                ++n;
                                up = min(up, key);
                            } else down = max(down, key);
                        }
                }
            });
            reduce(two(), one(), part, up, down);
            if (above + sum >= goal) {
                klo = up;
                count = n;
            } else {
                above += sum;
                khi = down;
                count -= n;
            }
        }
        if (klo >= khi) {
            cut = logit_of(klo);
            left = goal - above;
            equal = count;
            return;
        }
        Shared *const head = cluster.map_shared_rank(&sh, 0);
        const float flo = fmaxf(logit_of(klo), floor_l), fhi = logit_of(khi);
        each([&](const float(&l)[N], int) {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (l[e] >= flo && l[e] <= fhi) {
                    const int at = atomicAdd(&head->list_n, 1);
                    if (at < LIST) {
                        head->list_key[at] = key_of(l[e]);
                        head->list_mass[at] = measure(l[e]);
                    }
                }
        });
        cluster.sync();
        if (rank == 0) {
            const int n = min(sh.list_n, LIST);
            if (tid < n) {
                const uint32_t key = sh.list_key[tid];
                const u64 m = sh.list_mass[tid];
                u64 over = above, same = 0;
                bool first = true;
                for (int j = 0; j < n; ++j) {
                    const uint32_t kj = sh.list_key[j];
                    if (kj > key) over += sh.list_mass[j];
                    if (kj == key) {
                        ++same;
                        if (j < tid) first = false;
                    }
                }
                if (first && over < goal && goal <= over + same * m)
                    for (int c = 0; c < CS; ++c) {
                        Exchange &to = cluster.map_shared_rank(&sh, c)->ex;
                        to.found_key = key;
                        to.found_left = goal - over;
                        to.found_equal = same;
                    }
            }
            __syncthreads();
            if (tid == 0) sh.list_n = 0;
        }
        cluster.sync();
        cut = logit_of(sh.ex.found_key);
        left = sh.ex.found_left;
        equal = sh.ex.found_equal;
    };

    // ---- what is kept: logits above `cut`, and those equal to it among the first `ties` by index
    float cut = -INFINITY;
    u64 ties = ~0ull, equal = 0;
    if (k > 0 && k < V) {
        u64 finite = 0;
        each([&](const float(&l)[N], int) {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (l[e] > -INFINITY) {
                    ++finite;
                    atomicAdd(&sh.hist[bin_of(l[e])], 1u);
                }
        });
        reduce_sum(finite);
        if (static_cast<u64>(k) < finite) select(-INFINITY, false, static_cast<u64>(k), cut, ties, equal);
        cluster.sync();  // the others have read this histogram
        for (int i = tid; i < BINS; i += THREADS) sh.hist[i] = 0;
        __syncthreads();
    }
    if (p < 1.f) {
        // the masses that are left: their sum and histogram
        u64 sum = 0;
        in_mode([&](auto mode) {
            uint32_t his = 0, los = 0;
            each([&](const float(&l)[N], int) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float d = mass.depth(l[e]);
                    const float t = l[e] >= cut ? mass.template scaled<mode.value>(l[e]) : 0.f;
                    uint32_t hi, lo;
                    Masses::whole(l[e] > cut ? t : 0.f, hi, lo);
                    his += hi;
                    los += lo;
                    const int b = static_cast<int>(fminf(d, static_cast<float>(BINS - 1)));
                    const uint32_t v = static_cast<uint32_t>(t * __uint_as_float(static_cast<uint32_t>(127 - shift_of(b)) << 23));
                    if (v) atomicAdd(&sh.hist[b], v);
                }
            });
            sum += (static_cast<u64>(his) << 20) + los;
        });
        reduce_sum(sum);
        if (cut > -INFINITY) sum += (ties < equal ? ties : equal) * mass.of(cut);
        const u64 goal = max(share_of(sum, p > 0.f ? p : 0.f), 1ull);
        float cut2;
        u64 left, equal2;
        select(cut, true, goal, cut2, left, equal2);
        const u64 m = mass.of(cut2);
        const u64 n = m ? (left + m - 1) / m : 1ull;
        ties = cut2 == cut && ties < n ? ties : n;
        cut = cut2;
        equal = equal2;
    }
    int last_tie = 0x7fffffff;  // index of the last kept one of the equals
    if (cut > -INFINITY && ties < equal) {
        const u64 n = ties;
        u64 mine = 0;
        each([&](const float(&l)[N], int) {
#pragma unroll
            for (int e = 0; e < N; ++e) mine += l[e] == cut;
        });
        locate(mine, [&](int e) -> u64 { return logit(e) == cut; }, [&](u64) -> u64 { return n - 1; },
               [&](int index) {
                   for (int c = 0; c < CS; ++c) cluster.map_shared_rank(&sh, c)->ex.found_index = index;
               });
        cluster.sync();
        last_tie = sh.ex.found_index;
    }
    // logits below this have a mass under min_p's (or none): no exponential is
    // taken of them.  A little lower than the bound itself, which is rounded.
    float floor_l = cut;
    if (least > 0) {
        const float reach = -logf(fmaxf(min_p, 1e-30f)) * T;  // max - l at the bound
        const float lowest = mass.largest() - reach * 1.0001f - 1e-4f * (fabsf(mass.largest()) + T) - 1e-37f;
        floor_l = fmaxf(floor_l, lowest);
    }
    auto kept = [&](float l, int index) -> u64 {
        if (l < floor_l || (l == cut && index > last_tie)) return 0ull;
        const u64 m = mass.of(l);
        return m < least ? 0ull : m;
    };
    // the least scaled mass that rounds to `least`: least - 1/2 if that ties to
    // it, or the next above; from 2^23 on scaled masses are whole themselves
    const float least_t = least == 0             ? -1.f
                          : least < (1ull << 23) ? __uint_as_float(__float_as_uint(static_cast<float>(least) - 0.5f) + (least & 1u))
                                                 : __ull2float_ru(least);
    u64 mine = 0;
    in_mode([&](auto mode) {
        uint32_t his = 0, los = 0;
        each([&](const float(&l)[N], int e0) {
            // (l > -infinity too: cut and floor_l may be that)
            bool any = false;
#pragma unroll
            for (int e = 0; e < N; ++e) any |= l[e] >= floor_l;
            if (!any) return;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const bool in = l[e] >= floor_l && !(l[e] == cut && slice + e0 + e > last_tie);
                const float t = in ? mass.template scaled<mode.value>(l[e]) : 0.f;
                uint32_t hi, lo;
                Masses::whole(t >= least_t ? t : 0.f, hi, lo);
                his += hi;
                los += lo;
            }
        });
        mine += (static_cast<u64>(his) << 20) + los;
    });
    locate(mine, [&](int e) -> u64 { return kept(logit(e), slice + e); }, draw,
           [&](int index) { a.tokens[r] = index; });
}

template <bool BF16, int EPT>
cudaError_t launch_rows(const SampleArgs &a, int cs, cudaStream_t st, const DeviceInfo &dev) {
    const int smem = static_cast<int>((sizeof(Shared) + 127) / 128 * 128) + EPT * THREADS * (BF16 ? 2 : 4);
    static SmemLimit limit;
    if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(sample_kernel<BF16, EPT>), dev.device, smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * cs));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned>(cs);
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, sample_kernel<BF16, EPT>, a);
}

template <bool BF16>
cudaError_t launch_typed(const SampleArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    auto cluster = [&](int ept) {
        int cs = 1;
        while (cs * ept * THREADS < a.vocab) cs *= 2;
        return cs;
    };
    // A vocabulary that 8 CTAs hold at 16 logits a thread is spread thinner over
    // more SMs, unless rows alone are enough.  16 against 64, us, BF16:
    //     rows              1        16        64       128       256
    //     4096 logits    9.7/14.3  13/24     17/29     18/32     22/40
    //     32000         10.1/12.4  20/37     23/39     33/46     51/52
    //     65536         10.5/12.1  23/37     35/45     55/52     98/67
    if (cluster(16) <= 8 && a.rows * cluster(16) <= 6 * dev.num_sms) return launch_rows<BF16, 16>(a, cluster(16), st, dev);
    return launch_rows<BF16, 64>(a, cluster(64), st, dev);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    return a.bf16 ? launch_typed<true>(a, st, dev) : launch_typed<false>(a, st, dev);
}

}  // namespace w4
