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
// exchange.  Nothing is sorted but short lists.
//
// Small top-k (up to 256): a histogram of the threads' largest logits gives a
// bin that at least k of them reach, so everything kept lies in the bins up
// to it; those few candidates go to one CTA, which sorts them and does the
// rest alone.  Exponentials are taken of the candidates only.
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
    Exchange ex;
    uint32_t hist[BINS];
    u64 part[WARPS][3];
    uint32_t plo[WARPS], phi[WARPS];
    u64 scan[WARPS];
    u64 list_mass[LIST];
    uint32_t list_key[LIST];
    u64 cand[CANDIDATES];    // key << 32 | ~index
    u64 cand_mass[SMALL_K];
    int list_n, cand_n, bin;
};

// A row's exponentials.  The quotient l / T is the correctly rounded one: for
// T and 1 / T well inside the exponent range by Markstein's correction (P.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): with y the rounded reciprocal and q = l y rounded, the
// remainder l - q T is exact in a fused multiply-add and q + r y rounds to
// the quotient.
struct Masses {
    float T, inv, top;
    bool fused;
    __device__ __forceinline__ Masses(float temperature, float top_l) : T(temperature) {
        inv = __frcp_rn(T);
        fused = T > 1e-20f && T < 1e20f;
        top = __fdiv_rn(top_l, T);
    }
    __device__ __forceinline__ float quotient(float l) const {
        if (!fused || !(fabsf(l) < 1e15f)) return __fdiv_rn(l, T);
        const float q = l * inv;
        return fmaf(fmaf(-q, T, l), inv, q);
    }
    // mass before rounding; logits of -infinity have none
    __device__ __forceinline__ float scaled(float l) const {
        return l > -INFINITY ? expf(__fsub_rn(quotient(l), top)) * UNIT : 0.f;
    }
    __device__ __forceinline__ u64 of(float l) const { return static_cast<u64>(__float2ll_rn(scaled(l))); }
};

// EPT neighbouring logits per thread (EPT / 2 words of two BF16, or EPT of
// binary32): element e of the CTA's slice belongs to thread e / EPT.  The
// threads of a warp read their words rotated against each other, so that they
// fall into different banks.
template <bool BF16, int EPT>
__global__ void __launch_bounds__(THREADS) sample_kernel(const SampleArgs a) {
    constexpr int WORDS = BF16 ? EPT / 2 : EPT;
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    uint32_t *const row = reinterpret_cast<uint32_t *>(smem + (sizeof(Shared) + 127) / 128 * 128);
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int64_t r = blockIdx.x / CS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int V = a.vocab;
    const int slice = rank * EPT * THREADS;           // first index of the CTA
    const int rot = WORDS >= 32 ? lane : (lane * WORDS) >> 5;
    const uint32_t *const own = row + tid * WORDS;
    if (tid == 0) sh.list_n = sh.cand_n = 0;
    for (int i = tid; i < BINS; i += THREADS) sh.hist[i] = 0;
    // every CTA of the cluster has started (waited for before the first write
    // into another's shared memory)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_launch_dependents();
    pdl_wait();

    // ---- the row into shared memory, once; NaN as -infinity, -0 as +0
    float best = -INFINITY;
    {
        auto clean = [&](float v) -> float {
            v = v != v ? -INFINITY : v + 0.f;
            best = fmaxf(best, v);
            return v;
        };
        constexpr int PER = BF16 ? 8 : 4;  // logits of 16 bytes
        const unsigned char *p = static_cast<const unsigned char *>(a.logits) +
                                 (r * a.row_stride + slice) * (BF16 ? 2 : 4);
        const bool vec = (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
#pragma unroll 4
        for (int i = tid; i < EPT * THREADS / PER; i += THREADS) {
            const int left = V - slice - i * PER;  // logits from here on
            uint4 w;
            uint32_t *const x = reinterpret_cast<uint32_t *>(&w);
            if (vec && left >= PER) w = *reinterpret_cast<const uint4 *>(p + 16 * static_cast<int64_t>(i));
            else {
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    if (BF16) {
                        const uint32_t h = e < left ? reinterpret_cast<const uint16_t *>(p)[i * PER + e] : 0xff80u;
                        x[e / 2] = e & 1 ? x[e / 2] | h << 16 : h;
                    } else x[e & 3] = e < left ? reinterpret_cast<const uint32_t *>(p)[i * PER + e] : 0xff800000u;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (BF16) {
                    const float lo = clean(__uint_as_float(x[e] << 16)), hi = clean(__uint_as_float(x[e] & 0xffff0000u));
                    x[e] = __float_as_uint(lo) >> 16 | (__float_as_uint(hi) & 0xffff0000u);
                } else x[e] = __float_as_uint(clean(__uint_as_float(x[e])));
            }
            reinterpret_cast<uint4 *>(row)[i] = w;
        }
    }

    // f(logit) of every own element, in no particular order
    auto each = [&](auto f) {
#pragma unroll 4
        for (int j = 0; j < WORDS; ++j) {
            const uint32_t w = own[(j + rot) & (WORDS - 1)];
            if (BF16) {
                f(__uint_as_float(w << 16));
                f(__uint_as_float(w & 0xffff0000u));
            } else f(__uint_as_float(w));
        }
    };
    auto logit = [&](int e) -> float {  // own element e
        if (BF16) return __uint_as_float(e & 1 ? own[e >> 1] & 0xffff0000u : own[e >> 1] << 16);
        return __uint_as_float(own[e]);
    };

    // ---- sums of three numbers, and a least and a largest key, over the cluster
    int turn = 0;
    auto reduce = [&](u64 &s0, u64 &s1, u64 &s2, uint32_t &lo, uint32_t &hi) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, o);
            s1 += __shfl_xor_sync(0xffffffffu, s1, o);
            s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            sh.part[warp][0] = s0;
            sh.part[warp][1] = s1;
            sh.part[warp][2] = s2;
            sh.plo[warp] = lo;
            sh.phi[warp] = hi;
        }
        __syncthreads();
        if (warp == 0) {
            const bool on = lane < WARPS;
            s0 = on ? sh.part[lane & (WARPS - 1)][0] : 0;
            s1 = on ? sh.part[lane & (WARPS - 1)][1] : 0;
            s2 = on ? sh.part[lane & (WARPS - 1)][2] : 0;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                s0 += __shfl_xor_sync(0xffffffffu, s0, o);
                s1 += __shfl_xor_sync(0xffffffffu, s1, o);
                s2 += __shfl_xor_sync(0xffffffffu, s2, o);
            }
            lo = __reduce_min_sync(0xffffffffu, sh.plo[lane & (WARPS - 1)]);
            hi = __reduce_max_sync(0xffffffffu, sh.phi[lane & (WARPS - 1)]);
            if (lane < CS) {
                Exchange &to = cluster.map_shared_rank(&sh, lane)->ex;
                to.sums[turn][rank][0] = s0;
                to.sums[turn][rank][1] = s1;
                to.sums[turn][rank][2] = s2;
                to.lo[turn][rank] = lo;
                to.hi[turn][rank] = hi;
            }
        }
        cluster.sync();
        s0 = s1 = s2 = 0;
        lo = 0xffffffffu;
        hi = 0;
        for (int c = 0; c < CS; ++c) {
            s0 += sh.ex.sums[turn][c][0];
            s1 += sh.ex.sums[turn][c][1];
            s2 += sh.ex.sums[turn][c][2];
            lo = min(lo, sh.ex.lo[turn][c]);
            hi = max(hi, sh.ex.hi[turn][c]);
        }
        turn ^= 1;
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
    // goal(total); inside the thread that holds it, of value(element).
    auto locate = [&](u64 mine, auto value, auto goal_of, auto hit) {
        u64 all = mine, z1 = 0, z2 = 0;
        uint32_t lo = 0, hi = 0;
        const int t = turn;
        reduce(all, z1, z2, lo, hi);
        const u64 goal = goal_of(all);
        u64 before = 0;
        for (int c = 0; c < rank; ++c) before += sh.ex.sums[t][c][0];
        if (goal < before || goal >= before + sh.ex.sums[t][rank][0]) return;
        const u64 upto = before + block_scan(mine);
        if (goal >= upto || goal < upto - mine) return;
        u64 at = upto - mine;
        for (int e = 0; e < EPT; ++e) {
            at += value(e);
            if (at > goal) {
                hit(slice + tid * EPT + e);
                break;
            }
        }
    };

    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

    // ---- the largest logit
    float top_l;
    {
        u64 z0 = 0, z1 = 0, z2 = 0;
        uint32_t lo = 0, hi = key_of(best);
        reduce(z0, z1, z2, lo, hi);
        top_l = logit_of(hi);
    }
    if (top_l == -INFINITY) {  // nothing to choose from
        if (rank == 0 && tid == 0) a.tokens[r] = -1;
        return;                // every CTA of the cluster is past its last access to the others
    }
    const float T = a.temperature ? a.temperature[r] : 1.f;
    const Masses mass(T, top_l);
    if (!(T > 0.f) || !(fabsf(mass.top) < INFINITY)) {
        // the largest logit: the first index that holds it
        u64 n = 0;
        each([&](float l) { n += l == top_l; });
        locate(n, [&](int e) -> u64 { return logit(e) == top_l; }, [](u64) -> u64 { return 0; },
               [&](int index) { a.tokens[r] = index; });
        return;
    }
    const float per_bin = fminf(__fdividef(BINS_PER_UNIT, T), 1e30f);
    auto bin_of = [&](float v) -> int { return static_cast<int>(fminf((top_l - v) * per_bin, static_cast<float>(BINS - 1))); };
    // masses of bin b are below 2^(40 - 0.04 b): shortened to 15 bits
    auto shift_of = [](int b) -> int { return max(0, 26 - static_cast<int>(static_cast<float>(b) * 0.0400748f)); };
    const int k = a.top_k ? a.top_k[r] : 0;
    const float p = a.top_p ? a.top_p[r] : 1.f;
    const double least = static_cast<double>(a.min_p ? fminf(a.min_p[r], 1.f) : 0.f) * static_cast<double>(UNIT);
    const float u = a.u[r];
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
        constexpr int PER = BINS / THREADS;
        u64 part[PER], sum = 0;
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            u64 v = 0;
            for (int c = 0; c < CS; ++c) v += cluster.map_shared_rank(&sh, c)->hist[tid * PER + q];
            part[q] = shortened ? v << shift_of(tid * PER + q) : v;
            sum += part[q];
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
        const int bin = goal_bin(static_cast<u64>(k), false);
        Shared *const head = cluster.map_shared_rank(&sh, 0);
        for (int j = 0; j < WORDS; ++j) {
            const int q = (j + rot) & (WORDS - 1);
#pragma unroll
            for (int e = 0; e < (BF16 ? 2 : 1); ++e) {
                const float l = BF16 ? __uint_as_float(e ? own[q] & 0xffff0000u : own[q] << 16) : __uint_as_float(own[q]);
                if (l > -INFINITY && bin_of(l) <= bin) {
                    const int at = atomicAdd(&head->cand_n, 1);
                    const uint32_t index = static_cast<uint32_t>(slice + tid * EPT + (BF16 ? 2 * q + e : q));
                    if (at < CANDIDATES) head->cand[at] = static_cast<u64>(key_of(l)) << 32 | (0xffffffffu - index);
                }
            }
        }
        cluster.sync();
        const int n = *static_cast<volatile int *>(&head->cand_n);
        // (nobody may leave, or clear the count, while another still reads it)
        cluster.sync();
        if (n <= CANDIDATES) {
            if (rank != 0) return;
            int size = 2;
            while (size < n) size <<= 1;
            for (int i = n + tid; i < size; i += THREADS) sh.cand[i] = 0;
            __syncthreads();
            // falling order of key, rising order of index
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
            if (static_cast<double>(m) < least) m = 0;
            if (tid < top) sh.cand_mass[tid] = m;
            const u64 kept = block_scan(m);
            if (tid == THREADS - 1) sh.ex.found_equal = kept;
            __syncthreads();
            if (m) {
                const u64 goal = draw(sh.ex.found_equal);
                const uint32_t me = static_cast<uint32_t>(sh.cand[tid]);  // falls as the index rises
                u64 before = 0;
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
        u64 above, inside, count;
        uint32_t klo, khi;
        while (true) {
            above = inside = count = 0;
            klo = 0xffffffffu, khi = 0;
            each([&](float l) {
                if (l < floor_l || l == -INFINITY) return;
                const int b = bin_of(l);
                if (b > bin) return;
                const u64 m = measure(l);
                if (b < bin) above += m;
                else {
                    inside += m;
                    ++count;
                    klo = min(klo, key_of(l));
                    khi = max(khi, key_of(l));
                }
            });
            reduce(above, inside, count, klo, khi);
            if (above >= goal && bin > 0) --bin;
            else if (above + inside < goal && bin < BINS - 1) ++bin;
            else break;
        }
        while (count > LIST && klo < khi) {
            const uint32_t mid = klo + (khi - klo) / 2;
            u64 sum = 0, n = 0, none = 0;
            uint32_t up = 0xffffffffu, down = 0;
            each([&](float l) {
                const uint32_t key = key_of(l);
                if (key < klo || key > khi || l < floor_l) return;
                if (key > mid) {
                    sum += measure(l);
                    ++n;
                    up = min(up, key);
                } else down = max(down, key);
            });
            reduce(sum, n, none, up, down);
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
        each([&](float l) {
            const uint32_t key = key_of(l);
            if (key < klo || key > khi || l < floor_l) return;
            const int at = atomicAdd(&head->list_n, 1);
            if (at < LIST) {
                head->list_key[at] = key;
                head->list_mass[at] = measure(l);
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
        u64 finite = 0, z1 = 0, z2 = 0;
        uint32_t lo = 0, hi = 0;
        each([&](float l) {
            if (l > -INFINITY) {
                ++finite;
                atomicAdd(&sh.hist[bin_of(l)], 1u);
            }
        });
        reduce(finite, z1, z2, lo, hi);
        if (static_cast<u64>(k) < finite) select(-INFINITY, false, static_cast<u64>(k), cut, ties, equal);
        cluster.sync();  // the others have read this histogram
        for (int i = tid; i < BINS; i += THREADS) sh.hist[i] = 0;
        __syncthreads();
    }
    if (p < 1.f) {
        // the masses that are left: their sum and histogram
        u64 sum = 0, z1 = 0, z2 = 0;
        uint32_t lo = 0, hi = 0, small = 0;
        each([&](float l) {
            if (l < cut || l == -INFINITY) return;
            const float t = mass.scaled(l);
            const int b = bin_of(l);
            uint32_t v;
            if (t < 4194304.f) {  // below 2^22: rint by adding 2^23 (at most 2^6 such per thread)
                const uint32_t m = __float_as_uint(__fadd_rn(t, 8388608.f)) & 0x7fffffu;
                if (l > cut) small += m;
                v = m >> shift_of(b);
            } else {
                const u64 m = static_cast<u64>(__float2ll_rn(t));
                if (l > cut) sum += m;
                v = static_cast<uint32_t>(m >> shift_of(b));
            }
            if (v) atomicAdd(&sh.hist[b], v);
        });
        sum += small;
        reduce(sum, z1, z2, lo, hi);
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
        each([&](float l) { mine += l == cut; });
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
    if (least > 0.) {
        const float reach = -logf(fminf(fmaxf(a.min_p[r], 1e-30f), 1.f)) * T;  // max - l at the bound
        const float lowest = top_l - reach * 1.0001f - 1e-4f * (fabsf(top_l) + T);
        floor_l = fmaxf(floor_l, lowest);
    }
    auto kept = [&](float l, int index) -> u64 {
        if (l < floor_l || l == -INFINITY || (l == cut && index > last_tie)) return 0ull;
        const u64 m = mass.of(l);
        return static_cast<double>(m) < least ? 0ull : m;
    };
    u64 mine = 0;
    if (cut == -INFINITY && least <= 0.) {  // everything
        uint32_t small = 0;
        each([&](float l) {
            const float t = mass.scaled(l);
            if (t < 4194304.f) small += __float_as_uint(__fadd_rn(t, 8388608.f)) & 0x7fffffu;
            else mine += static_cast<u64>(__float2ll_rn(t));
        });
        mine += small;
    } else {
        const bool tie_here = slice + tid * EPT <= last_tie && last_tie < slice + (tid + 1) * EPT;
        if (tie_here) {
            for (int e = 0; e < EPT; ++e) mine += kept(logit(e), slice + tid * EPT + e);
        } else {
            const int index = slice + tid * EPT;  // all of this thread's are on one side of the last tie
            each([&](float l) { mine += kept(l, index); });
        }
    }
    locate(mine, [&](int e) -> u64 { return kept(logit(e), slice + tid * EPT + e); }, draw,
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
    // few rows of a small vocabulary: spread thinner over more SMs
    if (cluster(16) <= 8 && a.rows * cluster(16) <= dev.num_sms) return launch_rows<BF16, 16>(a, cluster(16), st, dev);
    return launch_rows<BF16, 64>(a, cluster(64), st, dev);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    return a.bf16 ? launch_typed<true>(a, st, dev) : launch_typed<false>(a, st, dev);
}

}  // namespace w4
