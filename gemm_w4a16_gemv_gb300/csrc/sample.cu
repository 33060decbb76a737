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
// A row is read once, by a cluster of up to 8 CTAs: the logits stay in
// registers (up to 32 a thread), exp(l / T - max) in shared memory, and what
// the CTAs need of one another (maxima, sums, histograms) goes through
// distributed shared memory.  Nothing is sorted.  The element at which a
// running count (top-k) or mass (top-p), in falling order, reaches its goal is
// found by
//   1. a histogram over (max - l) / T in 1024 bins, 36 to a unit: one shared
//      atomic per element, masses shortened to 16 bits with a shift per bin;
//   2. exact sums above and inside the bin found (moved by a bin where the
//      shortening misled);
//   3. halving the bin's range of keys while more than 128 elements with
//      different keys are left, and a comparison of all pairs of the rest.
// Ties at the cut are told apart by index, by the same search that picks the
// token: sums per warp in index order.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

#include <cooperative_groups.h>

namespace cg = cooperative_groups;

namespace w4 {
namespace {

typedef unsigned long long u64;

constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 1024;           // one per thread
constexpr int LIST = 128;            // candidates compared in pairs
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
__device__ __forceinline__ u64 mass_of(float w) { return static_cast<u64>(__float2ll_rn(w * UNIT)); }

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
    u64 wsum[4][WARPS];
    u64 scan[WARPS];
    u64 list_mass[LIST];
    uint32_t list_key[LIST];
    int list_n;
    int bin;
    u64 bin_above;
};

// EPT logits per thread, in blocks of 8 neighbours: block i of thread t holds
// the indices ((rank * EPT / 8 + i) * THREADS + t) * 8 .. + 7.
template <int EPT>
__global__ void __launch_bounds__(THREADS, 1) sample_kernel(const SampleArgs a) {
    constexpr int NB = EPT / 8;
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &sh = *reinterpret_cast<Shared *>(smem);
    float *const wbuf = reinterpret_cast<float *>(smem + (sizeof(Shared) + 127) / 128 * 128);  // [EPT][THREADS]
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int64_t row = blockIdx.x / CS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int V = a.vocab;
    const int base = rank * EPT * THREADS + tid * 8;
    if (tid == 0) sh.list_n = 0;
    // every CTA of the cluster has started (waited for before the first write
    // into another's shared memory)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_launch_dependents();
    pdl_wait();

    // ---- the row, once; NaN as -infinity, -0 as +0
    float l[EPT];
    {
        const unsigned char *p = static_cast<const unsigned char *>(a.logits) + row * a.row_stride * (a.bf16 ? 2 : 4);
        const bool vec = (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int at = base + i * 8 * THREADS;
            float *const v = l + 8 * i;
            if (vec && at + 8 <= V) {
                if (a.bf16) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(p + 2 * static_cast<int64_t>(at));
                    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[2 * e] = __uint_as_float(q[e] << 16);
                        v[2 * e + 1] = __uint_as_float(q[e] & 0xffff0000u);
                    }
                } else {
                    const float4 w0 = *reinterpret_cast<const float4 *>(p + 4 * static_cast<int64_t>(at));
                    const float4 w1 = *reinterpret_cast<const float4 *>(p + 4 * static_cast<int64_t>(at) + 16);
                    v[0] = w0.x, v[1] = w0.y, v[2] = w0.z, v[3] = w0.w;
                    v[4] = w1.x, v[5] = w1.y, v[6] = w1.z, v[7] = w1.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = at + e >= V ? -INFINITY
                           : a.bf16    ? bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(p)[at + e])
                                       : reinterpret_cast<const float *>(p)[at + e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] != v[e] ? -INFINITY : v[e] + 0.f;
        }
    }

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
            s0 = sh.part[lane][0];
            s1 = sh.part[lane][1];
            s2 = sh.part[lane][2];
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                s0 += __shfl_xor_sync(0xffffffffu, s0, o);
                s1 += __shfl_xor_sync(0xffffffffu, s1, o);
                s2 += __shfl_xor_sync(0xffffffffu, s2, o);
            }
            lo = __reduce_min_sync(0xffffffffu, sh.plo[lane]);
            hi = __reduce_max_sync(0xffffffffu, sh.phi[lane]);
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
        for (int r = 0; r < CS; ++r) {
            s0 += sh.ex.sums[turn][r][0];
            s1 += sh.ex.sums[turn][r][1];
            s2 += sh.ex.sums[turn][r][2];
            lo = min(lo, sh.ex.lo[turn][r]);
            hi = max(hi, sh.ex.hi[turn][r]);
        }
        turn ^= 1;
    };
    // The first index at which the running sum of value(element) exceeds
    // goal(total): each block's and warp's sum in index order, the CTAs'
    // totals through the cluster, then inside the one warp.  The thread that
    // holds it calls hit(index).
    auto locate = [&](auto value, auto goal_of, auto hit) {
        u64 own[NB], total = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            u64 s = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += value(8 * i + e);
            own[i] = s;
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) sh.wsum[i][warp] = s;
            total += s;
        }
        u64 all = lane == 0 ? total : 0, z1 = 0, z2 = 0;
        uint32_t lo = 0, hi = 0;
        const int t = turn;
        reduce(all, z1, z2, lo, hi);
        const u64 goal = goal_of(all);
        u64 before = 0;
        for (int r = 0; r < rank; ++r) before += sh.ex.sums[t][r][0];
        if (goal < before || goal >= before + sh.ex.sums[t][rank][0]) return;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            // where this warp's part of block i begins
            u64 s = sh.wsum[i][lane], upto = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const u64 mine = before + __shfl_sync(0xffffffffu, upto - s, warp);
            const u64 size = __shfl_sync(0xffffffffu, s, warp);
            before += __shfl_sync(0xffffffffu, upto, 31);
            if (goal < mine || goal >= mine + size) continue;
            u64 run = own[i];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            u64 at = mine + run - own[i];
            if (goal < at || goal >= at + own[i]) continue;
            int e_hit = -1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                at += value(8 * i + e);
                if (e_hit < 0 && at > goal) e_hit = e;
            }
            hit(base + i * 8 * THREADS + e_hit);
        }
    };

    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

    // ---- the largest logit
    float top_l = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPT; ++i) top_l = fmaxf(top_l, l[i]);
    {
        u64 z0 = 0, z1 = 0, z2 = 0;
        uint32_t lo = 0, hi = key_of(top_l);
        reduce(z0, z1, z2, lo, hi);
        top_l = logit_of(hi);
    }
    if (top_l == -INFINITY) {  // nothing to choose from
        if (rank == 0 && tid == 0) a.tokens[row] = -1;
        return;                // every CTA of the cluster is past its last access to the others
    }
    const float T = a.temperature ? a.temperature[row] : 1.f;
    const float top = __fdiv_rn(top_l, T);
    if (!(T > 0.f) || !(fabsf(top) < INFINITY)) {
        // the largest logit: the first index that holds it
        locate([&](int i) -> u64 { return l[i] == top_l; }, [](u64) -> u64 { return 0; },
               [&](int index) { a.tokens[row] = index; });
        return;
    }
    // ---- exp(l / T - max), kept in shared memory
    float *const w = wbuf + tid;
    if (T == 1.f) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) w[i * THREADS] = expf(__fsub_rn(l[i], top));
    } else {
#pragma unroll
        for (int i = 0; i < EPT; ++i)
            w[i * THREADS] = l[i] > -INFINITY ? expf(__fsub_rn(__fdiv_rn(l[i], T), top)) : 0.f;
    }
    const float per_bin = fminf(__fdividef(BINS_PER_UNIT, T), 1e30f);
    auto bin_of = [&](float v) -> int { return static_cast<int>(fminf((top_l - v) * per_bin, static_cast<float>(BINS - 1))); };
    // masses of bin b are below 2^(40 - 0.04 b): shortened to 15 bits
    auto shift_of = [](int b) -> int { return max(0, 26 - static_cast<int>(static_cast<float>(b) * 0.0400748f)); };

    // The logit at which the running count or mass, in falling order of the
    // logits not below `floor_l`, reaches `goal`; what of the goal is left
    // there, and how many elements are equal to it.
    auto select = [&](float floor_l, bool by_mass, u64 goal, float &cut, u64 &left, u64 &equal) {
        sh.hist[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            if (l[i] >= floor_l && l[i] > -INFINITY) {
                const int b = bin_of(l[i]);
                const uint32_t v = by_mass ? static_cast<uint32_t>(mass_of(w[i * THREADS]) >> shift_of(b)) : 1u;
                if (v) atomicAdd(&sh.hist[b], v);
            }
        }
        if (tid == 0) sh.bin = -1;
        cluster.sync();
        u64 mine = 0;
        for (int r = 0; r < CS; ++r) mine += cluster.map_shared_rank(&sh, r)->hist[tid];
        if (by_mass) mine <<= shift_of(tid);
        u64 upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) sh.scan[warp] = upto;
        __syncthreads();
        for (int k = 0; k < warp; ++k) upto += sh.scan[k];
        // the bin that holds the goal, or (sums shortened too far) the last one with anything
        if (upto >= goal && upto - mine < goal) sh.bin = tid;
        __syncthreads();
        if (sh.bin < 0) {
            __syncthreads();
            if (mine) atomicMax(&sh.bin, tid);
            __syncthreads();
        }
        int bin = max(sh.bin, 0);
        u64 above, inside, count;
        uint32_t klo, khi;
        while (true) {
            above = inside = count = 0;
            klo = 0xffffffffu, khi = 0;
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                if (l[i] >= floor_l && l[i] > -INFINITY) {
                    const int b = bin_of(l[i]);
                    if (b <= bin) {
                        const u64 m = by_mass ? mass_of(w[i * THREADS]) : 1ull;
                        if (b < bin) above += m;
                        else {
                            inside += m;
                            ++count;
                            klo = min(klo, key_of(l[i]));
                            khi = max(khi, key_of(l[i]));
                        }
                    }
                }
            }
            reduce(above, inside, count, klo, khi);
            if (above >= goal && bin > 0) --bin;
            else if (above + inside < goal && bin < BINS - 1) ++bin;
            else break;
        }
        // (count 0 cannot hold a goal that the kept elements reach)
        while (count > LIST && klo < khi) {
            const uint32_t mid = klo + (khi - klo) / 2;
            u64 sum = 0, n = 0, none = 0;
            uint32_t up = 0xffffffffu, down = 0;
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const uint32_t k = key_of(l[i]);
                if (k >= klo && k <= khi && l[i] >= floor_l) {
                    if (k > mid) {
                        sum += by_mass ? mass_of(w[i * THREADS]) : 1ull;
                        ++n;
                        up = min(up, k);
                    } else down = max(down, k);
                }
            }
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
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const uint32_t k = key_of(l[i]);
            if (k >= klo && k <= khi && l[i] >= floor_l) {
                const int at = atomicAdd(&head->list_n, 1);
                if (at < LIST) {
                    head->list_key[at] = k;
                    head->list_mass[at] = by_mass ? mass_of(w[i * THREADS]) : 1ull;
                }
            }
        }
        cluster.sync();
        if (rank == 0) {
            const int n = min(sh.list_n, LIST);
            if (tid < n) {
                const uint32_t k = sh.list_key[tid];
                const u64 m = sh.list_mass[tid];
                u64 over = above, same = 0;
                bool first = true;
                for (int j = 0; j < n; ++j) {
                    const uint32_t kj = sh.list_key[j];
                    if (kj > k) over += sh.list_mass[j];
                    if (kj == k) {
                        ++same;
                        if (j < tid) first = false;
                    }
                }
                if (first && over < goal && goal <= over + same * m) {
                    for (int r = 0; r < CS; ++r) {
                        Exchange &to = cluster.map_shared_rank(&sh, r)->ex;
                        to.found_key = k;
                        to.found_left = goal - over;
                        to.found_equal = same;
                    }
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
    const int k = a.top_k ? a.top_k[row] : 0;
    if (k > 0 && k < V) {
        u64 finite = 0, z1 = 0, z2 = 0;
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int i = 0; i < EPT; ++i) finite += l[i] > -INFINITY;
        reduce(finite, z1, z2, lo, hi);
        if (static_cast<u64>(k) < finite) select(-INFINITY, false, static_cast<u64>(k), cut, ties, equal);
    }
    const float p = a.top_p ? a.top_p[row] : 1.f;
    if (p < 1.f) {
        u64 sum = 0, z1 = 0, z2 = 0;
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int i = 0; i < EPT; ++i) sum += l[i] > cut ? mass_of(w[i * THREADS]) : 0ull;
        reduce(sum, z1, z2, lo, hi);
        if (cut > -INFINITY) sum += (ties < equal ? ties : equal) * mass_of(expf(__fsub_rn(__fdiv_rn(cut, T), top)));
        const float pc = p > 0.f ? p : 0.f;
        u64 goal = static_cast<u64>(__double2ll_rz(static_cast<double>(sum) * static_cast<double>(pc)));
        if (goal < 1) goal = 1;
        float cut2;
        u64 left, equal2;
        select(cut, true, goal, cut2, left, equal2);
        const u64 m = mass_of(expf(__fsub_rn(__fdiv_rn(cut2, T), top)));
        const u64 n = m ? (left + m - 1) / m : 1ull;
        ties = cut2 == cut && ties < n ? ties : n;
        cut = cut2;
        equal = equal2;
    }
    int last_tie = 0x7fffffff;  // index of the last kept one of the equals
    if (cut > -INFINITY && ties < equal) {
        const u64 n = ties;
        locate([&](int i) -> u64 { return l[i] == cut; }, [&](u64) -> u64 { return n - 1; },
               [&](int index) {
                   for (int r = 0; r < CS; ++r) cluster.map_shared_rank(&sh, r)->ex.found_index = index;
               });
        cluster.sync();
        last_tie = sh.ex.found_index;
    }
    const double least = static_cast<double>(a.min_p ? fminf(a.min_p[row], 1.f) : 0.f) * static_cast<double>(UNIT);
    const float u = a.u[row];
    locate(
        [&](int i) -> u64 {
            const int index = base + (i >> 3) * 8 * THREADS + (i & 7);
            if (!(l[i] > cut || (l[i] == cut && index <= last_tie))) return 0ull;
            const u64 m = mass_of(w[i * THREADS]);
            return static_cast<double>(m) >= least ? m : 0ull;
        },
        [&](u64 total) -> u64 {
            u64 g = u > 0.f ? static_cast<u64>(__double2ll_rz(static_cast<double>(total) * static_cast<double>(fminf(u, 1.f))))
                            : 0ull;
            return g < total ? g : total - 1;
        },
        [&](int index) { a.tokens[row] = index; });
}

template <int EPT>
cudaError_t launch_rows(const SampleArgs &a, int cs, cudaStream_t st, const DeviceInfo &dev) {
    const int smem = static_cast<int>((sizeof(Shared) + 127) / 128 * 128) + EPT * THREADS * 4;
    static SmemLimit limit;
    if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(sample_kernel<EPT>), dev.device, smem)) return e;
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
    return cudaLaunchKernelEx(&cfg, sample_kernel<EPT>, a);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    auto cluster = [&](int ept) {
        int cs = 1;
        while (cs * ept * THREADS < a.vocab) cs *= 2;
        return cs;
    };
    // few rows of a small vocabulary: spread thinner over more SMs
    if (a.vocab <= 8 * 8 * THREADS && a.rows * cluster(8) <= dev.num_sms) return launch_rows<8>(a, cluster(8), st, dev);
    return launch_rows<32>(a, cluster(32), st, dev);
}

}  // namespace w4
