// RMS norm of every query and key head with the position rotation in the same
// pass, the quantising write into the 4-bit cache, and its read-back
// (w4a16_qk_norm_rope, kv4_append, kv4_gather in the C header).
//
//   y = x * rsqrt(mean(x^2) + eps) * (w + offset)          per head, if w is given
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)   for the rot / 2 pairs
//   K and V to 4 bits by groups of 64 elements:
//     s = fl16((max(x, 0) - min(x, 0)) / 15), z = rint(-min(x, 0) / s),
//     code = clamp(rint(x / s) + z, 0, 15)
// The rotated value is rounded once, to BF16; a key is quantised from that
// BF16 value, so the fused call stores bit for bit what the norm followed by
// a plain append stores.
//
// All of it is bound by the launch for few tokens, and by its instructions and
// memory together for many.  A head is held by D / 8 lanes of a warp, 8 elements
// (one 16-byte load) per lane: the norm's sum, the rotation's partner (a lane
// rot / 16 away, or the lane itself for interleaved pairs) and a group's
// extremes are shuffles, and a lane's 8 codes are one 32-bit word of the
// cache's 32-byte rows.  A warp takes U x 256 / D heads of one token, all
// loads first: with U = 4 each lane has 64 bytes under way and a token's
// cosines, sines and addresses are found once for them; with few tokens U = 1
// spreads the heads over more warps.  Measured: 4099 tokens of 40 heads of 128,
// norm and rotation, 22.2 us (3.9 TB/s, issue slots 65% busy; four CTAs of 256
// threads per SM hold it best, with registers for three or five it was 28.4
// and 39.7 when it was 25.5); 8191 tokens of 8 heads of 256 appended and read
// back 41.5 us (4.1 TB/s, issue slots 78% busy); norm, rotation and write of
// 8191 tokens of 16 query heads and 8 of k and v in one pass 82.8 us (2.8 TB/s;
// its registers spill).
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {
namespace {

constexpr int ROPE_THREADS = 256;

__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Of each pair of BF16 the smaller, or a NaN where there is one.
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float min_or_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// 1 / s rounded, for every binary16 s > 0: one Newton step from the
// approximate reciprocal (the tests compare the codes of all scales with those
// of the division).
__device__ __forceinline__ float reciprocal(float s) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    return fmaf(fmaf(-s, y, 1.f), y, y);
}
// x / b correctly rounded, with y the rounded reciprocal of b, by Markstein's
// correction (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990): q = x y rounded, the remainder x - q b
// exact in a fused multiply-add, q + r y rounded.
__device__ __forceinline__ float divided(float x, float b, float y) {
    const float q = __fmul_rn(x, y);
    return fmaf(fmaf(-q, b, x), y, q);
}

// The least element, at most 0, and the greatest, at least 0, of a group of
// 64: 8 in each of the 8 lanes (`lanes` are those that take part).  They are
// found as BF16 pairs (a minimum of x and one of -x), and are NaN if the group
// holds one.
__device__ __forceinline__ void extremes(const uint4 raw, unsigned lanes, float &lo, float &hi) {
    const uint32_t low = min_bf16x2(min_bf16x2(raw.x, raw.y), min_bf16x2(raw.z, raw.w));
    const uint32_t neg = min_bf16x2(min_bf16x2(raw.x ^ 0x80008000u, raw.y ^ 0x80008000u),
                                    min_bf16x2(raw.z ^ 0x80008000u, raw.w ^ 0x80008000u));
    uint32_t both = min_bf16x2(__byte_perm(low, neg, 0x5410), __byte_perm(low, neg, 0x7632));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) both = min_bf16x2(both, __shfl_xor_sync(lanes, both, o));
    lo = min_or_nan(__uint_as_float(both << 16), 0.f);
    hi = -min_or_nan(__uint_as_float(both & 0xffff0000u), 0.f);
}
__device__ __forceinline__ __half scale_of(float lo, float hi) {  // of NaN: the limit
    return __float2half_rn(fminf(divided(__fsub_rn(hi, lo), 15.f, 1.f / 15.f), 65504.f));
}

// The code word and the parameters of a group whose scale is at its limit
// (values beyond 15 x 65504, infinities: the plain division) or that holds a
// NaN (which counts as zero).  A function of its own, whose registers are not
// the caller's: append and read-back of 8191 tokens 41.5 us, inlined 42.6.
__device__ __noinline__ uint2 quantise_rare(uint4 raw, float lo, float hi) {
    if (lo != lo) {  // (in all lanes of the group)
        auto clean = [](uint32_t w) -> uint32_t { return w & ~__vcmpgtu2(w & 0x7fff7fffu, 0x7f807f80u); };
        raw = make_uint4(clean(raw.x), clean(raw.y), clean(raw.z), clean(raw.w));
        extremes(raw, 0xffu << (threadIdx.x & 24), lo, hi);
    }
    const __half sh = scale_of(lo, hi);
    const float s = __half2float(sh);
    uint32_t word = 0;
    float z = 0.f;
    if (s > 0.f) {
        float x[8];
        unpack8(raw, x);
        z = __fadd_rn(fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f), 0.f);  // never -0
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = fminf(fmaxf(__fadd_rn(rintf(__fdiv_rn(x[i], s)), z), 0.f), 15.f);
            word |= static_cast<uint32_t>(c) << (4 * i);
        }
    }
    return make_uint2(word, static_cast<uint32_t>(__half_as_ushort(sh)) |
                                static_cast<uint32_t>(__half_as_ushort(__float2half_rn(z))) << 16);
}

// Quantises this lane's 8 BF16 elements (8 lanes hold a group of 64) and
// stores the code word and, from the group's first lane, the parameters, at
// `words` and `params` of the row.  Quotients are the correctly rounded ones of
// binary32.  Adding 1.5 2^23 rounds to the nearest whole number, ties to even,
// and leaves it in the low bits.
__device__ __forceinline__ void quantise_store(const uint4 raw, unsigned char *words, unsigned char *params, int l,
                                               bool store) {
    float lo, hi;
    extremes(raw, 0xffffffffu, lo, hi);
    const __half sh = scale_of(lo, hi);
    const float s = __half2float(sh);
    uint32_t word = 0, sz = __half_as_ushort(sh);
    if (s >= 65504.f) {
        const uint2 r = quantise_rare(raw, lo, hi);
        word = r.x;
        sz = r.y;
    } else if (s > 0.f) {
        float x[8];
        unpack8(raw, x);
        const float inv = reciprocal(s);
        auto whole = [&](float v) -> int { return __float_as_int(__fadd_rn(divided(v, s, inv), 12582912.f)); };
        const int zi = __vimin_s32_relu(whole(-lo) - 0x4b400000, 15);
        sz |= static_cast<uint32_t>(__half_as_ushort(__float2half_rn(static_cast<float>(zi)))) << 16;
#pragma unroll
        for (int i = 7; i >= 0; --i) word = word * 16 + __vimin_s32_relu(whole(x[i]) + (zi - 0x4b400000), 15);
    }
    if (!store) return;
    *reinterpret_cast<uint32_t *>(words) = word;
    if ((l & 7) == 0) *reinterpret_cast<uint32_t *>(params) = sz;
}

// A task is U x 32 / LPH heads of one token, in the order q heads, k heads, v
// heads; `tasks` of them per token.  TURN: with a norm or a rotation; KEEP:
// with a cache (instances of their own need fewer registers: 4099 tokens of 40
// heads of 128 take 24.0 us, 8191 tokens of 8 heads of 256 with their read-back
// 49.8, where one for all took 24.9 and 59.2).
template <int D, int U, bool TURN, bool KEEP>
__global__ void __launch_bounds__(ROPE_THREADS, 4) rope_kernel(const Kv4RopeArgs a, const unsigned tasks) {
    constexpr int LPH = D / 8;   // lanes per head
    constexpr int HPS = 32 / LPH;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int l = lane % LPH;
    const int heads = a.Hq + a.Hk + a.Hv;
    const int half = a.rot >> 1, hl = half >> 3;  // lanes of half a rotation
    bool bad = false;
    for (unsigned task = blockIdx.x * (ROPE_THREADS / 32) + (threadIdx.x >> 5); task < static_cast<unsigned>(a.T) * tasks;
         task += gridDim.x * (ROPE_THREADS / 32)) {
        const unsigned t = task / tasks;
        const int h0 = static_cast<int>(task - t * tasks) * (U * HPS) + lane / LPH;
        // the whole warp takes part in every shuffle: lanes past the last head
        // go along on it and store nothing
        uint4 raw[U];
        // (as if each tensor began with the heads before its own)
        const uint16_t *const qt = a.q + (t * a.q_stride + 8 * l), *const kt = a.k + (t * a.k_stride - a.Hq * D + 8 * l),
                       *const vt = a.v + (t * a.v_stride - (a.Hq + a.Hk) * D + 8 * l);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int h = min(h0 + k * HPS, heads - 1);
            raw[k] = *reinterpret_cast<const uint4 *>((h < a.Hq ? qt : h < a.Hq + a.Hk ? kt : vt) + h * D);
        }
        int64_t slot = -1;
        if (KEEP) slot = a.slots[t];
        // this lane's word of the slot's row in head 0, and its group's parameters from there
        const bool in = KEEP && slot >= 0 && slot < a.num_slots;
        if (KEEP) bad |= slot >= a.num_slots;
        unsigned char *row = nullptr;
        const int place = static_cast<int>(slot & 15), params = 16 * D + (l >> 3) * (KV4_TILE * 4) + place * 4 -
                                                               (((l >> 3) * KV4_TILE + place) * 32 + (l & 7) * 4);
        const int head_bytes = kv4_tile_bytes(D) << (a.bs_log2 - 4);
        if (KEEP)
            row = a.cache + kv4_tile_offset(in ? slot : 0, 0, a.Hv, a.bs_log2, D) + ((l >> 3) * KV4_TILE + place) * 32 + (l & 7) * 4;
        bool skip = false;  // a row whose position names none: written as zeros
        float cc[8], sn[8];
        const bool low = l < hl;
        if (TURN && a.cos_sin) {
            const int pos = a.positions[t];
            skip = pos < 0 || pos >= a.num_positions;
            bad |= pos >= a.num_positions;
            const float *cs = a.cos_sin + static_cast<size_t>(skip ? 0 : pos) * a.rot;
            const int at = a.interleaved ? 4 * l : 8 * (low ? l : l - hl);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
                if (l < 2 * hl && (i == 0 || !a.interleaved)) {
                    c = *reinterpret_cast<const float4 *>(cs + at + 4 * i);
                    s = *reinterpret_cast<const float4 *>(cs + half + at + 4 * i);
                }
                cc[4 * i] = c.x, cc[4 * i + 1] = c.y, cc[4 * i + 2] = c.z, cc[4 * i + 3] = c.w;
                sn[4 * i] = s.x, sn[4 * i + 1] = s.y, sn[4 * i + 2] = s.z, sn[4 * i + 3] = s.w;
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const bool live = h0 + k * HPS < heads;
            const int h = min(h0 + k * HPS, heads - 1);
            const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hk;
            // of the whole warp: no head to rotate, or none to quantise
            const int warp_h = h0 - lane / LPH + k * HPS;
            const bool all_v = warp_h >= a.Hq + a.Hk, all_q = warp_h + HPS <= a.Hq;
            uint4 packed = raw[k];
            float x[8];
            unpack8(packed, x);
            const uint16_t *w = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
            if (TURN && (a.q_weight || a.k_weight) && !all_v) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int o = 1; o < LPH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (w) {
                    const float r = rsqrtf(ss * (1.f / D) + a.eps);
                    float wv[8];
                    unpack8(*reinterpret_cast<const uint4 *>(w + 8 * l), wv);
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (wv[i] + a.weight_offset);
                }
            }
            if (TURN && a.cos_sin && !all_v) {
                if (a.interleaved) {
                    if (!is_v && l < 2 * hl) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p = x[2 * i], q = x[2 * i + 1];
                            x[2 * i] = p * cc[i] - q * sn[i];
                            x[2 * i + 1] = q * cc[i] + p * sn[i];
                        }
                    }
                } else {
                    const int from = (lane - l) + (l < 2 * hl ? (low ? l + hl : l - hl) : l);
                    float y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], from);
                    if (!is_v && l < 2 * hl) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = low ? x[i] * cc[i] - y[i] * sn[i] : x[i] * cc[i] + y[i] * sn[i];
                    }
                }
            }
            if (TURN && !is_v) packed = skip ? make_uint4(0, 0, 0, 0) : pack8(x);
            if (is_q) {
                if (live)
                    *reinterpret_cast<uint4 *>(a.q_out + (static_cast<size_t>(t) * a.Hq + h) * D + 8 * l) = packed;
            } else if (!KEEP) {
                if (live)
                    *reinterpret_cast<uint4 *>(a.k_out + (static_cast<size_t>(t) * a.Hk + (h - a.Hq)) * D + 8 * l) = packed;
            }
            if (KEEP && !all_q) {
                // all lanes form codes (the shuffles need the whole warp); heads of q among them and tokens
                // without a slot do not store
                const int hk = is_q ? 0 : is_v ? h - a.Hq - a.Hk : h - a.Hq;
                unsigned char *const at = row + hk * head_bytes + (is_v ? 8 * D : 0);
                quantise_store(packed, at, at + params + (is_v ? D - 8 * D : 0), l, live && in && !is_q);
            }
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kDevBadIndex);
}

// K and V of given slots as BF16 values (slots that name none: zeros); a task
// is U x 32 / LPH of the 2 Hkv heads of one slot.
template <int D, int U>
__global__ void __launch_bounds__(ROPE_THREADS, 4) gather_kernel(const Kv4GatherArgs a, const unsigned tasks) {
    constexpr int LPH = D / 8, HPS = 32 / LPH;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, l = lane % LPH;
    bool bad = false;
    for (unsigned task = blockIdx.x * (ROPE_THREADS / 32) + (threadIdx.x >> 5); task < static_cast<unsigned>(a.T) * tasks;
         task += gridDim.x * (ROPE_THREADS / 32)) {
        const unsigned t = task / tasks;
        const int h0 = static_cast<int>(task - t * tasks) * (U * HPS) + lane / LPH;
        const int64_t slot = a.slots[t];
        const bool in = slot >= 0 && slot < a.num_slots;
        bad |= slot >= a.num_slots;
        // the slot's tile in head 0, this lane's word and parameters in a tile of K
        const unsigned char *const tile = a.cache + kv4_tile_offset(in ? slot : 0, 0, a.Hkv, a.bs_log2, D);
        const int place = (l >> 3) * KV4_TILE + static_cast<int>(slot & 15);
        const int at = place * 32 + (l & 7) * 4, params = 16 * D + place * 4;
        const int head_bytes = kv4_tile_bytes(D) << (a.bs_log2 - 4);
        uint32_t word[U], sz[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            word[k] = sz[k] = 0;
            const int r = h0 + k * HPS, part = r >= a.Hkv;
            if (in && r < 2 * a.Hkv) {
                const int off = (part ? r - a.Hkv : r) * head_bytes;
                word[k] = *reinterpret_cast<const uint32_t *>(tile + (off + at + part * 8 * D));
                sz[k] = *reinterpret_cast<const uint32_t *>(tile + (off + params + part * D));
            }
        }
        const int64_t to = static_cast<int64_t>(t) * a.Hkv * D + 8 * l;
        uint16_t *const kt = a.k + to, *const vt = a.v + (to - static_cast<int64_t>(a.Hkv) * D);
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int r = h0 + k * HPS, part = r >= a.Hkv;
            if (r >= 2 * a.Hkv) continue;
            // a code in place in the significand of 2^23 is 2^23 + 16^i code; all
            // of it is exact (zero times scale has 15 bits)
            const float s = f16_lo(sz[k]), zs = -f16_hi(sz[k]) * s;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t w = i < 4 ? word[k] : word[k] >> 16;
                const float c = __fsub_rn(__uint_as_float((w & (15u << (4 * (i & 3)))) | 0x4b000000u), 8388608.f);
                x[i] = fmaf(c, s * (1.f / (1 << (4 * (i & 3)))), zs);
            }
            *reinterpret_cast<uint4 *>((part ? vt : kt) + r * D) = pack8(x);
        }
    }
    if (bad) atomicOr(a.status, kDevBadIndex);
}

// At most `per_sm` CTAs per SM: 4, one round of CTAs that go on with further
// tasks, for the norm alone (4099 tokens 23.4 -> 22.4 us), 16 where codes are
// formed or read (append and read-back of 8191 tokens 42.7 us, with 4 49.0).
template <typename Args>
cudaError_t launch_tasks(void (*kern)(Args, unsigned), const Args &a, int64_t tokens, int64_t heads, int per_task, int per_sm,
                         cudaStream_t st, const DeviceInfo &dev) {
    const int64_t tasks = (heads + per_task - 1) / per_task;
    int64_t grid = (tokens * tasks + ROPE_THREADS / 32 - 1) / (ROPE_THREADS / 32);
    const int64_t most = per_sm * static_cast<int64_t>(dev.num_sms);
    if (grid > most) grid = most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(ROPE_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, static_cast<unsigned>(tasks));
}

// Four heads in flight per lane once that still gives every SM enough warps.
// One against four, us: norm and rotation of 40 heads of 128, 512 tokens 5.3 /
// 6.3, 1024 8.3 / 8.4, 4096 31.9 / 25.1; append of 8 heads of 256, 512 tokens
// 7.3 / 11.0, 1024 11.8 / 11.7, 4096 38.5 / 32.4.
bool many(int64_t tokens, int64_t heads, int D, const DeviceInfo &dev) {
    return tokens * heads * D >= int64_t(dev.num_sms) * 32768;
}

template <int D, bool TURN, bool KEEP>
cudaError_t launch_form(const Kv4RopeArgs &a, cudaStream_t st, const DeviceInfo &dev) {
    const int64_t heads = a.Hq + a.Hk + a.Hv;
    if (many(a.T, heads, D, dev)) return launch_tasks(rope_kernel<D, 4, TURN, KEEP>, a, a.T, heads, 1024 / D, KEEP ? 16 : 4, st, dev);
    return launch_tasks(rope_kernel<D, 1, TURN, KEEP>, a, a.T, heads, 256 / D, 16, st, dev);
}

// (without a cache there is a norm or a rotation, or a plain copy of q and k)
template <int D>
cudaError_t launch_rope(const Kv4RopeArgs &a, bool turn, cudaStream_t st, const DeviceInfo &dev) {
    if (!a.cache) return launch_form<D, true, false>(a, st, dev);
    return turn ? launch_form<D, true, true>(a, st, dev) : launch_form<D, false, true>(a, st, dev);
}

}  // namespace

cudaError_t launch_kv4_rope(const Kv4RopeArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    const bool turn = a.q_weight || a.k_weight || a.cos_sin;
    if (D == 64) return launch_rope<64>(a, turn, st, dev);
    if (D == 128) return launch_rope<128>(a, turn, st, dev);
    return launch_rope<256>(a, turn, st, dev);
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    const int64_t heads = 2 * a.Hkv;
    if (many(a.T, heads, D, dev)) {
        if (D == 64) return launch_tasks(gather_kernel<64, 4>, a, a.T, heads, 16, 16, st, dev);
        if (D == 128) return launch_tasks(gather_kernel<128, 4>, a, a.T, heads, 8, 16, st, dev);
        return launch_tasks(gather_kernel<256, 4>, a, a.T, heads, 4, 16, st, dev);
    }
    if (D == 64) return launch_tasks(gather_kernel<64, 1>, a, a.T, heads, 4, 16, st, dev);
    if (D == 128) return launch_tasks(gather_kernel<128, 1>, a, a.T, heads, 2, 16, st, dev);
    return launch_tasks(gather_kernel<256, 1>, a, a.T, heads, 1, 16, st, dev);
}

}  // namespace w4
