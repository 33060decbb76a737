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
// All of it is bound by memory (a few operations per 2-byte element).  A head
// is held by D / 8 lanes of a warp, 8 elements (one 16-byte load) per lane:
// the norm's sum, the rotation's partner (a lane rot / 16 away, or the lane
// itself for interleaved pairs) and a group's extremes are shuffles, and a
// lane's 8 codes are one 32-bit word of the cache's 32-byte rows.
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
    for (int i = 0; i < 4; ++i)
        w[i] = static_cast<uint32_t>(f32_to_bf16_bits(x[2 * i])) |
               static_cast<uint32_t>(f32_to_bf16_bits(x[2 * i + 1])) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Quantises this lane's 8 elements (8 lanes hold a group of 64) and stores
// the code word and, from the group's first lane, the parameters.
// Division, rounding and addition are the IEEE operations one by one (no
// contraction), so that the codes are those of the formula in binary32.
template <int D>
__device__ __forceinline__ void quantise_store(const float (&x)[8], unsigned char *tile, int part, int l, int row,
                                               bool store) {
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const __half sh = __float2half_rn(fminf(__fdiv_rn(__fsub_rn(hi, lo), 15.f), 65504.f));
    const float s = __half2float(sh);
    uint32_t word = 0;
    float z = 0.f;
    if (s > 0.f) {
        z = __fadd_rn(fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f), 0.f);  // never -0
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = fminf(fmaxf(__fadd_rn(rintf(__fdiv_rn(x[i], s)), z), 0.f), 15.f);
            word |= static_cast<uint32_t>(c) << (4 * i);
        }
    }
    if (!store) return;
    const int group = l >> 3;
    *reinterpret_cast<uint32_t *>(tile + part * 8 * D + (group * KV4_TILE + row) * 32 + (l & 7) * 4) = word;
    if ((l & 7) == 0)
        *reinterpret_cast<uint32_t *>(tile + (16 + part) * D + (group * KV4_TILE + row) * 4) =
            static_cast<uint32_t>(__half_as_ushort(sh)) |
            static_cast<uint32_t>(__half_as_ushort(__float2half_rn(z))) << 16;
}

// A unit is one head of one token; 32 / LPH units per warp, in the order
// token, then q heads, k heads, v heads.
template <int D>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const Kv4RopeArgs a) {
    constexpr int LPH = D / 8;  // lanes per head
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int l = lane % LPH;
    const unsigned heads = a.Hq + a.Hk + a.Hv;
    const unsigned units = static_cast<unsigned>(a.T) * heads;
    const unsigned step = gridDim.x * (ROPE_THREADS / LPH);
    const unsigned first = blockIdx.x * (ROPE_THREADS / LPH) + (threadIdx.x >> 5) * (32 / LPH);
    bool bad = false;
    // the whole warp takes part in every shuffle: lanes without a unit go
    // along on the last one and store nothing
    for (unsigned u0 = first; u0 < units; u0 += step) {
        const unsigned mine = u0 + lane / LPH;
        const bool live = mine < units;
        const unsigned u = live ? mine : units - 1;
        const unsigned t = u / heads;
        const int h = static_cast<int>(u - t * heads);
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hk;
        const uint16_t *src = is_q   ? a.q + t * a.q_stride + h * D
                              : is_v ? a.v + t * a.v_stride + (h - a.Hq - a.Hk) * D
                                     : a.k + t * a.k_stride + (h - a.Hq) * D;
        float x[8];
        unpack8(*reinterpret_cast<const uint4 *>(src + 8 * l), x);
        const uint16_t *w = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
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
        bool skip = false;  // a row whose position names none: written as zeros
        if (a.cos_sin) {
            const int pos = a.positions[t];
            const bool in = pos >= 0 && pos < a.num_positions;
            bad |= live && pos >= a.num_positions;
            skip = !in;
            const float *cs = a.cos_sin + static_cast<size_t>(in ? pos : 0) * a.rot;
            const int half = a.rot >> 1;
            if (a.interleaved) {
                if (!is_v && 8 * l < a.rot) {
                    const float4 c = *reinterpret_cast<const float4 *>(cs + 4 * l);
                    const float4 s = *reinterpret_cast<const float4 *>(cs + half + 4 * l);
                    const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = x[2 * i], q = x[2 * i + 1];
                        x[2 * i] = p * cc[i] - q * sn[i];
                        x[2 * i + 1] = q * cc[i] + p * sn[i];
                    }
                }
            } else {
                const int hl = half >> 3;  // lanes of half a rotation
                const bool low = l < hl;
                const int from = (lane - l) + (l < 2 * hl ? (low ? l + hl : l - hl) : l);
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], from);
                if (!is_v && l < 2 * hl) {
                    const int at = 8 * (low ? l : l - hl);
                    float cc[8], sn[8];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 c = *reinterpret_cast<const float4 *>(cs + at + 4 * i);
                        const float4 s = *reinterpret_cast<const float4 *>(cs + half + at + 4 * i);
                        cc[4 * i] = c.x, cc[4 * i + 1] = c.y, cc[4 * i + 2] = c.z, cc[4 * i + 3] = c.w;
                        sn[4 * i] = s.x, sn[4 * i + 1] = s.y, sn[4 * i + 2] = s.z, sn[4 * i + 3] = s.w;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = low ? x[i] * cc[i] - y[i] * sn[i] : x[i] * cc[i] + y[i] * sn[i];
                }
            }
        }
        const uint4 packed = (skip && !is_v) ? make_uint4(0, 0, 0, 0) : pack8(x);
        if (is_q) {
            if (live)
                *reinterpret_cast<uint4 *>(a.q_out + (static_cast<size_t>(t) * a.Hq + h) * D + 8 * l) = packed;
        } else if (!a.cache) {
            if (live)
                *reinterpret_cast<uint4 *>(a.k_out + (static_cast<size_t>(t) * a.Hk + (h - a.Hq)) * D + 8 * l) = packed;
        }
        if (a.cache) {
            unpack8(packed, x);
            const int64_t slot = a.slots[t];
            const bool in = slot >= 0 && slot < a.num_slots;
            bad |= live && slot >= a.num_slots;
            // all lanes form codes (the shuffles need the whole warp); heads of q and tokens without a slot
            // point at the first tile and do not store
            const int hk = is_q ? 0 : is_v ? h - a.Hq - a.Hk : h - a.Hq;
            unsigned char *tile = a.cache + kv4_tile_offset(in ? slot : 0, hk, a.Hv, a.bs_log2, D);
            quantise_store<D>(x, tile, is_v ? 1 : 0, l, static_cast<int>(slot & 15), live && in && !is_q);
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kDevBadIndex);
}

// K and V of given slots as BF16 values (slots that name none: zeros).
template <int D>
__global__ void __launch_bounds__(ROPE_THREADS) gather_kernel(const Kv4GatherArgs a) {
    constexpr int LPH = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    const int l = threadIdx.x % LPH;
    const unsigned units = static_cast<unsigned>(a.T) * a.Hkv * 2;
    bool bad = false;
    for (unsigned u = blockIdx.x * (ROPE_THREADS / LPH) + threadIdx.x / LPH; u < units;
         u += gridDim.x * (ROPE_THREADS / LPH)) {
        const unsigned t = u / (2 * a.Hkv);
        const int r = static_cast<int>(u - t * 2 * a.Hkv);
        const int part = r >= a.Hkv, h = part ? r - a.Hkv : r;
        const int64_t slot = a.slots[t];
        uint4 out = make_uint4(0, 0, 0, 0);
        if (slot >= 0 && slot < a.num_slots) {
            const unsigned char *tile = a.cache + kv4_tile_offset(slot, h, a.Hkv, a.bs_log2, D);
            const int at = (l >> 3) * KV4_TILE + static_cast<int>(slot & 15);
            const uint32_t word = *reinterpret_cast<const uint32_t *>(tile + part * 8 * D + at * 32 + (l & 7) * 4);
            const uint32_t sz = *reinterpret_cast<const uint32_t *>(tile + (16 + part) * D + at * 4);
            const float s = f16_lo(sz), z = f16_hi(sz);
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (static_cast<float>((word >> (4 * i)) & 15u) - z) * s;
            out = pack8(x);
        } else if (slot >= 0) bad = true;
        *reinterpret_cast<uint4 *>((part ? a.v : a.k) + (static_cast<size_t>(t) * a.Hkv + h) * D + 8 * l) = out;
    }
    if (bad) atomicOr(a.status, kDevBadIndex);
}

template <typename Args>
cudaError_t launch_units(void (*kern)(Args), const Args &a, int64_t units, int lph, cudaStream_t st,
                         const DeviceInfo &dev) {
    const int64_t per = ROPE_THREADS / lph;
    int64_t grid = (units + per - 1) / per;
    const int64_t most = 8 * static_cast<int64_t>(dev.num_sms);
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
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_kv4_rope(const Kv4RopeArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    const int64_t units = a.T * (a.Hq + a.Hk + a.Hv);
    if (D == 64) return launch_units(rope_kernel<64>, a, units, 8, st, dev);
    if (D == 128) return launch_units(rope_kernel<128>, a, units, 16, st, dev);
    return launch_units(rope_kernel<256>, a, units, 32, st, dev);
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    const int64_t units = a.T * a.Hkv * 2;
    if (D == 64) return launch_units(gather_kernel<64>, a, units, 8, st, dev);
    if (D == 128) return launch_units(gather_kernel<128>, a, units, 16, st, dev);
    return launch_units(gather_kernel<256>, a, units, 32, st, dev);
}

}  // namespace w4
