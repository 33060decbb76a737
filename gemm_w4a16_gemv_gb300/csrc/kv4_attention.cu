// Attention over the paged 4-bit cache (kv4_attention in the C header).
//
//   o = sum_j softmax_j(scale q . k_j) v_j  over the keys j that query p sees:
//   j <= p, and with a window w also p - j < w or j < sinks.
//
// Simple form: a CTA per (token, query head), its warps take the visible keys
// in turn, a lane holds 8 dimensions; running maximum and sum in binary32.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace w4 {
namespace {

constexpr int ATTN_WARPS = 4;

template <int D>
__global__ void __launch_bounds__(ATTN_WARPS * 32) attn_simple_kernel(const Kv4AttnArgs a) {
    constexpr int LPH = D / 8;
    __shared__ float sm_m[ATTN_WARPS], sm_l[ATTN_WARPS], sm_o[ATTN_WARPS][D];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int hq = blockIdx.y, hk = hq / (a.Hq / a.Hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool on = lane < LPH;
    int lo = 0, hi = a.requests;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_new[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int b = lo;
    const bool mine = t >= a.cu_new[b] && t < a.cu_new[b + 1];
    const int64_t p = mine ? int64_t(a.seq_lens[b]) - a.cu_new[b + 1] + t : -1;
    float q[8] = {};
    if (on)
        for (int i = 0; i < 8; ++i) q[i] = bf16_bits_to_f32(a.q[t * a.q_stride + hq * D + 8 * lane + i]) * a.scale;
    float m = -INFINITY, l = 0.f, o[8] = {};
    const int64_t cap = a.max_blocks << a.bs_log2;
    const int64_t end = p + 1 < cap ? p + 1 : cap;
    for (int64_t j = warp; j < end; j += ATTN_WARPS) {
        if (a.window > 0 && p - j >= a.window && j >= a.sinks) continue;
        const int id = a.block_table[b * a.max_blocks + (j >> a.bs_log2)];
        if (id < 0 || id >= a.num_blocks) {
            if (lane == 0) atomicOr(a.status, kDevBadIndex);
            continue;
        }
        const int64_t slot = (int64_t(id) << a.bs_log2) + (j & ((int64_t(1) << a.bs_log2) - 1));
        const unsigned char *tile = a.cache + kv4_tile_offset(slot, hk, a.Hkv, a.bs_log2, D);
        const int at = (lane >> 3) * KV4_TILE + static_cast<int>(slot & 15);
        float x = 0.f;
        if (on) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(tile + at * 32 + (lane & 7) * 4);
            const uint32_t sz = *reinterpret_cast<const uint32_t *>(tile + 16 * D + at * 4);
            const float s = f16_lo(sz), z = f16_hi(sz);
            for (int i = 0; i < 8; ++i) x += q[i] * ((static_cast<float>((w >> (4 * i)) & 15u) - z) * s);
        }
        for (int k = 1; k < 32; k <<= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
        const float mn = fmaxf(m, x), f = __expf(m - mn), e = __expf(x - mn);
        m = mn;
        l = l * f + e;
        if (on) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(tile + 8 * D + at * 32 + (lane & 7) * 4);
            const uint32_t sz = *reinterpret_cast<const uint32_t *>(tile + 17 * D + at * 4);
            const float s = f16_lo(sz), z = f16_hi(sz);
            for (int i = 0; i < 8; ++i) o[i] = o[i] * f + e * ((static_cast<float>((w >> (4 * i)) & 15u) - z) * s);
        }
    }
    if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
    if (on)
        for (int i = 0; i < 8; ++i) sm_o[warp][8 * lane + i] = o[i];
    __syncthreads();
    float mm = -INFINITY;
    for (int w = 0; w < ATTN_WARPS; ++w) mm = fmaxf(mm, sm_m[w]);
    float ll = 0.f, f[ATTN_WARPS];
    for (int w = 0; w < ATTN_WARPS; ++w) {
        f[w] = mm == -INFINITY ? 0.f : __expf(sm_m[w] - mm);
        ll += sm_l[w] * f[w];
    }
    for (int d = threadIdx.x; d < D; d += ATTN_WARPS * 32) {
        float v = 0.f;
        for (int w = 0; w < ATTN_WARPS; ++w) v += sm_o[w][d] * f[w];
        a.out[(t * a.Hq + hq) * D + d] = f32_to_bf16_bits(ll > 0.f ? v / ll : 0.f);
    }
}

}  // namespace

int64_t kv4_attention_scratch(int, int, int) { return 256; }

cudaError_t launch_kv4_attention(const Kv4AttnArgs &a, int D, cudaStream_t st, const DeviceInfo &) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.T), static_cast<unsigned>(a.Hq));
    cfg.blockDim = dim3(ATTN_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    if (D == 64) return cudaLaunchKernelEx(&cfg, attn_simple_kernel<64>, a);
    if (D == 128) return cudaLaunchKernelEx(&cfg, attn_simple_kernel<128>, a);
    return cudaLaunchKernelEx(&cfg, attn_simple_kernel<256>, a);
}

}  // namespace w4
