// The 4-bit key/value cache: layout and helpers shared by the kernels that
// write and read it.
//
// The cache is uint8 [num_blocks, Hkv, block_size / 16, 18 D].  A page of one
// head is a row of tiles; a tile holds 16 tokens x D elements of K and V:
//   [0, 8 D)      codes of K  [D / 64][16 tokens][32 bytes], element 2 i of
//                 the 64 in the low nibble of byte i, 2 i + 1 in the high one
//   [8 D, 16 D)   codes of V, the same
//   [16 D, 17 D)  (scale, zero) of K, binary16 pairs [D / 64][16 tokens]
//   [17 D, 18 D)  (scale, zero) of V
// value = (code - zero) * scale, zero a whole number 0..15.  A tile is one
// contiguous run (4608 bytes at D = 256), so a kernel fetches everything it
// needs of 16 tokens with a single bulk copy whatever the page size, and the
// 32-byte rows let both operand layouts of the 16-bit MMA be read from
// shared memory without bank conflicts.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace w4 {

// Status bit of the operators on the cache (beside those in common.cuh): a
// position, slot, block id or length outside its range.
enum : unsigned int { kDevBadIndex = 4u };

constexpr int KV4_GROUP = 64;  // elements that share a scale and a zero
constexpr int KV4_TILE = 16;   // tokens of a tile

__host__ __device__ constexpr int kv4_tile_bytes(int D) { return 18 * D; }

// Tile of `slot` (block * block_size + offset) in head h; block_size = 1 << bs_log2.
__device__ __forceinline__ size_t kv4_tile_offset(int64_t slot, int h, int Hkv, int bs_log2, int D) {
    const int64_t block = slot >> bs_log2;
    const int64_t tile = (slot & ((int64_t(1) << bs_log2) - 1)) >> 4;
    return static_cast<size_t>(((block * Hkv + h) << (bs_log2 - 4)) + tile) * static_cast<size_t>(kv4_tile_bytes(D));
}

// Rows before request b; whatever the array holds, inside the tensors.
__device__ __forceinline__ int rows_before(const Kv4AttnArgs &a, int b) {
    return static_cast<int>(min(max(static_cast<int64_t>(a.cu_new[b]), int64_t(0)), a.T));
}

// Sets the status if request b's rows lie outside the tensors, or its length
// is negative or more than its row of the block table names (of a request
// with new tokens: of others it is not used).
__device__ __forceinline__ void check_lengths(const Kv4AttnArgs &a, int b) {
    const int64_t from = a.cu_new[b], to = a.cu_new[b + 1], len = a.seq_lens[b];
    if (from < 0 || to < from || to > a.T || (to > from && (len < 0 || len > a.max_blocks << a.bs_log2)))
        atomicOr(a.status, kDevBadIndex);
}

__device__ __forceinline__ float f16_lo(uint32_t w) { return __half2float(__ushort_as_half(static_cast<uint16_t>(w))); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return __half2float(__ushort_as_half(static_cast<uint16_t>(w >> 16))); }

}  // namespace w4
