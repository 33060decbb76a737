// kv4_sparse_attention (C header): attention of each new token over pages of its
// own, which it has in a table for each key head (kv4_select writes such tables).
//
// The streaming kernel of kv4_stream.cuh, with the tokens as its requests: a
// token and key head is a segment, the tiles of all segments are split evenly
// over the SMs, a tile is one bulk copy wherever its page lies.  Bound: memory,
// as there.  Measured: 128 tokens over 2048 others each, pages of 16, 16 heads of 256
// on 8: 104 us, 5.0 TB/s, 74% of the copy bandwidth; one such token 10.5 us (latency).
// 301 tokens of one request, 32 heads of 128 on 8, 1088 each: 100 us, the pages in L2,
// issue slots 65% and the ALU pipe 55% busy (the codes' logic).
#include "kv4_stream.cuh"

namespace w4 {

cudaError_t launch_kv4_sparse(const Kv4TableArgs &args, int D, cudaStream_t st, const DeviceInfo &dev) {
    // the running sums of a launch's tokens lie in shared memory
    constexpr int64_t MOST = 4096;
    Kv4TableArgs a = args;
    a.rows_least = 1;
    a.rows_most = 0x7fffffff;
    a.first_launch = 1;
    a.inject = dev.inject;
    for (int64_t t = 0; t < args.T; t += MOST) {
        a.T = a.requests = static_cast<int>(args.T - t < MOST ? args.T - t : MOST);
        if (cudaError_t e = stream(a, D, a.Hq / a.Hkv, st, dev)) return e;
        a.q += a.requests * a.q_stride;
        a.out += static_cast<int64_t>(a.requests) * a.Hq * D;
        a.block_table += a.requests * a.Hkv * a.max_blocks;
        a.seq_lens += a.requests;
    }
    return cudaSuccess;
}

}  // namespace w4
