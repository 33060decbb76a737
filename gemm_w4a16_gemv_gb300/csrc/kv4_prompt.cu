// Attention over the paged 4-bit cache for pieces of many new tokens, on the
// tcgen05 tensor cores (kv4_attention in the C header; the streaming form for
// few rows is kv4_stream.cuh).  For kv4_prefix_attention the same kernel has pieces
// of shared stretches of keys as its requests and leaves parts to be joined.
//
// An item is 128 rows (new tokens x the G query heads of one key head) of a
// request, or 256 for a pair of CTAs; its keys are taken 128 at a time:
//   S = Q K^T          N 128, K D       -> tensor memory (two buffers)
//   P = exp2(S' - M)   128 threads, one row each, back into tensor memory
//   O += P V           N D, K 128       P from tensor memory
//
// Bound.  At D = 256 the two products take 2 x 1024 cycles of an SM's tensor
// pipe per 128 x 128 tile.  One CTA alone also has to form 2 x 32768 codes as
// binary16 operands (14 instructions per 8 codes and lane), store them (128 KB
// at 128 bytes a cycle) and feed the products from shared memory (192 KB):
// 2500 cycles of its bandwidth, and the stages wait for one another.  So for
// D = 128 and 256 two CTAs work as a pair (cta_group::2): each keeps its own
// 128 rows of Q, S, P and O, but only half of K (64 of the 128 keys) and half
// of V (D / 2 of the dimensions), which halves the forming and the stores per
// SM, and leaves room for two buffers of each operand.  One CTA of the pair
// issues the products of both.  Measured on 6491 new tokens in three requests
// with up to 6000 tokens before them, 16 heads of 256 on 8: single CTAs 455 us,
// pairs 280 us, 1200 TFLOP/s.  A tile takes about 3700 cycles.  No stage does by
// itself (the tensor pipe 2048; the softmax 1290 with the SM to itself, of which the
// exponentials are 512 per SM quarter); they wait for one another, and the three roles
// share the issue slots, 55 % of them busy, and the instruction cache: the code is
// kept short (rolled loops, masks as 32-bit words: 341 -> 298 us).
// (D = 64 stays with single CTAs: half of its 64 dimensions is no whole
// swizzled row.)
//
// Items are handed out by a counter in scratch, the longest first (requests
// sorted by length, the last rows of a request first), and announced to the
// roles through a small ring in shared memory.
//
// Roles: warps 0-3 softmax and epilogue (warp w owns the tensor memory lanes
// 32 w ..), warps 4-7 form K and 8-11 V (16-byte loads of the codes one step
// ahead in registers) and together Q of the next item, warp 12 issues the
// products in the order Q K(i+1), P(i) V(i), so that the operands of one are
// formed while the other runs.
//
// Operands.  (code - zero) is exact in binary16; times the scale it is rounded
// once.  The scales of a cache tile are multiplied by a power of two that brings
// the largest to [2^10, 2^11), so that scales 2^25 apart keep all their bits; the
// power of K's goes into the factor of its 16 scores, that of V's into the
// exponent: P = exp2(x + e - M), and the sum of weights takes P 2^-e.  A row
// of Q enters after a power-of-two scale of its own.  K and V lie in shared
// memory as they come from the cache, a row of 64 dimensions per token and
// group with the 128-byte swizzle: K-major for the first product, MN-major
// (dimensions contiguous) for the second.  A word's codes leave in the order
// 0 4 1 5 2 6 3 7; Q is stored in the same order and the epilogue undoes it.
//
// The running reference M of a row puts its largest P into [2^6, 2^15] (binary16
// then keeps 11 bits of weights down to 2^-20 of it) and moves only when P would
// pass 2^15; then the softmax warps scale O in tensor memory themselves, between
// two products.
//
// Every wait is bounded.  On a timeout the roles still go through all their
// arrivals, except that one which is not told of its next item leaves; tensor
// memory is given back, and the CTAs end, when the products issued are done.
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "tc_common.cuh"

namespace w4 {
namespace {

constexpr int ROWS = 128;
constexpr int KEYS = 128;
constexpr int SOFT_THREADS = 128;
constexpr int FORM_WARPS = 4;         // of K, and as many of V
constexpr int THREADS = SOFT_THREADS + 2 * FORM_WARPS * 32 + 32;
// Registers: 128 a thread at launch (13 warps); of each SM quarter's three
// warps of four-warp groups 144 + 2 x 120 = 3 x 128.  With 128 the softmax
// spills, and the L1 left beside the operands does not hold what it spills.
constexpr int SOFT_REGS = 144, FORM_REGS = 120;
constexpr float NONE = -1e30f;       // reference of a row that has seen no key
constexpr int METAS = 4;             // buffers of what the softmax needs to know of a key tile: it is at most
                                     // two tiles behind the one whose operands are free to be written, of two
constexpr int QUEUE = 4;             // items announced ahead
constexpr int SORT_MOST = 512;       // requests that are put in order of length
constexpr int SUB = KEYS * 128;      // bytes of 128 rows x 64 binary16

// vfree goes by a key tile's number, not its buffer: where there is one buffer (D = 64), the
// softmax asks for the last tile's product when the one before may still run, and of a
// single barrier's phases every second looks the same.  Of two, what came before on the same
// one is the product of two tiles earlier, complete since this tile's scores are there.
struct Bars {
    uint64_t qfull, kfull[2], kfree[2], vfull[2], vfree[2], sfull[2], pfull[2], ifull[QUEUE], known[METAS];
    uint32_t tmem;
    int item[QUEUE];
    int late;  // key tiles worked on, where some wait has run out; else 0
};
// Of a key tile, from the warps that form it: the factors of its cache tiles
// and which of them there are.
struct alignas(16) Meta {
    float k_factor[8], v_exponent[8], v_factor[8];
    unsigned char held[8];
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

// ---- pairs of CTAs.  The leader (rank 0) issues the products and owns the
// barriers they wait for; the other CTA's warps arrive on them through the
// cluster's shared memory, and completions are announced to both.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One arrival of this (converged) warp on the leader's barrier, for operands
// that it wrote: the tensor core of its own CTA reads them, and the fence of the
// proxies (or of tensor memory) before this call orders them there.  So the
// arrival releases nothing to the other CTA's threads, and must not: a release
// of the cluster's scope waits for the warp's loads in flight (the whole kernel
// took 521 us with it and 410 without, at that step).
template <bool PAIR>
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
    __syncwarp();
    if (lane == 0) {
        if (PAIR) asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(peer(bar, 0)) : "memory");
        else mbar_arrive(bar);
    }
}
// mbar_wait that reads the timer (150 cycles) only when the phase is not there
// yet.  ACROSS: for data that a thread of the other CTA of a pair wrote.
template <bool ACROSS = false>
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, unsigned int *status) {
    const uint32_t a = smem_u32(bar);
    unsigned long long t0 = 0;
#pragma unroll 1
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 256; ++i) {
            uint32_t ok;
            if (ACROSS)
                asm volatile(
                    "{\n\t.reg .pred p;\n\t"
                    "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                    : "=r"(ok)
                    : "r"(a), "r"(parity)
                    : "memory");
            else
                asm volatile(
                    "{\n\t.reg .pred p;\n\t"
                    "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                    : "=r"(ok)
                    : "r"(a), "r"(parity)
                    : "memory");
            if (ok) return true;
        }
        if (status && (*reinterpret_cast<volatile unsigned int *>(status) & kDevTimeout)) return false;
        const unsigned long long now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) {
            if (status) atomicOr(status, kDevTimeout);
            return false;
        }
    }
}
template <bool PAIR>
__device__ __forceinline__ void product(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    if (!PAIR) {
        umma_f16_w(d, adesc, bdesc, idesc, accumulate);
        return;
    }
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void product_tmem(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    if (!PAIR) {
        umma_f16_tmem_a_w(d, a, bdesc, idesc, accumulate);
        return;
    }
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on `bar` (of both CTAs of a pair) when the products so far are done.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if (!PAIR) {
        umma_commit_w(bar);
        return;
    }
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tmem_take(uint32_t *holder) {
    if (!PAIR) {
        tmem_alloc(holder, 512);
        tmem_relinquish();
        return;
    }
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(holder)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tmem_give(uint32_t taddr) {
    if (!PAIR) tmem_dealloc(taddr, 512);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(512u) : "memory");
}

// The loads from tensor memory are complete; no use of x moves before this.
__device__ __forceinline__ void arrived(uint32_t (&x)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]),
                   "+r"(x[6]), "+r"(x[7]), "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]),
                   "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]), "+r"(x[16]), "+r"(x[17]),
                   "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]), "+r"(x[23]),
                   "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]), "+r"(x[28]), "+r"(x[29]),
                   "+r"(x[30]), "+r"(x[31])
                 :
                 : "memory");
}

// 2^x by the hardware's approximation (2 ulp): a weight is rounded to 11 bits
// after it.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
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
// 32 bytes, a whole sector.
__device__ __forceinline__ void store8(float *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f, uint32_t g,
                                       uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f),
                 "r"(g), "r"(h)
                 : "memory");
}
// (never zero, so that times -infinity it is no NaN)
__device__ __forceinline__ float factor(float f, float k) { return fmaxf(f * k, 1.2e-38f); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

struct Item {
    int b, h, tok0, r0, rows;   // rows [r0, r0 + rows) of the request; its row of the block table, its first token
    int64_t place;              // of the rows' parts (kv4_prefix_attention), or negative
    int base;                   // position of row r is base + r / G
    int end;                    // keys at or past this are seen by no row,
    int sink, first;            // nor are those from `sink` to before `first`
    int n, ns, low;             // key tiles: the first ns, then from `low` on
    __device__ __forceinline__ int key0(int i) const { return (i < ns ? i : i - ns + low) * KEYS; }
};

__device__ __forceinline__ bool taken(const Kv4AttnArgs &a, int rows) { return rows > a.rows_above; }

template <int ITEM>
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
    it.place = -1;
    it.tok0 = rows_before(a, lo);
    const int n = rows_before(a, lo + 1) - it.tok0;
    const int total = n * G, blocks = (total + ITEM - 1) / ITEM;
    it.h = local % a.Hkv;
    it.r0 = (blocks - 1 - local / a.Hkv) * ITEM;  // the rows that see most first
    it.rows = min(ITEM, total - it.r0);
    const int first = max(a.seq_lens[lo], 0) - n;
    it.base = first;
    const int cap = static_cast<int>(min(static_cast<long long>(a.max_blocks) << a.bs_log2, 0x7fffff00ll));
    const int p_lo = first + it.r0 / G, p_hi = first + (it.r0 + it.rows - 1) / G;
    const int end = max(min(p_hi + 1, cap), 0);
    int low = 0, ns = 0;
    it.sink = it.first = 0;
    if (a.window > 0) {
        it.first = static_cast<int>(max(p_lo - a.window + 1, int64_t(0)));
        it.sink = static_cast<int>(min(a.sinks, static_cast<int64_t>(end)));
        ns = (it.sink + KEYS - 1) / KEYS;
        low = max(it.first / KEYS, ns);
    }
    const int last = (end + KEYS - 1) / KEYS;
    it.end = end;
    it.ns = ns;
    it.low = low;
    // (rows that see nothing take one empty tile and come out as zeros)
    it.n = max(ns + max(last - low, 0), 1);
    return it;
}

// The same of a piece of kv4_prefix_attention's: its keys from `from` on (before
// them there may be some of the first key tile, whose cache tiles are not looked
// at).
template <int ITEM>
__device__ __forceinline__ Item item_of(const Kv4SharedArgs &a, const int *cum, const int *, int index, int G) {
    Item it;
    int lo = 0, hi = a.counts[0];
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= index) lo = mid;
        else hi = mid;
    }
    const int local = index - cum[lo];
    const Kv4Stretch s = a.pieces[lo];
    const int total = s.tokens * G, blocks = (total + ITEM - 1) / ITEM;
    it.b = s.row;
    it.tok0 = s.token;
    it.place = s.place;
    it.h = local % a.Hkv;
    it.r0 = (blocks - 1 - local / a.Hkv) * ITEM;
    it.rows = min(ITEM, total - it.r0);
    it.base = s.base;
    it.end = max(min(s.base + (it.r0 + it.rows - 1) / G + 1, s.end), 0);
    it.sink = it.ns = 0;
    it.first = s.from;
    it.low = s.from / KEYS;
    it.n = max((it.end + KEYS - 1) / KEYS - it.low, 1);
    return it;
}

template <int D, bool PAIR>
struct PromptSmem {
    static constexpr int G64 = D / 64;
    static constexpr int BUFS = PAIR ? 2 : 1;             // of K and of V
    static constexpr int K_ROWS = PAIR ? KEYS / 2 : KEYS; // keys of a tile that this CTA forms
    static constexpr int K_SUB = K_ROWS * 128;            // bytes of a group of them
    static constexpr int V_GROUPS = PAIR ? G64 / 2 : G64; // groups of V that this CTA forms
    static constexpr int q = 0, k = G64 * SUB, v = k + BUFS * G64 * K_SUB;
    static constexpr int meta = v + BUFS * V_GROUPS * SUB;  // [METAS] Meta
    static constexpr int factors = meta + METAS * static_cast<int>(sizeof(Meta));  // [2][ROWS] of the scores, per row
    static constexpr int bars = factors + 2 * ROWS * 4;
    static constexpr int cum = bars + 256;                // [requests + 1] ints, then [requests] order
};
static_assert(sizeof(Bars) <= 256, "shared memory map");

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

template <class Args, int D, bool PAIR>
__global__ void __launch_bounds__(THREADS, 1) attn_prompt_kernel(const Args a) {
    using L = PromptSmem<D, PAIR>;
    constexpr int G64 = L::G64, BUFS = L::BUFS, CTAS = PAIR ? 2 : 1, ITEM = CTAS * ROWS;
    constexpr uint32_t COL_S = D, IDESC_QK = idesc_kind_f16(ITEM, KEYS, 0u),
                       IDESC_PV = idesc_kind_f16(ITEM, D, 0u) | (1u << 16);
    const int rank = PAIR ? static_cast<int>(cluster_rank()) : 0;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Bars &bar = *reinterpret_cast<Bars *>(smem + L::bars);
    float *const q_factor = reinterpret_cast<float *>(smem + L::factors);
    int *const cum = reinterpret_cast<int *>(smem + L::cum);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.Hq / a.Hkv;

    if (tid == 0) {
        // arrivals: a warp each
        mbar_init(&bar.qfull, CTAS * 2 * FORM_WARPS);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.kfull[i], CTAS * FORM_WARPS);
            mbar_init(&bar.vfull[i], CTAS * FORM_WARPS);
            mbar_init(&bar.kfree[i], 1);
            mbar_init(&bar.vfree[i], 1);
            mbar_init(&bar.sfull[i], 1);
            mbar_init(&bar.pfull[i], CTAS * SOFT_THREADS / 32);
        }
        for (int i = 0; i < QUEUE; ++i) mbar_init(&bar.ifull[i], 1);
        for (int i = 0; i < METAS; ++i) mbar_init(&bar.known[i], 2 * FORM_WARPS);
        bar.late = 0;
        fence_barrier_init();
    }
    if (warp == 12) tmem_take<PAIR>(&bar.tmem);
    // (kv4_prefix_attention's next kernel does not need this one's results, but the plan,
    // which this one waits for: it begins when that is complete)
    if (!Args::kShared) pdl_launch_dependents();
    pdl_wait();
    if (Args::kShared) pdl_launch_dependents();
    int *const order = cum + a.requests + 1;
    if constexpr (Args::kShared) {
        for (int i = tid; i <= a.counts[0]; i += THREADS) cum[i] = a.items_before[i];
    } else {
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
                    n = taken(a, rows) ? (rows + ITEM - 1) / ITEM * a.Hkv : 0;
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
        if (blockIdx.x == 0)
            for (int b = tid; b < a.requests; b += THREADS) check_lengths(a, b);
        if (a.first_launch) {  // rows that belong to no request
            const int64_t from = static_cast<int64_t>(rows_before(a, a.requests)) * a.Hq * D / 8, to = a.T * a.Hq * D / 8;
            for (int64_t i = from + static_cast<int64_t>(blockIdx.x) * THREADS + tid; i < to;
                 i += static_cast<int64_t>(gridDim.x) * THREADS)
                reinterpret_cast<uint4 *>(a.out)[i] = make_uint4(0, 0, 0, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // the other CTA's barriers are there
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    int items;
    if constexpr (Args::kShared) items = cum[a.counts[0]];
    else items = cum[a.requests];
    unsigned int *const counter = reinterpret_cast<unsigned int *>(a.scratch + PROMPT_COUNTERS);
    // the k-th item of this CTA or pair (items or more: there is none, or it was not announced in time)
    auto item_at = [&](int k) -> int {
        const bool told = wait_for<PAIR>(&bar.ifull[k % QUEUE], (k / QUEUE) & 1, a.status);
        const int index = *static_cast<volatile int *>(&bar.item[k % QUEUE]);
        return __all_sync(0xffffffffu, told) ? index : items;
    };
    // until the products of so many key tiles are done
    auto finish = [&](int g) {
        if (g > 0) wait_for(&bar.vfree[(g - 1) % 2], ((g - 1) / 2) & 1, nullptr);
    };

    if (warp < 4) {
        // ------------------------------------------------ softmax, epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFT_REGS));
        const int r = tid;
        const uint32_t t_row = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        int g = 0;  // key tiles so far, over all items
        const int window = static_cast<int>(min(a.window, int64_t(0x7fffffff)));
        const int sinks = a.window > 0 ? static_cast<int>(min(a.sinks, int64_t(0x7fffffff))) : 0;
        for (int k_item = 0;; ++k_item) {
            const int index = item_at(k_item);
            if (index >= items) break;
            const Item cur = item_of<ITEM>(a, cum, order, index, G);
            float Fr = 0.f;
            float M = NONE, l = 0.f;
            // positions of this thread's row, of the CTA's first and of its last
            const int p = cur.base + (cur.r0 + min(rank * ROWS + r, cur.rows - 1)) / G;
            const int p_lo = cur.base + (cur.r0 + min(rank * ROWS, cur.rows - 1)) / G;
            const int p_hi = cur.base + (cur.r0 + min(rank * ROWS + ROWS, cur.rows) - 1) / G;
            for (int i = 0; i < cur.n; ++i, ++g) {
                const int j0 = cur.key0(i);
                const Meta &meta = reinterpret_cast<const Meta *>(smem + L::meta)[g % METAS];
                const uint32_t t_s = t_row + COL_S + (g & 1) * KEYS;
                wait_for(&bar.sfull[g & 1], (g >> 1) & 1, a.status);
                tc_fence_after();
                uint32_t x0[32];
                tmem_ld_32x32b_x32(t_s, x0);
                wait_for(&bar.known[g % METAS], (g / METAS) & 1, a.status);
                if (i == 0) Fr = q_factor[(k_item & 1) * ROWS + r];
                const uint2 held = *reinterpret_cast<const uint2 *>(meta.held);
                const bool free = (held.x & held.y) == 0x01010101u && j0 + KEYS <= p_lo + 1 &&
                                  (window == 0 || p_hi - j0 < window || j0 + KEYS <= sinks);
                // 32 keys at a time: scores in, weights out into the columns of scores already read (half as wide)
                float m = M, scaled = 1.f, added = 0.f;
                // -infinity for the keys of chunk c that this row does not see
                auto hide = [&](uint32_t(&x)[32], int c) {
                    // keys from .. upto of these 32 are seen, and those before `first`
                    const int at = j0 + 32 * c;
                    auto below = [](int n) -> uint32_t { return n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1 : 0u; };
                    const uint32_t pages = (c & 2 ? held.y : held.x) >> (16 * (c & 1));
                    uint32_t see = window == 0 ? 0xffffffffu : ~below(p - window + 1 - at) | below(sinks - at);
                    see &= below(min(p + 1, cur.end) - at) & ((pages & 1u) * 0xffffu | (pages >> 8 & 1u) * 0xffff0000u);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = see >> e & 1u ? x[e] : 0xff800000u;  // -infinity
                };
                float4 kf4 = {}, ve4 = {}, vf4 = {};  // factors of two chunks' cache tiles
                auto weigh = [&](uint32_t(&x)[32], int c) {
                    float top[2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t *const y = x + q * 16;
                        float t[2] = {fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1])),
                                      fmaxf(__uint_as_float(y[2]), __uint_as_float(y[3]))};
#pragma unroll
                        for (int e = 4; e < 16; e += 2)
                            t[e / 2 & 1] = max3(t[e / 2 & 1], __uint_as_float(y[e]), __uint_as_float(y[e + 1]));
                        top[q] = fmaxf(t[0], t[1]);
                    }
                    const float2 kf = c & 1 ? make_float2(kf4.z, kf4.w) : make_float2(kf4.x, kf4.y);
                    const float2 B = c & 1 ? make_float2(ve4.z, ve4.w) : make_float2(ve4.x, ve4.y);
                    const float2 vf = c & 1 ? make_float2(vf4.z, vf4.w) : make_float2(vf4.x, vf4.y);
                    const float A[2] = {factor(Fr, kf.x), factor(Fr, kf.y)};
                    const float mx = fmaxf(fmaf(top[0], A[0], B.x), fmaf(top[1], A[1], B.y));
                    if (__any_sync(0xffffffffu, mx > m + 15.f)) {
                        // the reference moves: what this tile has written so far, its
                        // sum, and (below) what earlier tiles left shrink with it
                        const float up = fmaxf(m, ceilf(mx) - 7.f), f = ex2(m - up);  // whole numbers: f is a power of two
                        m = up;
                        added *= f;
                        scaled *= f;
                        if (c > 0) {
                            // (in binary32: f may lie below binary16's smallest number
                            // where its product with a weight does not)
                            tmem_st_wait();
#pragma unroll 1
                            for (int q = 0; q < c; ++q) {
                                uint32_t w[16];
                                tmem_ld_32x32b_x16(t_s + 16 * q, w);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 16; ++e) w[e] = pack_f16(f16_lo(w[e]) * f, f16_hi(w[e]) * f);
                                tmem_st_32x32b_x16(t_s + 16 * q, w);
                            }
                        }
                    }
                    const float Bm[2] = {B.x - m, B.y - m}, of[2] = {vf.x, vf.y};
                    uint32_t w[16];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float2 sum[2];
                        const uint32_t *const y = x + q * 16;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float2 v = fma2(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])),
                                            make_float2(A[q], A[q]), make_float2(Bm[q], Bm[q]));
                            v.x = ex2(v.x);
                            v.y = ex2(v.y);
                            if (e < 4) sum[e / 2] = v;
                            else sum[(e / 2) & 1] = add2(sum[(e / 2) & 1], v);
                            w[8 * q + e / 2] = pack_f16(v.x, v.y);
                        }
                        sum[0] = add2(sum[0], sum[1]);
                        added = fmaf(sum[0].x + sum[0].y, of[q], added);
                    }
                    tmem_st_32x32b_x16(t_s + 16 * c, w);
                };
                if (!free) {
                    // in tensor memory, so that the loop below has no branch for it (alone on
                    // the SM it takes 1520 cycles a tile with one, 1360 without; the factors
                    // asked for before the scores are there, 1290)
                    arrived(x0);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        if (c > 0) {
                            tmem_ld_32x32b_x32(t_s + 32 * c, x0);
                            arrived(x0);
                        }
                        hide(x0, c);
                        tmem_st_32x32b_x32(t_s + 32 * c, x0);
                    }
                    tmem_st_wait();
                    tmem_ld_32x32b_x32(t_s, x0);
                }
                // the next scores are on their way while these are worked on
                uint32_t x1[32];
#pragma unroll 1
                for (int c = 0; c < 4; c += 2) {
                    kf4 = *reinterpret_cast<const float4 *>(meta.k_factor + 2 * c);
                    ve4 = *reinterpret_cast<const float4 *>(meta.v_exponent + 2 * c);
                    vf4 = *reinterpret_cast<const float4 *>(meta.v_factor + 2 * c);
                    arrived(x0);
                    tmem_ld_32x32b_x32(t_s + 32 * c + 32, x1);
                    weigh(x0, c & 2);
                    arrived(x1);
                    if (c == 0) tmem_ld_32x32b_x32(t_s + 64, x0);
                    weigh(x1, (c & 2) + 1);
                }
                if (__any_sync(0xffffffffu, m != M)) {
                    l *= scaled;
                    if (i > 0) {  // O holds the earlier tiles once their product is done
                        wait_for(&bar.vfree[(g - 1) % 2], ((g - 1) / 2) & 1, a.status);
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
                l += added;
                tmem_st_wait();
                tc_fence_before();
                warp_arrive<PAIR>(&bar.pfull[g & 1], lane);
            }
            wait_for(&bar.vfree[(g - 1) % 2], ((g - 1) / 2) & 1, a.status);
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const bool on = rank * ROWS + r < cur.rows;
            const int row = cur.r0 + (on ? rank * ROWS + r : 0);
            uint16_t *const dst = a.out + (static_cast<int64_t>(cur.tok0 + row / G) * a.Hq + cur.h * G + row % G) * D;
            float *part = nullptr;
            if constexpr (Args::kShared)
                if (cur.place >= 0) {
                    const int64_t at = cur.place + static_cast<int64_t>(row / G) * a.Hq + cur.h * G + row % G;
                    part = a.values + at * D;
                    if (on) a.weights[at] = make_float2(M, l);
                }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld_32x32b_x32(t_row + 32 * c, o);
                tmem_ld_wait();
                if (on) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
                        const uint32_t *x = o + 8 * e;  // dimensions 0 4 1 5 2 6 3 7
                        const int at[8] = {0, 2, 4, 6, 1, 3, 5, 7};
                        if (Args::kShared && part) {
                            store8(part + 32 * c + 8 * e, x[at[0]], x[at[1]], x[at[2]], x[at[3]], x[at[4]], x[at[5]], x[at[6]], x[at[7]]);
                            continue;
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_bf16(__uint_as_float(x[at[2 * k]]) * inv, __uint_as_float(x[at[2 * k + 1]]) * inv);
                        *reinterpret_cast<uint4 *>(dst + 32 * c + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            tc_fence_before();
        }
    } else if (warp < 4 + 2 * FORM_WARPS) {
        // ------------------------------------------- operands from the cache
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(FORM_REGS));
        // Q of an item: 16 rows a warp, D / 8 lanes a row with 16 bytes each, and
        // the factors of their scores.
        auto build = [&](const Item &it, int k_item) {
            constexpr int LANES = D / 8, AT_ONCE = 32 / LANES, STEPS = 16 / AT_ONCE, BATCH = STEPS < 8 ? STEPS : 8;
            const int first = (warp - 4) * 16 + lane / LANES, col = lane % LANES;
#pragma unroll 1
            for (int s = 0; s < STEPS; s += BATCH) {
                uint4 rows[BATCH];  // all on their way together
#pragma unroll
                for (int e = 0; e < BATCH; ++e) {
                    const int row = it.r0 + min(rank * ROWS + first + (s + e) * AT_ONCE, it.rows - 1), t = row / G;
                    rows[e] = *reinterpret_cast<const uint4 *>(a.q + static_cast<int64_t>(it.tok0 + t) * a.q_stride +
                                                               (it.h * G + row - t * G) * D + col * 8);
                }
#pragma unroll
                for (int e = 0; e < BATCH; ++e) {
                    const int r = first + (s + e) * AT_ONCE;
                    const uint4 v = rank * ROWS + r < it.rows ? rows[e] : make_uint4(0, 0, 0, 0);
                    // the largest |q| by its exponent: without signs, as whole numbers
                    const unsigned big2 = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                   __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                    unsigned big = max(big2 & 0xffffu, big2 >> 16);
                    if (LANES == 32) big = __reduce_max_sync(0xffffffffu, big);
                    else
#pragma unroll
                        for (int o = 1; o < LANES; o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
                    int kappa = big ? 13 - (static_cast<int>(big >> 7) - 127) : 0;
                    kappa = min(max(kappa, -110), 110);
                    if (col == 0)
                        q_factor[(k_item & 1) * ROWS + r] = fmaxf(fabsf(a.scale) * 1.4426950408889634f * pow2(-kappa), 1e-37f);
                    const float up = a.scale < 0.f ? -pow2(kappa) : pow2(kappa);
                    const float x0 = __uint_as_float(v.x << 16) * up, x1 = __uint_as_float(v.x & 0xffff0000u) * up;
                    const float x2 = __uint_as_float(v.y << 16) * up, x3 = __uint_as_float(v.y & 0xffff0000u) * up;
                    const float x4 = __uint_as_float(v.z << 16) * up, x5 = __uint_as_float(v.z & 0xffff0000u) * up;
                    const float x6 = __uint_as_float(v.w << 16) * up, x7 = __uint_as_float(v.w & 0xffff0000u) * up;
                    *reinterpret_cast<uint4 *>(smem + L::q + r * 128 + (col >> 3) * SUB + (((col & 7) ^ (r & 7)) << 4)) =
                        make_uint4(pack_f16(x0, x4), pack_f16(x1, x5), pack_f16(x2, x6), pack_f16(x3, x7));
                }
            }
            fence_proxy_async_smem();
            warp_arrive<PAIR>(&bar.qfull, lane);
        };
        // Four warps for K and four for V run the same code.  Of a key tile a
        // warp forms two parts (h = 0, 1) of HALF pieces, a piece being the 16
        // tokens of a cache tile in one group of 64 dimensions:
        //   K, a pair's   cache tile 4 rank + w; part h: its groups HALF h ..
        //   K, alone      part h: cache tile 2 w + h, its one group
        //   V             part h: cache tile 2 w + h, this CTA's groups
        // and finds the largest scale of two cache tiles (of a pair's K the other
        // CTA's tile 4 (1 - rank) + w as second), for the softmax of its CTA.
        constexpr int HALF = D / 128 > 0 ? D / 128 : 1;
        static_assert(PAIR ? L::V_GROUPS == HALF && G64 == 2 * HALF : G64 == 1, "pieces");
        const bool is_v = warp >= 4 + FORM_WARPS, shared = PAIR && !is_v;  // (a K tile of a pair: both parts of one tile)
        const int w = (warp - 4) % FORM_WARPS, token = lane >> 1, half = lane & 1, x7 = token & 7;
        const int c0 = shared ? 4 * rank + w : 2 * w, c1 = shared ? 4 * (rank ^ 1) + w : 2 * w + 1;
        const int g0 = is_v && PAIR ? rank * HALF : 0, g1 = shared ? HALF : g0;  // first group of each part
        const int row = (shared ? w * 16 : 2 * w * 16) + token;
        const int step = is_v ? SUB : L::K_SUB;                     // shared memory of the next group,
        const int part = shared ? HALF * step : 16 * 128;           // of part 1,
        const int next_buf = is_v ? L::V_GROUPS * SUB : G64 * L::K_SUB;  // of the other buffer
        unsigned char *const dst = smem + (is_v ? L::v : L::k) + row * 128;
        uint64_t *const full = is_v ? bar.vfull : bar.kfull, *const empty = is_v ? bar.vfree : bar.kfree;
        const unsigned char *const codes = a.cache + (is_v ? 8 * D : 0) + token * 32 + half * 16;
        const unsigned char *const params = a.cache + (is_v ? 17 * D : 16 * D);
        const int shift = a.bs_log2 - 4;                  // cache tiles of a page and head
        const int in_page = (1 << shift) - 1;
        int g = 0;
        bool bad = false;
        for (int k_item = 0;; ++k_item) {
            const int index = item_at(k_item);
            if (index >= items) break;
            const Item it = item_of<ITEM>(a, cum, order, index, G);
            const int32_t *const pages = a.block_table + static_cast<int64_t>(it.b) * a.max_blocks;
            // Lane 0 looks after cache tile c0, lane 1 after c1 (and so on): its
            // tokens in key tile i (none if no row sees any of them: the caller may
            // have given such a page back), the page (asked for a step before it is looked
            // at), its number among all cache tiles (of 18 D bytes: 32 bits are
            // enough for terabytes).
            const int c = lane & 1 ? c1 : c0;
            const int from = it.first - 15 - c * 16, upto = it.sink - c * 16, end = it.end - c * 16;  // of key0
            auto tokens = [&](int i) -> int {
                const int at = it.key0(i);
                return i < it.n && (at >= from || at < upto) ? min(max(end - at, 0), 16) : 0;
            };
            auto page_of = [&](int i) -> int { return tokens(i) > 0 ? pages[(it.key0(i) + c * 16) >> a.bs_log2] : -1; };
            auto number = [&](int i, int id) -> unsigned {
                const int at = (it.key0(i) >> 4) + c;
                return ((static_cast<unsigned>(id) * a.Hkv + it.h) << shift) + (at & in_page);
            };
            struct Tile {
                uint4 raw[2][HALF];
                uint32_t par[2][HALF];  // (scale, zero) of this lane's token
                uint2 all[2];           // of tokens 2 (lane % 8) and one more in group lane / 8, of both cache tiles
                int n0, n1;             // tokens there are
            };
            // (without branches: where the tokens end is looked at when the values are
            // used.  With the loads behind a test of it a tile's ten of them waited for
            // one another, 1400 cycles of each tile's 3900)
            auto load = [&](int i, int id) -> Tile {
                Tile t;
                int n = tokens(i);
                if (n > 0 && (id < 0 || id >= a.num_blocks)) {
                    bad = true;
                    n = 0;
                }
                const unsigned mine = n > 0 ? number(i, id) : 0u;  // (nothing there: some tile)
                t.n0 = __shfl_sync(0xffffffffu, n, 0);
                t.n1 = __shfl_sync(0xffffffffu, n, 1);
                const size_t o0 = static_cast<size_t>(__shfl_sync(0xffffffffu, mine, 0)) * kv4_tile_bytes(D);
                const size_t o1 = static_cast<size_t>(__shfl_sync(0xffffffffu, mine, 1)) * kv4_tile_bytes(D);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const size_t o = h && !shared ? o1 : o0;
                    const int grp = h ? g1 : g0;
#pragma unroll
                    for (int q = 0; q < HALF; ++q) {
                        t.raw[h][q] = *reinterpret_cast<const uint4 *>(codes + o + (grp + q) * 512);
                        t.par[h][q] = *reinterpret_cast<const uint32_t *>(params + o + ((grp + q) * 16 + token) * 4);
                    }
                    t.all[h] = *reinterpret_cast<const uint2 *>(params + (h ? o1 : o0) + lane % (8 * G64) * 8);
                }
                return t;
            };
            // e such that every scale of a cache tile < 2^(e + 11)
            auto exponent = [&](uint2 x, int n) -> int {
                // (no stale scale past the end)
                const unsigned first = 2 * (lane & 7) < n ? x.x & 0x7fffu : 0u, second = 2 * (lane & 7) + 1 < n ? x.y & 0x7fffu : 0u;
                const unsigned bits = __reduce_max_sync(0xffffffffu, max(first, second));
                return bits ? static_cast<int>(__float_as_uint(f16_lo(bits)) >> 23) - 137 : -11;
            };
            Tile tile = load(0, page_of(0));
            int id = page_of(1);
            // (Q's place is free when the last product Q K of the item before is done)
            if (g > 0) wait_for(&bar.kfree[(g - 1) % BUFS], ((g - 1) / BUFS) & 1, a.status);
            build(it, k_item);
#pragma unroll 1
            for (int i = 0; i < it.n; ++i) {
                const int gi = g + i, buf = gi % BUFS, id2 = page_of(i + 2);
                const Tile next = load(i + 1, id);  // on its way while this one is formed
                Meta &meta = reinterpret_cast<Meta *>(smem + L::meta)[gi % METAS];
                const int e0 = exponent(tile.all[0], tile.n0), e1 = exponent(tile.all[1], tile.n1);
                if (is_v) {
                    // (that the operands of the tile before could be written shows that
                    // the softmax is past the tile that had this entry)
                    if (lane < 2) {
                        const int e = lane ? e1 : e0;
                        meta.v_exponent[c] = static_cast<float>(e);
                        meta.v_factor[c] = pow2(-e);
                        meta.held[c] = (lane ? tile.n1 : tile.n0) > 0;
                    }
                }
                if (!is_v) {
                    // (that the operands of two tiles before have been used shows the same)
                    if (gi >= BUFS) wait_for(&empty[buf], (gi / BUFS - 1) & 1, a.status);
                    if (lane < 2) meta.k_factor[c] = pow2(lane ? e1 : e0);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.known[gi % METAS]);
                if (is_v && gi >= BUFS) wait_for(&empty[(gi + 2 - BUFS) % 2], ((gi + 2 - BUFS) / 2 - 1) & 1, a.status);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float up = pow2(-(h && !shared ? e1 : e0));
                    const bool there = token < (h && !shared ? tile.n1 : tile.n0);
#pragma unroll
                    for (int q = 0; q < HALF; ++q) {
                        const uint32_t par = there ? tile.par[h][q] : 0u;
                        const float s = f16_lo(par) * up, z = f16_hi(par);
                        form(tile.raw[h][q], pack_f16(s, s), pack_f16(-1024.f - z, -1024.f - z), pack_f16(-64.f - z, -64.f - z),
                             dst + buf * next_buf + h * part + q * step, x7, half);
                    }
                }
                fence_proxy_async_smem();
                warp_arrive<PAIR>(&full[buf], lane);
                tile = next;
                id = id2;
            }
            g += it.n;
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kDevBadIndex);
    } else {
        // ------------------------------------------------------- products
        // (the second CTA of a pair leaves all of it to the first)
        const uint32_t qa = smem_u32(smem + L::q), ka = smem_u32(smem + L::k), va = smem_u32(smem + L::v);
        int g = 0;
        auto qk = [&](int gi) {
            const int buf = gi % BUFS;
            wait_for(&bar.kfull[buf], (gi / BUFS) & 1, a.status);
            tc_fence_after();
            const uint32_t kb = ka + buf * G64 * L::K_SUB;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                product<PAIR>(tmem + COL_S + (gi & 1) * KEYS, smem_desc_sw128_kmajor(qa + (k >> 2) * SUB + (k & 3) * 32),
                              smem_desc_sw128_kmajor(kb + (k >> 2) * L::K_SUB + (k & 3) * 32), IDESC_QK, k != 0);
            commit<PAIR>(&bar.sfull[gi & 1]);
            commit<PAIR>(&bar.kfree[buf]);
        };
        auto pv = [&](int gi, bool first) {
            const int buf = gi % BUFS;
            wait_for(&bar.vfull[buf], (gi / BUFS) & 1, a.status);
            wait_for(&bar.pfull[gi & 1], (gi >> 1) & 1, a.status);
            tc_fence_after();
            const uint32_t vb = va + buf * L::V_GROUPS * SUB;
#pragma unroll
            for (int k = 0; k < KEYS / 16; ++k)
                product_tmem<PAIR>(tmem, tmem + COL_S + (gi & 1) * KEYS + 8 * k, desc_sw128_mn(vb + k * 2048, SUB), IDESC_PV,
                                   !(first && k == 0));
            commit<PAIR>(&bar.vfree[gi % 2]);
        };
        auto announce = [&](int k, int index) {
            if (lane == 0) {
                bar.item[k % QUEUE] = index;
                if (PAIR) {
                    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer(&bar.item[k % QUEUE], 1)), "r"(index) : "memory");
                    arrive_at(peer(&bar.ifull[k % QUEUE], 0));
                    arrive_at(peer(&bar.ifull[k % QUEUE], 1));
                } else mbar_arrive(&bar.ifull[k % QUEUE]);
            }
            __syncwarp();
        };
        if (rank == 0) {
            // the first item is the CTA's (pair's) number, the others come from the
            // counter; one is fetched ahead.  A slot of the ring is written again
            // four items later, when every role has left it: the softmax is at
            // most an item behind, and the forming warps are ahead.
            const int workers = static_cast<int>(gridDim.x) / CTAS;
            int index = static_cast<int>(blockIdx.x) / CTAS;
            if (!(a.inject & kInjectStallPipeline)) announce(0, index);
            if (a.inject) index = items;  // test-only injection: no item announced, or none worked on
            for (int k = 0; index < items; ++k) {
                int next = 0;
                if (lane == 0) next = workers + static_cast<int>(atomicAdd(counter, 1u));
                next = __shfl_sync(0xffffffffu, next, 0);
                announce(k + 1, next);
                const Item it = item_of<ITEM>(a, cum, order, index, G);
                index = next;
                wait_for(&bar.qfull, k & 1, a.status);
#pragma unroll 1
                for (int i = 0; i <= it.n; ++i) {
                    if (i < it.n) qk(g + i);
                    if (i > 0) pv(g + i - 1, i == 1);
                }
                g += it.n;
            }
            // the last to run out of items leaves the counters at zero
            if (lane == 0) {
                __threadfence();
                if (atomicAdd(counter + 1, 1u) == static_cast<unsigned>(workers) - 1) {
                    counter[0] = 0;
                    counter[1] = 0;
                }
                if (PAIR && (*reinterpret_cast<volatile unsigned int *>(a.status) & kDevTimeout)) {
                    bar.late = g;
                    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer(&bar.late, 1)), "r"(g) : "memory");
                }
            }
            __syncwarp();
        }
        // tensor memory is released only when every product has completed
        finish(g);
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) {
        cluster_sync();  // nothing of the other CTA's is in use any more
        if (bar.late) {
            // a role of the second CTA may have left early: it ends when it too has been
            // told that the last products are done
            if (rank == 1 && warp == 12) finish(bar.late);
            cluster_sync();
        }
    }
    if (warp == 12) {
        tc_fence_after();
        tmem_give<PAIR>(tmem);
    }
}

template <int D, bool PAIR, class Args>
cudaError_t launch(const Args &a, cudaStream_t st, const DeviceInfo &dev) {
    // (of kv4_prefix_attention `requests` is the most pieces there can be)
    const int smem = 1024 + PromptSmem<D, PAIR>::cum + ((Args::kShared ? 1 : 2) * a.requests + 1) * 4;
    if (smem > dev.max_smem_optin) return cudaErrorNotSupported;
    static SmemLimit limit;
    if (cudaError_t e = limit.ensure(reinterpret_cast<const void *>(attn_prompt_kernel<Args, D, PAIR>), dev.device, smem)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(PAIR ? dev.num_sms & ~1 : dev.num_sms));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, attn_prompt_kernel<Args, D, PAIR>, a);
}

}  // namespace

cudaError_t launch_kv4_prompt(const Kv4AttnArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    if (D == 64) return launch<64, false>(a, st, dev);
    if (D == 128) return launch<128, true>(a, st, dev);
    return launch<256, true>(a, st, dev);
}

cudaError_t launch_kv4_prompt(const Kv4SharedArgs &a, int D, cudaStream_t st, const DeviceInfo &dev) {
    if (D == 64) return launch<64, false>(a, st, dev);
    if (D == 128) return launch<128, true>(a, st, dev);
    return launch<256, true>(a, st, dev);
}

}  // namespace w4
