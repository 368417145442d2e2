// tg_tree_attention.cu -- attention of drafted token trees (or single tokens)
// over a paged cache for sm_100a (tcgen05 + TMEM + TMA); tg_tree_attention of
// include/tg_cache.h.
//
// Rows.  The query heads that share a key head see the same keys, so a tile of
// 128 query rows holds (token, head) pairs of one request and key head:
// 128 / group tokens with all their heads, one TMA box of the packed queries.
// Keys come in tiles of 128: first the request's cached tokens, page by page
// (a TMA box each, the block table's entry as a coordinate), then its drafted
// tokens from their dense tensor.
//
// Work division.  A unit is (request, key head, pair of query tiles); its
// length is the request's number of key tiles.  Only the device knows the
// lengths, so each CTA sums them up itself and takes an equal share of all key
// tiles, wherever units begin and end: the last unit of a CTA's share may go
// on in the next CTA.  A unit that lies in one CTA is finished there; the
// parts of a divided one leave their unnormalised output, maxima and sums in
// the workspace, and a second kernel joins them in the CTAs' order.
//
// One CTA per SM, twelve warps:
//   warps 0-3, 4-7  two softmax groups, thread r of a group owns query row r
//                   (TMEM lane r).  A unit with two query tiles gives one to
//                   each group, both over all key tiles; a unit with one gives
//                   it to both, one group taking the even key tiles and the
//                   other the odd ones, each with its own maximum, sum and
//                   output, joined at the end in tensor memory.  Either way
//                   one group's exponentials run beside the other's products.
//   warps 8, 10, 11 TMA producers: queries, and keys and values through one
//                   ring in the order in which the products need them, each
//                   a third of a tile's pages (with pages of 16 tokens one
//                   alone held the stream of 64 requests to 4.0 TB/s, three
//                   gave 5.4, and 5.9 with what was made faster since).
//   warp 9          TMEM allocator and MMA issuer.
// Step i (a key tile of a query tile) belongs to group t = i mod 2 and has two
// halves of 64 keys, each with its own score columns.  The issuer's order is
// S_0 S_1, then for i = 0, 1, ... and each half h: P_i,h V, S_i+2,h.  P_i,h (16
// bits) overwrites S_i,h in tensor memory, and S_i+2,h follows P_i,h V in the
// tensor pipe's order; while a group exponentiates one half, the other half's
// product and next scores are made, so it does not wait for them.  A half that
// lies past the last key is left out by all.
// TMEM: S_t,h / P_t,h at columns 128 t + 64 h, O_t at 256 + D t.
//
// Masked places.  A masked score becomes -inf before the maximum.  A masked
// key's value still enters the product with weight 0, so values that are not
// finite there would spread: in a tile that is not wholly visible the group
// zeroes, in shared memory, the values of rows past the end, and elements
// that are not finite; what visible drafted tokens lose by that is added
// back to the written output from global memory (a rare path behind a flag).
//
// Without a mask a token sees its request's drafted tokens up to itself, but a
// unit's length does not depend on its query tiles: tiles above the diagonal are
// computed and masked, so a long prompt takes about twice the products of its
// definition (2048 tokens of 32 heads 104 us, floor 21).
//
// What bounds it (bursts from a captured graph; then back to back, at the power
// limit).  HBM where a key head has one or two tiles of rows and the cache is
// long: 151 and 170 us for 872 MB (2 requests over up to 131072 tokens, 27 tokens
// x 4 heads a key head), 213 and 249 us for 1238 MB (64 requests, up to 16
// tokens, up to 8192, pages of 16).  With many rows the tensor core's 64-key
// products and the softmax, both near 1800 cycles per 64 keys of both groups:
// 169 and 200 us for 139.6 GFLOP (16 requests over 4096, 64 tokens x 8 heads),
// where these products are 206,000 of an SM's 254,000 active cycles.  With short
// contexts the latencies of a CTA's start, of a part's end and of the join.
//
// Every wait is bounded; see tg_attention.cu.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "tg_attn.cuh"
#include "tg_cache.h"
#include "tg_cache_internal.h"
#include "tg_internal.h"

namespace tgt {

using namespace tga;

constexpr int kRows = 128;         // query rows of a tile (TMEM lanes)
constexpr int kKeys = 128;         // keys of a tile
constexpr int kHalf = 64;          // keys of a half step (score columns)
constexpr int kAtom = 64;          // head-dim elements per 128-byte swizzle atom
constexpr int kAtomBytes = 128 * 128;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kWarps = 12;
constexpr int kProducers = 3;      // warps 8, 10 and 11
constexpr int kLongPart = 16;      // key tiles of a part whose unused query rows are zeroed
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOBase = 256;
constexpr int kMaxCtas = 148;      // one per SM of a B200; the workspace's size goes by it

// Error word bits (shared with the other kernels of the library).
constexpr unsigned kErrTreeProducer = 1024u;
constexpr unsigned kErrTreeMma = 2048u;
constexpr unsigned kErrTreeSoftmax = 4096u;
constexpr unsigned kErrTreeDrain = 8192u;
constexpr unsigned kErrTreeSmem = 16384u;

// What a CTA leaves for the joining kernel: the unit that begins in its share
// and goes on behind it (first row of the packing, its key head, rows of its
// two query tiles), and how many CTAs have a part of it (0: none).
struct Split {
    int ctas, head, first, rows[2], pad[3];
};

struct TreeParams {
    const int32_t *lens, *starts, *tables, *mask;
    const uint16_t *q, *k, *v;    // queries, drafted keys and values
    uint16_t *out;
    int64_t q_token_stride, q_head_stride;
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    int64_t out_token_stride, out_head_stride;
    int64_t table_stride, max_len, mask_stride;
    int tokens, batch, kv_heads, group, tile_tokens, words, page_shift;
    float scale_log2, lag;        // scale * log2(e); scores that make 8 of it
    Split *split;                 // [CTAs]
    float *part;                  // [CTAs][first, last part][query tile][D + 2][128]
    int inject;
    uint64_t wait_limit_ns;
    unsigned *error_word;
};

template <int D>
struct TreeShape {
    static_assert(D == 64 || D == 128, "head_dim 64 or 128");
    static constexpr int kAtoms = D / kAtom;
    static constexpr int kTileBytes = kAtoms * kAtomBytes;   // one 128-row tile
    static constexpr int kStages = D == 128 ? 5 : 10;        // ring of key and value tiles
    static constexpr int kQOff = 0;                          // two query tiles
    static constexpr int kKVOff = 2 * kTileBytes;
    static constexpr int kMlOff = kKVOff + kStages * kTileBytes;   // (m, l) of both groups
    static constexpr int kBarOff = kMlOff + 2 * kRows * 8;
    // q_full[2], q_empty[2], kv_full[], kv_empty[], s_full[2][2], p_full[2][2],
    // pv_done[2][2], o_free, ml_full, drain
    static constexpr int kNumBars = 4 + 2 * kStages + 12 + 3;
    static constexpr int kTmemSlotOff = kBarOff + kNumBars * 8;
    static constexpr int kAbortOff = kTmemSlotOff + 4;
    static constexpr int kFlagOff = kAbortOff + 4;
    static constexpr int kItemsOff = kFlagOff + 4;           // ring items of each producer
    static constexpr int kIdsOff = kItemsOff + 4 * kProducers;   // page entries, 2 x 32 each
    static constexpr int kDynamicBytes = kIdsOff + 256 * kProducers;
    static_assert(kDynamicBytes <= 232448, "shared-memory budget");
    // Floats of one part of a divided unit's query tile: O (by columns), m, l.
    static constexpr int kPartFloats = (D + 2) * kRows;
};

constexpr size_t split_bytes() { return (sizeof(Split) * kMaxCtas + 255) / 256 * 256; }

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (BF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        return pack_half2(lo, hi);
    }
}

// Probabilities, and their sum beside them, are 2^((score - m) sl2 + kLift).
// In fp16 that is 2^15 at most (m may lag 8 log2 units behind), and weights
// down to 2^-32 of the largest count; without the lift those below 2^-25 would be
// zero in the product and yet part of the sum (32768 keys of weight 2^-25.2
// beside two of weight 1, whose values were 0, gave 0 instead of 4.1e-4).  bf16
// has fp32's range.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;

// Instruction descriptor bits that select bf16 for A and B.
template <bool BF16>
constexpr uint32_t kTypeBits = BF16 ? (1u << 7) | (1u << 10) : 0u;

// True in one lane of the (converged) warp, the same one every time.  A branch
// on it tells the compiler that one thread runs it, so that the descriptors of
// the products are kept in uniform registers; behind `lane == 0` each product
// took about 110 cycles to issue, more than the tensor core needs for it.
__device__ __forceinline__ bool elect_lane()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// The largest of three, NaN if one is (one instruction on sm_100).
__device__ __forceinline__ float max3_nan(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst_smem, const CUtensorMap *tm,
                                            uint64_t *bar, int32_t x, int32_t y, int32_t z,
                                            int32_t w)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst_smem),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// An element of a 16-bit tensor.
template <bool BF16>
__device__ __forceinline__ float value_of(uint16_t bits)
{
    if constexpr (BF16)
        return __uint_as_float(static_cast<uint32_t>(bits) << 16);
    else
        return __half2float(__ushort_as_half(bits));
}

// True for infinities and NaN: an exponent of all ones.
template <bool BF16>
__device__ __forceinline__ bool not_finite(uint16_t bits)
{
    constexpr uint16_t kExp = BF16 ? 0x7F80u : 0x7C00u;
    return (bits & kExp) == kExp;
}

// a / b for a >= 0, b > 0.  A 64-bit division takes several hundred cycles and as
// many instructions, which are kept out of the way.
__device__ __noinline__ int64_t quotient64(int64_t a, int64_t b) { return a / b; }

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return quotient64(a, b);
}

// A request: its drafted rows, cached tokens, tiles and work.
struct Request {
    int s0, n, ctx;      // first drafted row, drafted tokens, cached tokens
    int ctx_tiles, nk;   // key tiles of the cache, and of all keys
    int q_tiles, pairs;  // query tiles, and pairs of them
    int64_t work;        // key tiles of all its units
};

__device__ __forceinline__ Request request(const TreeParams &p, int b)
{
    Request r;
    int s0 = p.starts[b], s1 = p.starts[b + 1];
    const int64_t len = p.lens[b];
    s0 = min(max(s0, 0), p.tokens);
    s1 = min(max(s1, s0), p.tokens);
    r.s0 = s0;
    r.n = s1 - s0;
    r.ctx = static_cast<int>(len < 0 ? 0 : (len < p.max_len ? len : p.max_len));
    r.ctx_tiles = (r.ctx + kKeys - 1) / kKeys;
    r.nk = r.ctx_tiles + (r.n + kKeys - 1) / kKeys;
    r.q_tiles = (r.n + p.tile_tokens - 1) / p.tile_tokens;
    r.pairs = (r.q_tiles + 1) >> 1;
    r.work = static_cast<int64_t>(p.kv_heads) * r.pairs * r.nk;
    return r;
}

// The parts of units in a CTA's share, in order; every warp walks through them
// by itself, all lanes together.  Where a share begins is found once per CTA.
struct Walk {
    int64_t left;        // key tiles left of the share, from the current part's end
    int b;
    Request r;
    // the current part: key tiles [k0, k1) of a unit
    int head, pair, k0, k1;
    bool two;            // both query tiles of the pair exist

    __device__ __forceinline__ void part()
    {
        k1 = left < r.nk - k0 ? k0 + static_cast<int>(left) : r.nk;
        left -= k1 - k0;
        two = 2 * pair + 1 < r.q_tiles;
    }
    // The next part (k0 == k1 < nk: the first one, set up by the caller).
    __device__ __forceinline__ bool next(const TreeParams &p, int lane)
    {
        if (left <= 0) return false;
        if (k1 == r.nk) {
            k0 = 0;
            if (++pair == r.pairs) {
                pair = 0;
                ++head;
            }
            if (head == p.kv_heads) {
                head = 0;
                // the next request that has work
                for (;;) {
                    const int mine = b + 1 + lane;
                    const bool has = mine < p.batch && request(p, mine).work > 0;
                    const unsigned any = __ballot_sync(0xffffffffu, has);
                    if (any) {
                        b += __ffs(any);
                        break;
                    }
                    b += 32;
                    if (b >= p.batch) return false;
                }
                r = request(p, b);
            }
        }
        part();
        return true;
    }
    __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == r.nk; }
    // Keys of key tile kj from its first on (more than 128 where it is full),
    // and its halves that have any.
    __device__ __forceinline__ int keys(int kj) const
    {
        return kj >= r.ctx_tiles ? r.n - (kj - r.ctx_tiles) * kKeys : r.ctx - kj * kKeys;
    }
    __device__ __forceinline__ int halves(int kj) const { return keys(kj) > kHalf ? 2 : 1; }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmKC,
                     const __grid_constant__ CUtensorMap tmVC,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const TreeParams p)
{
    using S = TreeShape<D>;
    constexpr int NS = S::kStages;

    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kBarOff);
    uint64_t *q_full = bars;
    uint64_t *q_empty = bars + 2;
    uint64_t *kv_full = bars + 4;
    uint64_t *kv_empty = kv_full + NS;
    uint64_t *s_full = kv_empty + NS;    // [2 t + h]: S_t,h is in TMEM
    uint64_t *p_full = s_full + 4;       // [2 t + h]: P_t,h is in TMEM (4 arrivals)
    uint64_t *pv_done = p_full + 4;      // [2 t + k mod 2]: group t's product number k is complete
    uint64_t *o_free = pv_done + 4;      // both O read (8 arrivals)
    uint64_t *ml_full = o_free + 1;      // both groups' m and l written (8 arrivals)
    uint64_t *drain_bar = ml_full + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kTmemSlotOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kAbortOff);
    volatile int *odd_values = reinterpret_cast<volatile int *>(smem + S::kFlagOff);
    volatile uint32_t *items = reinterpret_cast<volatile uint32_t *>(smem + S::kItemsOff);
    float2 *ml = reinterpret_cast<float2 *>(smem + S::kMlOff);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint64_t limit = p.wait_limit_ns;
    const int cta = static_cast<int>(blockIdx.x);
    grid_launch_dependents();

    // The swizzled tiles need a 1024-byte aligned base (the alignment asked for
    // above); uniform over the CTA.
    if (sbase & 1023u) {
        if (threadIdx.x == 0) {
            p.split[cta].ctas = 0;
            atomicOr(p.error_word, kErrTreeSmem);
        }
        return;
    }

    // A thread's run of requests; the loads are on their way during the set-up.
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.batch), b1 = min(b0 + per, p.batch);
    int64_t work = 0;
    for (int b = b0; b < b1; ++b) work += request(p, b).work;
    if (threadIdx.x < S::kNumBars) {
        uint64_t *bar = &bars[threadIdx.x];
        const uint32_t count = (bar >= kv_full && bar < kv_empty)  ? kProducers
                               : (bar >= p_full && bar < pv_done)  ? 4u
                               : (bar == o_free || bar == ml_full) ? 8u
                                                                   : 1u;
        mbar_init(bar, count);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        *odd_values = 0;
    }
    if (warp == kProducerWarp && lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmKC);
        tma_prefetch_desc(&tmVC);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == kMmaWarp) {
        tmem_alloc<1>(tmem_slot, kTmemCols);
        tmem_relinquish<1>();
    }

    // Share of this CTA, from the sums of the requests' work over the threads.
    // Scratch in the ring, which is not in use yet.
    struct Scratch {
        int64_t sum[kWarps];
        Walk walk;
    };
    Scratch &scr = *reinterpret_cast<Scratch *>(smem + S::kKVOff);
    int64_t incl = work;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) scr.sum[warp] = incl;
    __syncthreads();
    int64_t hi = incl, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) hi += scr.sum[w];
        total += scr.sum[w];
    }
    const int64_t share = quotient(total + gridDim.x - 1, gridDim.x);
    const int64_t pos0 = min(total, cta * share);
    const int64_t pos1 = min(total, pos0 + share);
    if (pos0 == pos1 && threadIdx.x == 0) p.split[cta].ctas = 0;
    // The threads whose runs hold the share's first and last key tile.
    int64_t lo = hi - work;
    if (pos0 < pos1 && lo < pos1 && hi > pos0) {
        for (int b = b0; b < b1 && lo < pos1; ++b) {
            const Request r = request(p, b);
            const int64_t end = lo + r.work;
            if (lo <= pos0 && pos0 < end) {
                Walk w;
                const int64_t rel = pos0 - lo;
                const int unit = static_cast<int>(quotient(rel, r.nk));
                w.left = pos1 - pos0;
                w.b = b;
                w.r = r;
                w.head = unit / r.pairs;
                w.pair = unit - w.head * r.pairs;
                w.k0 = w.k1 = static_cast<int>(rel - static_cast<int64_t>(unit) * r.nk);
                w.two = false;
                scr.walk = w;
            }
            if (lo < pos1 && pos1 <= end) {
                // The unit that holds the share's last key tile.
                const int64_t u = quotient(pos1 - 1 - lo, r.nk);
                const int64_t ubegin = lo + u * r.nk, uend = ubegin + r.nk;
                Split sp = {};
                if (ubegin >= pos0 && uend > pos1)
                    sp.ctas = static_cast<int>(quotient(uend - 1, share)) - cta + 1;
                sp.head = static_cast<int>(u) / r.pairs;
                const int tok0 = 2 * (static_cast<int>(u) - sp.head * r.pairs) * p.tile_tokens;
                sp.first = r.s0 + tok0;
                for (int t = 0; t < 2; ++t)
                    sp.rows[t] =
                        max(0, min(p.tile_tokens, r.n - tok0 - t * p.tile_tokens)) * p.group;
                p.split[cta] = sp;
            }
            lo = end;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    Walk walk;
    walk.left = 0;
    if (pos0 < pos1) walk = scr.walk;
    // The scratch is read before the ring's first copies land on it.
    fence_proxy_async_smem();
    __syncthreads();

    auto wait_all = [&](uint64_t *bar, uint32_t parity, unsigned site) -> bool {
        const bool ok = mbar_wait_bounded(bar, parity, abort_flag, limit, p.error_word, site);
        return __all_sync(0xffffffffu, ok);
    };

    if (warp == kProducerWarp || warp > kMmaWarp) {
        // Producer `me` of kProducers; each announces the bytes of its own copies,
        // the first one also those of whole tiles and of the queries.
        const int me = warp == kProducerWarp ? 0 : warp - kMmaWarp;
        uint32_t qc = 0, ic = 0;       // query tiles and ring items so far
        bool ok = true;
        const int shift = p.page_shift;
        const bool small = shift < 7;                     // pages of less than a tile
        const int per_tile = small ? kKeys >> shift : 1;  // pages of a tile
        const int run_shift = small ? shift - 2 : 5;      // log2 of the tiles that 32 pages fill
        volatile int *ids = reinterpret_cast<volatile int *>(smem + S::kIdsOff) + me * 64;
        while (ok && walk.next(p, lane)) {
            const Request &r = walk.r;
            const int n = walk.k1 - walk.k0;
            const int32_t *table = p.tables + static_cast<int64_t>(walk.b) * p.table_stride;
            // Lane i: page i of the run of tiles that begins with tile j of the part
            // (-1: none).
            auto page_of = [&](int j) -> int {
                const int kj = walk.k0 + j;
                if (kj >= r.ctx_tiles) return -1;
                const int64_t pi = small ? static_cast<int64_t>(kj) * per_tile + lane
                                         : (static_cast<int64_t>(kj + lane) * kKeys) >> shift;
                return (pi << shift) < r.ctx ? table[pi] : -1;
            };
            int page = page_of(0);
            for (int t = 0; me == 0 && t < (walk.two ? 2 : 1) && ok; ++t, ++qc) {
                const uint32_t slot = qc & 1u;
                if (qc >= 2) ok = wait_all(&q_empty[slot], ((qc >> 1) - 1) & 1, kErrTreeProducer);
                if (!ok) break;
                if (elect_lane()) {
                    mbar_arrive_expect_tx(&q_full[slot],
                                          p.group * p.tile_tokens * S::kAtoms * 128);
#pragma unroll
                    for (int a = 0; a < S::kAtoms; ++a)
                        tma_load_3d(sbase + S::kQOff + slot * S::kTileBytes + a * kAtomBytes, &tmQ,
                                    &q_full[slot], a * kAtom, walk.head * p.group,
                                    r.s0 + (2 * walk.pair + t) * p.tile_tokens);
                }
                __syncwarp();
            }
            // Tile j of the part into the next ring stage.  Page entries outside the
            // cache read as zeros (out of the map's range).
            auto load = [&](int j, bool value) -> bool {
                const uint32_t st = ic % NS;
                if (ic >= NS && !mbar_wait_bounded(&kv_empty[st], (ic / NS - 1) & 1, abort_flag,
                                                   limit, p.error_word, kErrTreeProducer))
                    return false;
                const uint32_t dst = sbase + S::kKVOff + st * S::kTileBytes;
                const int kj = walk.k0 + j;
                const bool skip = p.inject == 1 && cta == 0 && ic == 0;
                if (kj < r.ctx_tiles) {
                    const int left = r.ctx - kj * kKeys;
                    const int pages =
                        small ? min(per_tile, (left + (1 << shift) - 1) >> shift) : 1;
                    // rows of this producer's pages
                    const int rows = small ? (pages - me + kProducers - 1) / kProducers << shift
                                           : (me == 0 ? kKeys : 0);
                    const int y = small ? 0 : (kj * kKeys) & ((1 << shift) - 1);
                    const CUtensorMap *map = value ? &tmVC : &tmKC;
                    const int id0 = ((j >> run_shift) & 1) * 32 +
                                    (j & ((1 << run_shift) - 1)) * per_tile;
                    mbar_arrive_expect_tx(&kv_full[st], rows * S::kAtoms * 128);
                    for (int i = me; i < pages && !skip; i += kProducers) {
                        const int id = ids[id0 + i];
#pragma unroll
                        for (int a = 0; a < S::kAtoms; ++a)
                            tma_load_4d(dst + a * kAtomBytes + (i << (shift + 7)), map,
                                        &kv_full[st], a * kAtom, y, walk.head, id);
                    }
                } else {
                    mbar_arrive_expect_tx(&kv_full[st], me == 0 ? S::kTileBytes : 0);
                    const CUtensorMap *map = value ? &tmV : &tmK;
                    if (me == 0 && !skip)
#pragma unroll
                        for (int a = 0; a < S::kAtoms; ++a)
                            tma_load_3d(dst + a * kAtomBytes, map, &kv_full[st], a * kAtom,
                                        r.s0 + (kj - r.ctx_tiles) * kKeys, walk.head);
                }
                ++ic;
                return true;
            };
            // Items K_0 | K_1 V_0 | K_2 V_1 | ... | V_n-1.  The page entries of a run of
            // tiles go through shared memory, those of the next run are on their way
            // meanwhile; one elected thread waits and issues for the run.  (With the
            // entries handed from lane to lane an item took the warp about 1000
            // cycles, and 64 requests of one token and 4 heads a key head 227 us in
            // bursts; so 211.)
            for (int j0 = 0; ok && j0 < n; j0 += 1 << run_shift) {
                ids[((j0 >> run_shift) & 1) * 32 + lane] = page;
                __syncwarp();
                const int j1 = min(n, j0 + (1 << run_shift));
                if (j1 < n) page = page_of(j1);
                if (elect_lane()) {
                    for (int j = j0; ok && j < j1; ++j) {
                        ok = load(j, false);
                        if (ok && j > 0) ok = load(j - 1, true);
                    }
                    if (ok && j1 == n) ok = load(n - 1, true);
                }
                ok = __all_sync(0xffffffffu, ok);
                ic = __reduce_max_sync(0xffffffffu, ic);
            }
        }
        // Every copy lands before shared memory goes away.  After an expiry the
        // producers may have stopped at different items: each makes up for those
        // it has not arrived at, so that all phases that were begun end.  (The
        // injected test skips one load, whose barrier never completes.)
        if (lane == 0) items[me] = ic;
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kProducers) : "memory");
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < kProducers; ++i) most = max(most, items[i]);
        if (lane == 0) {
            for (uint32_t i = ic; i < most; ++i) mbar_arrive(&kv_full[i % NS]);
            if (me == 0) {
                for (uint32_t s = 0; s < 2; ++s)
                    if (qc > s && !mbar_wait_drain(&q_full[s], ((qc - 1 - s) >> 1) & 1, limit))
                        atomicOr(p.error_word, kErrTreeDrain);
                for (uint32_t s = 0; s < NS; ++s)
                    if (most > s && !(p.inject == 1 && cta == 0 && s == 0 && most <= NS) &&
                        !mbar_wait_drain(&kv_full[s], ((most - 1 - s) / NS) & 1, limit))
                        atomicOr(p.error_word, kErrTreeDrain);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        constexpr uint32_t kIdescS = idesc_f16_f32_kk(kRows, kHalf) | kTypeBits<BF16>;
        constexpr uint32_t kIdescO = idesc_f16_f32(kRows, D) | kTypeBits<BF16>;
        constexpr uint32_t kHalfBytes = kHalf * 128;      // 64 rows of a 128-byte atom
        uint32_t qc = 0, ic = 0, parts = 0;
        uint32_t p_phase = 0;           // bit 2 t + h: parity of the next P_t,h
        uint32_t pv_next = 0;           // bit t: parity of group t's next product's number
        bool ok = true, issued = false;
        while (ok && walk.next(p, lane)) {
            const bool two = walk.two;
            const int n = walk.k1 - walk.k0;
            const int N = two ? 2 * n : n;
            // Rows of the query tiles that no token of the request has (what the box
            // brought of the next request, or an earlier part's) become zero in long
            // parts: the products with them cost power, and with it clock, for
            // nothing.  Without and with it, back to back at the 1000 W limit: 64 requests
            // of 16 tokens 256 and 246 us a call (bursts 218 and 212), of 4 tokens 234 and
            // 224, 16 requests over 8192 (head width 128) 125 and 124, two long trees
            // 168 and 169 (bursts 151 both).  The limit of 16 tiles is not sharp: with
            // parts of 10 tiles zeroing took 38.3 to 40.6 us when it was measured there,
            // and zeroing in all parts gains 0 to 1.5% in the cases above.
            for (int t = 0; ok && n >= kLongPart && t < (two ? 2 : 1); ++t) {
                const int rows =
                    min(p.tile_tokens, walk.r.n - (2 * walk.pair + t) * p.tile_tokens) * p.group;
                if (rows == kRows) continue;
                const uint32_t qs = (qc + t) & 1u;
                ok = wait_all(&q_full[qs], ((qc + t) >> 1) & 1, kErrTreeMma);
                uint8_t *q = smem + S::kQOff + qs * S::kTileBytes;
                for (int c = rows * 8 + lane; ok && c < kRows * 8; c += 32)
#pragma unroll
                    for (int a = 0; a < S::kAtoms; ++a)
                        *reinterpret_cast<uint4 *>(q + a * kAtomBytes + c * 16) =
                            make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            // One thread waits and issues for the whole part.  The tensor core
            // takes few products ahead, so what lies between two of them is kept
            // short: nothing is waited for twice.
            if (ok && elect_lane()) {
                auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
                    return mbar_wait_bounded(bar, parity, abort_flag, limit, p.error_word,
                                             kErrTreeMma);
                };
                auto tile_of = [&](int i) { return two ? i >> 1 : i; };
                // Ring stages of K_j and V_j; true once they are loaded (the second
                // group of a pair of query tiles finds them so).
                auto k_item = [&](int j) { return j == 0 ? ic : ic + 2 * j - 1; };
                auto v_item = [&](int j) { return j == n - 1 ? ic + 2 * n - 1 : ic + 2 * j + 2; };
                auto ready = [&](int i, uint32_t item) -> bool {
                    return (two && (i & 1)) || wait(&kv_full[item % NS], (item / NS) & 1);
                };
                auto halves_of = [&](int i) { return walk.halves(walk.k0 + tile_of(i)); };
                // S_i,h = Q K_h^T, K ready
                auto issue_s = [&](int i, int h, int halves) {
                    const int t = i & 1;
                    const uint32_t qs = (two ? qc + t : qc) & 1u;
                    const uint32_t st = k_item(tile_of(i)) % NS;
                    const uint64_t qd =
                        smem_desc_sw128(sbase + S::kQOff + qs * S::kTileBytes, 16, 1024);
                    const uint64_t kd = smem_desc_sw128(
                        sbase + S::kKVOff + st * S::kTileBytes + h * kHalfBytes, 16, 1024);
                    const uint32_t ds = tmem_base + t * kKeys + h * kHalf;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        // a descriptor counts in 16 bytes
                        const uint64_t off = ((kk >> 2) * kAtomBytes + (kk & 3) * 32) / 16;
                        mma_f16_ss<1>(ds, qd + off, kd + off, kIdescS, kk > 0);
                    }
                    mma_commit<1>(&s_full[2 * t + h]);
                    if (h + 1 == halves) {
                        if (!two || t == 1) mma_commit<1>(&kv_empty[st]);
                        if (two ? i + 2 >= N : i + 1 == N) mma_commit<1>(&q_empty[qs]);
                    }
                };
                // O_t += P_i,h V_h, V ready
                auto issue_pv = [&](int i, int h, int halves, uint32_t st, uint64_t vd) -> bool {
                    const int t = i & 1;
                    const uint32_t pb = 2 * t + h;
                    const uint32_t od = tmem_base + kOBase + t * D;
                    const uint32_t pa = tmem_base + t * kKeys + h * kHalf;
                    const uint32_t more = i >= 2 || h > 0;
                    if (!wait(&p_full[pb], (p_phase >> pb) & 1)) return false;
                    p_phase ^= 1u << pb;
                    tc_fence_after_sync();
#pragma unroll
                    for (int kk = 0; kk < kHalf / 16; ++kk)
                        mma_f16_ts(od, pa + kk * 8, vd + (h * kHalfBytes + kk * 2048) / 16,
                                   kIdescO, kk > 0 ? 1u : more);
                    mma_commit<1>(&pv_done[2 * t + ((pv_next >> t) & 1)]);
                    pv_next ^= 1u << t;
                    if (h + 1 == halves && (!two || t == 1)) mma_commit<1>(&kv_empty[st]);
                    return true;
                };
                bool good = true;
                for (int i = 0; good && i < 2 && i < N; ++i) {
                    const uint32_t qi = two ? qc + i : qc;
                    good = (i > 0 && !two) || wait(&q_full[qi & 1u], (qi >> 1) & 1);
                    if (good) good = ready(i, k_item(tile_of(i)));
                    if (!good) break;
                    tc_fence_after_sync();
                    const int hn = halves_of(i);
                    for (int h = 0; h < hn; ++h) issue_s(i, h, hn);
                }
                // The previous part's outputs have been read.
                if (good && parts > 0) good = wait(o_free, (parts - 1) & 1);
                int hn = halves_of(0);
                uint32_t st = v_item(0) % NS;
                if (good) good = ready(0, v_item(0));
                for (int i = 0; good && i < N; ++i) {
                    // Between a product P V and the scores behind it the tensor core is
                    // busy: there the next tiles are waited for.
                    const uint64_t vd =
                        smem_desc_sw128(sbase + S::kKVOff + st * S::kTileBytes, kAtomBytes, 1024);
                    const int hs = i + 2 < N ? halves_of(i + 2) : 0;
                    good = issue_pv(i, 0, hn, st, vd);
                    if (good && hs > 0) {
                        good = ready(i, k_item(tile_of(i + 2)));
                        if (!good) break;
                        tc_fence_after_sync();
                        issue_s(i + 2, 0, hs);
                    }
                    if (good && hn > 1) good = issue_pv(i, 1, hn, st, vd);
                    if (good && i + 1 < N) {
                        hn = halves_of(i + 1);
                        st = v_item(tile_of(i + 1)) % NS;
                        good = ready(i + 1, v_item(tile_of(i + 1)));
                    }
                    if (good && hs > 1) issue_s(i + 2, 1, hs);
                }
                ok = good;
            }
            ok = __all_sync(0xffffffffu, ok);
            issued = true;
            qc += two ? 2 : 1;
            ic += 2 * n;
            ++parts;
        }
        if (issued && elect_lane()) {
            mma_commit<1>(drain_bar);
            if (!mbar_wait_drain(drain_bar, 0, limit)) atomicOr(p.error_word, kErrTreeDrain);
        }
        __syncwarp();
    } else {
        const int t = warp >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t t_lanes = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t t_s = t_lanes + t * kKeys;
        const float sl2 = p.scale_log2;
        const int tl = row / p.group, hd = row - tl * p.group;
        uint32_t ic = 0, joins = 0;
        uint32_t s_phase = 0;           // bit h: parity of the next S_t,h
        uint32_t pv = 0;                // products P V of this group in the parts before
        uint32_t parts = 0;
        bool ok = true;
        // Waits for this group's product number k.  Scores k came after product
        // k - 2, so the barrier that k shares with k - 2 is in k's phase or past it.
        auto wait_pv = [&](uint32_t k) -> bool {
            ok = wait_all(&pv_done[2 * t + (k & 1)], (k >> 1) & 1, kErrTreeSoftmax);
            return ok;
        };
        while (ok && walk.next(p, lane)) {
            const Request &r = walk.r;
            const bool two = walk.two;
            const int n = walk.k1 - walk.k0;
            const int N = two ? 2 * n : n;
            const int tok0 = (2 * walk.pair + (two ? t : 0)) * p.tile_tokens;
            const int rows = min(p.tile_tokens, r.n - tok0) * p.group;
            const bool act = quarter * 32 < rows;        // uniform over the warp
            const int tok = tok0 + tl;                   // of the request
            const int64_t grow = static_cast<int64_t>(r.s0) + tok;
            const int32_t *mrow = p.mask ? p.mask + grow * p.mask_stride : nullptr;
            uint32_t done = pv;     // products of this group before the next
            // The row's mask words for the first tile of drafted keys, fetched ahead.
            uint32_t bits[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                bits[q] = mrow && row < rows && q < p.words ? static_cast<uint32_t>(mrow[q]) : 0u;
            float m = -INFINITY;    // running maximum of the scores, before the scale
            float l = 0.f;          // running sum of 2^((score - m) sl2 + lift)
            for (int i = t; ok && i < N; i += 2) {
                const int j = two ? i >> 1 : i;
                const int kj = walk.k0 + j;
                const bool tree = kj >= r.ctx_tiles;
                const int lim = walk.keys(kj);
                const bool edge = tree || lim < kKeys;             // not wholly visible
                const int key0 = (kj - r.ctx_tiles) * kKeys;       // first drafted key (tree)
#pragma unroll 1
                for (int h = 0; h < (lim > kHalf ? 2 : 1); ++h) {
                    if (!wait_all(&s_full[2 * t + h], (s_phase >> h) & 1, kErrTreeSoftmax)) {
                        ok = false;
                        break;
                    }
                    s_phase ^= 1u << h;
                    tc_fence_after_sync();
                    if (act) {
                        const uint32_t t_h = t_s + h * kHalf;
                        uint32_t s[2][32];
                        tmem_ld_32x32b_x32(t_h, s[0]);
                        tmem_ld_32x32b_x32(t_h + 32u, s[1]);
                        tmem_wait_ld_dep(s[0]);
                        tmem_wait_ld_dep(s[1]);
                        if (edge) {
                            // Visible columns: keys that exist, and for drafted ones
                            // the row's mask (or, without one, keys up to its own).
                            const int lim_row = tree && !mrow ? min(lim, tok + 1 - key0) : lim;
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const int v = lim_row - h * kHalf - 32 * q;
                                uint32_t vis =
                                    v >= 32 ? 0xffffffffu : (v <= 0 ? 0u : (1u << v) - 1u);
                                if (tree && mrow) {
                                    const int w = (key0 >> 5) + 2 * h + q;
                                    vis &= key0 == 0 ? (h ? bits[2 + q] : bits[q])
                                           : row < rows && w < p.words
                                               ? static_cast<uint32_t>(mrow[w])
                                               : 0u;
                                }
#pragma unroll
                                for (int c = 0; c < 32; ++c)
                                    if (!((vis >> c) & 1u)) s[q][c] = __float_as_uint(-INFINITY);
                            }
                        }
                        // The maximum keeps NaN (a NaN score makes the row NaN).
                        float mx[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            mx[u] = max_nan(__uint_as_float(s[0][u]), __uint_as_float(s[1][u]));
#pragma unroll
                        for (int c = 4; c < 32; ++c)
                            mx[c & 3] = max3_nan(mx[c & 3], __uint_as_float(s[0][c]),
                                                 __uint_as_float(s[1][c]));
                        const float smax = max_nan(max_nan(mx[0], mx[1]), max_nan(mx[2], mx[3]));
                        // Lazy rescale: m moves only when a half raises it by more than
                        // 8 log2 units (as a difference: m + lag may round up far from 0).
                        float alpha = 1.f;
                        const bool raise = !(smax - m <= p.lag) && smax != -INFINITY;
                        if (raise) {
                            alpha = m == -INFINITY ? 0.f : ex2((m - smax) * sl2);
                            m = smax;
                        }
                        if (done != pv && __any_sync(0xffffffffu, raise && row < rows)) {
                            if (!wait_pv(done - 1)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                const uint32_t t_o = t_lanes + kOBase + t * D + c * 32;
                                tmem_ld_32x32b_x32(t_o, o);
                                tmem_wait_ld_dep(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st_32x32b_x32(t_o, o);
                            }
                        }
                        // The difference to the maximum first, then the scale: as one
                        // multiply-add with a rounded product as the maximum, scores
                        // from 2^27 on overflowed fp16 (wide trees 165.5 us so, 167.5 as
                        // it is).
                        const float nm = m == -INFINITY ? 0.f : -m;
                        const uint64_t nm2 = f2(nm, nm), sl2x2 = f2(sl2, sl2),
                                       lift2 = f2(kLift<BF16>, kLift<BF16>);
                        uint64_t ps2[4] = {0, 0, 0, 0};
                        // P takes the first 32 columns of S, two keys per column.
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t hp[16];
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                const uint64_t d2 = fadd2(f2(__uint_as_float(s[q][c]),
                                                             __uint_as_float(s[q][c + 1])),
                                                          nm2);
                                const uint64_t a2 = ffma2(d2, sl2x2, lift2);
                                float a0, a1;
                                f2split(a2, a0, a1);
                                const float e0 = ex2(a0), e1 = ex2(a1);
                                ps2[(c >> 1) & 3] = fadd2(ps2[(c >> 1) & 3], f2(e0, e1));
                                hp[c >> 1] = pack2<BF16>(e0, e1);
                            }
                            tmem_st_32x32b_x16(t_h + q * 16, hp);
                        }
                        float q0, q1, q2, q3;
                        f2split(fadd2(ps2[0], ps2[1]), q0, q1);
                        f2split(fadd2(ps2[2], ps2[3]), q2, q3);
                        l = fmaf(l, alpha, (q0 + q1) + (q2 + q3));
                        tmem_wait_st();
                    }
                    ++done;
                    if (edge && h == 0 && (!two || t == 0)) {
                        // Values of this tile that no row may meet, see the head of
                        // the file.  Thread r looks after key r.
                        const uint32_t item = j == n - 1 ? ic + 2 * n - 1 : ic + 2 * j + 2;
                        const uint32_t st = item % NS;
                        if (!wait_all(&kv_full[st], (item / NS) & 1, kErrTreeSoftmax)) {
                            ok = false;
                            break;
                        }
                        uint8_t *vrow = smem + S::kKVOff + st * S::kTileBytes + row * 128;
                        if (row >= lim) {
                            if (lim > kHalf || row < kHalf)      // else no product reads it
#pragma unroll
                                for (int a = 0; a < S::kAtoms * 8; ++a)
                                    *reinterpret_cast<uint4 *>(vrow + (a >> 3) * kAtomBytes +
                                                               (((a + row) & 7) << 4)) =
                                        make_uint4(0, 0, 0, 0);
                        } else if (tree) {
                            // An exponent of all ones carries into the sign's place.
                            constexpr uint32_t kExp = BF16 ? 0x7F807F80u : 0x7C007C00u;
                            constexpr uint32_t kOne = BF16 ? 0x00800080u : 0x04000400u;
                            uint32_t odd = 0;
#pragma unroll 8
                            for (int a = 0; a < S::kAtoms * 8; ++a) {
                                const uint4 x = *reinterpret_cast<const uint4 *>(
                                    vrow + (a >> 3) * kAtomBytes + (((a + row) & 7) << 4));
                                odd |= ((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) |
                                       ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne);
                            }
                            if (odd & 0x80008000u) {
                                *odd_values = 1;
#pragma unroll 1
                                for (int a = 0; a < S::kAtoms * 32; ++a) {
                                    uint32_t *w = reinterpret_cast<uint32_t *>(
                                        vrow + (a >> 5) * kAtomBytes + (a & 31) * 4);
                                    const uint32_t hit = ((*w & kExp) + kOne) & 0x80008000u;
                                    if (hit & 0x00008000u) *w &= 0xFFFF0000u;
                                    if (hit & 0x80000000u) *w &= 0x0000FFFFu;
                                }
                            }
                        }
                        fence_proxy_async_smem();     // the tensor core reads the tile next
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[2 * t + h]);
                }
            }
            if (!ok) break;
            // End of the part.  A single query tile: both groups' outputs are
            // joined, each group doing half of the columns.
            const bool second = N > 1;     // group 1 had steps
            if (done != pv && !wait_pv(done - 1)) break;
            pv = done;
            float w0 = t == 0 ? 1.f : 0.f, w1 = t == 1 ? 1.f : 0.f;
            if (!two) {
                // The previous part's m and l have been read by both groups.
                if (parts > 0 && !wait_all(o_free, (parts - 1) & 1, kErrTreeSoftmax)) {
                    ok = false;
                    break;
                }
                ml[t * kRows + row] = make_float2(m, l);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(ml_full);
                if (!wait_all(ml_full, joins & 1, kErrTreeSoftmax)) {
                    ok = false;
                    break;
                }
                ++joins;
                const float2 a = ml[row], b = ml[kRows + row];
                m = max_nan(a.x, b.x);
                w0 = a.x == -INFINITY ? 0.f : ex2((a.x - m) * sl2);
                w1 = b.x == -INFINITY ? 0.f : ex2((b.x - m) * sl2);
                l = fmaf(a.y, w0, b.y * w1);
            }
            ++parts;
            tc_fence_after_sync();
            if (act) {
                const bool whole = walk.whole();
                const float inv = l > 0.f ? 1.f / l : 0.f;
                const int c_lo = two ? 0 : t * (D / 64), c_hi = two ? D / 32 : c_lo + D / 64;
                uint16_t *orow = p.out + grow * p.out_token_stride +
                                 static_cast<int64_t>(walk.head * p.group + hd) *
                                     p.out_head_stride;
                // The part's slot: the CTA's first part, or the one that begins a unit.
                float *part = p.part + (static_cast<int64_t>(cta) * 4 + (walk.k0 == 0 ? 2 : 0) +
                                        (two ? t : 0)) *
                                           S::kPartFloats;
#pragma unroll 1
                for (int c = c_lo; c < c_hi; ++c) {
                    uint32_t o[32];
                    float x[32];
                    if (two || second) {
                        const int g = two ? t : 1;
                        tmem_ld_32x32b_x32(t_lanes + kOBase + g * D + c * 32, o);
                        tmem_wait_ld_dep(o);
                        const float w = two ? 1.f : w1;
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(o[e]) * w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = 0.f;
                    }
                    if (!two) {
                        tmem_ld_32x32b_x32(t_lanes + kOBase + c * 32, o);
                        tmem_wait_ld_dep(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            x[e] = fmaf(__uint_as_float(o[e]), w0, x[e]);
                    }
                    if (whole) {
                        if (row < rows) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                uint4 u;
                                u.x = pack2<BF16>(x[q * 8 + 0] * inv, x[q * 8 + 1] * inv);
                                u.y = pack2<BF16>(x[q * 8 + 2] * inv, x[q * 8 + 3] * inv);
                                u.z = pack2<BF16>(x[q * 8 + 4] * inv, x[q * 8 + 5] * inv);
                                u.w = pack2<BF16>(x[q * 8 + 6] * inv, x[q * 8 + 7] * inv);
                                *reinterpret_cast<uint4 *>(orow + c * 32 + q * 8) = u;
                            }
                        }
                    } else if (row < rows) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) __stcg(part + (c * 32 + e) * kRows + row, x[e]);
                    }
                }
                if (!whole && row < rows && (two || t == 0)) {
                    __stcg(part + D * kRows + row, m);
                    __stcg(part + (D + 1) * kRows + row, l);
                }
                if (*odd_values != 0 && row < rows) {
                    // Values that are not finite, of drafted tokens that this row
                    // sees, are added to what has just been written: a positive
                    // weight leaves them what they are, and the weight 0 of a
                    // score of -inf makes them NaN.
                    const int jlo = max(walk.k0 - r.ctx_tiles, 0) * kKeys;
                    const int jhi = min((walk.k1 - r.ctx_tiles) * kKeys, r.n);
#pragma unroll 1
                    for (int jj = jlo; jj < jhi; ++jj) {
                        const bool sees =
                            mrow ? (jj >> 5) < p.words && ((mrow[jj >> 5] >> (jj & 31)) & 1)
                                 : jj <= tok;
                        if (!sees) continue;
                        const int64_t krow = static_cast<int64_t>(r.s0) + jj;
                        const uint16_t *vr =
                            p.v + krow * p.v_token_stride + walk.head * p.v_head_stride;
                        float odd_weight = -1.f;
#pragma unroll 1
                        for (int e = c_lo * 32; e < c_hi * 32; ++e) {
                            if (!not_finite<BF16>(vr[e])) continue;
                            if (odd_weight < 0.f) {
                                const uint16_t *qr =
                                    p.q + grow * p.q_token_stride +
                                    static_cast<int64_t>(walk.head * p.group + hd) *
                                        p.q_head_stride;
                                const uint16_t *kr =
                                    p.k + krow * p.k_token_stride + walk.head * p.k_head_stride;
                                float score = 0.f;
#pragma unroll 1
                                for (int i = 0; i < D; ++i)
                                    score =
                                        fmaf(value_of<BF16>(qr[i]), value_of<BF16>(kr[i]), score);
                                odd_weight = sl2 * score == -INFINITY ? 0.f : 1.f;
                            }
                            const float v = value_of<BF16>(vr[e]) * odd_weight;
                            float *pe = part + e * kRows + row;
                            if (whole)
                                orow[e] = static_cast<uint16_t>(
                                    pack2<BF16>(value_of<BF16>(orow[e]) + v, 0.f));
                            else
                                __stcg(pe, __ldcg(pe) + v);
                        }
                    }
                }
            }
            // Outputs read: the next part's products may overwrite them.
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_free);
            ic += 2 * n;
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem_base, kTmemCols);
    }
}

// The weight of a partial result with maximum m beside a maximum mn >= m; at least
// fp32's smallest number where the part saw anything, so that an infinite output
// stays infinite however small its weight: how a unit is divided must not show.
__device__ __forceinline__ float part_weight(float m, float mn, float sl2)
{
    return m == -INFINITY ? 0.f : max_nan(ex2((m - mn) * sl2), 1.401298464e-45f);
}

// Joins the parts of the units that more than one CTA worked on:
//   O = sum_s O_s w_s / sum_s l_s w_s,  w_s = 2^((m_s - m) sl2),  m = max_s m_s.
// Block (c, y): the unit that began in CTA c's share, 16 columns of one of its
// query tiles.  A thread has 8 columns of a row for one of `groups` runs of
// parts, in one pass with a running maximum: rp (a power of two that covers the
// rows in use) x 2 x groups threads.  The groups are then joined in order
// through shared memory.  Bound by the latency of the partial results' loads
// (they lie in L2), hence the single pass, and the many groups where there are
// few rows.  Five blocks to an SM (48 registers): with four, units of 74 parts took
// 2.5 us longer.
constexpr int kJoinThreads = 256;
constexpr int kJoinCols = 16;

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads, 5) tree_join_kernel(const TreeParams p)
{
    using S = TreeShape<D>;
    __shared__ float s_part[10][kJoinThreads];      // 8 columns, maximum and sum
    const int c = blockIdx.x, tid = threadIdx.x;
    const int t = static_cast<int>(blockIdx.y) / (D / kJoinCols);
    const int col0 = (static_cast<int>(blockIdx.y) % (D / kJoinCols)) * kJoinCols;
    grid_dependency_wait();
    const Split *sp = p.split + c;
    const int ctas = sp->ctas, head = sp->head, first = sp->first, rows = sp->rows[t];
    if (ctas < 2 || rows <= 0) return;
    const int shift = rows <= 8 ? 3 : 32 - __clz(rows - 1);
    const int row = tid & ((1 << shift) - 1), cg = (tid >> shift) & 1, g = tid >> (shift + 1);
    const int groups = kJoinThreads >> (shift + 1);
    const int per = (ctas + groups - 1) / groups;
    const int s0 = min(g * per, ctas), s1 = min(s0 + per, ctas);
    const float sl2 = p.scale_log2;
    float m = -INFINITY, acc[9];
#pragma unroll
    for (int e = 0; e < 9; ++e) acc[e] = 0.f;
    if (row < rows) {
#pragma unroll 2
        for (int s = s0; s < s1; ++s) {
            // Part s lies in CTA c + s: the one that begins a unit, then first parts.
            const float *part =
                p.part +
                (static_cast<int64_t>(c + s) * 4 + (s == 0 ? 2 : 0) + t) * S::kPartFloats + row;
            const float ms = __ldcg(part + D * kRows), ls = __ldcg(part + (D + 1) * kRows);
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __ldcg(part + (col0 + cg * 8 + e) * kRows);
            const float mn = max_nan(m, ms);
            const float w0 = part_weight(m, mn, sl2);
            const float w1 = part_weight(ms, mn, sl2);
            m = mn;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(x[e], w1, acc[e] * w0);
            acc[8] = fmaf(ls, w1, acc[8] * w0);
        }
    }
    if (groups > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_part[e][tid] = acc[e];
        s_part[8][tid] = acc[8];
        s_part[9][tid] = m;
        __syncthreads();
        if (g > 0) return;
        for (int i = 1; i < groups; ++i) {
            const int o = (i << (shift + 1)) + tid;
            const float ms = s_part[9][o];
            const float mn = max_nan(m, ms);
            const float w0 = part_weight(m, mn, sl2);
            const float w1 = part_weight(ms, mn, sl2);
            m = mn;
#pragma unroll
            for (int e = 0; e < 9; ++e) acc[e] = fmaf(s_part[e][o], w1, acc[e] * w0);
        }
    }
    if (row < rows) {
        const float inv = acc[8] > 0.f ? 1.f / acc[8] : 0.f;
        const int tl = row / p.group, hd = row - tl * p.group;
        uint4 u;
        u.x = pack2<BF16>(acc[0] * inv, acc[1] * inv);
        u.y = pack2<BF16>(acc[2] * inv, acc[3] * inv);
        u.z = pack2<BF16>(acc[4] * inv, acc[5] * inv);
        u.w = pack2<BF16>(acc[6] * inv, acc[7] * inv);
        *reinterpret_cast<uint4 *>(
            p.out + (static_cast<int64_t>(first) + t * p.tile_tokens + tl) * p.out_token_stride +
            static_cast<int64_t>(head * p.group + hd) * p.out_head_stride + col0 + cg * 8) = u;
    }
}

}  // namespace tgt

namespace {

using namespace tgc;

constexpr uint64_t kDefaultWaitLimitNs = 2000000000ull;

// A tensor map of 16-bit elements: dims from the head dimension outwards with
// the strides (in elements) of all but the first; a box of 64 elements by
// `rows` along the dimensions that have a box extent.
bool encode_map(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *tm, const void *base,
                bool bf16, int rank, const int64_t *dims, const int64_t *strides,
                const uint32_t *box)
{
    cuuint64_t d[4], st[3];
    cuuint32_t bx[4], es[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        d[i] = static_cast<cuuint64_t>(dims[i]);
        bx[i] = box[i];
    }
    // The stride of a dimension of extent 1 is never used; it only has to be valid.
    for (int i = 0; i + 1 < rank; ++i)
        st[i] = dims[i + 1] > 1 ? static_cast<cuuint64_t>(strides[i]) * 2 : 128;
    return encode(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  rank, const_cast<void *>(base), d, st, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap q, kc, vc, k, v;
};

template <int D, bool BF16>
tg_status_t launch(const Maps &maps, const tgt::TreeParams &p, int grid, cudaStream_t stream)
{
    using S = tgt::TreeShape<D>;
    // One bit per device: the kernel's dynamic shared-memory limit is raised.
    static std::atomic<uint64_t> attr_set{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return TG_ERR_UNSUPPORTED_DEVICE;
    }
    const uint64_t bit = uint64_t(1) << dev;
    if (!(attr_set.load() & bit)) {
        if (cudaFuncSetAttribute(tgt::tree_attn_kernel<D, BF16>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 S::kDynamicBytes) != cudaSuccess) {
            cudaGetLastError();
            return TG_ERR_LAUNCH;
        }
        attr_set.fetch_or(bit);
    }
    tgt::tree_attn_kernel<D, BF16><<<grid, tgt::kThreads, S::kDynamicBytes, stream>>>(
        maps.q, maps.kc, maps.vc, maps.k, maps.v, p);
    if (cudaGetLastError() != cudaSuccess) return TG_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 2 * (D / tgt::kJoinCols));
    cfg.blockDim = dim3(tgt::kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, tgt::tree_join_kernel<D, BF16>, p) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_LAUNCH;
    }
    return TG_OK;
}

constexpr int64_t kMaxStride = int64_t(1) << 38;    // elements; a map's strides are below 2^40 bytes

tg_status_t tree_attention_impl(const tg_tree_attention_t &a, cudaStream_t stream)
{
    const int shift = page_shift_of(a.page_size);
    if ((a.type != TG_TYPE_FP16 && a.type != TG_TYPE_BF16) || a.tokens < 0 || a.tokens >= kInt32 ||
        a.batch < 0 || a.batch >= kInt32 - 1024 || a.kv_heads < 0 || a.kv_heads > (1 << 20) ||
        a.group < 1 || a.group > 128 || (a.head_dim != 64 && a.head_dim != 128) || shift < 0 ||
        a.num_pages < 0 || a.num_pages >= kInt32 || a.max_pages < 0 ||
        a.max_pages >= (kInt32 - 256) >> shift || a.table_stride < a.max_pages ||
        a.table_stride >= kInt32 || !std::isfinite(a.scale) || a.scale < 0.f ||
        (a.scale != 0.f && (a.scale < 1e-30f || a.scale > 1e30f)) ||
        (a.inject != 0 && a.inject != TG_INJECT_SKIP_FIRST_LOAD))
        return TG_ERR_INVALID_ARG;
    if (a.mask && (a.words < 1 || a.words > (1 << 26) || a.mask_stride < a.words ||
                   a.mask_stride >= kInt32))
        return TG_ERR_INVALID_ARG;
    // Query tiles of all key heads, and 32-bit key indexes.
    const int64_t tile_tokens = tgt::kRows / a.group;
    if (a.kv_heads * (a.tokens / tile_tokens + 2) >= kInt32 || a.tokens >= kInt32 - 256)
        return TG_ERR_INVALID_ARG;
    if (a.tokens == 0 || a.batch == 0 || a.kv_heads == 0) return TG_OK;
    if (!a.q || !a.k || !a.v || !a.out || !a.lens || !a.starts || !a.workspace ||
        a.workspace_bytes < tg_tree_attention_workspace_size(a.head_dim))
        return TG_ERR_INVALID_ARG;
    const bool cache = a.num_pages > 0 && a.max_pages > 0;
    if (cache && (!a.k_cache || !a.v_cache || !a.block_tables)) return TG_ERR_INVALID_ARG;

    const int64_t heads = a.kv_heads * a.group, D = a.head_dim;
    const int64_t v_token_stride = a.own_v_strides ? a.v_token_stride : a.kv_token_stride;
    const int64_t v_head_stride = a.own_v_strides ? a.v_head_stride : a.kv_head_stride;
    // Strides of dimensions with more than one element.
    const Dim strides[] = {{a.tokens, a.q_token_stride},
                             {heads, a.q_head_stride},
                             {a.tokens, a.kv_token_stride},
                             {a.kv_heads, a.kv_head_stride},
                             {a.tokens, v_token_stride},
                             {a.kv_heads, v_head_stride},
                             {a.tokens, a.out_token_stride},
                             {heads, a.out_head_stride},
                             {cache ? a.num_pages : 1, a.page_stride},
                             {cache ? a.page_size : 1, a.slot_stride},
                             {cache ? a.kv_heads : 1, a.cache_head_stride}};
    for (const Dim &c : strides)
        if (c.n > 1 && (c.stride < D || c.stride >= kMaxStride)) return TG_ERR_INVALID_ARG;
    for (const Dim &c : strides)
        if (c.n > 1 && (c.stride & 7)) return TG_ERR_MISALIGNED;
    const void *vec[] = {a.q, a.k, a.v, a.out};
    for (const void *q : vec)
        if (misaligned(q, 16)) return TG_ERR_MISALIGNED;
    if (cache && (misaligned(a.k_cache, 16) || misaligned(a.v_cache, 16))) return TG_ERR_MISALIGNED;
    if (misaligned(a.workspace, 256) || misaligned(a.lens, 4) || misaligned(a.starts, 4) ||
        misaligned(a.block_tables, 4) || misaligned(a.mask, 4))
        return TG_ERR_MISALIGNED;

    const size_t cache_bytes = cache ? extent({{a.num_pages, a.page_stride},
                                               {a.page_size, a.slot_stride},
                                               {a.kv_heads, a.cache_head_stride}},
                                              D)
                                     : 0;
    const Range in[] = {
        {a.q, extent({{a.tokens, a.q_token_stride}, {heads, a.q_head_stride}}, D)},
        {a.k, extent({{a.tokens, a.kv_token_stride}, {a.kv_heads, a.kv_head_stride}}, D)},
        {a.v, extent({{a.tokens, v_token_stride}, {a.kv_heads, v_head_stride}}, D)},
        {a.k_cache, cache_bytes},
        {a.v_cache, cache_bytes},
        {a.block_tables,
         cache ? static_cast<size_t>((a.batch - 1) * a.table_stride + a.max_pages) * 4 : 0},
        {a.lens, static_cast<size_t>(a.batch) * 4},
        {a.starts, static_cast<size_t>(a.batch + 1) * 4},
        {a.mask, a.mask ? static_cast<size_t>((a.tokens - 1) * a.mask_stride + a.words) * 4 : 0}};
    const Range out = {a.out,
                       extent({{a.tokens, a.out_token_stride}, {heads, a.out_head_stride}}, D)};
    const Range ws = {a.workspace, tg_tree_attention_workspace_size(a.head_dim)};
    for (const Range &i : in)
        if (overlap(out, i) || overlap(ws, i)) return TG_ERR_INVALID_ARG;
    if (overlap(out, ws)) return TG_ERR_INVALID_ARG;

    int num_sms = 0;
    unsigned *error_word = nullptr;
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const tg_status_t st = tg_internal_device(&num_sms, &error_word, &encode);
    if (st != TG_OK) return st;

    const bool bf16 = a.type == TG_TYPE_BF16;
    Maps maps;
    {
        const int64_t dims[] = {D, heads, a.tokens};
        const int64_t str[] = {a.q_head_stride, a.q_token_stride};
        const uint32_t box[] = {tgt::kAtom, static_cast<uint32_t>(a.group),
                                static_cast<uint32_t>(tile_tokens)};
        if (!encode_map(encode, &maps.q, a.q, bf16, 3, dims, str, box)) return TG_ERR_CUDA;
    }
    {
        const int64_t dims[] = {D, a.tokens, a.kv_heads};
        const int64_t k_str[] = {a.kv_token_stride, a.kv_head_stride};
        const int64_t v_str[] = {v_token_stride, v_head_stride};
        const uint32_t box[] = {tgt::kAtom, tgt::kKeys, 1};
        if (!encode_map(encode, &maps.k, a.k, bf16, 3, dims, k_str, box) ||
            !encode_map(encode, &maps.v, a.v, bf16, 3, dims, v_str, box))
            return TG_ERR_CUDA;
    }
    if (cache) {
        const int64_t dims[] = {D, a.page_size, a.kv_heads, a.num_pages};
        const int64_t str[] = {a.slot_stride, a.cache_head_stride, a.page_stride};
        const uint32_t box[] = {
            tgt::kAtom, static_cast<uint32_t>(a.page_size < tgt::kKeys ? a.page_size : tgt::kKeys),
            1, 1};
        if (!encode_map(encode, &maps.kc, a.k_cache, bf16, 4, dims, str, box) ||
            !encode_map(encode, &maps.vc, a.v_cache, bf16, 4, dims, str, box))
            return TG_ERR_CUDA;
    } else {
        maps.kc = maps.k;     // not read: every context is empty
        maps.vc = maps.v;
    }

    tgt::TreeParams p;
    p.lens = a.lens;
    p.starts = a.starts;
    p.tables = a.block_tables;
    p.mask = a.mask;
    p.q = static_cast<const uint16_t *>(a.q);
    p.k = static_cast<const uint16_t *>(a.k);
    p.v = static_cast<const uint16_t *>(a.v);
    p.out = static_cast<uint16_t *>(a.out);
    p.q_token_stride = a.q_token_stride;
    p.q_head_stride = a.q_head_stride;
    p.k_token_stride = a.kv_token_stride;
    p.k_head_stride = a.kv_head_stride;
    p.v_token_stride = v_token_stride;
    p.v_head_stride = v_head_stride;
    p.out_token_stride = a.out_token_stride;
    p.out_head_stride = a.out_head_stride;
    p.table_stride = a.table_stride;
    p.max_len = cache ? a.max_pages << shift : 0;
    p.mask_stride = a.mask_stride;
    p.tokens = static_cast<int>(a.tokens);
    p.batch = static_cast<int>(a.batch);
    p.kv_heads = static_cast<int>(a.kv_heads);
    p.group = static_cast<int>(a.group);
    p.tile_tokens = static_cast<int>(tile_tokens);
    p.words = static_cast<int>(a.words);
    p.page_shift = shift;
    const float scale = a.scale != 0.f ? a.scale : 1.0f / std::sqrt(static_cast<float>(D));
    p.scale_log2 = scale * 1.4426950408889634f;
    p.lag = 8.0f / p.scale_log2;
    p.split = static_cast<tgt::Split *>(a.workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + tgt::split_bytes());
    p.inject = a.inject;
    p.wait_limit_ns = a.wait_limit_ns ? a.wait_limit_ns : kDefaultWaitLimitNs;
    p.error_word = error_word;
    const int grid = num_sms < tgt::kMaxCtas ? num_sms : tgt::kMaxCtas;
    if (D == 64)
        return bf16 ? launch<64, true>(maps, p, grid, stream)
                    : launch<64, false>(maps, p, grid, stream);
    return bf16 ? launch<128, true>(maps, p, grid, stream)
                : launch<128, false>(maps, p, grid, stream);
}

}  // namespace

extern "C" {

size_t tg_tree_attention_workspace_size(int64_t head_dim)
{
    if (head_dim != 64 && head_dim != 128) return 0;
    return tgt::split_bytes() + sizeof(float) * static_cast<size_t>(tgt::kMaxCtas) * 4 *
                                    static_cast<size_t>((head_dim + 2) * tgt::kRows);
}

tg_status_t tg_tree_attention(const tg_tree_attention_t *args, void *stream)
{
    if (!args) return TG_ERR_INVALID_ARG;
    return tree_attention_impl(*args, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
