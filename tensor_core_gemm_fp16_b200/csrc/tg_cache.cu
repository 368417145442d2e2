// tg_cache.cu -- the small operators of include/tg_cache.h for sm_100a: block
// tables and slot maps (tg_cache_plan), keys and values into pages
// (tg_cache_write), ancestor masks (tg_tree_mask).
#include <cuda_runtime.h>

#include <cstdint>

#include "tg_cache.h"
#include "tg_cache_internal.h"
#include "tg_internal.h"

namespace tgc {

// ---------------------------------------------------------------- tg_cache_plan
// With have = ceil(len / P), want = ceil((len + add) / P), grow = max(want - have, 0),
// drop = max(have - want, 0) and exclusive prefix sums G, D over the requests:
//   table[b][have + i] = free[(head + G_b + i) mod cap]             i < grow_b
//   free[(head + count + D_b + i) mod cap] = table[b][want + i]     i < drop_b
//   slot of token p = page(p / P) * P + p mod P
// The taken and the given-back ring entries never overlap (count + sum of drop
// <= cap is checked), and a token's page is taken from the ring itself where
// its table entry is new, so nothing a CTA reads is written by another: every
// CTA makes the sums over all requests for itself (at most 8192, from L2) and
// then takes its share of the pages and tokens; no CTA waits for another.
// Bound by latency: launch, two rounds of loads, one scan.
// Threads of a CTA: about one per request, 128 to 1024 (a decode step of 64 requests
// spends its time in the barriers, 4096 requests in the loads of the sums).
constexpr int kPlanMinThreads = 128;
constexpr int kPlanMaxThreads = 1024;

struct PlanParams {
    const int32_t *lens, *add, *starts, *offsets, *ring;
    int32_t *tables, *free_pages, *lens_out, *ring_out, *starts_out, *positions, *status;
    int64_t *slots;
    int64_t table_stride, max_pages, num_pages;
    int batch, tokens, page_shift;
};

struct Sums {
    int64_t grow, drop, toks;
};

__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b)
{
    return {a.grow + b.grow, a.drop + b.drop, a.toks + b.toks};
}

__device__ __forceinline__ Sums shfl_up(const Sums &a, int d)
{
    return {__shfl_up_sync(0xffffffffu, a.grow, d), __shfl_up_sync(0xffffffffu, a.drop, d),
            __shfl_up_sync(0xffffffffu, a.toks, d)};
}

__device__ __forceinline__ int64_t pages_of(int64_t len, int shift)
{
    return (len + (int64_t(1) << shift) - 1) >> shift;
}

__device__ __forceinline__ int32_t saturate(int64_t v)
{
    return v > 0x7fffffff ? 0x7fffffff : static_cast<int32_t>(v);
}

// Entry of the ring that lies at `at`, for 0 <= at < 3 cap (a 64-bit remainder
// takes several hundred cycles).
__device__ __forceinline__ int64_t in_ring(int64_t at, int64_t cap)
{
    if (at >= cap) at -= cap;
    return at >= cap ? at - cap : at;
}

// Last index i in [0, n) with a[i] <= v, for ascending a with a[0] <= v.
__device__ __forceinline__ int last_at_most(const int32_t *a, int n, int32_t v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanMaxThreads) cache_plan_kernel(const PlanParams p)
{
    extern __shared__ int32_t smem[];
    const int B = p.batch;
    int32_t *s_grow = smem;             // exclusive prefixes, [B]
    int32_t *s_drop = s_grow + B;
    int32_t *s_start = s_drop + B;      // [B + 1]
    __shared__ Sums s_warp[kPlanMaxThreads / 32 + 1];
    __shared__ int s_status;

    const int threads = blockDim.x, warps = threads >> 5;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (B + threads - 1) / threads;
    const int b0 = min(tid * per, B), b1 = min(b0 + per, B);

    const int64_t head = p.ring[0], count = p.ring[1];
    int bad = 0;
    if (head < 0 || head >= p.num_pages || count < 0 || count > p.num_pages)
        bad |= TG_PLAN_BAD_RING;
    Sums mine{0, 0, 0};
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
        const int64_t len = p.lens[b], after = len + p.add[b];
        if (len < 0 || after < 0 || after > 0x7fffffff) bad |= TG_PLAN_BAD_LENGTH;
        const int64_t have = pages_of(len < 0 ? 0 : len, p.page_shift);
        const int64_t want = pages_of(after < 0 ? 0 : after, p.page_shift);
        if (have > p.max_pages || want > p.max_pages) bad |= TG_PLAN_TABLE_FULL;
        mine.grow += want > have ? want - have : 0;
        mine.drop += have > want ? have - want : 0;
        if (p.starts) {
            const int32_t s = p.starts[b], e = p.starts[b + 1];
            if (s < 0 || e < s || e > p.tokens || p.add[b] > int64_t(e) - s)
                bad |= TG_PLAN_BAD_TOKENS;
            s_start[b] = s;
            if (b == B - 1) s_start[B] = e;
        } else {
            mine.toks += after > len ? after - len : 0;
        }
    }
    // Inclusive scan over the threads.
    Sums incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums o = shfl_up(incl, d);
        if (lane >= d) incl = incl + o;
    }
    if (lane == 31) s_warp[warp + 1] = incl;
    if (tid == 0) {
        s_warp[0] = {0, 0, 0};
        s_status = 0;
    }
    __syncthreads();
    if (warp == 0) {
        Sums w = lane < warps ? s_warp[lane + 1] : Sums{0, 0, 0};
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sums o = shfl_up(w, d);
            if (lane >= d) w = w + o;
        }
        __syncwarp();
        if (lane < warps) s_warp[lane + 1] = w;
    }
    __syncthreads();
    const Sums total = s_warp[warps];
    if (total.grow > count) bad |= TG_PLAN_NO_PAGES;
    if (count + total.drop > p.num_pages) bad |= TG_PLAN_BAD_RING;
    if (!p.starts && total.toks > p.tokens) bad |= TG_PLAN_BAD_TOKENS;

    Sums run = s_warp[warp] + incl;   // exclusive: this thread's own sums taken off again
    run = {run.grow - mine.grow, run.drop - mine.drop, run.toks - mine.toks};
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
        const int64_t len = p.lens[b], after = len + p.add[b];
        const int64_t have = pages_of(len < 0 ? 0 : len, p.page_shift);
        const int64_t want = pages_of(after < 0 ? 0 : after, p.page_shift);
        s_grow[b] = saturate(run.grow);
        s_drop[b] = saturate(run.drop);
        run.grow += want > have ? want - have : 0;
        run.drop += have > want ? have - want : 0;
        if (!p.starts) {
            s_start[b] = saturate(run.toks);
            run.toks += after > len ? after - len : 0;
            if (b == B - 1) s_start[B] = saturate(run.toks);
        }
    }
    if (B == 0 && tid == 0) s_start[0] = p.starts ? p.starts[0] : 0;
    // Bits that any thread has seen (the barrier also publishes the prefixes).
    if (bad) atomicOr(&s_status, bad);
    __syncthreads();
    const int status = s_status;
    const bool fine = status == 0;

    const int64_t t0 = blockIdx.x * int64_t(threads) + tid;
    const int64_t stride = int64_t(gridDim.x) * threads;
    for (int64_t b = t0; b < B; b += stride)
        p.lens_out[b] = p.lens[b] + (fine ? p.add[b] : 0);
    if (p.starts_out)
        for (int64_t b = t0; b <= B; b += stride) p.starts_out[b] = s_start[b];
    if (t0 == 0) {
        p.status[0] = status;
        p.ring_out[0] =
            static_cast<int32_t>(fine ? in_ring(head + total.grow, p.num_pages) : head);
        p.ring_out[1] = static_cast<int32_t>(fine ? count - total.grow + total.drop : count);
    }
    // Pages taken, pages given back and tokens in one loop over all three: a
    // thread that has one of each would make the three chains of loads one after
    // the other (4096 requests with 25,000 pages given back: 11.1 us so, 10.2
    // in one loop).
    const int64_t taken = fine ? total.grow : 0, moved = taken + (fine ? total.drop : 0);
    const int64_t page_mask = (int64_t(1) << p.page_shift) - 1;
    for (int64_t at = t0; at < moved + p.tokens; at += stride) {
        if (at < taken) {
            const int64_t i = at;
            const int b = last_at_most(s_grow, B, static_cast<int32_t>(i));
            const int64_t col = pages_of(p.lens[b], p.page_shift) + (i - s_grow[b]);
            p.tables[b * p.table_stride + col] = p.free_pages[in_ring(head + i, p.num_pages)];
            continue;
        }
        if (at < moved) {
            const int64_t i = at - taken;
            const int b = last_at_most(s_drop, B, static_cast<int32_t>(i));
            const int64_t col =
                pages_of(int64_t(p.lens[b]) + p.add[b], p.page_shift) + (i - s_drop[b]);
            p.free_pages[in_ring(head + count + i, p.num_pages)] =
                p.tables[b * p.table_stride + col];
            continue;
        }
        const int64_t i = at - moved;
        int64_t slot = -1, pos = -1;
        if (fine && B > 0 && i >= s_start[0] && i < s_start[B]) {
            const int b = last_at_most(s_start, B, static_cast<int32_t>(i));
            const int64_t off = p.offsets ? p.offsets[i] : i - s_start[b];
            if (off >= 0 && off < p.add[b]) {
                const int64_t len = p.lens[b];
                pos = len + off;
                const int64_t col = pos >> p.page_shift, have = pages_of(len, p.page_shift);
                const int64_t page =
                    col < have ? p.tables[b * p.table_stride + col]
                               : p.free_pages[in_ring(head + s_grow[b] + (col - have), p.num_pages)];
                slot = (page << p.page_shift) + (pos & page_mask);
            }
        }
        p.slots[i] = slot;
        p.positions[i] = static_cast<int32_t>(pos);
    }
}

// ---------------------------------------------------------------- tg_cache_write
// A copy, bound by HBM (keys and values read once, written once).  A warp takes
// a token: its keys' and values' 16-byte pieces, up to 8 per lane in flight
// together; the pieces of a head are contiguous on both sides.
constexpr int kWriteThreads = 256;
constexpr int kWriteUnroll = 8;

struct WriteParams {
    const uint4 *k, *v;
    uint4 *kc, *vc;
    const int64_t *slots;
    int64_t tokens, num_slots;
    int64_t k_token_stride, k_head_stride;                  // in 16-byte pieces
    int64_t v_token_stride, v_head_stride;                  // in 16-byte pieces
    int64_t page_stride, slot_stride, cache_head_stride;    // in 16-byte pieces
    int page_shift, dim_shift;                              // log2(page size), log2(head_dim / 8)
    int pieces;                                             // 2 * heads * head_dim / 8
};

__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const WriteParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (kWriteThreads / 32);
    const int half = p.pieces >> 1, dmask = (1 << p.dim_shift) - 1;
    for (int64_t t = (blockIdx.x * int64_t(kWriteThreads) + threadIdx.x) >> 5; t < p.tokens;
         t += warps) {
        const int64_t slot = p.slots[t];
        if (slot < 0 || slot >= p.num_slots) continue;
        const uint4 *k = p.k + t * p.k_token_stride, *v = p.v + t * p.v_token_stride;
        const int64_t dst0 = (slot >> p.page_shift) * p.page_stride +
                             (slot & ((int64_t(1) << p.page_shift) - 1)) * p.slot_stride;
        for (int c0 = lane; c0 < p.pieces; c0 += 32 * kWriteUnroll) {
            uint4 x[kWriteUnroll];
#pragma unroll
            for (int u = 0; u < kWriteUnroll; ++u) {
                const int c = c0 + 32 * u;
                if (c < p.pieces) {
                    const int e = c < half ? c : c - half;
                    const int64_t head = (e >> p.dim_shift) *
                                         (c < half ? p.k_head_stride : p.v_head_stride);
                    x[u] = __ldg((c < half ? k : v) + head + (e & dmask));
                }
            }
#pragma unroll
            for (int u = 0; u < kWriteUnroll; ++u) {
                const int c = c0 + 32 * u;
                if (c < p.pieces) {
                    const int e = c < half ? c : c - half;
                    const int64_t off =
                        dst0 + (e >> p.dim_shift) * p.cache_head_stride + (e & dmask);
                    (c < half ? p.kc : p.vc)[off] = x[u];
                }
            }
        }
    }
}

// ---------------------------------------------------------------- tg_tree_mask
// A mask row is its parent's row and one bit more.  Tokens are taken in chunks
// of 32, a mask word each.  First each chunk by itself, a warp per chunk: by
// doubling over shuffles every token gets the bits of its ancestors within the
// chunk and `exit`, the first one before it.  Then, chunk after chunk,
//   row(i) = row(exit(i)) | own word,   count(i) = count(exit(i)) + bits of it,
// a thread per token and word.  The words are independent of one another: a CTA
// has 16 of them, for all tokens of a request.  Bound by latency: a barrier and
// three dependent shared-memory loads per chunk (a walk along the ancestors of
// a tree of 1000 tokens some 300 generations deep took 110 us, with eight
// ancestors a step 20 us).
constexpr int kMaskThreads = 512;
constexpr int kMaskWords = 16;       // words of a CTA
static_assert(kMaskThreads == 32 * kMaskWords, "a thread per token of a chunk and word");

struct MaskParams {
    const int32_t *parents, *starts;
    int32_t *mask, *depth;
    int tokens, batch, words, slices;     // slices = ceil(words / kMaskWords)
};

// Shared memory of a CTA: rows, own words, exits and counts of 32 * words tokens.
constexpr size_t mask_smem(int64_t words)
{
    return static_cast<size_t>(words) * 32 * (kMaskWords + 3) * 4;
}

__device__ __forceinline__ int clamp_row(int v, int tokens)
{
    return v < 0 ? 0 : (v > tokens ? tokens : v);
}

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const MaskParams p)
{
    constexpr int kRoot = -1, kBad = -2;       // parents above a root; of no tree
    extern __shared__ uint32_t s_rows[];       // [tokens][kMaskWords]
    const int tid = threadIdx.x, lane = tid & 31;
    const int W = p.words, room = 32 * W;
    uint32_t *s_own = s_rows + room * kMaskWords;
    int *s_exit = reinterpret_cast<int *>(s_own + room);
    int *s_count = s_exit + room;
    const int b = blockIdx.x / p.slices, w0 = blockIdx.x % p.slices * kMaskWords;
    if (b == p.batch) {
        // Rows before the first request and behind the last.
        if (w0 > 0) return;
        const int first = clamp_row(p.starts[0], p.tokens);
        const int last = clamp_row(p.starts[p.batch], p.tokens);
        for (int64_t i = tid; i < p.tokens; i += kMaskThreads) {
            if (i >= first && i < last) {
                i += (last - 1 - i) / kMaskThreads * kMaskThreads;     // past the requests
                continue;
            }
            p.depth[i] = -1;
            for (int w = 0; w < W; ++w) p.mask[i * W + w] = 0;
        }
        return;
    }
    const int row0 = clamp_row(p.starts[b], p.tokens);
    const int n = clamp_row(p.starts[b + 1], p.tokens) - row0;
    const int n_tree = min(n, room);
    // Tokens past the mask's width.
    if (w0 == 0)
        for (int64_t i = n_tree + tid; i < n; i += kMaskThreads) {
            p.depth[row0 + i] = -1;
            for (int w = 0; w < W; ++w) p.mask[(row0 + i) * W + w] = 0;
        }
    for (int i = tid; i - lane < n_tree; i += kMaskThreads) {
        const int base = i - lane;             // the warp's chunk
        int up = kBad;
        if (i < n_tree) {
            const int u = p.parents[row0 + i];
            up = u >= kRoot && u < i ? u : kBad;
        }
        uint32_t own = 1u << lane;
#pragma unroll
        for (int r = 0; r < 5; ++r) {
            const bool in = up >= base;
            const int src = in ? up - base : lane;
            const uint32_t bits = __shfl_sync(0xffffffffu, own, src);
            const int next = __shfl_sync(0xffffffffu, up, src);
            if (in) {
                own |= bits;
                up = next;
            }
        }
        s_own[i] = own;
        s_exit[i] = up;
    }
    __syncthreads();
    const int tok = tid / kMaskWords, w = w0 + tid % kMaskWords;
    // Entries of rows past the tree's end are never read by others.
    int up = s_exit[tok];
    uint32_t own = s_own[tok];
    for (int c = 0; 32 * c < n_tree; ++c) {
        const int i = 32 * c + tok;
        if (i < n_tree) {
            const int above = up >= 0 ? s_count[up] : (up == kRoot ? 0 : -1);
            uint32_t row = 0;
            if (above >= 0) {
                if (w == c)
                    row = own;
                else if (up >= 0)
                    row = s_rows[up * kMaskWords + tid % kMaskWords];
            }
            const int count = above >= 0 ? above + __popc(own) : -1;
            s_rows[i * kMaskWords + tid % kMaskWords] = row;
            if (w == w0) s_count[i] = count;
            if (w < W) p.mask[static_cast<int64_t>(row0 + i) * W + w] = static_cast<int32_t>(row);
            if (w == 0) p.depth[row0 + i] = count > 0 ? count - 1 : -1;
        }
        if (i + 32 < n_tree) {
            up = s_exit[i + 32];
            own = s_own[i + 32];
        }
        __syncthreads();
    }
}

}  // namespace tgc

namespace {

using namespace tgc;

int grid_for(int64_t items, int per_cta, int num_sms, int ctas_per_sm)
{
    const int64_t want = (items + per_cta - 1) / per_cta;
    const int64_t most = static_cast<int64_t>(num_sms) * ctas_per_sm;
    return static_cast<int>(want < 1 ? 1 : (want < most ? want : most));
}

}  // namespace

extern "C" {

tg_status_t tg_cache_plan(const int32_t *lens, const int32_t *add, int64_t batch,
                          const int32_t *starts, const int32_t *offsets, int64_t tokens,
                          int32_t *block_tables, int64_t table_stride, int64_t max_pages,
                          int64_t page_size, int32_t *free_pages, int64_t num_pages,
                          const int32_t *ring, int32_t *lens_out, int32_t *ring_out,
                          int32_t *starts_out, int64_t *slots, int32_t *positions,
                          int32_t *status, void *stream)
{
    const int shift = page_shift_of(page_size);
    if (batch < 0 || batch > TG_CACHE_MAX_BATCH || tokens < 0 || tokens >= kInt32 || shift < 0 ||
        max_pages < 0 || max_pages >= kInt32 || table_stride < max_pages ||
        table_stride >= kInt32 || num_pages < 1 || num_pages >= kInt32 || (offsets && !starts))
        return TG_ERR_INVALID_ARG;
    if (!ring || !ring_out || !status || !free_pages || (batch > 0 && (!lens || !add || !lens_out)) ||
        (batch > 0 && max_pages > 0 && !block_tables) || (tokens > 0 && (!slots || !positions)))
        return TG_ERR_INVALID_ARG;
    const void *word[] = {lens,       add,  starts,   offsets,  block_tables, free_pages,
                          ring,       lens_out, ring_out, starts_out, positions, status};
    for (const void *q : word)
        if (misaligned(q, 4)) return TG_ERR_MISALIGNED;
    if (misaligned(slots, 8)) return TG_ERR_MISALIGNED;
    const size_t nb = static_cast<size_t>(batch) * 4, nt = static_cast<size_t>(tokens) * 4;
    const size_t table_bytes =
        batch > 0 ? static_cast<size_t>((batch - 1) * table_stride + max_pages) * 4 : 0;
    const Range in[] = {{lens, nb}, {add, nb}, {starts, nb + 4}, {offsets, nt}, {ring, 8}};
    const Range out[] = {{block_tables, table_bytes},
                         {free_pages, static_cast<size_t>(num_pages) * 4},
                         {lens_out, nb},
                         {ring_out, 8},
                         {starts_out, nb + 4},
                         {slots, 2 * nt},
                         {positions, nt},
                         {status, 4}};
    for (const Range &o : out) {
        for (const Range &i : in)
            if (overlap(o, i)) return TG_ERR_INVALID_ARG;
        for (const Range &o2 : out)
            if (&o != &o2 && overlap(o, o2)) return TG_ERR_INVALID_ARG;
    }
    int num_sms = 0;
    unsigned *error_word = nullptr;
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const tg_status_t st = tg_internal_device(&num_sms, &error_word, &encode);
    if (st != TG_OK) return st;

    tgc::PlanParams p;
    p.lens = lens;
    p.add = add;
    p.starts = starts;
    p.offsets = offsets;
    p.ring = ring;
    p.tables = block_tables;
    p.free_pages = free_pages;
    p.lens_out = lens_out;
    p.ring_out = ring_out;
    p.starts_out = starts_out;
    p.positions = positions;
    p.status = status;
    p.slots = slots;
    p.table_stride = table_stride;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.batch = static_cast<int>(batch);
    p.tokens = static_cast<int>(tokens);
    p.page_shift = shift;
    const int smem = static_cast<int>(3 * batch + 1) * 4;
    // More than the default limit of shared memory (the scan's sums take some too).
    if (smem > 47 * 1024 &&
        cudaFuncSetAttribute(tgc::cache_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (3 * TG_CACHE_MAX_BATCH + 1) * 4) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_LAUNCH;
    }
    int threads = static_cast<int>((batch + 31) / 32 * 32);
    threads = threads < tgc::kPlanMinThreads   ? tgc::kPlanMinThreads
              : threads > tgc::kPlanMaxThreads ? tgc::kPlanMaxThreads
                                               : threads;
    // How many pages move only the device knows; a few per request are likely.
    const int grid = grid_for(tokens + 4 * batch, threads, num_sms, 1);
    tgc::cache_plan_kernel<<<grid, threads, smem,
                             static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? TG_OK : TG_ERR_LAUNCH;
}

tg_status_t tg_cache_write(const void *k, const void *v, int64_t tokens, int64_t heads,
                           int64_t head_dim, int64_t token_stride, int64_t head_stride,
                           const int64_t *slots, void *k_cache, void *v_cache, int64_t num_pages,
                           int64_t page_size, int64_t page_stride, int64_t slot_stride,
                           int64_t cache_head_stride, void *stream)
{
    return tg_cache_write_ex(k, token_stride, head_stride, v, token_stride, head_stride, tokens,
                             heads, head_dim, slots, k_cache, v_cache, num_pages, page_size,
                             page_stride, slot_stride, cache_head_stride, stream);
}

tg_status_t tg_cache_write_ex(const void *k, int64_t k_token_stride, int64_t k_head_stride,
                              const void *v, int64_t v_token_stride, int64_t v_head_stride,
                              int64_t tokens, int64_t heads, int64_t head_dim,
                              const int64_t *slots, void *k_cache, void *v_cache,
                              int64_t num_pages, int64_t page_size, int64_t page_stride,
                              int64_t slot_stride, int64_t cache_head_stride, void *stream)
{
    const int shift = page_shift_of(page_size);
    if (tokens < 0 || heads < 0 || heads > (1 << 20) || num_pages < 0 || num_pages >= kInt32 ||
        shift < 0 || (head_dim != 64 && head_dim != 128))
        return TG_ERR_INVALID_ARG;
    if (tokens >= kInt32) return TG_ERR_INVALID_ARG;
    if (tokens == 0 || heads == 0 || num_pages == 0) return TG_OK;
    if (!k || !v || !slots || !k_cache || !v_cache) return TG_ERR_INVALID_ARG;
    // Strides of dimensions with more than one element.  Rows of a cache may be
    // interleaved with others, not with one another.
    const Dim src_dims[] = {{tokens, k_token_stride},
                            {heads, k_head_stride},
                            {tokens, v_token_stride},
                            {heads, v_head_stride}};
    const Dim dst_dims[] = {
        {num_pages, page_stride}, {page_size, slot_stride}, {heads, cache_head_stride}};
    for (const Dim &d : src_dims)
        if (d.n > 1 && (d.stride < 0 || d.stride >= (int64_t(1) << 40))) return TG_ERR_INVALID_ARG;
    for (const Dim &d : dst_dims)
        if (d.n > 1 && (d.stride < head_dim || d.stride >= (int64_t(1) << 40)))
            return TG_ERR_INVALID_ARG;
    for (const Dim &d : src_dims)
        if (d.n > 1 && (d.stride & 7)) return TG_ERR_MISALIGNED;
    for (const Dim &d : dst_dims)
        if (d.n > 1 && (d.stride & 7)) return TG_ERR_MISALIGNED;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_cache, 16) ||
        misaligned(v_cache, 16) || misaligned(slots, 8))
        return TG_ERR_MISALIGNED;
    const size_t k_src = extent({{tokens, k_token_stride}, {heads, k_head_stride}}, head_dim);
    const size_t v_src = extent({{tokens, v_token_stride}, {heads, v_head_stride}}, head_dim);
    const size_t dst = extent({{num_pages, page_stride},
                               {page_size, slot_stride},
                               {heads, cache_head_stride}},
                              head_dim);
    const Range in[] = {{k, k_src}, {v, v_src}, {slots, 8 * static_cast<size_t>(tokens)}};
    for (const Range &i : in)
        if (overlap(i, {k_cache, dst}) || overlap(i, {v_cache, dst})) return TG_ERR_INVALID_ARG;
    // The two caches may be interleaved (slices of one tensor), not the same.
    if (k_cache == v_cache) return TG_ERR_INVALID_ARG;
    int num_sms = 0;
    unsigned *error_word = nullptr;
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const tg_status_t st = tg_internal_device(&num_sms, &error_word, &encode);
    if (st != TG_OK) return st;

    tgc::WriteParams p;
    p.k = static_cast<const uint4 *>(k);
    p.v = static_cast<const uint4 *>(v);
    p.kc = static_cast<uint4 *>(k_cache);
    p.vc = static_cast<uint4 *>(v_cache);
    p.slots = slots;
    p.tokens = tokens;
    p.num_slots = num_pages << shift;
    p.k_token_stride = k_token_stride / 8;
    p.k_head_stride = k_head_stride / 8;
    p.v_token_stride = v_token_stride / 8;
    p.v_head_stride = v_head_stride / 8;
    p.page_stride = page_stride / 8;
    p.slot_stride = slot_stride / 8;
    p.cache_head_stride = cache_head_stride / 8;
    p.page_shift = shift;
    p.dim_shift = head_dim == 64 ? 3 : 4;
    p.pieces = static_cast<int>(2 * heads * (head_dim / 8));
    const int grid = grid_for(tokens, tgc::kWriteThreads / 32, num_sms, 8);
    tgc::cache_write_kernel<<<grid, tgc::kWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? TG_OK : TG_ERR_LAUNCH;
}

tg_status_t tg_tree_mask(const int32_t *parents, int64_t tokens, const int32_t *starts,
                         int64_t batch, int64_t words, int32_t *mask, int32_t *depth,
                         void *stream)
{
    if (tokens < 0 || tokens >= kInt32 || batch < 0 || words < 1 || words > TG_TREE_MAX_WORDS ||
        (batch + 1) * words >= kInt32)
        return TG_ERR_INVALID_ARG;
    if (tokens == 0) return TG_OK;
    if (!parents || !starts || !mask || !depth) return TG_ERR_INVALID_ARG;
    if (misaligned(parents, 4) || misaligned(starts, 4) || misaligned(mask, 4) ||
        misaligned(depth, 4))
        return TG_ERR_MISALIGNED;
    const size_t nt = static_cast<size_t>(tokens) * 4;
    const Range in[] = {{parents, nt}, {starts, static_cast<size_t>(batch + 1) * 4}};
    const Range out[] = {{mask, nt * static_cast<size_t>(words)}, {depth, nt}};
    for (const Range &o : out)
        for (const Range &i : in)
            if (overlap(o, i)) return TG_ERR_INVALID_ARG;
    if (overlap(out[0], out[1])) return TG_ERR_INVALID_ARG;
    int num_sms = 0;
    unsigned *error_word = nullptr;
    PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    const tg_status_t st = tg_internal_device(&num_sms, &error_word, &encode);
    if (st != TG_OK) return st;

    tgc::MaskParams p;
    p.parents = parents;
    p.starts = starts;
    p.mask = mask;
    p.depth = depth;
    p.tokens = static_cast<int>(tokens);
    p.batch = static_cast<int>(batch);
    p.words = static_cast<int>(words);
    p.slices = static_cast<int>((words + tgc::kMaskWords - 1) / tgc::kMaskWords);
    const size_t smem = tgc::mask_smem(words);
    // More than the default limit of shared memory above 20 words.
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(tgc::tree_mask_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(tgc::mask_smem(TG_TREE_MAX_WORDS))) != cudaSuccess) {
        cudaGetLastError();
        return TG_ERR_LAUNCH;
    }
    const int grid = (p.batch + 1) * p.slices;
    tgc::tree_mask_kernel<<<grid, tgc::kMaskThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? TG_OK : TG_ERR_LAUNCH;
}

}  // extern "C"
