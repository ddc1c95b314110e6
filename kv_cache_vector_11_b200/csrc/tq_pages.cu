// Block tables and slot maps from request lengths (tq_page_tables).
//
// With held = ceil(ctx / P), want = ceil((ctx + new) / P), need = want - held
// per request, two exclusive sums over the requests place everything: cu (of
// new) gives a token's request, base (of need) gives its pages.  One launch:
// every CTA takes 2048 entries of the slot map and computes the sums for itself
// (8 bytes of lengths a request, from L2), which is cheaper than a second
// launch or a grid-wide wait up to the 16384 requests that fit its shared
// memory.  A token finds its request by binary search over cu in shared memory.
// Nothing is exchanged between CTAs: an entry of the table that a token needs
// is either one that was there before the call or free[base + ..], and the
// token that opens a page writes that page's entry.
//
// Bound by launch latency: 2 MB of slots are 0.4 us of HBM time.

#include <cuda_runtime.h>

#include <climits>

#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kPtThreads = 512;
constexpr int kPtWarps = kPtThreads / 32;
constexpr int kPtTokens = 4 * kPtThreads;     // slot-map entries per CTA
constexpr int kPtMaxBatch = 16384;

struct PageTablesArgs {
    const int32_t * ctx;
    const int32_t * add;
    int32_t batch;
    int32_t page_shift;
    int32_t n_pages;
    const int32_t * free_pages;
    int32_t n_free;
    int32_t * table;
    int32_t max_pages;
    int32_t * cu;
    int32_t * total;
    int64_t * slots;
    int32_t * positions;
    int32_t n_slots;
    int32_t * n_taken;
    uint32_t * status;
};

// Inclusive sum over the CTA's threads of 64-bit values (a request's length can
// be 2^31 - 1, so a sum of 16384 of them needs 45 bits); *all gets the total.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t * warp_sums, int64_t * all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();                     // the last scan's reads of warp_sums are done
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int64_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kPtWarps; ++w) {
        const int64_t s = warp_sums[w];
        if (w < warp) before += s;
        sum += s;
    }
    *all = sum;
    return v + before;
}

__device__ __forceinline__ int32_t clamp31(int64_t v) {
    return (int32_t)min(v, (int64_t)INT32_MAX);
}

__global__ void __launch_bounds__(kPtThreads) page_tables_kernel(const PageTablesArgs a) {
    // cu[batch + 1], then base[batch]: the first free-list index of a request's
    // new pages, or -1 for a request that was not placed
    extern __shared__ int32_t s_lens[];
    __shared__ int64_t s_sums[kPtWarps];
    int32_t * s_cu = s_lens;
    int32_t * s_base = s_lens + a.batch + 1;
    const int tid = threadIdx.x;
    const int P1 = (1 << a.page_shift) - 1;
    const bool first = blockIdx.x == 0;
    uint32_t status = 0u;

    int64_t tokens = 0, pages = 0;       // sums of the requests before this chunk
    for (int b0 = 0; b0 < a.batch; b0 += kPtThreads) {
        const int b = b0 + tid;
        const bool live = b < a.batch;
        const int64_t ctx = live ? max(a.ctx[b], 0) : 0;
        const int64_t add = live ? max(a.add[b], 0) : 0;
        int64_t all;
        const int64_t cu_end = tokens + cta_scan(add, s_sums, &all);
        tokens += all;
        const int64_t held = (ctx + P1) >> a.page_shift, want = (ctx + add + P1) >> a.page_shift;
        bool fits = want <= a.max_pages && cu_end <= a.n_slots && ctx + add <= INT32_MAX;
        const int64_t need = live && fits ? want - held : 0;
        const int64_t end = pages + cta_scan(need, s_sums, &all);
        // the sums only grow, so the requests whose pages fit are the first
        // ones that need any, and their pages a prefix of the free list
        fits = fits && (need == 0 || end <= a.n_free);
        pages += all;
        if (live) {
            s_cu[b] = clamp31(cu_end - add);
            s_base[b] = fits ? (int32_t)min(end - need, (int64_t)INT32_MAX) : -1;
            if (b == a.batch - 1) s_cu[a.batch] = clamp31(cu_end);
            if (first) {
                a.cu[b] = clamp31(cu_end - add);
                if (b == a.batch - 1) a.cu[a.batch] = clamp31(cu_end);
                a.total[b] = (int32_t)(fits ? ctx + add : ctx);
                if (!fits) status |= TQ_STATUS_NO_PAGES;
            }
        }
        if (first) {
            // pages taken: the placed requests' needs, a prefix of the sums
            int64_t taken;
            cta_scan(fits ? need : 0, s_sums, &taken);
            if (tid == 0) *a.n_taken = (int32_t)(taken + (b0 > 0 ? *a.n_taken : 0));
        }
    }
    __syncthreads();

    const int n_tok = s_cu[a.batch];
    for (int k = 0; k < kPtTokens / kPtThreads; ++k) {
        const int64_t i64 = (int64_t)blockIdx.x * kPtTokens + k * kPtThreads + tid;
        if (i64 >= a.n_slots) break;
        const int i = (int)i64;
        int64_t slot = -1;
        int32_t pos = -1;
        if (i < n_tok) {
            // the last request that starts at or before i (an empty request
            // starts where the next one does, so it is never the last)
            int lo = 0, hi = a.batch;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_cu[mid] <= i) lo = mid; else hi = mid;
            }
            const int32_t base = s_base[lo];
            if (base >= 0) {
                const int ctx = max(a.ctx[lo], 0);
                pos = ctx + (i - s_cu[lo]);
                const int j = pos >> a.page_shift, off = pos & P1;
                const int held = (int)(((int64_t)ctx + P1) >> a.page_shift);
                int32_t * entry = a.table + (int64_t)lo * a.max_pages + j;
                int32_t page;
                if (j < held) {
                    page = *entry;
                } else {
                    page = a.free_pages[base + j - held];
                    if (off == 0) *entry = page;
                }
                if (page >= 0 && page < a.n_pages)
                    slot = ((int64_t)page << a.page_shift) + off;
                else
                    status |= TQ_STATUS_BAD_PAGE;
            }
        }
        a.slots[i] = slot;
        if (a.positions != nullptr) a.positions[i] = pos;
    }
    if (status != 0u && a.status != nullptr) atomicOr(a.status, status);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" tq_status tq_page_tables(const int32_t * ctx_lens, const int32_t * new_lens, int32_t batch,
                                    int32_t page_size, int32_t n_pages, const int32_t * free_pages,
                                    int32_t n_free, int32_t * block_table, int32_t max_pages,
                                    int32_t * cu_new, int32_t * total_lens, int64_t * slots,
                                    int32_t * positions, int32_t n_slots, int32_t * n_taken,
                                    uint32_t * status_dev, void * stream) {
    if (batch < 1) return fail(TQ_ERR_INVALID_ARG, "batch must be >= 1");
    if (batch > kPtMaxBatch) return fail(TQ_ERR_UNSUPPORTED, "batch above 16384");
    if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
        return fail(TQ_ERR_UNSUPPORTED, "page_size must be a power of two in [16, 65536]");
    if (n_pages < 1 || max_pages < 1) return fail(TQ_ERR_INVALID_ARG, "n_pages and max_pages must be >= 1");
    if (n_free < 0 || n_slots < 0) return fail(TQ_ERR_INVALID_ARG, "n_free and n_slots must be >= 0");
    if (!ctx_lens || !new_lens || !block_table || !cu_new || !total_lens || !n_taken)
        return fail(TQ_ERR_INVALID_ARG, "null lengths / block_table / cu_new / total_lens / n_taken");
    if (total_lens == ctx_lens || total_lens == new_lens || cu_new == ctx_lens || cu_new == new_lens)
        return fail(TQ_ERR_INVALID_ARG, "total_lens and cu_new must not be input arrays");
    if ((n_free > 0 && !free_pages) || (n_slots > 0 && !slots))
        return fail(TQ_ERR_INVALID_ARG, "null free_pages / slots");
    if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(free_pages, 4) || !aligned(block_table, 4) ||
        !aligned(cu_new, 4) || !aligned(total_lens, 4) || !aligned(slots, 8) || !aligned(positions, 4) ||
        !aligned(n_taken, 4) || !aligned(status_dev, 4))
        return fail(TQ_ERR_INVALID_ARG, "int32 arrays 4-byte, slots 8-byte aligned");
    PageTablesArgs a{};
    a.ctx = ctx_lens;
    a.add = new_lens;
    a.batch = batch;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.n_pages = n_pages;
    a.free_pages = free_pages;
    a.n_free = n_free;
    a.table = block_table;
    a.max_pages = max_pages;
    a.cu = cu_new;
    a.total = total_lens;
    a.slots = slots;
    a.positions = positions;
    a.n_slots = n_slots;
    a.n_taken = n_taken;
    a.status = status_dev;
    const int smem = (2 * batch + 1) * 4;
    if (int e = ensure_dynamic_smem(reinterpret_cast<const void *>(page_tables_kernel), smem))
        return cuda_status(e, "page tables shared memory");
    const int64_t grid = n_slots > 0 ? ((int64_t)n_slots + kPtTokens - 1) / kPtTokens : 1;
    page_tables_kernel<<<(unsigned)grid, kPtThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
    return cuda_status((int)cudaGetLastError(), "page tables launch");
}
