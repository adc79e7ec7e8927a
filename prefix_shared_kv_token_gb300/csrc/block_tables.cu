// build_block_tables: a step's page table entries, slot map, positions and query offsets from
// the requests' lengths, on the device.
//
// Request r has seq[r] context positions after the step, new[r] of them new.  With
// had = ceil((seq - new) / P) pages before and has = ceil(seq / P) after, it takes
// need = has - had pages off the free list, in request order:
//     table[row[r]][had + j] = free[head + off[r] + j],   off = exclusive sum of need,
// and its new token i (position t = seq - new + i, query row indptr[r] + i) goes to slot
// table[row[r]][t / P] * P + t mod P.
//
// A page id that no pool can have (negative, or its slots past 2^31) is flagged, its tokens' slots are -1.
// A step with a bad request (or more pages than the list has, or more tokens than the maps
// hold) is refused whole: the error word is set, no table entry is written, every map entry is
// -1 and the list's head stays.
//
// Bound: latency.  A decode step moves a few KB; the chain lengths -> scan -> page -> slot is
// three dependent loads.  So there is one launch: every CTA scans all lengths (4 bytes each, from
// L2) instead of waiting for another CTA's sums, then takes its share of the tokens and fresh
// pages, finding each one's request by bisection of the sums in shared memory.  The head is
// written by the CTA that finishes last, so that it may be read and written in place.

#include <algorithm>
#include <atomic>

#include "block.cuh"

namespace pkv {

constexpr int kTabThreads = 512;
constexpr int kMaxTableBatch = 16384;
constexpr int kTicketWord = 16;  // of the workspace header

struct TableParams {
    int32_t *table;
    int64_t stride;
    int32_t num_rows, shift, batch;
    const int32_t *rows, *seq, *fresh;  // fresh: new tokens per request
    const int32_t *free_pages;
    int64_t num_free;
    const int32_t *head;
    int32_t *head_out;
    int32_t *loc, *pos, *indptr;
    int64_t cap;
    int32_t *err;
    uint32_t *ticket;
};

// pages of n positions
PKV_DEV int32_t pages_of(int32_t n, int shift) { return (int32_t)(((int64_t)n + (1 << shift) - 1) >> shift); }
// last r in [0, n) with a[r] <= x (a ascending, a[0] <= x)
PKV_DEV int last_at_most(const int32_t *a, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) block_tables_kernel(const TableParams p) {
    extern __shared__ int32_t sums[];  // token sums [batch + 1], page sums [batch + 1]
    int32_t *tok = sums, *pg = sums + p.batch + 1;
    __shared__ int64_t warp_tok[kTabThreads / 32], warp_pg[kTabThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mask = (1 << p.shift) - 1;
    const int32_t head = __ldcg(p.head);

    // exclusive sums of new tokens and fresh pages: a chunk of requests a thread, then the block
    const int chunk = (p.batch + kTabThreads - 1) / kTabThreads;
    const int r0 = min(tid * chunk, p.batch), r1 = min(r0 + chunk, p.batch);
    int64_t my_tok = 0, my_pg = 0;  // 64 bits: a bad step may ask for more than 2^31
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const int32_t seq = ld(p.seq + r), n = ld(p.fresh + r), row = ld(p.rows + r);
        const bool ok = n >= 0 && seq >= n && (int64_t)seq <= (p.stride << p.shift) && row >= 0 && row < p.num_rows;
        bad |= !ok;
        if (ok) {
            my_tok += n;
            my_pg += pages_of(seq, p.shift) - pages_of(seq - n, p.shift);
        }
    }
    int64_t scan_tok = my_tok, scan_pg = my_pg;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, scan_tok, d), y = __shfl_up_sync(0xffffffffu, scan_pg, d);
        if (lane >= d) {
            scan_tok += x;
            scan_pg += y;
        }
    }
    if (lane == 31) {
        warp_tok[warp] = scan_tok;
        warp_pg[warp] = scan_pg;
    }
    bad = __syncthreads_or(bad);
    int64_t tokens = 0, pages = 0, base_tok = 0, base_pg = 0;
    for (int w = 0; w < kTabThreads / 32; ++w) {
        if (w == warp) {
            base_tok = tokens;
            base_pg = pages;
        }
        tokens += warp_tok[w];
        pages += warp_pg[w];
    }
    bad |= tokens > p.cap;
    const bool refuse = bad || head < 0 || (int64_t)head + pages > p.num_free;
    if (refuse) {
        if (tid == 0 && blockIdx.x == 0)
            set_error(p.err, bad ? DERR_POSITION : DERR_NO_PAGES);
    } else {
        int64_t at_tok = base_tok + scan_tok - my_tok, at_pg = base_pg + scan_pg - my_pg;
        for (int r = r0; r < r1; ++r) {
            const int32_t seq = ld(p.seq + r), n = ld(p.fresh + r);
            tok[r] = (int32_t)at_tok;
            pg[r] = (int32_t)at_pg;
            at_tok += n;
            at_pg += pages_of(seq, p.shift) - pages_of(seq - n, p.shift);
        }
        if (tid == 0) {
            tok[p.batch] = (int32_t)tokens;
            pg[p.batch] = (int32_t)pages;
        }
    }
    __syncthreads();

    const int64_t step = (int64_t)gridDim.x * kTabThreads;
    const int64_t first = (int64_t)blockIdx.x * kTabThreads + tid;
    for (int64_t i = first; i <= p.batch; i += step) p.indptr[i] = refuse ? 0 : tok[i];
    for (int64_t i = first; i < p.cap; i += step) {
        int32_t slot = -1, t = -1;
        if (!refuse && i < tokens) {
            const int r = last_at_most(tok, p.batch, (int32_t)i);
            const int32_t old = ld(p.seq + r) - ld(p.fresh + r);
            t = old + (int32_t)(i - tok[r]);
            const int32_t had = pages_of(old, p.shift), b = t >> p.shift;
            const int32_t page = b < had ? p.table[(int64_t)ld(p.rows + r) * p.stride + b]
                                         : ld(p.free_pages + head + pg[r] + (b - had));
            if ((uint32_t)page <= (uint32_t)0x7FFFFFFF >> p.shift)
                slot = (page << p.shift) + (t & mask);
            else
                set_error(p.err, DERR_SLOT_RANGE);  // no page: its slots do not fit
        }
        p.loc[i] = slot;
        p.pos[i] = t;
    }
    if (!refuse) {
        for (int64_t i = first; i < pages; i += step) {
            const int r = last_at_most(pg, p.batch, (int32_t)i);
            const int32_t old = ld(p.seq + r) - ld(p.fresh + r);
            const int64_t b = pages_of(old, p.shift) + (i - pg[r]);
            p.table[(int64_t)ld(p.rows + r) * p.stride + b] = ld(p.free_pages + head + i);
        }
    }
    // every CTA has read the head before it draws its ticket; the counter wraps to 0 by itself
    if (tid == 0) {
        bool last = gridDim.x == 1;
        if (!last) {
            __threadfence();
            last = atomicInc(p.ticket, gridDim.x - 1) == gridDim.x - 1;
        }
        if (last) *p.head_out = refuse ? head : head + (int32_t)pages;
    }
}

}  // namespace pkv

extern "C" int pkv_build_block_tables(const pkv_batch *batch, const int32_t *new_lens, const int32_t *free_pages,
                                      int64_t num_free, const int32_t *free_head, int32_t *free_head_out,
                                      int32_t *out_cache_loc, int32_t *positions, int64_t cap, int32_t *qo_indptr,
                                      void *workspace, size_t ws_bytes, void *stream) {
    using namespace pkv;
    if (!batch || !batch->req_to_token || !free_head || !free_head_out || !qo_indptr || !workspace)
        return PKV_E_INVALID;
    if (batch->batch < 0 || batch->num_rows < 0 || batch->stride < 0 || num_free < 0 || cap < 0) return PKV_E_INVALID;
    if (batch->batch > 0 && (!batch->req_pool_indices || !batch->seq_lens || !new_lens)) return PKV_E_INVALID;
    if ((cap > 0 && (!out_cache_loc || !positions)) || (num_free > 0 && !free_pages)) return PKV_E_INVALID;
    const int shift = page_shift_of(batch);
    if (shift < 0 || num_free >= ((int64_t)1 << 31) || cap >= ((int64_t)1 << 31) || batch->stride >= ((int64_t)1 << 31))
        return PKV_E_INVALID;
    if (batch->batch > kMaxTableBatch) return PKV_E_UNSUPPORTED;
    if (ws_bytes < kWorkspaceHeader) return PKV_E_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 3) return PKV_E_INVALID;
    TableParams p;
    p.table = const_cast<int32_t *>(batch->req_to_token);
    p.stride = batch->stride;
    p.num_rows = batch->num_rows;
    p.shift = shift;
    p.batch = batch->batch;
    p.rows = batch->req_pool_indices;
    p.seq = batch->seq_lens;
    p.fresh = new_lens;
    p.free_pages = free_pages;
    p.num_free = num_free;
    p.head = free_head;
    p.head_out = free_head_out;
    p.loc = out_cache_loc;
    p.pos = positions;
    p.indptr = qo_indptr;
    p.cap = cap;
    p.err = static_cast<int32_t *>(workspace);
    p.ticket = reinterpret_cast<uint32_t *>(workspace) + kTicketWord;
    const int64_t want = (std::max<int64_t>(cap, batch->batch + 1) + kTabThreads - 1) / kTabThreads;
    const int grid = (int)std::min<int64_t>(want, num_sms());
    const size_t smem = 2 * ((size_t)batch->batch + 1) * sizeof(int32_t);
    // Leave for the largest batch's sums, given once a device and never lowered: a size of this call's own could be
    // taken back by another thread's smaller call before the launch.  (The 48 KB a kernel may use without it
    // count its static shared memory too.)
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_E_CUDA;
    if (dev >= 64 || !((allowed.load(std::memory_order_relaxed) >> dev) & 1)) {
        constexpr int most = 2 * (kMaxTableBatch + 1) * (int)sizeof(int32_t);
        if (cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return PKV_E_CUDA;
        if (dev < 64) allowed.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    }
    return launch_pdl(block_tables_kernel, dim3(grid), dim3(kTabThreads), smem, reinterpret_cast<cudaStream_t>(stream),
                      true, p) == cudaSuccess
               ? PKV_OK
               : PKV_E_CUDA;
}
