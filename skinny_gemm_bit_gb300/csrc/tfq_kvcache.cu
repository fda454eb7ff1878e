// The paged K/V cache: descriptor, and the page operations on the device.
//
//   extend  one block: validates the call, takes free pages, writes each new row's slot
//   fork    plan (one block: who copies what, lengths) -> apply (page tables, reference
//           counts and the copies of the unfilled pages, side by side)
//   keep    plan (one block: lengths, freed pages, the pages of each block) -> move (rows)
//
// The books are small (a few thousand integers), so one block of 1024 threads, one thread a
// slot, decides everything from one consistent state and the calls can be all or nothing; the
// rows, which are the bytes (a 64-sequence keep over 28 layers moves 26 MB), are moved by
// the whole GPU from what the plan left in the workspace.
//
// That keep takes 16.8 us, plan and move (and a copy of the book, as in the next); the moves are scattered rows of
// 256 bytes, each read and written once. A fork of 32 slots that copies 38 MB takes 19.3 us, an extend 3.4 to 5.4. Plans are chains of a few dependent
// reads and barriers (some 4 us); the second kernel's launch hides behind them.
#include "tfq_cache.h"
#include "tfq_ptx.cuh"

namespace tfq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFreeList = 4096;   // fresh pages of a call held in shared memory
constexpr int kForkCols = 16;     // page-table columns a block of the fork's apply kernel takes
constexpr int kCopyThreads = 256;
constexpr int kBlockPages = kMaxDraftRows / 16 + 1;  // pages that a block of drafts can touch
constexpr size_t kPlanHeader = 256;                  // after the status word's 256 bytes

// One slot's (fork) or sequence's (keep) part of a plan.
struct SlotPlan {
    int32_t parent;     // fork: the slot it takes (itself: unchanged)
    int32_t old_len;    // fork: the slot's length before the call; keep: the length before the block
    int32_t new_len;    // fork: its length after; keep: rows kept, -1: leave the sequence alone
    int32_t fresh;      // fork: the fresh page that takes the unfilled page's place, or -1; keep: q_start[b]
    int32_t pages[kBlockPages + 1];  // keep: the block's pages
};
struct PlanHeader2 {
    int32_t ok;        // fork: the plan is to be carried out
    int32_t n_copies;  // fork
    int32_t max_cols;  // fork: page-table columns that any slot uses, before or after
};
struct CopyItem {
    int32_t src, dst, rows;
};

size_t plan_bytes(int n_seqs)
{
    return 256 + kPlanHeader + (size_t)n_seqs * (sizeof(SlotPlan) + sizeof(CopyItem));
}

__device__ __forceinline__ SlotPlan* plan_slots(void* ws) { return reinterpret_cast<SlotPlan*>((uint8_t*)ws + 256 + kPlanHeader); }
__device__ __forceinline__ PlanHeader2* plan_header(void* ws) { return reinterpret_cast<PlanHeader2*>((uint8_t*)ws + 256); }
__device__ __forceinline__ CopyItem* plan_copies(void* ws, int n_seqs)
{
    return reinterpret_cast<CopyItem*>(plan_slots(ws) + n_seqs);
}

// Exclusive prefix sum of one value a thread over the block; *total is the sum. `buf` holds 33.
__device__ int64_t block_scan(int64_t v, int64_t* buf, int64_t* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o)
            x += y;
    }
    __syncthreads();  // the last use of buf is over
    if (lane == 31)
        buf[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t s = buf[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o)
                s += y;
        }
        buf[lane] = s;
    }
    __syncthreads();
    *total = buf[31];
    return x - v + (warp > 0 ? buf[warp - 1] : 0);
}

// Calls emit(rank, page) for the `want` lowest free pages (fewer if there are not so many)
// and returns how many there were, at most want. All threads of the block.
template <class Emit>
__device__ int64_t scan_free(const CacheView& c, int64_t want, int64_t* buf, Emit&& emit)
{
    int64_t found = 0;
    for (int64_t p0 = 0; p0 < c.n_pages && found < want; p0 += 4 * kPlanThreads) {
        const int64_t p = p0 + 4 * (int64_t)threadIdx.x;
        unsigned free_bits = 0;
        for (int i = 0; i < 4; ++i)
            if (p + i < c.n_pages && c.refs[p + i] == 0)
                free_bits |= 1u << i;
        int64_t total;
        int64_t rank = found + block_scan(__popc(free_bits), buf, &total);
        for (int i = 0; i < 4; ++i)
            if (free_bits >> i & 1) {
                if (rank < want)
                    emit(rank, (int)(p + i));
                ++rank;
            }
        found += total;
    }
    return found < want ? found : want;
}

__device__ __forceinline__ bool page_ok(const CacheView& c, int page) { return page >= 0 && page < c.n_pages; }

// ---------------------------------------------------------------- extend

__global__ void __launch_bounds__(kPlanThreads) extend_kernel(CacheView c, const int32_t* seqs, const int32_t* q_start,
                                                              int B, int64_t M, const uint64_t* masks, int32_t* slots,
                                                              int32_t* positions, int* status)
{
    __shared__ int64_t buf[33];
    __shared__ int64_t offs[kPlanThreads];  // first fresh page (by rank) of each sequence
    __shared__ int32_t start[kPlanThreads + 1], base[kPlanThreads], slot_of[kPlanThreads];
    __shared__ int32_t list[kFreeList];
    __shared__ unsigned seen[kMaxSeqs / 32];
    __shared__ int bad;
    const int b = threadIdx.x;
    if (b < kMaxSeqs / 32)
        seen[b] = 0;
    if (b == 0)
        bad = 0;
    if (b <= B)
        start[b] = q_start[b];
    if (b == 0 && B == kPlanThreads)
        start[B] = q_start[B];
    __syncthreads();
    int s = 0, len = 0;
    int64_t need = 0, fresh_len = 0;
    if (b < B) {
        s = seqs[b];
        bool ok = s >= 0 && s < c.n_seqs && start[b] >= 0 && start[b] <= start[b + 1] && start[b + 1] <= M;
        if (ok)
            ok = !(atomicOr(&seen[s >> 5], 1u << (s & 31)) >> (s & 31) & 1);
        if (ok) {
            len = c.len[s];
            fresh_len = (int64_t)len + start[b + 1] - start[b];
            ok = len >= 0 && fresh_len <= (int64_t)c.max_pages << c.page_shift;
        }
        const int fill = len & (c.page_size - 1);
        if (ok && fill && fresh_len > len) {  // an unfilled last page must be this slot's alone
            const int p = c.table[(int64_t)s * c.max_pages + (len >> c.page_shift)];
            ok = page_ok(c, p) && c.refs[p] == 1;
        }
        if (!ok)
            bad = 1;
        need = ((fresh_len + c.page_size - 1) >> c.page_shift) - (((int64_t)len + c.page_size - 1) >> c.page_shift);
        base[b] = len;
        slot_of[b] = s;
    }
    int64_t total;
    const int64_t at = block_scan(b < B ? need : 0, buf, &total);  // its barriers also publish `bad`
    if (b < B)
        offs[b] = at;
    __syncthreads();
    int code = bad ? TF_E_INVALID_ARG : TF_OK;
    if (code == TF_OK && total > 0) {
        const bool small = total <= kFreeList;
        const int64_t got = scan_free(c, total, buf, [&](int64_t rank, int page) {
            if (small)
                list[rank] = page;
        });
        if (got < total)
            code = TF_E_CACHE_FULL;
        __syncthreads();
        auto assign = [&](int64_t rank, int page) {
            int lo = 0, hi = B - 1;  // the last sequence whose first fresh page is not behind `rank`
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (offs[mid] <= rank)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int64_t col = (((int64_t)base[lo] + c.page_size - 1) >> c.page_shift) + (rank - offs[lo]);
            c.table[(int64_t)slot_of[lo] * c.max_pages + col] = page;
            c.refs[page] = 1;
        };
        if (code == TF_OK) {
            if (small) {
                for (int64_t r = b; r < total; r += kPlanThreads)
                    assign(r, list[r]);
            } else {
                // a thread marks pages that it alone has read in this scan
                scan_free(c, total, buf, assign);
            }
        }
    }
    __syncthreads();
    if (code == TF_OK && b < B)
        c.len[s] = (int)fresh_len;
    if (code != TF_OK && b == 0)
        record_status(status, code);
    for (int64_t m = b; m < M; m += kPlanThreads) {
        int32_t slot = -1, pos = 0;
        if (code == TF_OK && m >= start[0] && m < start[B]) {
            int lo = 0, hi = B - 1;  // the last sequence that starts at or before m
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (start[mid] <= m)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int j = (int)(m - start[lo]);
            const int at_row = base[lo] + j;
            const int page = c.table[(int64_t)slot_of[lo] * c.max_pages + (at_row >> c.page_shift)];
            slot = page * c.page_size + (at_row & (c.page_size - 1));
            pos = masks == nullptr ? at_row : base[lo] + max(__popcll(masks[m]) - 1, 0);
        }
        slots[m] = slot;
        if (positions != nullptr)
            positions[m] = pos;
    }
}

// ---------------------------------------------------------------- fork

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(CacheView c, const int32_t* parent, void* ws)
{
    pdl_launch_dependents();  // its blocks wait for this one's plan
    __shared__ int64_t buf[33];
    __shared__ int32_t keeper[kMaxSeqs];  // the slot that keeps each parent's unfilled page (-1: itself)
    __shared__ int32_t list[kMaxSeqs];
    __shared__ int32_t lens[kMaxSeqs];
    __shared__ unsigned taken[kMaxSeqs / 32];  // slots that another one takes
    __shared__ int bad, cols;
    const int s = threadIdx.x;
    if (s == 0) {
        bad = 0;
        cols = 0;
    }
    if (s < kMaxSeqs / 32)
        taken[s] = 0;
    if (s < c.n_seqs)
        keeper[s] = INT32_MAX;
    __syncthreads();
    int p = s, len = 0, new_len = 0, tail = -1;
    if (s < c.n_seqs) {
        p = parent[s];
        lens[s] = len = c.len[s];
        bool ok = p >= -1 && p < c.n_seqs && len >= 0 && len <= (int64_t)c.max_pages << c.page_shift;
        new_len = len;
        if (ok && p >= 0) {
            new_len = c.len[p];
            ok = new_len >= 0 && new_len <= (int64_t)c.max_pages << c.page_shift;
            atomicMin(&keeper[p], p == s ? -1 : s);
            if (ok && p != s)
                atomicOr(&taken[p >> 5], 1u << (p & 31));
        } else if (ok) {
            new_len = 0;
        }
        if (!ok)
            bad = 1;
        else
            atomicMax(&cols, (max(len, new_len) + c.page_size - 1) >> c.page_shift);
    }
    __syncthreads();
    const int fill = new_len & (c.page_size - 1);
    bool copy = s < c.n_seqs && !bad && p >= 0 && p != s && fill != 0 && keeper[p] != s;
    if (copy)
        tail = c.table[(int64_t)p * c.max_pages + (new_len >> c.page_shift)];
    // nothing is taken over with an entry that is no page: the pages of the slots taken, a warp a slot. Costs a fork
    // of 32 slots of 8 pages 0.2 us, of 64 of 512 2.5, of 1024 of 500 35.
    for (int t = s >> 5; t < c.n_seqs; t += kPlanThreads / 32)
        if (taken[t >> 5] >> (t & 31) & 1) {
            const int used = (int)(((int64_t)lens[t] + c.page_size - 1) >> c.page_shift);
            const int32_t* row = c.table + (int64_t)t * c.max_pages;
            bool ok = true;
            for (int c0 = s & 31; c0 < used; c0 += 32 * 8) {  // eight loads under way
                int page[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    page[i] = c0 + 32 * i < used ? row[c0 + 32 * i] : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    ok &= page_ok(c, page[i]);
            }
            if (!ok)
                bad = 1;
        }
    int64_t total;
    const int64_t rank = block_scan(copy ? 1 : 0, buf, &total);
    const bool refused = bad != 0;  // every write of `bad` is before the scan's barriers
    const int64_t got = refused ? 0 : scan_free(c, total, buf, [&](int64_t r, int page) { list[r] = page; });
    __syncthreads();
    const int code = refused ? TF_E_INVALID_ARG : got < total ? TF_E_CACHE_FULL : TF_OK;
    if (s < c.n_seqs) {
        SlotPlan* pl = plan_slots(ws) + s;
        pl->parent = p;
        pl->old_len = len;
        pl->new_len = new_len;
        pl->fresh = code == TF_OK && copy ? list[rank] : -1;
        if (code == TF_OK) {
            if (copy)
                plan_copies(ws, c.n_seqs)[rank] = CopyItem{tail, list[rank], fill};
            c.len[s] = new_len;
        }
    }
    if (s == 0) {
        PlanHeader2* h = plan_header(ws);
        h->ok = code == TF_OK;
        h->n_copies = code == TF_OK ? (int)total : 0;
        h->max_cols = cols;
        if (code != TF_OK)
            record_status(static_cast<int*>(ws), code);
    }
}

// Copies `rows` rows of every head of a page, in all layers, K and V. A unit is one
// (copy, layer, kv, head): rows * head_dim elements in a row on both sides.
__device__ void copy_pages(const CacheView& c, const CopyItem* items, int n_items, int block, int n_blocks)
{
    const int units_per = c.n_layers * 2 * c.n_kv;
    const int64_t units = (int64_t)n_items * units_per;
    const int row16 = c.head_dim / 8;
    for (int64_t u = block; u < units; u += n_blocks) {
        const CopyItem it = items[u / units_per];
        const int lkh = (int)(u % units_per), head = lkh % c.n_kv, lk = lkh / c.n_kv;
        const uint4* src = reinterpret_cast<const uint4*>(c.data + c.row_of(lk >> 1, lk & 1, it.src, head) * c.head_dim);
        uint4* dst = reinterpret_cast<uint4*>(c.data + c.row_of(lk >> 1, lk & 1, it.dst, head) * c.head_dim);
        const int n = it.rows * row16;
        for (int i = threadIdx.x; i < n; i += 4 * kCopyThreads) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j * kCopyThreads < n)
                    v[j] = __ldcg(src + i + j * kCopyThreads);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j * kCopyThreads < n)
                    dst[i + j * kCopyThreads] = v[j];
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(CacheView c, int col_blocks, void* ws)
{
    extern __shared__ int32_t tile[];  // [n_seqs][kForkCols]
    pdl_wait();
    const PlanHeader2 h = *plan_header(ws);
    if (!h.ok)
        return;
    if ((int)blockIdx.x >= col_blocks) {
        copy_pages(c, plan_copies(ws, c.n_seqs), h.n_copies, blockIdx.x - col_blocks, gridDim.x - col_blocks);
        return;
    }
    // a column of the page table depends on the same column alone, so a block holds its
    // columns of every slot as they were and then writes them anew
    const SlotPlan* pl = plan_slots(ws);
    for (int c0 = blockIdx.x * kForkCols; c0 < h.max_cols; c0 += col_blocks * kForkCols) {
        for (int i = threadIdx.x; i < c.n_seqs * kForkCols; i += blockDim.x) {
            const int s = i / kForkCols, col = c0 + i % kForkCols;
            const int used = (pl[s].old_len + c.page_size - 1) >> c.page_shift;
            tile[i] = col < used ? c.table[(int64_t)s * c.max_pages + col] : -1;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < c.n_seqs * kForkCols; i += blockDim.x) {
            const int s = i / kForkCols, col = c0 + i % kForkCols;
            const int p = pl[s].parent;
            if (p == s || col >= c.max_pages)
                continue;
            const int was = tile[i];
            int now = p < 0 ? -1 : tile[p * kForkCols + i % kForkCols];
            if (now >= 0 && pl[s].fresh >= 0 && col == pl[s].new_len >> c.page_shift)
                now = pl[s].fresh;
            if (page_ok(c, was))
                atomicAdd(&c.refs[was], -1);
            if (page_ok(c, now))
                atomicAdd(&c.refs[now], 1);
            if (now != was)
                c.table[(int64_t)s * c.max_pages + col] = now;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- keep

__global__ void __launch_bounds__(kPlanThreads) keep_plan_kernel(CacheView c, const int32_t* seqs, const int32_t* q_start,
                                                                 const int32_t* keep, const int32_t* n_keep, int B,
                                                                 int64_t M, void* ws)
{
    pdl_launch_dependents();  // its blocks wait for this one's plan
    __shared__ unsigned seen[kMaxSeqs / 32];
    __shared__ int twice, bad;
    const int b = threadIdx.x;
    if (b < kMaxSeqs / 32)
        seen[b] = 0;
    if (b == 0)
        twice = bad = 0;
    __syncthreads();
    bool ok = false;
    int s = 0, r0 = 0, T = 0, len = 0, n = 0;
    SlotPlan pl;
    if (b < B) {
        s = seqs[b];
        r0 = q_start[b];
        const int r1 = q_start[b + 1];
        n = n_keep[b];
        const bool slot_ok = s >= 0 && s < c.n_seqs;
        if (slot_ok && (atomicOr(&seen[s >> 5], 1u << (s & 31)) >> (s & 31) & 1))
            twice = 1;
        ok = slot_ok && r0 >= 0 && r0 <= r1 && r1 <= M && r1 - r0 <= kMaxDraftRows;
        if (ok) {
            T = r1 - r0;
            len = c.len[s];
            ok = len >= T && len <= (int64_t)c.max_pages << c.page_shift && n >= 0 && n <= T;
        }
        int last = -1;
        for (int j = 0; ok && j < n; ++j) {
            const int k = keep[r0 + j];
            ok = k > last && k < T;
            last = k;
        }
        const int first = (len - T) >> c.page_shift;
        for (int i = 0; ok && T > 0 && i < kBlockPages && first + i <= (len - 1) >> c.page_shift; ++i) {
            const int p = c.table[(int64_t)s * c.max_pages + first + i];
            ok = page_ok(c, p) && c.refs[p] == 1;
            pl.pages[i] = p;
        }
        if (!ok)
            bad = 1;
    }
    __syncthreads();
    if (twice)
        ok = false;
    if (b == 0 && (twice || bad))
        record_status(static_cast<int*>(ws), TF_E_INVALID_ARG);
    if (b >= B)
        return;
    const int base = len - T;
    pl.parent = s;
    pl.old_len = base;
    pl.new_len = ok ? n : -1;
    pl.fresh = r0;
    plan_slots(ws)[b] = pl;
    if (!ok)
        return;
    // the pages of the block are this slot's alone: no other thread touches them
    for (int64_t col = ((int64_t)base + n + c.page_size - 1) >> c.page_shift;
         col < ((int64_t)len + c.page_size - 1) >> c.page_shift; ++col) {
        int32_t* e = &c.table[(int64_t)s * c.max_pages + col];
        c.refs[*e] = 0;
        *e = -1;
    }
    c.len[s] = base + n;
}

// A thread moves one 16-byte column of a sequence's rows (layer, K or V, head, 16 bytes of a row)
// from the kept rows up to the rows behind the base, eight rows at a time: loads first, then stores.
// A kept row lies at or behind its place and the kept rows increase, so no store reaches a row
// that a later batch still reads. The rows' places are the same for every column but for its start.
__global__ void __launch_bounds__(kCopyThreads) keep_move_kernel(CacheView c, const int32_t* __restrict__ q_start,
                                                                 const int32_t* __restrict__ keep, int64_t M, void* ws)
{
    __shared__ SlotPlan pl;
    __shared__ int64_t src[kMaxDraftRows], dst[kMaxDraftRows];  // elements; src < 0: stays
    // the lists are the caller's; the plan is the kernel's before this one
    const int64_t at = (int64_t)q_start[blockIdx.y] + threadIdx.x;
    const int from = threadIdx.x < kMaxDraftRows && at >= 0 && at < M ? keep[at] : 0;
    const int row16 = c.head_dim / 8, cols = c.n_layers * 2 * c.n_kv * row16;
    const int col = blockIdx.x * kCopyThreads + threadIdx.x;
    const int lkh = col / row16, head = lkh % c.n_kv, lk = lkh / c.n_kv;
    uint16_t* base = c.data + c.row_of(lk >> 1, lk & 1, 0, head) * c.head_dim + (col - lkh * row16) * 8;
    pdl_wait();
    if (threadIdx.x < sizeof(SlotPlan) / 4)
        reinterpret_cast<int32_t*>(&pl)[threadIdx.x] = __ldcg(reinterpret_cast<const int32_t*>(plan_slots(ws) + blockIdx.y) + threadIdx.x);
    __syncthreads();
    const int n = pl.new_len;
    if (n <= 0)
        return;
    if ((int)threadIdx.x < n) {
        const int first = pl.old_len >> c.page_shift, j = threadIdx.x;
        auto place = [&](int i) {
            const int row = pl.old_len + i;
            return ((int64_t)pl.pages[(row >> c.page_shift) - first] * c.n_kv * c.page_size + (row & (c.page_size - 1))) * c.head_dim;
        };
        src[j] = from == j ? -1 : place(from);
        dst[j] = place(j);
    }
    __syncthreads();
    if (col >= cols)
        return;
    for (int j0 = 0; j0 < n; j0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < n && src[j0 + j] >= 0)
                v[j] = *reinterpret_cast<const uint4*>(base + src[j0 + j]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j0 + j < n && src[j0 + j] >= 0)
                *reinterpret_cast<uint4*>(base + dst[j0 + j]) = v[j];
    }
}

__global__ void reset_kernel(CacheView c, int64_t n)
{
    const int64_t zeros = (int64_t)c.n_seqs + c.n_pages;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
        c.len[i] = i < zeros ? 0 : -1;
}

bool shape_ok(int64_t n_layers, int64_t n_kv, int64_t head_dim, int64_t page_size, int64_t n_pages)
{
    return n_layers >= 1 && n_layers <= 4096 && n_kv >= 1 && n_kv <= 256 &&
           (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
           (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128) && n_pages >= 1 &&
           n_pages < ((int64_t)1 << 31) / page_size &&
           n_pages < ((int64_t)1 << 31) / (n_layers * 2 * n_kv * page_size);
}

bool book_ok(int64_t n_seqs, int64_t max_pages, int64_t page_size)
{
    return n_seqs >= 1 && n_seqs <= kMaxSeqs && max_pages >= 1 && max_pages < ((int64_t)1 << 31) / page_size;
}

}  // namespace

int check_cache(const tf_kvcache* c, const char* name, CacheView* v)
{
    if (c == nullptr)
        return report_error(TF_E_INVALID_ARG, "%s: cache descriptor is NULL", name);
    if (c->magic != TF_KVCACHE_MAGIC)
        return report_error(TF_E_INVALID_ARG, "%s: cache descriptor not filled by tf_kvcache_init", name);
    if (!shape_ok(c->n_layers, c->n_kv, c->head_dim, c->page_size, c->n_pages) ||
        !book_ok(c->n_seqs, c->max_pages, c->page_size))
        return report_error(TF_E_UNSUPPORTED_SHAPE, "%s: cache shape out of range", name);
    if (c->data == nullptr || c->book == nullptr || !is_aligned(c->data, 16) || !is_aligned(c->book, 4))
        return report_error(TF_E_INVALID_ARG, "%s: cache data or book NULL or misaligned", name);
    v->data = static_cast<uint16_t*>(c->data);
    v->len = c->book;
    v->refs = c->book + c->n_seqs;
    v->table = v->refs + c->n_pages;
    v->n_layers = c->n_layers;
    v->n_kv = c->n_kv;
    v->head_dim = c->head_dim;
    v->page_size = c->page_size;
    v->page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
    v->n_seqs = c->n_seqs;
    v->n_pages = c->n_pages;
    v->max_pages = c->max_pages;
    return TF_OK;
}

int check_ws(const void* ws, size_t ws_bytes, size_t need, const char* name)
{
    if (ws == nullptr || !is_aligned(ws, 256))
        return report_error(TF_E_INVALID_ARG, "%s: workspace NULL or not 256-byte aligned", name);
    if (ws_bytes < need)
        return report_error(TF_E_WORKSPACE_TOO_SMALL, "%s: workspace has %zu bytes, needs %zu", name, ws_bytes, need);
    return TF_OK;
}

}  // namespace tfq

using namespace tfq;

namespace {

int launched(cudaError_t e, const char* name)
{
    return e == cudaSuccess ? TF_OK : report_error(TF_E_CUDA, "%s: %s", name, cudaGetErrorString(e));
}

int check_batch(const CacheView& v, const int32_t* seqs, const int32_t* q_start, int64_t B, int64_t M, const char* name)
{
    if (seqs == nullptr || q_start == nullptr)
        return report_error(TF_E_INVALID_ARG, "%s: seqs or q_start is NULL", name);
    if (B < 1 || B > v.n_seqs || M < 1 || M > INT32_MAX)
        return report_error(TF_E_UNSUPPORTED_SHAPE, "%s: need 1 <= B <= n_seqs and 1 <= M < 2^31", name);
    return TF_OK;
}

}  // namespace

extern "C" {

size_t tf_kvcache_data_bytes(int n_layers, int n_kv, int head_dim, int page_size, int64_t n_pages)
{
    if (!shape_ok(n_layers, n_kv, head_dim, page_size, n_pages))
        return 0;
    return (size_t)n_layers * 2 * n_pages * n_kv * page_size * head_dim * sizeof(uint16_t);
}

size_t tf_kvcache_book_elems(int64_t n_pages, int n_seqs, int64_t max_pages)
{
    if (n_pages < 1 || n_pages > INT32_MAX || !book_ok(n_seqs, max_pages, 16))
        return 0;
    return (size_t)n_seqs + n_pages + (size_t)n_seqs * max_pages;
}

int tf_kvcache_init(int n_layers, int n_kv, int head_dim, int page_size, int64_t n_pages, int n_seqs,
                    int64_t max_pages, void* data, size_t data_bytes, int32_t* book, size_t book_elems,
                    tf_kvcache* desc)
{
    const char* name = "tf_kvcache_init";
    if (desc == nullptr)
        return report_error(TF_E_INVALID_ARG, "%s: desc is NULL", name);
    if (!shape_ok(n_layers, n_kv, head_dim, page_size, n_pages))
        return report_error(TF_E_UNSUPPORTED_SHAPE,
                            "%s: need head_dim 64, 128 or 256, page_size 16, 32, 64 or 128, 1 <= n_kv <= 256 and fewer "
                            "than 2^31 slots and rows",
                            name);
    if (!book_ok(n_seqs, max_pages, page_size))
        return report_error(TF_E_UNSUPPORTED_SHAPE, "%s: need 1 <= n_seqs <= %d and 1 <= max_pages * page_size < 2^31",
                            name, kMaxSeqs);
    if (data == nullptr || book == nullptr || !is_aligned(data, 16) || !is_aligned(book, 4))
        return report_error(TF_E_INVALID_ARG, "%s: data (16-byte) or book (4-byte) NULL or misaligned", name);
    if (data_bytes < tf_kvcache_data_bytes(n_layers, n_kv, head_dim, page_size, n_pages) ||
        book_elems < tf_kvcache_book_elems(n_pages, n_seqs, max_pages))
        return report_error(TF_E_WORKSPACE_TOO_SMALL, "%s: data or book too small for the shape", name);
    desc->magic = TF_KVCACHE_MAGIC;
    desc->n_layers = n_layers;
    desc->n_kv = n_kv;
    desc->head_dim = head_dim;
    desc->page_size = page_size;
    desc->n_seqs = n_seqs;
    desc->n_pages = (int32_t)n_pages;
    desc->max_pages = (int32_t)max_pages;
    desc->data = data;
    desc->book = book;
    return TF_OK;
}

int tf_kvcache_reset(const tf_kvcache* c, void* stream)
{
    CacheView v;
    if (int rc = check_cache(c, "tf_kvcache_reset", &v))
        return rc;
    const int64_t n = (int64_t)tf_kvcache_book_elems(v.n_pages, v.n_seqs, v.max_pages);
    const unsigned blocks = (unsigned)(n < 256 * 1024 ? (n + 255) / 256 : 1024);
    reset_kernel<<<blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(v, n);
    return launched(cudaGetLastError(), "tf_kvcache_reset");
}

size_t tf_kvcache_workspace_bytes(const tf_kvcache* c)
{
    CacheView v;
    return check_cache(c, "tf_kvcache_workspace_bytes", &v) ? 0 : plan_bytes(v.n_seqs);
}

int tf_kvcache_extend(const tf_kvcache* c, const int32_t* seqs, const int32_t* q_start, int64_t B, int64_t M,
                      const uint64_t* masks, int32_t* slots, int32_t* positions, void* ws, size_t ws_bytes,
                      void* stream)
{
    const char* name = "tf_kvcache_extend";
    CacheView v;
    int rc = check_cache(c, name, &v);
    if (rc || (rc = check_batch(v, seqs, q_start, B, M, name)) || (rc = check_ws(ws, ws_bytes, plan_bytes(v.n_seqs), name)))
        return rc;
    if (slots == nullptr)
        return report_error(TF_E_INVALID_ARG, "%s: slots is NULL", name);
    const MemRange ranges[] = {{slots, (size_t)M * 4}, {positions, (size_t)M * 4}, {seqs, (size_t)B * 4},
                            {q_start, (size_t)(B + 1) * 4}, {masks, (size_t)M * 8}};
    if (outputs_overlap(ranges, 2, 5) || in_cache(v, ranges[0]) || in_cache(v, ranges[1]))
        return report_error(TF_E_INVALID_ARG, "%s: slots or positions overlaps another argument", name);
    extend_kernel<<<1, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(v, seqs, q_start, (int)B, M, masks, slots,
                                                                             positions, static_cast<int*>(ws));
    return launched(cudaGetLastError(), name);
}

int tf_kvcache_fork(const tf_kvcache* c, const int32_t* parent, void* ws, size_t ws_bytes, void* stream)
{
    const char* name = "tf_kvcache_fork";
    CacheView v;
    int rc = check_cache(c, name, &v);
    if (rc || (rc = check_ws(ws, ws_bytes, plan_bytes(v.n_seqs), name)))
        return rc;
    if (parent == nullptr)
        return report_error(TF_E_INVALID_ARG, "%s: parent is NULL", name);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    fork_plan_kernel<<<1, kPlanThreads, 0, s>>>(v, parent, ws);
    if ((rc = launched(cudaGetLastError(), name)))
        return rc;
    const size_t smem = (size_t)v.n_seqs * kForkCols * sizeof(int32_t);
    if (smem > 48 * 1024) {
        static std::atomic<uint64_t> done{0};
        const cudaError_t e = allow_smem(fork_apply_kernel, kMaxSeqs * kForkCols * (int)sizeof(int32_t), done);
        if (e != cudaSuccess)
            return launched(e, name);
    }
    const int sms = device_sms();  // 16 blocks an SM for the copies: 18.9 us where 8 take 19.6 and 64 take 20.3
    const int col_blocks = v.max_pages <= kForkCols * sms ? (v.max_pages + kForkCols - 1) / kForkCols : sms;
    return launched(launch_pdl(fork_apply_kernel, dim3(col_blocks + 16 * sms), dim3(kCopyThreads), smem, s, true, v,
                               col_blocks, ws),
                    name);
}

int tf_kvcache_keep(const tf_kvcache* c, const int32_t* seqs, const int32_t* q_start, const int32_t* keep,
                    const int32_t* n_keep, int64_t B, int64_t M, void* ws, size_t ws_bytes, void* stream)
{
    const char* name = "tf_kvcache_keep";
    CacheView v;
    int rc = check_cache(c, name, &v);
    if (rc || (rc = check_batch(v, seqs, q_start, B, M, name)) || (rc = check_ws(ws, ws_bytes, plan_bytes(v.n_seqs), name)))
        return rc;
    if (keep == nullptr || n_keep == nullptr)
        return report_error(TF_E_INVALID_ARG, "%s: keep or n_keep is NULL", name);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    keep_plan_kernel<<<1, kPlanThreads, 0, s>>>(v, seqs, q_start, keep, n_keep, (int)B, M, ws);
    if ((rc = launched(cudaGetLastError(), name)))
        return rc;
    const int64_t cols = (int64_t)v.n_layers * 2 * v.n_kv * (v.head_dim / 8), per = kCopyThreads;
    return launched(launch_pdl(keep_move_kernel, dim3((unsigned)((cols + per - 1) / per), (unsigned)B), dim3(kCopyThreads), 0, s,
                               true, v, q_start, keep, M, ws),
                    name);
}

}  // extern "C"
