// What the attention kernels share: their parameters, the split of a call's work over the
// CTAs, and the joining of partial results.
//
// A call is a list of items, one for each (sequence, key/value head, tile of query rows), and
// an item's keys come in tiles of kKeyTile. The CTAs of a persistent grid take equal shares of
// all (item, key tile) units in that order, so the load is even whatever the lengths are, and
// few rows over a long context still use the whole GPU. A CTA that holds all of an item writes
// its output; otherwise each writes its part (running maximum, sum and unscaled output) to the
// workspace, and once all of an item's parts are there each of its CTAs joins a slice of the
// output, parts in key order: 8 rows over 32,771 tokens, some 19 parts to an item, take 32 us so and
// 35.6 when the last CTA to arrive joins them all. CTAs wait for one another at their very end only, when all their parts are
// written; the launch is cooperative, so all of them run. The lengths are read on the device: a
// captured call follows them.
#pragma once

#include <cuda.h>

#include "tfq_cache.h"
#include "tfq_ptx.cuh"

namespace tfq {

constexpr int kMaxAttnSeqs = 1024;

struct AttnParams {
    const uint16_t* q;
    int64_t ldq, M;
    int n_q, group;  // query heads; query heads of a key/value head
    unsigned group_inv;  // 2^31 / group, rounded up
    CacheView c;
    int layer;
    int total_rows;  // rows of the pool: a row coordinate that the tensor map fills with zeros
    const int32_t *seqs, *q_start;
    int B, max_rows;
    int over;  // a segment's own cost, in key tiles
    bool few;  // no more items than SMs, where one CTA or two run on each, and no more sequences than threads
    const uint64_t* masks;
    float scale_log2;  // scale * log2(e)
    uint16_t* o;
    bool q_boxes;  // prompts: an item's queries are a tensor map's box
    int* status;
    unsigned* counters;  // [CTAs][2], zero between calls: parts written, CTAs done with them
    float* parts;        // [2 * CTAs] of a part: [head_dim / 4][ROWS] float4, then [ROWS] (m, l)
    uint64_t limit_ns;

    // Query row r of a key/value head is head r % group of its sequence's row r / group. The quotient
    // is exact for r < 2^25 and group <= 64: it is over by less than r * 63 / 2^31 / group < 1 / group.
    __device__ __forceinline__ int token_of(int r) const { return (int)__umulhi((unsigned)r << 1, group_inv); }
    __device__ __forceinline__ int head_of(int r) const { return r - token_of(r) * group; }
};

// Sequence b of the call: its rows and tokens, or why it has none.
struct SeqRows {
    int slot, r0, rows, base;  // rows r0 .. r0 + rows of q; tokens base .. base + rows of the slot
    __host__ __device__ __forceinline__ int len() const { return base + rows; }
};

// base < 0: the sequence's arguments do not hold. rows is 0 where the rows themselves do not.
__device__ __forceinline__ SeqRows seq_rows(const AttnParams& p, int b)
{
    SeqRows s;
    s.slot = p.seqs[b];
    s.r0 = p.q_start[b];
    const int r1 = p.q_start[b + 1];
    const bool rows_ok = s.r0 >= 0 && s.r0 <= r1 && r1 <= p.M;
    s.rows = rows_ok ? r1 - s.r0 : 0;
    s.base = -1;
    if (rows_ok && s.rows <= p.max_rows && s.slot >= 0 && s.slot < p.c.n_seqs) {
        const int len = p.c.len[s.slot];
        if (len >= s.rows && len <= (int64_t)p.c.max_pages << p.c.page_shift)
            s.base = len - s.rows;
    }
    return s;
}

// A sequence of the call's schedule, in shared memory.
struct SeqEntry {
    int first;      // units before it
    int r0, base;   // as in SeqRows
    int slot_rows;  // slot | rows << 16
};
constexpr size_t schedule_bytes(int B) { return (size_t)(B + 8) * sizeof(SeqEntry); }  // the last 7: build() uses them

struct Segment {
    SeqRows q;       // item: sequence, key/value head, row tile
    int h, rt;
    int t0, t1, nt;  // key tiles t0 .. t1 of nt; none of them: t0 == t1
    int units;       // units it takes
    int first;       // the item's first key tile, in units
};

// An item counts p.over units before its key tiles: what a segment costs apart from them (its
// queries, joining the warps' parts, the hand-over), so that CTAs with many short items get no more
// than their share. A CTA has kLeast units or more, so that a short item is not torn apart.
//
// Joining an item's parts costs what kJoin key tiles do (0: not looked at), and more the more CTAs have parts
// of two. If there are no more items than CTAs, and the longest has no more tiles than an even share and
// that, each has a CTA: their units are then one number, whatever the lengths, so that shares and items
// coincide. A sequence of kMostTiles or more is always split: counts stop there, so that they fit 32 bits.
template <int ROWS, int KEYS, int kLeast, int kJoin>
struct Shares {
    SeqEntry* seq;  // [B + 1]
    const AttnParams& p;
    unsigned total, ctas;  // units; CTAs that have some: every one of them has at least one
    unsigned share, rest;  // total = ctas * share + rest
    int whole;             // units of an item when each has a CTA, else 0
    // Tiles that an item more costs a split call, over all CTAs (6: two an SM). Two an SM with 24, and with another number: 8
    // sequences' single rows over 768 tokens, 8 heads, 14.0 us and (64) 17.6, 16 over 1536 24.9 and 27.7; 8 of 8 rows over 544
    // 14.05 and (8, 0) 14.4, single rows there 13.5 and 13.4
    static constexpr int kTorn = kLeast == 6 ? 24 : 64;
    static constexpr int kMostTiles = 1 << 20;

    __host__ __device__ Shares(const AttnParams& params, void* smem)
        : seq(static_cast<SeqEntry*>(smem)), p(params), total(0), ctas(0), share(0), rest(0), whole(0)
    {
    }

    __host__ __device__ __forceinline__ int row_tiles(int rows) const { return (rows * p.group + ROWS - 1) / ROWS; }
    __host__ __device__ __forceinline__ int key_tiles(int len) const { return (int)(((int64_t)len + KEYS - 1) / KEYS); }

    __host__ __device__ __forceinline__ int units_of(int nt) const { return whole ? whole : nt + p.over; }

    __host__ __device__ __forceinline__ int items_of(const SeqRows& q) const { return p.c.n_kv * row_tiles(q.rows); }
    __host__ __device__ __forceinline__ int all_units(const SeqRows& q) const
    {
        const int64_t n = (int64_t)items_of(q) * units_of(key_tiles(q.len()));
        return n < INT32_MAX ? (int)n : INT32_MAX;
    }

    // What a sequence adds to the choice of `whole`: its tiles, and over its items their sum and kTorn each
    // (at most one item a CTA in all, so 32 bits).
    __host__ __device__ __forceinline__ int2 counted(const SeqRows& q) const
    {
        const int nt = key_tiles(q.len()), tiles = nt < kMostTiles ? nt : kMostTiles;
        return q.base < 0 || q.rows == 0 ? make_int2(0, 0) : make_int2(tiles, (tiles + kTorn) * items_of(q));
    }
    __host__ __device__ __forceinline__ int whole_of(int most, int sum, unsigned grid) const
    {
        return most < kMostTiles && (int64_t)(most - kJoin) * grid <= sum ? most + 1 : 0;
    }

    // The CTAs' shares of `total` units.
    __host__ __device__ __forceinline__ void deal(unsigned grid)
    {
        const unsigned least = (total + kLeast - 1) / kLeast;
        ctas = whole ? total / whole : least < grid ? least : grid;
        if (ctas > 0) {
            share = total / ctas;
            rest = total - share * ctas;
        }
    }

    template <class Enter>
    __device__ __forceinline__ void sum_up(const SeqRows& first, Enter& enter)
    {
        if (kJoin > 0 && p.few) {  // a sequence a thread
            const int2 mine = counted(first);
            int2* found = reinterpret_cast<int2*>(seq + p.B + 1);  // of each warp
            const int most = __reduce_max_sync(0xffffffffu, mine.x), sum = __reduce_add_sync(0xffffffffu, mine.y);
            if (threadIdx.x % 32 == 0 && (int)threadIdx.x < p.B)  // 8 warps at most: the call looks at 256 sequences or fewer
                found[threadIdx.x / 32] = make_int2(most, sum);
            __syncthreads();
            int2 all = make_int2(0, 0);
            for (int w = 0; w * 32 < p.B; ++w) {
                all.x = max(all.x, found[w].x);
                all.y += found[w].y;
            }
            whole = whole_of(all.x, all.y, gridDim.x);
        }
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const SeqRows q = b < (int)blockDim.x ? first : seq_rows(p, b);
            enter(b, q, q.base >= 0 ? all_units(q) : 0);
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            unsigned sum = 0;  // sums stop at INT32_MAX, as do their terms
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int b = b0 + threadIdx.x;
                unsigned x = b < p.B ? seq[b].first : 0;
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
                    if ((int)threadIdx.x >= o)
                        x = min(x + y, (unsigned)INT32_MAX);
                }
                const unsigned before = __shfl_up_sync(0xffffffffu, x, 1);
                if (b < p.B)
                    seq[b].first = (int)min(threadIdx.x > 0 ? sum + before : sum, (unsigned)INT32_MAX);
                sum = min(sum + __shfl_sync(0xffffffffu, x, 31), (unsigned)INT32_MAX);
            }
            if (threadIdx.x == 0)
                seq[p.B].first = (int)sum;
        }
        __syncthreads();
        total = seq[p.B].first;
    }

    // All threads of the CTA (a multiple of 32); has barriers.
    __device__ void build()
    {
        auto enter = [&](int b, const SeqRows& q, int units) {
            SeqEntry e{0, q.r0, q.base, 0};
            if (q.base >= 0) {
                e.slot_rows = q.slot | q.rows << 16;
                e.first = units;
            } else {
                // arguments that do not hold: zero rows, a share of them a CTA (20,000 of 16 heads of 128 beside a
                // good sequence: 168 us from the host's view; by one thread, 15,251)
                if (blockIdx.x == 0)
                    record_status(p.status, TF_E_INVALID_ARG);
                const int64_t n = (int64_t)q.rows * p.n_q * p.c.head_dim / 8;
                uint4* o = reinterpret_cast<uint4*>(p.o + (int64_t)q.r0 * p.n_q * p.c.head_dim);
                const uint4* end = o + n * (blockIdx.x + 1) / gridDim.x;
                for (o += n * blockIdx.x / gridDim.x; o < end; ++o)
                    *o = make_uint4(0, 0, 0, 0);
            }
            seq[b] = e;
        };
        SeqRows first{0, 0, 0, -1};
        if ((int)threadIdx.x < p.B || p.B == 1)
            first = seq_rows(p, p.B == 1 ? 0 : threadIdx.x);
        if (p.B == 1) {  // nothing to be summed up: every thread has the answer
            if (first.base >= 0) {
                const int2 mine = counted(first);
                if (kJoin > 0 && p.few && mine.y > 0)
                    whole = whole_of(mine.x, mine.y, gridDim.x);
                total = all_units(first);
            }
            if (threadIdx.x == 0)
                enter(0, first, 0);
            __syncthreads();
        } else {
            sum_up(first, enter);
        }
        if (total == INT32_MAX) {  // more than the units' 31 bits: nothing is done
            if (blockIdx.x == 0 && threadIdx.x == 0)
                record_status(p.status, TF_E_UNSUPPORTED_SHAPE);
            total = 0;
        }
        deal(gridDim.x);
    }

    // total * cta / ctas, in 32 bits
    __host__ __device__ __forceinline__ int start_of(unsigned cta) const { return (int)(cta >= ctas ? total : share * cta + rest * cta / ctas); }
    // the CTA that takes unit u
    __host__ __device__ __forceinline__ int cta_of(int u) const { return (int)((((uint64_t)u + 1) * ctas - 1) / total); }

    __host__ __device__ __forceinline__ Segment segment(int u, int end) const
    {
        int lo = 0, hi = p.B - 1;  // the last sequence whose first unit is not behind u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq[mid].first <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const SeqEntry e = seq[lo];
        Segment g;
        g.q = SeqRows{e.slot_rows & 0xFFFF, e.r0, e.slot_rows >> 16, e.base};
        g.nt = key_tiles(g.q.len());
        const int rt = row_tiles(g.q.rows), per = units_of(g.nt), over = per - g.nt;
        const int local = u - e.first, item = local / per, off = local - item * per;
        g.h = item / rt;
        g.rt = item - g.h * rt;
        g.units = min(end - u, per - off);
        g.t0 = max(off - over, 0);
        g.t1 = max(off + g.units - over, 0);
        g.first = u - off + over;
        return g;
    }
};

// The same for causal rows without a limit to their number, where a row tile sees the tokens up to its last row's: its
// key tiles grow with the rows before it. The units before row tile rt of a head are
//   P(rt) = rt * (over + 1) + floor((rt * base + A * rt * (rt + 1) / 2) / KEYS),   A = ROWS / group, rounded up, tokens,
// in closed form, so an item is found without a list of them. Its own P(rt + 1) - P(rt) is over - 1 at least above its
// key tiles ceil((base + last row's token + 1) / KEYS), since A (rt + 1) >= that token + 1; over >= 2.
template <int ROWS, int KEYS, int PER = 1>  // PER: shares a CTA
struct PromptShares {
    struct Entry {
        int first, r0, base, rows;
    };
    Entry* seq;  // [B + 1], base < 0: none
    const AttnParams& p;
    unsigned total, ctas, share, rest;
    static_assert(sizeof(Entry) == sizeof(SeqEntry), "schedule_bytes");

    __host__ __device__ PromptShares(const AttnParams& params, void* smem)
        : seq(static_cast<Entry*>(smem)), p(params), total(0), ctas(0), share(0), rest(0)
    {
    }

    __host__ __device__ __forceinline__ int row_tiles(int rows) const { return (rows * p.group + ROWS - 1) / ROWS; }
    __host__ __device__ __forceinline__ int64_t before(int base, int rt) const
    {
        const int64_t a = (ROWS + p.group - 1) / p.group;
        return (int64_t)rt * (p.over + 1) + ((int64_t)rt * base + a * rt * (rt + 1) / 2) / KEYS;
    }
    // tokens that row tile rt's last row, the last of them, sees
    __host__ __device__ __forceinline__ int seen_by(int base, int rows, int rt) const
    {
        const int last = ((rt + 1) * ROWS + p.group - 1) / p.group;
        return base + (last < rows ? last : rows);
    }
    __host__ __device__ __forceinline__ int all_units(int base, int rows) const
    {
        const int64_t n = p.c.n_kv * before(base, row_tiles(rows));  // below 2^8 * 2^43
        return n < INT32_MAX ? (int)n : INT32_MAX;
    }
    __host__ __device__ __forceinline__ void deal(unsigned grid)
    {
        ctas = total < grid ? total : grid;
        if (ctas > 0) {
            share = total / ctas;
            rest = total - share * ctas;
        }
    }

    // All threads of the CTA (a multiple of 32); has barriers.
    __device__ void build()
    {
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const SeqRows q = seq_rows(p, b);
            seq[b] = Entry{q.base >= 0 ? all_units(q.base, q.rows) : 0, q.r0, q.base, q.rows};
            if (q.base < 0 && blockIdx.x == 0)
                record_status(p.status, TF_E_INVALID_ARG);
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            unsigned sum = 0;  // sums stop at INT32_MAX, as do their terms
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int b = b0 + threadIdx.x;
                const unsigned own = b < p.B ? seq[b].first : 0;
                unsigned x = own;
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
                    if ((int)threadIdx.x >= o)
                        x = min(x + y, (unsigned)INT32_MAX);
                }
                const unsigned upto = __shfl_up_sync(0xffffffffu, x, 1);
                if (b < p.B)
                    seq[b].first = (int)min(threadIdx.x > 0 ? sum + upto : sum, (unsigned)INT32_MAX);
                sum = min(sum + __shfl_sync(0xffffffffu, x, 31), (unsigned)INT32_MAX);
            }
            if (threadIdx.x == 0)
                seq[p.B].first = (int)sum;
        }
        __syncthreads();
        total = seq[p.B].first;
        // rows of a sequence whose arguments do not hold become zeros, a share of them a CTA
        for (int b = 0; b < p.B; ++b) {
            if (seq[b].base >= 0)
                continue;
            const int64_t row = (int64_t)p.n_q * p.c.head_dim / 8, n = seq[b].rows * row;
            uint4* o = reinterpret_cast<uint4*>(p.o) + seq[b].r0 * row;
            for (int64_t i = n * blockIdx.x / gridDim.x + threadIdx.x; i < n * (blockIdx.x + 1) / gridDim.x; i += blockDim.x)
                o[i] = make_uint4(0, 0, 0, 0);
        }
        if (total == INT32_MAX) {  // more than the units' 31 bits: nothing is done
            if (blockIdx.x == 0 && threadIdx.x == 0)
                record_status(p.status, TF_E_UNSUPPORTED_SHAPE);
            total = 0;
        }
        deal(gridDim.x * PER);
    }

    __host__ __device__ __forceinline__ int start_of(unsigned cta) const { return (int)(cta >= ctas ? total : share * cta + rest * cta / ctas); }
    __host__ __device__ __forceinline__ int cta_of(int u) const { return (int)((((uint64_t)u + 1) * ctas - 1) / total); }

    __host__ __device__ __forceinline__ Segment segment(int u, int end) const
    {
        int lo = 0, hi = p.B - 1;  // the last sequence whose first unit is not behind u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq[mid].first <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const Entry e = seq[lo];
        const int tiles = row_tiles(e.rows), head = (int)before(e.base, tiles), local = u - e.first;
        Segment g;
        g.h = local / head;
        const int off = local - g.h * head;
        // the last rt with P(rt) <= off: the root of the parabola, then the step or so that it is off
        const float b = (ROWS + p.group - 1) / p.group * (0.5f / KEYS), a = p.over + 1 + (float)e.base / KEYS + b;
        int rt = (int)((sqrtf(a * a + 4.f * b * off) - a) / (2.f * b));
        rt = rt < 0 ? 0 : rt > tiles - 1 ? tiles - 1 : rt;
        while (rt > 0 && before(e.base, rt) > off)
            --rt;
        while (rt < tiles - 1 && before(e.base, rt + 1) <= off)
            ++rt;
        const int at = (int)before(e.base, rt), per = (int)before(e.base, rt + 1) - at;
        g.rt = rt;
        g.q = SeqRows{0, e.r0, e.rows, e.base};
#ifdef __CUDA_ARCH__
        g.q.slot = p.seqs[lo];
#endif
        g.nt = (seen_by(e.base, e.rows, rt) + KEYS - 1) / KEYS;
        const int over = per - g.nt;
        g.units = end - u < per - (off - at) ? end - u : per - (off - at);
        g.t0 = off - at - over > 0 ? off - at - over : 0;
        g.t1 = off - at + g.units - over > 0 ? off - at + g.units - over : 0;
        g.first = u - (off - at) + over;
        return g;
    }
};

// A row's mask of the block of `rows` tokens, bits behind them taken out.
__device__ __forceinline__ uint64_t block_mask(const AttnParams& p, const SeqRows& q, int t)
{
    return p.masks == nullptr ? ~0ull >> (63 - t) : p.masks[q.r0 + t] & (~0ull >> (64 - q.rows));
}

// What a row sees of a tile that begins at token d of its block (d > -64: before it), from bit 0.
__device__ __forceinline__ uint64_t tile_mask(uint64_t mask, int d)
{
    return d >= 0 ? (d < 64 ? mask >> d : 0ull) : mask << -d | ((1ull << -d) - 1);
}

// 2^x: scores are scaled by log2(e), so that a weight is one instruction
__device__ __forceinline__ float attn_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Launch with all CTAs running at once (they wait for one another).
template <class... KArgs, class... Args>
cudaError_t launch_coop(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Bounded wait that also ends when another thread of the CTA has given up.
__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          uint64_t limit_ns)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const long long start = clock64(), limit = (long long)(limit_ns * 2);  // 2 cycles per ns
    while (true) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (*abort_flag)
            return false;
        if (clock64() - start > limit) {
            *abort_flag = 1;
            record_status(status, TF_E_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ uint2 bf16x4(float4 a) { return make_uint2(f32x2_to_bf16x2(a.x, a.y), f32x2_to_bf16x2(a.z, a.w)); }

// An item that several CTAs have parts of: c0 .. c1 (part c0 is the slot 2 c0 + 1, which starts the
// item; the others continue it in slot 2 c).
struct SplitItem {
    SeqRows q;
    int h, row0, rows;  // head; first row and rows of the item
    int c0, c1;         // c0 > c1: none
};

// All the CTA's output threads have written its part; one thread of them says so.
__device__ __forceinline__ void part_written(const AttnParams& p, const SplitItem& s)
{
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p.counters + 2 * s.c0), "r"(1u) : "memory");
}

__device__ __forceinline__ const float* part_of(const AttnParams& p, const SplitItem& s, int c, int floats)
{
    return p.parts + (int64_t)(c == s.c0 ? 2 * c + 1 : 2 * c) * floats;
}

// A slice of more items (four columns of a row) than there are threads: i0 .. i1 of few parts. A thread's items
// are all of one row, so it forms the parts' weights once, and what it will add comes by asynchronous
// copies of its own into `buf`, all under way at once: loaded into registers item by item, 2 or 3 parts of
// 256 rows took a CTA 8 us. buf: ROWS * HD * 4 bytes + 1024 for each part and thread, at most.
template <int ROWS, int HD, int THREADS>
__device__ __forceinline__ void join_many(const AttnParams& p, const SplitItem& s, int i0, int i1, uint8_t* buf, int tid)
{
    static_assert(THREADS % ROWS == 0, "a thread keeps its row");
    constexpr int kFloats = ROWS * (HD + 2);
    const int n = s.c1 - s.c0 + 1, items = i1 - i0, first = i0 + tid, row = first % ROWS;
    if (row >= s.rows)
        return;
    float4* data = reinterpret_cast<float4*>(buf) + tid;                       // [n][items]
    float* weight = reinterpret_cast<float*>(buf + (size_t)n * items * 16) + tid;  // [n][THREADS]
    for (int c = 0; c < n; ++c) {
        const float* part = part_of(p, s, s.c0 + c, kFloats);
        for (int i = tid; i < items; i += THREADS)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(data + c * items + i - tid)),
                         "l"(part + (size_t)(i0 + i) * 4)
                         : "memory");
    }
    float top = -INFINITY, l = 0.f;
    for (int c0 = 0; c0 < n; c0 += 4) {
        float2 ml[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c0 + i < n)
                ml[i] = __ldcg(reinterpret_cast<const float2*>(part_of(p, s, s.c0 + c0 + i, kFloats) + ROWS * HD + 2 * row));
        const float was = top;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c0 + i < n)
                top = fmaxf(top, ml[i].x);
        const float ref = top == -INFINITY ? 0.f : top;
        l *= attn_ex2(was - ref);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c0 + i < n) {
                l = fmaf(attn_ex2(ml[i].x - ref), ml[i].y, l);
                weight[(c0 + i) * THREADS] = ml[i].x;
            }
    }
    const float ref = top == -INFINITY ? 0.f : top, inv = l == 0.f ? 0.f : 1.f / l;
    for (int c = 0; c < n; ++c)
        weight[c * THREADS] = attn_ex2(weight[c * THREADS] - ref);
    asm volatile("cp.async.wait_all;" ::: "memory");
    const int r = s.row0 + row;
    uint16_t* o = p.o + ((int64_t)(s.q.r0 + p.token_of(r)) * p.n_q + s.h * p.group + p.head_of(r)) * HD;
    for (int i = 0; i + tid < items; i += THREADS) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < n; ++c) {
            const float w = weight[c * THREADS];
            const float4 v = data[c * items + i];
            a.x = fmaf(w, v.x, a.x), a.y = fmaf(w, v.y, a.y), a.z = fmaf(w, v.z, a.z), a.w = fmaf(w, v.w, a.w);
        }
        *reinterpret_cast<uint2*>(o + (first + i) / ROWS * 4) = bf16x4(make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
    }
}

// Waits for the item's parts and writes this CTA's (or group's) slice of its output. THREADS threads, which
// share named barrier `bar`; several lanes share four columns of a row and take every lp-th part, so
// that all parts are asked for at once. The order in which they are added depends on the call alone.
// buf: shared memory that nobody uses any more, as join_many wants it (ROWS >= 128).
template <int ROWS, int HD, int THREADS>
__device__ __forceinline__ void join_slice(const AttnParams& p, const SplitItem& s, volatile int* abort_flag, uint8_t* buf, int tid, int cta, int bar)
{
    constexpr int kFloats = ROWS * (HD + 2), kQuads = HD / 4;
    const int n = s.c1 - s.c0 + 1, me = cta - s.c0;
    if (tid == 0) {
        const long long start = clock64(), limit = (long long)(p.limit_ns * 2);
        unsigned there = 0;
        while (true) {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(there) : "l"(p.counters + 2 * s.c0) : "memory");
            if (there >= (unsigned)n || *abort_flag)
                break;
            if (clock64() - start > limit) {
                *abort_flag = 1;
                record_status(p.status, TF_E_TIMEOUT);
                break;
            }
        }
    }
    named_bar_sync(bar, THREADS);
    // item: four columns of a row, whether the sequence has that row or not: no division by a length here
    constexpr unsigned kItems = ROWS * kQuads;
    const int i0 = (int)(kItems * (unsigned)me / (unsigned)n), i1 = (int)(kItems * (unsigned)(me + 1) / (unsigned)n);
    bool done = false;
    if constexpr (ROWS >= 128) {
        done = i1 - i0 > THREADS;
        if (done)
            join_many<ROWS, HD, THREADS>(p, s, i0, i1, buf, tid);
    }
    int lp = 1;
    while (lp < 8 && (i1 - i0) * lp * 2 <= THREADS && lp < n)
        lp *= 2;
    const int sub = tid % lp;
    for (int at = done ? i1 : i0; at < i1; at += THREADS / lp) {
        const int item = at + tid / lp;
        const int quad = item / ROWS, row = item % ROWS, col = quad * 4;
        const bool in = item < i1 && row < s.rows;
        float m = -INFINITY, l = 0.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = in ? s.c0 + sub : s.c1 + 1; c <= s.c1; c += 4 * lp) {
            float2 ml[4];
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i * lp <= s.c1) {
                    const int cc = c + i * lp;
                    const float* part = part_of(p, s, cc, kFloats);
                    ml[i] = __ldcg(reinterpret_cast<const float2*>(part + ROWS * HD + 2 * row));
                    v[i] = __ldcg(reinterpret_cast<const float4*>(part + (quad * ROWS + row) * 4));
                }
            float top = m;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i * lp <= s.c1)
                    top = fmaxf(top, ml[i].x);
            const float ref = top == -INFINITY ? 0.f : top, f = attn_ex2(m - ref);
            m = top;
            l *= f;
            a.x *= f, a.y *= f, a.z *= f, a.w *= f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i * lp <= s.c1) {
                    const float w = attn_ex2(ml[i].x - ref);
                    l = fmaf(w, ml[i].y, l);
                    a.x = fmaf(w, v[i].x, a.x), a.y = fmaf(w, v[i].y, a.y), a.z = fmaf(w, v[i].z, a.z), a.w = fmaf(w, v[i].w, a.w);
                }
        }
        for (int o = 1; o < lp; o *= 2) {
            const float om = __shfl_xor_sync(0xffffffffu, m, o), top = fmaxf(m, om), ref = top == -INFINITY ? 0.f : top;
            const float f = attn_ex2(m - ref), g = attn_ex2(om - ref);
            l = l * f + __shfl_xor_sync(0xffffffffu, l, o) * g;
            a.x = a.x * f + __shfl_xor_sync(0xffffffffu, a.x, o) * g;
            a.y = a.y * f + __shfl_xor_sync(0xffffffffu, a.y, o) * g;
            a.z = a.z * f + __shfl_xor_sync(0xffffffffu, a.z, o) * g;
            a.w = a.w * f + __shfl_xor_sync(0xffffffffu, a.w, o) * g;
            m = top;
        }
        if (in && sub == 0) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int r = s.row0 + row;
            *reinterpret_cast<uint2*>(p.o + ((int64_t)(s.q.r0 + p.token_of(r)) * p.n_q + s.h * p.group + p.head_of(r)) * HD + col) =
                bf16x4(make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
        }
    }
    // the last CTA to have read the parts leaves the counters as the next call wants them
    named_bar_sync(bar, THREADS);
    if (tid == 0 && !*abort_flag && atom_add_acq_rel_gpu(p.counters + 2 * s.c0 + 1, 1u) == (unsigned)(n - 1)) {
        p.counters[2 * s.c0] = 0;
        p.counters[2 * s.c0 + 1] = 0;
    }
}

// rows: query rows of an item. tfq_attn_warp.cu: 16, and up to head_dim 128 also 32;
// tfq_attn_tc.cu: 128 or 256, head_dim 64 or 128; causal: the rows of prompts. *Tile: keys of a tile.
cudaError_t launch_attn_warp(const AttnParams& p, int rows, const CUtensorMap& map, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnParams& p, int rows, bool causal, const CUtensorMap& map, const CUtensorMap& q_map, cudaStream_t stream);
int attn_warp_tile(const CacheView& c);
int attn_warp_ctas(const CacheView& c, int rows);  // an SM
int attn_warp_threads(const CacheView& c, int rows);
constexpr int kTcTile = 64;

}  // namespace tfq
