// What the attention kernels share: their parameters, the split of a call's work over the
// CTAs, and the joining of partial results.
//
// A call is a list of items, one for each (sequence, key/value head, tile of query rows), and
// an item's keys come in tiles of kKeyTile. The CTAs of a persistent grid take equal shares of
// all (item, key tile) units in that order, so the load is even whatever the lengths are, and
// few rows over a long context still use the whole GPU. A CTA that holds all of an item writes
// its output; otherwise each writes its part (running maximum, sum and unscaled output) to
// the workspace and the last to arrive joins them in key order, so the result does not depend
// on who that is. The lengths are read on the device: a captured call follows them.
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
    CacheView c;
    int layer;
    int total_rows;  // rows of the pool: a row coordinate that the tensor map fills with zeros
    const int32_t *seqs, *q_start;
    int B, max_rows;
    const uint64_t* masks;
    float scale_log2;  // scale * log2(e)
    uint16_t* o;
    int* status;
    unsigned* counters;  // [CTAs], zero between calls
    float* parts;        // [2 * CTAs][part_floats]
    uint64_t limit_ns;
};

// Sequence b of the call: its rows and tokens, or why it has none.
struct SeqRows {
    int slot, r0, rows, base;  // rows r0 .. r0 + rows of q; tokens base .. base + rows of the slot
    __device__ __forceinline__ int len() const { return base + rows; }
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

// Shared memory of a call's schedule: the units before each sequence.
constexpr size_t schedule_bytes(int B) { return (size_t)(B + 1) * 8; }

struct Segment {
    int b, h, rt;    // item: sequence, key/value head, row tile
    int t0, t1, nt;  // key tiles t0 .. t1 of nt
    int64_t u;       // the first unit
};

template <int ROWS, int KEYS>
struct Shares {
    int64_t* first;  // [B + 1], shared memory: units before each sequence
    const AttnParams& p;
    int64_t total, ctas;  // units; CTAs that have some: every one of them has at least one

    __device__ Shares(const AttnParams& params, void* smem) : first(static_cast<int64_t*>(smem)), p(params), total(0), ctas(0) {}

    // Read anew from the cache that build() has filled: shared memory is the ring's.
    __device__ __forceinline__ SeqRows seq(int b) const { return seq_rows(p, b); }

    __device__ __forceinline__ int row_tiles(const SeqRows& q) const { return (q.rows * p.group + ROWS - 1) / ROWS; }
    __device__ __forceinline__ int key_tiles(const SeqRows& q) const { return (q.len() + KEYS - 1) / KEYS; }

    // All threads of the CTA (a multiple of 32); ends with a barrier.
    __device__ void build()
    {
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const SeqRows q = seq(b);
            first[b + 1] = q.base < 0 ? 0 : (int64_t)p.c.n_kv * row_tiles(q) * key_tiles(q);
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            int64_t sum = 0;
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                const int b = b0 + threadIdx.x;
                int64_t x = b < p.B ? first[b + 1] : 0;
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                    if ((int)threadIdx.x >= o)
                        x += y;
                }
                if (b < p.B)
                    first[b + 1] = sum + x;
                sum += __shfl_sync(0xffffffffu, x, 31);
            }
            if (threadIdx.x == 0)
                first[0] = 0;
        }
        __syncthreads();
        total = first[p.B];
        ctas = total < gridDim.x ? total : gridDim.x;
        // sequences whose arguments do not hold: zero rows
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            const SeqRows q = seq(b);
            if (q.base >= 0)
                continue;
            if (threadIdx.x == 0)
                record_status(p.status, TF_E_INVALID_ARG);
            const int64_t n = (int64_t)q.rows * p.n_q * p.c.head_dim / 8;
            uint4* o = reinterpret_cast<uint4*>(p.o + (int64_t)q.r0 * p.n_q * p.c.head_dim);
            for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
                o[i] = make_uint4(0, 0, 0, 0);
        }
    }

    __device__ __forceinline__ int64_t start_of(int64_t cta) const { return cta >= ctas ? total : total * cta / ctas; }
    // the CTA that takes unit u
    __device__ __forceinline__ int cta_of(int64_t u) const { return (int)(((u + 1) * ctas - 1) / total); }

    __device__ __forceinline__ Segment segment(int64_t u, int64_t end) const
    {
        int lo = 0, hi = p.B - 1;  // the last sequence whose first unit is not behind u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        Segment g;
        g.b = lo;
        g.u = u;
        const SeqRows q = seq(lo);
        g.nt = key_tiles(q);
        const int rt = row_tiles(q);
        const int64_t local = u - first[lo];
        const int64_t item = local / g.nt;
        g.t0 = (int)(local - item * g.nt);
        g.h = (int)(item / rt);
        g.rt = (int)(item - (int64_t)g.h * rt);
        const int64_t left = end - u;
        g.t1 = left < g.nt - g.t0 ? g.t0 + (int)left : g.nt;
        return g;
    }
};

// The scaled score of a row and a key in the softmax's running form.
__device__ __forceinline__ float attn_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// The joined output of one row's four columns over parts c0 .. c1 of an item (part c0 is the
// slot 2 c0 + 1, which starts the item; the others continue it in slot 2 c).
template <int ROWS, int HD>
__device__ __forceinline__ float4 join_parts(const float* parts, int c0, int c1, int row, int col)
{
    constexpr int kFloats = ROWS * (HD + 2);
    auto at = [&](int c) { return parts + (int64_t)(c == c0 ? 2 * c0 + 1 : 2 * c) * kFloats; };
    // eight parts at a time, in order: their loads together, then the running softmax over them
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; c += 8) {
        float2 ml[8];
        float4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i <= c1) {
                ml[i] = __ldcg(reinterpret_cast<const float2*>(at(c + i) + ROWS * HD + 2 * row));
                v[i] = __ldcg(reinterpret_cast<const float4*>(at(c + i) + row * HD + col));
            }
        float top = m;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i <= c1)
                top = fmaxf(top, ml[i].x);
        const float ref = top == -INFINITY ? 0.f : top, f = attn_ex2(m - ref);
        m = top;
        l *= f;
        a.x *= f, a.y *= f, a.z *= f, a.w *= f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i <= c1) {
                const float w = attn_ex2(ml[i].x - ref);
                l = fmaf(w, ml[i].y, l);
                a.x = fmaf(w, v[i].x, a.x), a.y = fmaf(w, v[i].y, a.y), a.z = fmaf(w, v[i].z, a.z), a.w = fmaf(w, v[i].w, a.w);
            }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    return make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
}

__device__ __forceinline__ uint2 bf16x4(float4 a) { return make_uint2(f32x2_to_bf16x2(a.x, a.y), f32x2_to_bf16x2(a.z, a.w)); }

// rows: query rows of an item. tfq_attn_warp.cu: 16, and up to head_dim 128 also 32;
// tfq_attn_tc.cu: 128 or 256, head_dim 64 or 128. *_box: cache rows of a tensor-map box.
cudaError_t launch_attn_warp(const AttnParams& p, int rows, const CUtensorMap& map, cudaStream_t stream, bool pdl);
cudaError_t launch_attn_tc(const AttnParams& p, int rows, const CUtensorMap& map, cudaStream_t stream, bool pdl);
int attn_warp_box(int head_dim, int page_size);
int attn_tc_box(int rows, int page_size);

}  // namespace tfq
