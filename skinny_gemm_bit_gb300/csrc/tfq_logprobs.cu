// Log probabilities of given tokens, entropy and top alternatives of rows of logits, in one
// pass over them.
//
// A row's softmax statistics are kept as (m, n, r, w): the largest value m, how many elements
// equal it, and over the others r = sum e^(x - m) and w = sum e^(x - m) (x - m). Then
//   lse = m + log(n + r),  logp = (x - m) - log(n + r),  entropy = log(n + r) - w / (n + r)
// and for n = 1 log(n + r) is log1p(r): the largest element's own 1 never meets the sum of
// the rest, so a sure row's entropy keeps its digits.
//
// Bound by memory for many rows (two or four bytes a logit against about six instructions) and
// by latency for few. A row is cut into 16-byte units; few rows are spread over a thread-block
// cluster each, whose first block joins the parts through distributed shared memory. A warp
// shares one m, so the sums need no test per element: a batch of kBatch units a lane whose
// largest value lies below m (all but a few of them) takes the straight path. The next batch's
// loads are under way while one is summed.
//
// The top k: each thread notes its largest value. The k-th largest of the warps' largest few of
// those (32 in all) is a bound that k elements of the row (or the block's part of it) reach, and
// seldom many more do. Only threads whose largest reaches it can hold one, and nearly always in
// the one batch that their largest came from (they note which, and their second largest batch): those
// batches are read again (from L2), eight a warp at once, and what reaches the bound is collected
// and sorted as (value, lower index first) keys, 32 a warp. That costs a row's latency, not its
// bandwidth: 1000 rows of 151,936 in bf16 take 67.2 us with 20 alternatives (4.5 TB/s), 54 without (5.6). A thread whose second batch
// reaches the bound too has all its units read. Rows with more than kMaxCand such elements (ties
// without end, NaN) take their units through sorted lists instead, one key a lane.
#include <cmath>
#include <type_traits>
#include <cooperative_groups.h>

#include "tfq_cache.h"
#include "tfq_ptx.cuh"

namespace cg = cooperative_groups;

namespace tfq {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxCand = kLpThreads;  // collected keys: 32 a warp
static_assert(kLpThreads == 256, "a thread's index in eight bits");
constexpr int kBatch = 4;        // 16-byte units a lane takes at once
constexpr int kMaxCluster = 8;  // at most kLpWarps: a warp reads a part's list
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LpParams {
    const void* v;
    int64_t ld, M, N;
    const int32_t* targets;
    int n_targets, top_k;
    float *logp, *entropy;
    int32_t* top_idx;
    float* top_logp;
    int* status;
};

struct Stats {
    float m, n, r, w;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Takes the sums of (m, n, r, w) over to a larger reference.
__device__ __forceinline__ void rebase(Stats& s, float m)
{
    if (s.m == m)
        return;
    if (s.m == -INFINITY) {  // nothing yet
        s = Stats{m, 0.f, s.r, s.w};  // r, w are 0, or NaN
        return;
    }
    const float d = s.m - m, all = s.n + s.r, f = expf(d);
    s.w = f == 0.f ? 0.f * s.w : (s.w + d * all) * f;
    s.r = all * f;
    s.n = 0.f;
    s.m = m;
}

__device__ __forceinline__ Stats join(Stats a, Stats b)
{
    const float m = fmaxf(a.m, b.m);
    rebase(a, m);
    rebase(b, m);
    return Stats{m, a.n + b.n, a.r + b.r, a.w + b.w};
}

// A value as an unsigned integer of the same order; -0 as +0, NaN as 0, below every number.
__device__ __forceinline__ uint32_t order_of(float x)
{
    if (x != x)
        return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float of_order(uint32_t u)
{
    return u == 0u ? NAN : __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// (order, lower index first); 0 is no element
__device__ __forceinline__ uint64_t key_of(float x, int64_t n) { return (uint64_t)order_of(x) << 32 | (0xFFFFFFFFu - (uint32_t)n); }

template <class K>
__device__ __forceinline__ K shfl_xor(K v, int o)
{
    return __shfl_xor_sync(0xffffffffu, v, o);
}

// The lanes' keys, largest first (bitonic sort of 32).
template <class K>
__device__ __forceinline__ K sort32(K v, int lane)
{
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int o = size / 2; o > 0; o /= 2) {
            const K u = shfl_xor(v, o);
            const bool up = ((lane & size) != 0) == ((lane & o) == 0);  // keep the smaller
            v = (u < v) == up ? u : v;
        }
    return v;
}

// The 32 largest of two sorted lists, sorted.
template <class K>
__device__ __forceinline__ K merge32(K a, K b, int lane)
{
    const K br = __shfl_sync(0xffffffffu, b, 31 - lane);
    K v = a > br ? a : br;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const K u = shfl_xor(v, o);
        const bool up = (lane & o) != 0;
        v = (u < v) == up ? u : v;
    }
    return v;
}

// Joins the warps' sorted lists in shared memory; the result is in lists[0]. All threads.
template <class K>
__device__ void join_lists(K (*lists)[32], int warp, int lane)
{
    for (int half = kLpWarps / 2; half > 0; half /= 2) {
        __syncthreads();
        if (warp < half)
            lists[warp][lane] = merge32(lists[warp][lane], lists[warp + half][lane], lane);
    }
    __syncthreads();
}

template <class T>
struct Unit;  // 16 bytes of logits

template <>
struct Unit<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void widen(const uint4& u, float (&f)[8])
    {
        f[0] = bf16lo_f32(u.x), f[1] = bf16hi_f32(u.x), f[2] = bf16lo_f32(u.y), f[3] = bf16hi_f32(u.y);
        f[4] = bf16lo_f32(u.z), f[5] = bf16hi_f32(u.z), f[6] = bf16lo_f32(u.w), f[7] = bf16hi_f32(u.w);
    }
    // largest and smallest of the units a, b (pairs at once; NaN is passed over)
    struct Range {
        __nv_bfloat162 hi, lo;
    };
    static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
    static __device__ __forceinline__ Range range(const uint4& u)
    {
        const __nv_bfloat162 a = pair(u.x), b = pair(u.y), c = pair(u.z), d = pair(u.w);
        return {__hmax2(__hmax2(a, b), __hmax2(c, d)), __hmin2(__hmin2(a, b), __hmin2(c, d))};
    }
    static __device__ __forceinline__ Range both(const Range& a, const Range& b) { return {__hmax2(a.hi, b.hi), __hmin2(a.lo, b.lo)}; }
    static __device__ __forceinline__ float top(const Range& r) { return fmaxf(__low2float(r.hi), __high2float(r.hi)); }
    static __device__ __forceinline__ float low(const Range& r) { return fminf(__low2float(r.lo), __high2float(r.lo)); }
    static __device__ __forceinline__ float one(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
};

template <>
struct Unit<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void widen(const uint4& u, float (&f)[4])
    {
        f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
    }
    struct Range {
        float hi, lo;
    };
    static __device__ __forceinline__ Range range(const uint4& u)
    {
        float f[4];
        widen(u, f);
        return {fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), fminf(fminf(f[0], f[1]), fminf(f[2], f[3]))};
    }
    static __device__ __forceinline__ Range both(const Range& a, const Range& b) { return {fmaxf(a.hi, b.hi), fminf(a.lo, b.lo)}; }
    static __device__ __forceinline__ float top(const Range& r) { return r.hi; }
    static __device__ __forceinline__ float low(const Range& r) { return r.lo; }
    static __device__ __forceinline__ float one(const float* p) { return *p; }
};

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
        v = fmaxf(v, shfl_xor(v, o));
    return v;
}

__device__ __forceinline__ Stats warp_join(Stats s)
{
    for (int o = 16; o > 0; o /= 2) {
        const Stats t{shfl_xor(s.m, o), shfl_xor(s.n, o), shfl_xor(s.r, o), shfl_xor(s.w, o)};
        s = join(s, t);
    }
    return s;
}

struct Shared {
    uint64_t lists[kLpWarps][32];
    uint32_t maxima[kLpWarps][32];
    Stats stats[kLpWarps];
    // what the cluster's first block reads of the others
    Stats part;
    uint64_t top[32];
    int once, flagged, found;
    int batch[kLpThreads];  // thread | batch << 8: read that batch again
    int flags[kLpThreads];  // thread: read all its units again
};

// The sums of a batch against the warp's m. COUNT: an element may equal m.
template <class T, bool COUNT, bool WHOLE>
__device__ __forceinline__ void add_batch(Stats& s, const uint4 (&raw)[kBatch], int units)
{
    constexpr int N = Unit<T>::N;
    // z = x log2 e - ref is rounded once; what rounding m log2 e to ref left over is the same for
    // every element and put right on the batch's sums
    const float ref = s.m * kLog2e, left = fmaf(s.m, kLog2e, -ref);
    const float2 log2e2 = make_float2(kLog2e, kLog2e), ref2 = make_float2(-ref, -ref);
    float2 r[2] = {}, w[2] = {};  // pairs in the packed fp32 instructions
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
        if (!WHOLE && b >= units)
            continue;
        float f[N];
        Unit<T>::widen(raw[b], f);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 z = __ffma2_rn(make_float2(f[i], f[i + 1]), log2e2, ref2);
            float2 e = make_float2(ex2(z.x), ex2(z.y));
            if (COUNT) {
                if (f[i] == s.m) {
                    e.x = 0.f;
                    s.n += 1.f;
                }
                if (f[i + 1] == s.m) {
                    e.y = 0.f;
                    s.n += 1.f;
                }
            }
            r[i >> 1 & 1] = __fadd2_rn(r[i >> 1 & 1], e);
            w[i >> 1 & 1] = __ffma2_rn(e, z, w[i >> 1 & 1]);
        }
    }
    const float rs = (r[0].x + r[0].y) + (r[1].x + r[1].y), ws = (w[0].x + w[0].y) + (w[1].x + w[1].y);
    const float fix = 1.f - left * kLn2;
    s.r = fmaf(rs, fix, s.r);
    s.w = fmaf(fmaf(-left, rs, ws) * fix, kLn2, s.w);
}

template <class T>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_kernel(const __grid_constant__ LpParams p)
{
    using U = Unit<T>;
    constexpr int N = U::N;
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = cluster.num_blocks(), part = cluster.block_rank();
    const int64_t m = blockIdx.x / parts;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T* row = static_cast<const T*>(p.v) + m * p.ld;
    // elements before the first and behind the last whole unit go one by one (block 0)
    const int head = (int)min((int64_t)((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T)), p.N);
    const int64_t units = (p.N - head) / N;
    const int tail = (int)(p.N - head - units * N);
    const uint4* body = reinterpret_cast<const uint4*>(row + head);
    const int64_t u0 = units * part / parts, u1 = units * (part + 1) / parts;

    Stats s{-INFINITY, 0.f, 0.f, 0.f};
    float big = -INFINITY, second = -INFINITY;  // this thread's largest, and its largest of other batches
    int where = 0;                              // the largest's batch
    // one batch of the warp: `have` units a lane, fewer than kBatch only in the last
    auto take = [&](const uint4 (&raw)[kBatch], auto whole, int have, int batch) {
        constexpr bool kWhole = decltype(whole)::value;
        float top = -INFINITY, low = INFINITY;
        if (kWhole) {
            const typename U::Range x = U::both(U::both(U::range(raw[0]), U::range(raw[1])), U::both(U::range(raw[2]), U::range(raw[3])));
            top = fmaxf(top, U::top(x));
            low = fminf(low, U::low(x));
        } else {
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (b < have) {
                    const typename U::Range x = U::range(raw[b]);
                    top = fmaxf(top, U::top(x));
                    low = fminf(low, U::low(x));
                }
        }
        second = fmaxf(second, fminf(top, big));
        where = top > big ? batch : where;
        big = fmaxf(big, top);
        // nothing overflows below (-inf and the type's lowest value, as masks write them, go the
        // last way), and m is not so far from 0 that the rounding of m log2 e (2^-11 at 1e4) is
        // more than a first-order matter
        if (kWhole && __all_sync(0xffffffffu, top < s.m && low > -1e38f && fabsf(s.m) < 1e4f)) {
            add_batch<T, false, true>(s, raw, kBatch);
            return;
        }
        const float wm = warp_max(top);
        if (wm > s.m)
            rebase(s, wm);
        if (__all_sync(0xffffffffu, low > -1e38f && fabsf(s.m) < 1e4f)) {
            add_batch<T, true, kWhole>(s, raw, have);
            return;
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (b >= have)
                continue;
            float f[N];
            U::widen(raw[b], f);
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                float x = f[0];  // a rotation of the array keeps this loop small
#pragma unroll
                for (int j = 0; j + 1 < N; ++j)
                    f[j] = f[j + 1];
                if (x == s.m && x != -INFINITY) {
                    s.n += 1.f;
                } else if (x != -INFINITY) {  // NaN takes this way
                    const float z = x - s.m, e = expf(z);
                    s.r += e;
                    s.w = fmaf(e, fmaxf(z, -200.f), s.w);
                }
            }
        }
    };
    const int mine_units = (int)(u1 - u0), batches = mine_units / (kBatch * kLpThreads);
    const uint4* at = body + u0 + threadIdx.x;
    if (batches > 0) {
        uint4 raw[kBatch], next[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            next[b] = __ldg(at + b * kLpThreads);
#pragma unroll 1
        for (int i = 0; i < batches; ++i) {
            at += kBatch * kLpThreads;
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                raw[b] = next[b];
            if (i + 1 < batches) {
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    next[b] = __ldg(at + b * kLpThreads);
            }
            take(raw, std::true_type{}, kBatch, i);
        }
    }
    {
        const int rest = mine_units - batches * kBatch * kLpThreads;  // units of the last batch
        if (rest - ((int)threadIdx.x - lane) > 0) {
            const int have = rest > (int)threadIdx.x ? (rest - (int)threadIdx.x + kLpThreads - 1) / kLpThreads : 0;
            uint4 raw[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch - 1; ++b)
                if (b < have)
                    raw[b] = __ldg(at + b * kLpThreads);
            // the first lanes of a short batch can have all of theirs
            if (have == kBatch)
                raw[kBatch - 1] = __ldg(at + (kBatch - 1) * kLpThreads);
            take(raw, std::false_type{}, have, batches);
        }
    }
    const bool nan = s.r != s.r;
    // the single elements: one a lane of warp 0
    uint64_t single = 0;
    if (part == 0 && warp == 0 && lane < head + tail) {
        const int64_t at = lane < head ? lane : p.N - tail + (lane - head);
        const float x = U::one(row + at);
        single = key_of(x, at);
        s = join(s, x == x ? Stats{x, x == -INFINITY ? 0.f : 1.f, 0.f, 0.f} : Stats{-INFINITY, 0.f, x, x});
    }
    // +inf: no finite statistics
    if (s.m == INFINITY)
        s.r = NAN;
    s = warp_join(s);
    if (lane == 0)
        sh.stats[warp] = s;
    if (threadIdx.x == 0)
        sh.once = sh.flagged = sh.found = 0;

    if (p.top_k > 0) {
        const bool has = (int64_t)threadIdx.x < u1 - u0;
        const uint32_t mine = has ? order_of(big) : 0u;
        // over the warps whose lanes all have a unit; without one, the few elements there are all reach 0
        const int warps = (int)min((u1 - u0) / 32, (int64_t)kLpWarps);
        sh.maxima[warp][lane] = sort32(mine, lane);
        const bool any_nan = __syncthreads_or(nan);
        uint32_t bound = 0u;
        if (warps > 0)
            bound = __shfl_sync(0xffffffffu, sort32(sh.maxima[lane % warps][lane / warps], lane), p.top_k - 1);
        if (any_nan)  // it may hide an element that the bound does not count
            bound = 0u;
        // (bound 0 is reached by NaN as well, which the largest do not tell of)
        if (has && mine >= bound) {
            if (bound != 0u && order_of(second) < bound)
                sh.batch[atomicAdd(&sh.once, 1)] = threadIdx.x | where << 8;
            else
                sh.flags[atomicAdd(&sh.flagged, 1)] = threadIdx.x;
        }
        uint64_t* cand = &sh.lists[0][0];
        auto collect = [&](uint64_t key) {  // keys of the lanes, 0 for none
            const unsigned come = __ballot_sync(0xffffffffu, key != 0);
            if (come == 0)
                return;
            int at = 0;
            if (lane == 0)
                at = atomicAdd(&sh.found, __popc(come));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(come & ((1u << lane) - 1));
            if (key != 0 && at < kMaxCand)
                cand[at] = key;
        };
        __syncthreads();
        if (part == 0 && warp == 0)
            collect((uint32_t)(single >> 32) >= bound ? single : 0);
        auto collect_unit = [&](bool there, const uint4& raw4, int64_t unit) {
            const bool reaches = there && (bound == 0u || order_of(U::top(U::range(raw4))) >= bound);
            if (!__any_sync(0xffffffffu, reaches))
                return;
            float y[N];
            U::widen(raw4, y);
#pragma unroll
            for (int i = 0; i < N; ++i)
                collect(reaches && order_of(y[i]) >= bound ? key_of(y[i], head + unit * N + i) : 0);
        };
        // one batch of a thread: four lanes, a unit each
        const int once = sh.once;
        for (int e0 = 0; e0 < once; e0 += 8 * kLpWarps) {
            const int e = e0 + warp + (lane >> 2) * kLpWarps;
            int64_t unit = u1;
            if (e < once) {
                const int who = sh.batch[e];
                unit = u0 + (who & 255) + ((int64_t)(who >> 8) * kBatch + (lane & 3)) * kLpThreads;
            }
            uint4 raw4 = {};
            if (unit < u1)
                raw4 = __ldg(body + unit);
            collect_unit(unit < u1, raw4, unit);
        }
        // all units of a thread: 32 of them an item
        const int flagged = sh.flagged, rounds = (int)((u1 - u0 + 32 * kLpThreads - 1) / (32 * kLpThreads));
        for (int f = warp; f < flagged * rounds; f += kLpWarps) {
            const int64_t unit = u0 + sh.flags[f / rounds] + ((int64_t)(f % rounds) * 32 + lane) * kLpThreads;
            uint4 raw4 = {};
            if (unit < u1)
                raw4 = __ldg(body + unit);
            collect_unit(unit < u1, raw4, unit);
        }
        __syncthreads();
        const int found = sh.found;
        if (found <= kMaxCand) {
            uint64_t list = 0;
            if (warp * 32 < found)
                list = sort32(warp * 32 + lane < found ? cand[warp * 32 + lane] : 0, lane);
            if (found > 32) {
                sh.lists[warp][lane] = list;  // each warp its own 32
                join_lists(sh.lists, warp, lane);
            } else if (warp == 0) {
                sh.lists[0][lane] = list;
            }
        } else {
            uint64_t list = part == 0 && warp == 0 ? sort32(single, lane) : 0;  // lane i: the warp's i-th largest key
            uint64_t last = __shfl_sync(0xffffffffu, list, p.top_k - 1);
            for (int f = warp; f < once + flagged; f += kLpWarps) {
                const int64_t own = u0 + (f < once ? sh.batch[f] & 255 : sh.flags[f - once]);
                for (int64_t v0 = own; v0 < u1; v0 += 32 * kLpThreads) {
                    const int64_t v = v0 + (int64_t)lane * kLpThreads;
                    float x[N];
                    if (v < u1)
                        U::widen(__ldg(body + v), x);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        uint64_t key = 0;
                        if (v < u1 && order_of(x[i]) >= bound)
                            key = key_of(x[i], head + v * N + i);
                        unsigned come = __ballot_sync(0xffffffffu, key > last);
                        while (come) {
                            const uint64_t k = __shfl_sync(0xffffffffu, key, __ffs(come) - 1);
                            come &= come - 1;
                            if (k <= last)
                                continue;
                            const int before = __popc(__ballot_sync(0xffffffffu, list > k));
                            const uint64_t up = __shfl_up_sync(0xffffffffu, list, 1);
                            list = lane < before ? list : lane == before ? k : up;
                            last = __shfl_sync(0xffffffffu, list, p.top_k - 1);
                        }
                    }
                }
            }
            __syncthreads();  // the collected keys have been dropped
            sh.lists[warp][lane] = list;
            join_lists(sh.lists, warp, lane);
        }
        if (warp == 0)
            sh.top[lane] = sh.lists[0][lane];
    } else {
        __syncthreads();
    }
    if (warp == 0) {
        s = warp_join(lane < kLpWarps ? sh.stats[lane] : Stats{-INFINITY, 0.f, 0.f, 0.f});
        if (lane == 0)
            sh.part = s;
    }
    if (parts > 1) {
        cluster.sync();
        if (part != 0) {
            cluster.sync();  // this shared memory stays until block 0 has read it
            return;
        }
        {  // the parts' lists and statistics, a warp or a lane each
            if (p.top_k > 0) {
                sh.lists[warp][lane] = warp < parts ? cluster.map_shared_rank(&sh, warp)->top[lane] : 0;
                join_lists(sh.lists, warp, lane);
            }
            if (warp == 0)
                s = warp_join(lane < parts ? cluster.map_shared_rank(&sh, lane)->part : Stats{-INFINITY, 0.f, 0.f, 0.f});
            cluster.barrier_arrive();  // what it needs of the others it has
        }
    }
    if (warp == 0) {
        const uint64_t list = p.top_k > 0 ? sh.lists[0][lane] : 0;
        // n is 0 only for a row without numbers above -inf
        const bool none = s.m == -INFINITY && s.r == 0.f;
        const float log_total = s.n == 1.f ? log1pf(s.r) : logf(s.n) + log1pf(s.r / s.n);
        const bool odd = !(s.r == s.r) || (s.n == 0.f && !none);  // NaN or +inf in the row
        if (p.entropy != nullptr && lane == 0)
            p.entropy[m] = odd ? NAN : none ? 0.f : log_total - s.w / (s.n + s.r);
        for (int i = lane; i < p.n_targets; i += 32) {
            const int64_t t = p.targets[m * p.n_targets + i];
            float y;
            if (t >= 0 && t < p.N) {
                y = odd ? NAN : none ? -INFINITY : U::one(row + t) - s.m - log_total;
            } else {
                y = t == -1 ? 0.f : NAN;
                if (t != -1)
                    record_status(p.status, TF_E_INVALID_ARG);
            }
            p.logp[m * p.n_targets + i] = y;
        }
        if (lane < p.top_k) {
            p.top_idx[m * p.top_k + lane] = (int32_t)(0xFFFFFFFFu - (uint32_t)list);
            p.top_logp[m * p.top_k + lane] = odd ? NAN : none ? -INFINITY : of_order((uint32_t)(list >> 32)) - s.m - log_total;
        }
    }
}

bool logprobs_shape_ok(int64_t M, int64_t N, int top_k)
{
    return M >= 1 && M < ((int64_t)1 << 31) / 64 && N >= 1 && N <= INT32_MAX && top_k >= 0 && top_k <= 32 && top_k <= N;
}

}  // namespace
}  // namespace tfq

using namespace tfq;

extern "C" {

size_t tf_logprobs_workspace_bytes(int64_t M, int64_t N, int top_k)
{
    if (!logprobs_shape_ok(M, N, top_k)) {
        report_error(TF_E_UNSUPPORTED_SHAPE, "tf_logprobs_workspace_bytes: M, N or top_k out of range");
        return 0;
    }
    return 256;
}

int tf_logprobs_rows(const void* v, int dtype, int64_t ld, int64_t M, int64_t N, const int32_t* targets,
                     int n_targets, int top_k, float* logp, float* entropy, int32_t* top_idx, float* top_logp,
                     void* ws, size_t ws_bytes, void* stream)
{
    const char* name = "tf_logprobs_rows";
    if (v == nullptr)
        return report_error(TF_E_INVALID_ARG, "%s: v is NULL", name);
    if (dtype != TF_DTYPE_BF16 && dtype != TF_DTYPE_F32)
        return report_error(TF_E_INVALID_ARG, "%s: dtype must be TF_DTYPE_BF16 or TF_DTYPE_F32", name);
    if (!logprobs_shape_ok(M, N, top_k) || n_targets < 0 || n_targets > 1024 || ld < N)
        return report_error(TF_E_UNSUPPORTED_SHAPE,
                            "%s: need 1 <= M < 2^25, 1 <= N < 2^31, ld >= N, 0 <= top_k <= min(32, N), 0 <= n_targets <= 1024",
                            name);
    if (!is_aligned(v, dtype == TF_DTYPE_F32 ? 4 : 2))
        return report_error(TF_E_INVALID_ARG, "%s: v misaligned", name);
    if ((n_targets > 0 && (targets == nullptr || logp == nullptr)) ||
        (top_k > 0 && (top_idx == nullptr || top_logp == nullptr)))
        return report_error(TF_E_INVALID_ARG, "%s: NULL output or targets", name);
    int rc = check_ws(ws, ws_bytes, 256, name);
    if (rc)
        return rc;
    const MemRange ranges[] = {{logp, (size_t)M * n_targets * 4},
                            {entropy, (size_t)M * 4},
                            {top_idx, (size_t)M * top_k * 4},
                            {top_logp, (size_t)M * top_k * 4},
                            {v, (size_t)((M - 1) * ld + N) * (dtype == TF_DTYPE_F32 ? 4 : 2)},
                            {targets, (size_t)M * n_targets * 4}};
    if (outputs_overlap(ranges, 4, 6))
        return report_error(TF_E_INVALID_ARG, "%s: an output overlaps another argument", name);
    const LpParams p{v, ld, M, N, targets, n_targets, top_k, logp, entropy, top_idx, top_logp, static_cast<int*>(ws)};
    // few rows: as many blocks a row (a power of two up to 8) as the SMs hold, if each still
    // has a batch of units a thread. Rows of 151,936 in us, with 1, 2, 4, 8 blocks: one row 13.0,
    // 11.8, 10.8, 9.4; 24 rows 14.2, 12.9, 11.4, 11.8; 60 rows 14.3, 13.3, 13.4, 15.5.
    int parts = 1;
    const int64_t batch = (int64_t)kLpThreads * kBatch * (dtype == TF_DTYPE_F32 ? 4 : 8);
    while (parts < kMaxCluster && M * parts * 2 <= device_sms() && N >= batch * parts)
        parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(M * parts));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = dtype == TF_DTYPE_F32 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<float>, p)
                                                : cudaLaunchKernelEx(&cfg, logprobs_kernel<uint16_t>, p);
    return e == cudaSuccess ? TF_OK : report_error(TF_E_CUDA, "%s: %s", name, cudaGetErrorString(e));
}

}  // extern "C"
