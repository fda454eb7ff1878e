// Attention of few query rows: warp MMAs (m16n8k16), a ring of key tiles filled by TMA.
//
// What bounds it is the cache's bytes: a key/value head of 128 is 512 bytes a token for 4 * 128
// operations a query row, so up to some 64 rows the arithmetic has room. A CTA an SM: one
// producer warp keeps a ring of 64-key tiles (K and V, 32 KB at head_dim 128) full, eight warps
// take the tiles apart: a warp holds 16 query rows (fragments in registers) and takes 16 keys
// at a time, with its own running maximum, sum and output, so that nothing is exchanged until
// the segment ends and the warps' parts are joined through shared memory. More than 16 query
// rows: 2 or 4 warps share a piece of keys, each with 16 rows of its own.
//
// Tiles land with the 128-byte swizzle (16-byte piece c of row r at c ^ (r % 8)), so the eight
// rows of an ldmatrix fall in different banks. A box is one page's rows of a tile.
#include "tfq_attn.cuh"

namespace tfq {
namespace {

constexpr int kKeys = 64;         // keys of a tile
constexpr int kWarps = 8;         // consumer warps
constexpr int kCtaThreads = (kWarps + 1) * 32;
constexpr int kRingBytes = 128 * 1024;
constexpr int kOutCols = 128;     // columns joined at once
constexpr int kOutStride = 136;   // floats; 8 banks on a row, so that a fragment's rows do not collide
constexpr int kOutBytes = kWarps * 16 * kOutStride * 4;

template <int HD>
struct Cfg {
    static constexpr int kTileBytes = 2 * kKeys * HD * 2;
    static constexpr int kStages = kRingBytes / kTileBytes;
    static constexpr int kMlOff = 0;                                  // [kWarps][16][2] floats
    static constexpr int kBarOff = kMlOff + kWarps * 16 * 2 * 4;      // full[kStages], empty[kStages]
    static constexpr int kFlagOff = kBarOff + 2 * 16 * 8;             // [0] abort [1] last [2] abort, as of a segment's end
    static constexpr int kOutOff = 2048;
    static constexpr int kSchedOff = kOutOff + kOutBytes;
    static size_t smem(int B)
    {
        return 1024 + ((kSchedOff + Schedule::bytes(B) + 1023) / 1024 * 1024) + (size_t)kStages * kTileBytes;
    }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// A box {64 columns, rows, head_dim / 64} of the pool at row `y`, all of a row's columns.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int y, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(0), "r"(y), "r"(0), "r"(smem_u32(bar))
        : "memory");
}

// 0xFFFF in each half of x whose bf16 is infinite or NaN.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x)
{
    return ((x & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// RW row tiles of 16 (16 RW query rows an item); 8 / RW groups of warps share out the keys.
template <int HD, int RW>
__global__ void __launch_bounds__(kCtaThreads, 1)
    tree_attn_warp_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map)
{
    using C = Cfg<HD>;
    constexpr int ROWS = 16 * RW, KG = kWarps / RW, NC = HD / 8, KS = HD / 16;
    constexpr int CH = RW == 4 ? 2 : 1;       // 16-key pieces a warp takes of a tile
    constexpr int TEAMS = RW == 1 ? 2 : 1;    // warps that take turns on the tiles
    constexpr int kUsers = kWarps / TEAMS;    // warps that read a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    float* ml = reinterpret_cast<float*>(smem + C::kMlOff);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
    uint64_t* empty = full + C::kStages;
    volatile int* flags = reinterpret_cast<volatile int*>(smem + C::kFlagOff);
    float* outbuf = reinterpret_cast<float*>(smem + C::kOutOff);
    uint8_t* ring = smem + (C::kSchedOff + Schedule::bytes(p.B) + 1023) / 1024 * 1024;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kUsers);
        }
        flags[0] = 0;
        fence_mbar_init();
    }
    pdl_wait();
    Shares<ROWS, kKeys> shares(p, smem + C::kSchedOff);
    shares.build();
    pdl_launch_dependents();
    const int64_t u0 = shares.start_of(blockIdx.x), u1 = shares.start_of(blockIdx.x + 1);
    const int box = min(p.c.page_size, kKeys);

    if (warp == kWarps) {
        // ---- producer: lanes 0 .. boxes - 1 take the tile's K boxes, the next as many its V boxes
        const int boxes = kKeys / box, kv = lane / boxes, mine = lane % boxes;
        const bool active = lane < 2 * boxes;
        int n = 0;
        bool gone = false;
        for (int64_t u = u0; u < u1 && !gone;) {
            const Segment g = shares.segment(u, u1);
            const SeqRows q = shares.s.seq[g.b];
            const int32_t* table = p.c.table + (int64_t)q.slot * p.c.max_pages;
            const int len = q.len();
            // the table entry of the lane's box of the next tile is read a tile ahead
            auto page_at = [&](int t) {
                const int row = t * kKeys + mine * box;
                return active && t < g.t1 && row < len ? __ldcg(table + (row >> p.c.page_shift)) : -1;
            };
            int page = page_at(g.t0);
            for (int t = g.t0; t < g.t1; ++t, ++n) {
                const int next = page_at(t + 1);
                const int st = n % C::kStages;
                const bool ok = n < C::kStages || attn_wait(&empty[st], (n / C::kStages - 1) & 1, flags, p.status, p.limit_ns);
                if (!__all_sync(0xffffffffu, ok)) {
                    gone = true;
                    break;
                }
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[st], C::kTileBytes);
                __syncwarp();
                if (active) {
                    const int row = t * kKeys + mine * box;
                    int y = p.total_rows;  // zeros
                    if (row < len) {
                        if (page >= 0 && page < p.c.n_pages)
                            y = (int)p.c.row_of(p.layer, kv, page, g.h) + (row & (p.c.page_size - 1));
                        else
                            record_status(p.status, TF_E_INVALID_ARG);
                    }
                    tma_rows(smem_u32(ring + (size_t)st * C::kTileBytes + kv * (C::kTileBytes / 2) + mine * box * HD * 2), &map,
                             y, &full[st]);
                }
                page = next;
            }
            u += g.t1 - g.t0;
        }
        if (gone)  // no copy may be in flight when the CTA leaves
            for (int i = max(0, n - C::kStages); i < n; ++i)
                mbar_wait_bounded(&full[i % C::kStages], (i / C::kStages) & 1, p.limit_ns);
        return;
    }

    // ---- consumers
    const int rw = warp % RW, kg = warp / RW;
    const int gi = lane >> 2, ti = lane & 3;
    const int team = TEAMS == 2 ? kg / 4 : 0, piece = TEAMS == 2 ? kg % 4 : kg * CH;
    const int k_row = (lane >> 4) * 8 + (lane & 7), k_bit = (lane >> 3) & 1;  // ldmatrix rows: K
    const int v_row = ((lane >> 3) & 1) * 8 + (lane & 7), v_bit = lane >> 4;  // V (transposed)
    const int half = box * 128;                                              // bytes of a box's 64 columns
    int n = 0;
    for (int64_t u = u0; u < u1;) {
        const Segment g = shares.segment(u, u1);
        const SeqRows q = shares.s.seq[g.b];
        const int len = q.len(), n_rows = q.rows * p.group;
        // the lane's two query rows, their masks and the A fragments
        const int row0 = g.rt * ROWS + rw * 16 + gi, row1 = row0 + 8;
        uint64_t mask0 = 0, mask1 = 0;
        uint32_t qa[KS][4];
        {
            const bool in0 = row0 < n_rows, in1 = row1 < n_rows;
            const int t0 = in0 ? row0 / p.group : 0, t1 = in1 ? row1 / p.group : 0;
            const uint16_t* q0 = p.q + (q.r0 + t0) * p.ldq + (int64_t)(g.h * p.group + (in0 ? row0 % p.group : 0)) * HD;
            const uint16_t* q1 = p.q + (q.r0 + t1) * p.ldq + (int64_t)(g.h * p.group + (in1 ? row1 % p.group : 0)) * HD;
            if (in0)
                mask0 = p.masks == nullptr ? ~0ull >> (63 - t0) : p.masks[q.r0 + t0];
            if (in1)
                mask1 = p.masks == nullptr ? ~0ull >> (63 - t1) : p.masks[q.r0 + t1];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int col = ks * 16 + ti * 2;
                qa[ks][0] = in0 ? __ldcg(reinterpret_cast<const uint32_t*>(q0 + col)) : 0u;
                qa[ks][1] = in1 ? __ldcg(reinterpret_cast<const uint32_t*>(q1 + col)) : 0u;
                qa[ks][2] = in0 ? __ldcg(reinterpret_cast<const uint32_t*>(q0 + col + 8)) : 0u;
                qa[ks][3] = in1 ? __ldcg(reinterpret_cast<const uint32_t*>(q1 + col + 8)) : 0u;
            }
        }
        float o[NC][4];
#pragma unroll
        for (int i = 0; i < NC; ++i)
            o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        for (int t = g.t0; t < g.t1; ++t, ++n) {
            if (TEAMS == 2 && (n & 1) != team)
                continue;
            const int st = n % C::kStages;
            const bool ok = attn_wait(&full[st], (n / C::kStages) & 1, flags, p.status, p.limit_ns);
            if (!__all_sync(0xffffffffu, ok))
                break;
            const uint32_t tile = smem_u32(ring + (size_t)st * C::kTileBytes);
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                const int r0 = (piece + ch) * 16, k0 = t * kKeys + r0;
                if (k0 >= len)
                    break;
                const uint32_t at = tile + (r0 / box) * (box * HD * 2) + (r0 % box) * 128;
                // S = Q K^T
                float s[2][4] = {};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t b[4];
                    ldsm4(b, at + (ks >> 2) * half + k_row * 128 + ((((ks & 3) * 2 + k_bit) ^ (k_row & 7)) << 4));
                    mma_bf16_16816(s[0], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b[0], b[1]);
                    mma_bf16_16816(s[1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b[2], b[3]);
                }
                const bool edge = k0 + 16 > q.base;  // the block's own tokens, or what lies behind them
                unsigned see0 = 0xFu, see1 = 0xFu;   // bits: keys 2 ti, 2 ti + 1, 2 ti + 8, 2 ti + 9
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] *= p.scale_log2;
                if (edge) {
                    see0 = see1 = 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = k0 + (i >> 1) * 8 + ti * 2 + (i & 1), j = k - q.base;
                        const bool ctx = j < 0, in = k < len;
                        if (ctx || (in && (mask0 >> (j & 63) & 1)))
                            see0 |= 1u << i;
                        else
                            s[i >> 1][i & 1] = -INFINITY;
                        if (ctx || (in && (mask1 >> (j & 63) & 1)))
                            see1 |= 1u << i;
                        else
                            s[i >> 1][2 + (i & 1)] = -INFINITY;
                    }
                }
                // running maximum of each row, over its four lanes
                float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
                float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
                if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
                    const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                    const float f0 = n0 == -INFINITY ? 1.f : attn_ex2(m0 - n0), f1 = n1 == -INFINITY ? 1.f : attn_ex2(m1 - n1);
                    m0 = n0, m1 = n1;
                    l0 *= f0, l1 *= f1;
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        o[i][0] *= f0, o[i][1] *= f0;
                        o[i][2] *= f1, o[i][3] *= f1;
                    }
                }
                const float ref0 = m0 == -INFINITY ? 0.f : m0, ref1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    s[i][0] = attn_ex2(s[i][0] - ref0), s[i][1] = attn_ex2(s[i][1] - ref0);
                    s[i][2] = attn_ex2(s[i][2] - ref1), s[i][3] = attn_ex2(s[i][3] - ref1);
                    l0 += s[i][0] + s[i][1];
                    l1 += s[i][2] + s[i][3];
                }
                // weights rounded to bf16, the type of V: 2^-8 each, under the output's own rounding
                const uint32_t a0 = f32x2_to_bf16x2(s[0][0], s[0][1]), a1 = f32x2_to_bf16x2(s[0][2], s[0][3]);
                const uint32_t a2 = f32x2_to_bf16x2(s[1][0], s[1][1]), a3 = f32x2_to_bf16x2(s[1][2], s[1][3]);
                const uint32_t vat = at + C::kTileBytes / 2;
                uint32_t odd = 0;
                const int left = len - k0;  // keys of the piece that exist
                // nothing behind the sequence's end takes part: not even as 0 times NaN
                const uint32_t in_lo = (2 * ti < left ? 0xFFFFu : 0u) | (2 * ti + 1 < left ? 0xFFFF0000u : 0u);
                const uint32_t in_hi = (2 * ti + 8 < left ? 0xFFFFu : 0u) | (2 * ti + 9 < left ? 0xFFFF0000u : 0u);
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) {
                    uint32_t b[4];
                    ldsm4_trans(b, vat + (i >> 2) * half + v_row * 128 + ((((i & 3) * 2 + v_bit) ^ (v_row & 7)) << 4));
                    if (edge) {
                        b[0] &= in_lo, b[1] &= in_hi, b[2] &= in_lo, b[3] &= in_hi;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t x = nonfinite2(b[j]);
                            odd |= x;
                            b[j] &= ~x;
                        }
                    }
                    mma_bf16_16816(o[2 * i], a0, a1, a2, a3, b[0], b[1]);
                    mma_bf16_16816(o[2 * i + 1], a0, a1, a2, a3, b[2], b[3]);
                }
                if (edge && __any_sync(0xffffffffu, odd != 0)) {
                    // infinities and NaN among the values: they reach the rows that see their key alone
                    for (int k = 0; k < 16 && k < left; ++k) {
                        const int src = (lane & ~3) | ((k & 7) >> 1), bit = (k >> 3) * 2 + (k & 1);
                        const uint32_t w01 = k < 8 ? a0 : a2, w23 = k < 8 ? a1 : a3;
                        const uint32_t p0 = __shfl_sync(0xffffffffu, w01, src), p1 = __shfl_sync(0xffffffffu, w23, src);
                        const bool r0s = __shfl_sync(0xffffffffu, see0, src) >> bit & 1, r1s = __shfl_sync(0xffffffffu, see1, src) >> bit & 1;
                        const float w0 = k & 1 ? bf16hi_f32(p0) : bf16lo_f32(p0), w1 = k & 1 ? bf16hi_f32(p1) : bf16lo_f32(p1);
#pragma unroll
                        for (int i = 0; i < NC; ++i) {
                            uint32_t v;
                            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(vat + (i >> 3) * half + k * 128 + (((i & 7) ^ (k & 7)) << 4) + ti * 4) : "memory");
                            const uint32_t x = nonfinite2(v);
                            if (x & 0xFFFFu) {
                                if (r0s) o[i][0] += w0 * bf16lo_f32(v);
                                if (r1s) o[i][2] += w1 * bf16lo_f32(v);
                            }
                            if (x >> 16) {
                                if (r0s) o[i][1] += w0 * bf16hi_f32(v);
                                if (r1s) o[i][3] += w1 * bf16hi_f32(v);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&empty[st]);
        }

        // ---- the segment's end: the key groups' parts of each row joined
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (ti == 0) {
            ml[(warp * 16 + gi) * 2] = m0;
            ml[(warp * 16 + gi) * 2 + 1] = l0;
            ml[(warp * 16 + gi + 8) * 2] = m1;
            ml[(warp * 16 + gi + 8) * 2 + 1] = l1;
        }
        named_bar_sync(1, kWarps * 32);
        float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
        for (int k = 0; k < KG; ++k) {
            top0 = fmaxf(top0, ml[((k * RW + rw) * 16 + gi) * 2]);
            top1 = fmaxf(top1, ml[((k * RW + rw) * 16 + gi + 8) * 2]);
        }
        const float f0 = top0 == -INFINITY ? 1.f : attn_ex2(m0 - top0), f1 = top1 == -INFINITY ? 1.f : attn_ex2(m1 - top1);
        const bool whole = g.t0 == 0 && g.t1 == g.nt;
        const int slot = g.t0 > 0 ? 2 * blockIdx.x : 2 * blockIdx.x + 1;
        float* part = p.parts + (int64_t)slot * (ROWS * (HD + 2));
        for (int c0 = 0; c0 < HD; c0 += kOutCols) {
            if (c0 > 0)
                named_bar_sync(1, kWarps * 32);  // the last columns have been read
            float* mine = outbuf + (warp * 16 + gi) * kOutStride + ti * 2;
#pragma unroll
            for (int i = 0; i < NC; ++i)
                if (i * 8 >= c0 && i * 8 < c0 + kOutCols) {
                    *reinterpret_cast<float2*>(mine + i * 8 - c0) = make_float2(o[i][0] * f0, o[i][1] * f0);
                    *reinterpret_cast<float2*>(mine + 8 * kOutStride + i * 8 - c0) = make_float2(o[i][2] * f1, o[i][3] * f1);
                }
            named_bar_sync(1, kWarps * 32);
            constexpr int kQuads = (HD < kOutCols ? HD : kOutCols) / 4;
            for (int i = threadIdx.x; i < ROWS * kQuads; i += kWarps * 32) {
                const int r = i / kQuads, c = i % kQuads * 4, w = r / 16, rr = r % 16;
                float top = -INFINITY, l = 0.f;
#pragma unroll
                for (int k = 0; k < KG; ++k)
                    top = fmaxf(top, ml[((k * RW + w) * 16 + rr) * 2]);
                const float ref = top == -INFINITY ? 0.f : top;
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < KG; ++k) {
                    const int wk = k * RW + w;
                    l = fmaf(attn_ex2(ml[(wk * 16 + rr) * 2] - ref), ml[(wk * 16 + rr) * 2 + 1], l);
                    const float4 v = *reinterpret_cast<const float4*>(outbuf + (wk * 16 + rr) * kOutStride + c);
                    a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
                }
                const int row = g.rt * ROWS + r;
                if (row >= n_rows)
                    continue;
                if (whole) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    *reinterpret_cast<uint2*>(p.o + ((int64_t)(q.r0 + row / p.group) * p.n_q + g.h * p.group + row % p.group) * HD + c0 + c) =
                        bf16x4(make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
                } else {
                    __stcg(reinterpret_cast<float4*>(part + r * HD + c0 + c), a);
                    if (c0 + c == 0)
                        __stcg(reinterpret_cast<float2*>(part + ROWS * HD + 2 * r), make_float2(top, l));
                }
            }
        }
        if (!whole) {
            const int64_t first = g.u - g.t0;  // the item's first unit
            const int ca = shares.cta_of(first), cz = shares.cta_of(first + g.nt - 1);
            __threadfence();
            named_bar_sync(1, kWarps * 32);
            if (threadIdx.x == 0) {
                const int last = !flags[0] && atom_add_acq_rel_gpu(&p.counters[ca], 1u) == (unsigned)(cz - ca);
                if (last)
                    p.counters[ca] = 0;
                flags[1] = last;
            }
            named_bar_sync(1, kWarps * 32);
            if (flags[1]) {
                __threadfence();
                for (int i = threadIdx.x; i < ROWS * (HD / 4); i += kWarps * 32) {
                    const int r = i / (HD / 4), c = i % (HD / 4) * 4, row = g.rt * ROWS + r;
                    if (row < n_rows)
                        *reinterpret_cast<uint2*>(p.o + ((int64_t)(q.r0 + row / p.group) * p.n_q + g.h * p.group + row % p.group) * HD + c) =
                            bf16x4(join_parts<ROWS, HD>(p.parts, ca, cz, r, c));
                }
            }
        }
        if (threadIdx.x == 0)
            flags[2] = flags[0];
        named_bar_sync(1, kWarps * 32);  // the buffers may be written again
        if (flags[2])                    // one answer for all warps
            break;
        u += g.t1 - g.t0;
    }
}

template <int HD, int RW>
cudaError_t launch(const AttnParams& p, const CUtensorMap& map, cudaStream_t stream, bool pdl)
{
    const size_t smem = Cfg<HD>::smem(p.B);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(tree_attn_warp_kernel<HD, RW>, (int)Cfg<HD>::smem(kMaxAttnSeqs), done);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(tree_attn_warp_kernel<HD, RW>, dim3(device_sms()), dim3(kCtaThreads), smem, stream, pdl, p, map);
}

}  // namespace

cudaError_t launch_attn_warp(const AttnParams& p, int rows, const CUtensorMap& map, cudaStream_t stream, bool pdl)
{
    if (p.c.head_dim == 64)
        return rows == 16 ? launch<64, 1>(p, map, stream, pdl) : rows == 32 ? launch<64, 2>(p, map, stream, pdl) : launch<64, 4>(p, map, stream, pdl);
    if (p.c.head_dim == 128)
        return rows == 16 ? launch<128, 1>(p, map, stream, pdl) : rows == 32 ? launch<128, 2>(p, map, stream, pdl) : launch<128, 4>(p, map, stream, pdl);
    return rows == 16 ? launch<256, 1>(p, map, stream, pdl) : rows == 32 ? launch<256, 2>(p, map, stream, pdl) : launch<256, 4>(p, map, stream, pdl);
}

}  // namespace tfq
