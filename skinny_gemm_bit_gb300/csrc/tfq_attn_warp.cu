// Attention of few query rows: warp MMAs (m16n8k16), every warp with a ring of its own.
//
// What bounds it is the cache's bytes: a key/value head of 128 is 512 bytes a token for 4 * 128
// operations a query row, so up to some 32 rows the arithmetic has room. One CTA of eight warps an
// SM; of a segment's key tiles (32 keys; 16 at head_dim 256) warp w takes every eighth. A
// warp fetches its own tiles: as soon as it has read a K or V tile it asks the TMA for the
// next one into the same slot (three slots of 8 KB a warp, 192 KB an SM), so there is no
// producer to wait for and the ring is full while a segment ends or the next begins. Each
// warp keeps its own running maximum, sum and output; they meet in shared memory once a
// segment.
//
// 64 ragged sequences of up to 8190 tokens, 16 query and 8 key/value heads of 128: 174 us, 6.2 TB/s of
// K and V; 64 of 8192 tokens 320 us, 6.7 TB/s. A ring shared by the warps, filled by a producer warp, kept a
// tile 1700 cycles from its release and took 242 us. Few tokens are bound by the chain of latencies
// (queries, tiles, the warps' join, the CTAs' join): one token over 4097 takes 10.7 us, 8 over 32,771 31.6.
//
// Tiles land with the 128-byte swizzle (16-byte piece c of row r at c ^ (r % 8)), so the eight
// rows of an ldmatrix fall in different banks. A box is one page's rows of a tile.
#include "tfq_attn.cuh"

namespace tfq {
namespace {

constexpr int kWarps = 8;
constexpr int kCtaThreads = kWarps * 32;
constexpr float kGrow = 8.f;  // the reference of a row moves when its maximum has grown by 2^8

template <int HD, int RW>
struct Cfg {
    static constexpr int CH = HD == 256 ? 1 : 2;          // 16-key pieces of a tile
    static constexpr int KT = 16 * CH;
    static constexpr int ROWS = 16 * RW;
    static constexpr int kSlotBytes = KT * HD * 2;        // K or V of a tile
    static constexpr int kSlots = 24576 / kSlotBytes;     // of a warp: 3, or 6 at head_dim 64
    static constexpr int kCols = RW == 2 ? 8 : 16;         // output columns joined at once, as shared memory allows
    static constexpr int kStride = kCols + 4;             // floats
    static constexpr int kMlOff = 0;                      // [kWarps][ROWS][2] floats
    static constexpr int kBarOff = kMlOff + kWarps * ROWS * 2 * 4;
    static constexpr int kFlagOff = kBarOff + kWarps * kSlots * 8;  // [0] abort [2] abort, as of a segment's end
    // the item's queries, and after its last tile what the warps hand over
    static constexpr int kQOff = (kFlagOff + 16 + 1023) / 1024 * 1024;
    static constexpr int kOutBytes = kWarps * ROWS * kStride * 4;
    static constexpr int kSchedOff = kQOff + (ROWS * HD * 2 > kOutBytes ? ROWS * HD * 2 : kOutBytes);
    static constexpr __host__ __device__ size_t ring(int B) { return (kSchedOff + schedule_bytes(B) + 1023) / 1024 * 1024; }
    static constexpr __host__ __device__ size_t smem(int B) { return 1024 + ring(B) + (size_t)kWarps * kSlots * kSlotBytes; }
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

// RW row tiles of 16 (16 RW query rows an item).
template <int HD, int RW>
__global__ void __launch_bounds__(kCtaThreads, 1)
    tree_attn_warp_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map)
{
    using C = Cfg<HD, RW>;
    constexpr int ROWS = C::ROWS, KT = C::KT, CH = C::CH, NC = HD / 8, KS = HD / 16, NS = C::kSlots;
    constexpr bool kQRegs = RW == 1 && HD <= 128;  // the rows' A fragments in registers
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* ml = reinterpret_cast<float*>(smem + C::kMlOff);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff) + warp * NS;  // the warp's own
    volatile int* flags = reinterpret_cast<volatile int*>(smem + C::kFlagOff);
    uint8_t* qbuf = smem + C::kQOff;
    float* outbuf = reinterpret_cast<float*>(qbuf);
    uint8_t* ring = smem + C::ring(p.B) + (size_t)warp * NS * C::kSlotBytes;

    if (lane == 0) {
        for (int i = 0; i < NS; ++i)
            mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) {
        flags[0] = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    }
    pdl_wait();
    // 8 key/value heads of 128, in us, an item a CTA against split and joined: one row over 200 tokens 7.1, 10.2;
    // over 500 9.7, 10.5, but in a decoder step, its code not in the caches, 28 layers 787, 769; eight
    // sequences of eight rows over 500 tokens 11.3, 14.7, over 1000 13.9, 18.7, over 3000 27.5, 26.0
    Shares<ROWS, KT, kWarps, RW == 2 ? 8 : 10> shares(p, smem + C::kSchedOff);
    shares.build();
    pdl_launch_dependents();
    const int u0 = shares.start_of(blockIdx.x), u1 = shares.start_of(blockIdx.x + 1);

    // ---- the warp's loads, in the order it will read them: K, V of its first tile, of its next ...
    const int box = min(p.c.page_size, KT), bs = KT / box - 1;  // a tile is 1 << bs boxes, one or two
    const int ahead = 32 >> bs;  // tiles whose pages the lanes hold at once
    int lu = u0;                   // first unit of the segment that the next load belongs to
    Segment lg{};                  // that segment
    int lt = 0, lkv = 0;           // the next load: tile, K or V
    int lpages = -1, lj = 0;       // the lane's page (tile lane >> bs of those, box lane & bs); which of them is next
    uint32_t issued = 0, taken = 0;
    auto look = [&]() {
        const int t = lt + kWarps * (lane >> bs), row = t * KT + (lane & bs) * box;
        lpages = t < lg.t1 && row < lg.q.len() ? p.c.table[(int64_t)lg.q.slot * p.c.max_pages + (row >> p.c.page_shift)] : -1;
        lj = 0;
    };
    auto settle = [&]() {  // from a tile behind its segment's end to the next segment that has one
        while (lt >= lg.t1) {
            lu += lg.units;
            if (lu >= u1)
                return;
            lg = shares.segment(lu, u1);
            lt = lg.t0 + warp;
            lj = ahead;
        }
        if (lj == ahead)
            look();
    };
    auto load = [&]() {
        if (lu >= u1)
            return;
        const uint32_t slot = issued % NS;
        const int page = __shfl_sync(0xffffffffu, lpages, ((lj << bs) + lane) & 31);
        if (lane == 0)
            mbar_arrive_expect_tx(&full[slot], C::kSlotBytes);
        __syncwarp();
        if (lane <= bs) {
            const int row = lt * KT + lane * box;
            int y = p.total_rows;  // zeros
            if (row < lg.q.len()) {
                if (page >= 0 && page < p.c.n_pages)
                    y = (int)p.c.row_of(p.layer, lkv, page, lg.h) + (row & (p.c.page_size - 1));
                else
                    record_status(p.status, TF_E_INVALID_ARG);
            }
            tma_rows(smem_u32(ring + slot * C::kSlotBytes + lane * box * HD * 2), &map, y, &full[slot]);
        }
        ++issued;
        if (lkv == 0) {
            lkv = 1;
        } else {
            lkv = 0;
            lt += kWarps;
            ++lj;
            settle();
        }
    };
    // an item's rows of q: a thread's pieces, on their way while the first tiles are asked for
    constexpr int kPieces = ROWS * (HD / 8), kMine = (kPieces + kCtaThreads - 1) / kCtaThreads;
    uint4 mine[kMine];
    auto fetch = [&](const Segment& s) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int piece = threadIdx.x + i * kCtaThreads, row = s.rt * ROWS + piece / (HD / 8);
            mine[i] = make_uint4(0, 0, 0, 0);
            if (piece < kPieces && row < s.q.rows * p.group)
                mine[i] = __ldcg(reinterpret_cast<const uint4*>(p.q + (s.q.r0 + p.token_of(row)) * p.ldq +
                                                                (int64_t)(s.h * p.group + p.head_of(row)) * HD + piece % (HD / 8) * 8));
        }
    };
    Segment g{};
    if (u0 < u1) {
        g = lg = shares.segment(u0, u1);
        fetch(g);
        lt = lg.t0 + warp;
        lj = ahead;
        settle();
#pragma unroll 1
        for (int i = 0; i < NS; ++i)
            load();
    }

    const int gi = lane >> 2, ti = lane & 3;
    const int k_row = (lane >> 4) * 8 + (lane & 7), k_bit = (lane >> 3) & 1;  // ldmatrix rows: K
    const int v_row = ((lane >> 3) & 1) * 8 + (lane & 7), v_bit = lane >> 4;  // V (transposed), and Q
    const int half = box * 128;                                              // bytes of a box's 64 columns
    SplitItem split[2];  // the item that the CTA continues, the one that it starts
    split[0].c0 = split[1].c0 = 1;
    split[0].c1 = split[1].c1 = 0;
    bool alive = true;
    for (int u = u0; u < u1;) {
        if (u != u0) {
            g = shares.segment(u, u1);
            fetch(g);
        }
        u += g.units;
        if (g.t0 == g.t1)
            continue;
        const SeqRows& q = g.q;
        const int len = q.len(), n_rows = q.rows * p.group;
        // the item's rows of q, swizzled as the tiles are
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const int piece = threadIdx.x + i * kCtaThreads, r = piece / (HD / 8), c = piece % (HD / 8);
            if (piece < kPieces)
                *reinterpret_cast<uint4*>(qbuf + (c >> 3) * (ROWS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = mine[i];
        }
        // the masks of the lane's rows
        uint64_t mask[RW][2];
#pragma unroll
        for (int i = 0; i < 2 * RW; ++i) {
            const int row = g.rt * ROWS + (i >> 1) * 16 + (i & 1) * 8 + gi, t = p.token_of(row);
            mask[i >> 1][i & 1] = row >= n_rows ? 0 : block_mask(p, q, t);
        }
        named_bar_sync(1, kCtaThreads);
        const uint32_t q_at = smem_u32(qbuf);
        auto q_frag = [&](uint32_t (&a)[4], int rw, int ks) {
            ldsm4(a, q_at + (ks >> 2) * (ROWS * 128) + (rw * 16 + v_row) * 128 + ((((ks & 3) * 2 + v_bit) ^ (v_row & 7)) << 4));
        };
        uint32_t qa[kQRegs ? KS : 1][4];
        if (kQRegs) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                q_frag(qa[kQRegs ? ks : 0], 0, ks);
        }
        float o[RW][NC][4];
        float m[RW][2], l[RW][2];  // the rows' references and sums
#pragma unroll
        for (int r = 0; r < RW; ++r) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
                o[r][i][0] = o[r][i][1] = o[r][i][2] = o[r][i][3] = 0.f;
            m[r][0] = m[r][1] = -INFINITY;
            l[r][0] = l[r][1] = 0.f;
        }

        for (int t = g.t0 + warp; t < g.t1 && alive; t += kWarps) {
            const int k0 = t * KT;
            const uint32_t ks_slot = taken % NS;
            alive = __all_sync(0xffffffffu, attn_wait(&full[ks_slot], (taken / NS) & 1, flags, p.status, p.limit_ns));
            if (!alive)
                break;
            // S = Q K^T
            const uint32_t k_at = smem_u32(ring + ks_slot * C::kSlotBytes);
            float s[RW][2 * CH][4] = {};
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                const uint32_t at = k_at + (ch * 16 / box) * (box * HD * 2) + (ch * 16 % box) * 128 + k_row * 128;
#pragma unroll
                for (int kq = 0; kq < KS; kq += 4) {  // four fragments ahead of the MMAs that take them
                    uint32_t b[4][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        ldsm4(b[j], at + (kq >> 2) * half + (((j * 2 + k_bit) ^ (k_row & 7)) << 4));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int r = 0; r < RW; ++r) {
                            uint32_t a[4];
                            if (kQRegs)
                                a[0] = qa[kQRegs ? kq + j : 0][0], a[1] = qa[kQRegs ? kq + j : 0][1], a[2] = qa[kQRegs ? kq + j : 0][2], a[3] = qa[kQRegs ? kq + j : 0][3];
                            else
                                q_frag(a, r, kq + j);
                            mma_bf16_16816(s[r][2 * ch], a[0], a[1], a[2], a[3], b[j][0], b[j][1]);
                            mma_bf16_16816(s[r][2 * ch + 1], a[0], a[1], a[2], a[3], b[j][2], b[j][3]);
                        }
                }
            }
            ++taken;
            __syncwarp();
            load();  // into the slot just read

            const bool edge = k0 + KT > q.base;  // the block's own tokens, or what lies behind them
            unsigned see[RW][2];                 // bit 2 i + j: key 8 i + 2 ti + j
#pragma unroll
            for (int r = 0; r < RW; ++r) {
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[r][i][j] *= p.scale_log2;
                if (edge) {
                    see[r][0] = see[r][1] = 0u;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t of = (uint32_t)tile_mask(mask[r][h], k0 - q.base) >> (ti * 2);
#pragma unroll
                        for (int i = 0; i < 4 * CH; ++i) {
                            if (of >> ((i >> 1) * 8 + (i & 1)) & 1)
                                see[r][h] |= 1u << i;
                            else
                                s[r][i >> 1][2 * h + (i & 1)] = -INFINITY;
                        }
                    }
                }
                // each row's largest, over its four lanes
                float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i) {
                    x[0] = fmaxf(x[0], fmaxf(s[r][i][0], s[r][i][1]));
                    x[1] = fmaxf(x[1], fmaxf(s[r][i][2], s[r][i][3]));
                }
#pragma unroll
                for (int f = 1; f < 4; f *= 2) {
                    x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], f));
                    x[1] = fmaxf(x[1], __shfl_xor_sync(0xffffffffu, x[1], f));
                }
                if (__any_sync(0xffffffffu, x[0] > m[r][0] + kGrow || x[1] > m[r][1] + kGrow)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float now = fmaxf(m[r][h], x[h]), f = now == -INFINITY ? 1.f : attn_ex2(m[r][h] - now);
                        m[r][h] = now;
                        l[r][h] *= f;
#pragma unroll
                        for (int i = 0; i < NC; ++i)
                            o[r][i][2 * h] *= f, o[r][i][2 * h + 1] *= f;
                    }
                }
                const float ref0 = m[r][0] == -INFINITY ? 0.f : m[r][0], ref1 = m[r][1] == -INFINITY ? 0.f : m[r][1];
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i) {
                    s[r][i][0] = attn_ex2(s[r][i][0] - ref0), s[r][i][1] = attn_ex2(s[r][i][1] - ref0);
                    s[r][i][2] = attn_ex2(s[r][i][2] - ref1), s[r][i][3] = attn_ex2(s[r][i][3] - ref1);
                    l[r][0] += s[r][i][0] + s[r][i][1];
                    l[r][1] += s[r][i][2] + s[r][i][3];
                }
            }
            // weights rounded to bf16, as the product with V takes them: up to 2^-8 of each, 2^-8 of sum p |v| in
            // all. Rounding to nearest, independent errors: 8 rows over 32,771 tokens 0.0022 of the output's norm
            // against 64 bits, 0.0017 of it the output's own rounding. Their sum is of the unrounded ones. A second
            // product with what the rounding left took 64 ragged sequences from 174 to 176 us, one token over 4097
            // from 10.6 to 10.8 and 8 x 8 rows over 2000 from 20.0 to 21.8.
            uint32_t w[RW][CH][4];
#pragma unroll
            for (int r = 0; r < RW; ++r)
#pragma unroll
                for (int ch = 0; ch < CH; ++ch) {
                    w[r][ch][0] = f32x2_to_bf16x2(s[r][2 * ch][0], s[r][2 * ch][1]);
                    w[r][ch][1] = f32x2_to_bf16x2(s[r][2 * ch][2], s[r][2 * ch][3]);
                    w[r][ch][2] = f32x2_to_bf16x2(s[r][2 * ch + 1][0], s[r][2 * ch + 1][1]);
                    w[r][ch][3] = f32x2_to_bf16x2(s[r][2 * ch + 1][2], s[r][2 * ch + 1][3]);
                }

            // O += P V
            const uint32_t vs = taken % NS;
            alive = __all_sync(0xffffffffu, attn_wait(&full[vs], (taken / NS) & 1, flags, p.status, p.limit_ns));
            if (!alive)
                break;
            const uint32_t v_at = smem_u32(ring + vs * C::kSlotBytes);
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
                const uint32_t at = v_at + (ch * 16 / box) * (box * HD * 2) + (ch * 16 % box) * 128;
                if (!edge) {
#pragma unroll
                    for (int i = 0; i < NC / 2; i += 4) {
                        uint32_t b[4][4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            ldsm4_trans(b[j], at + (i >> 2) * half + v_row * 128 + (((j * 2 + v_bit) ^ (v_row & 7)) << 4));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int r = 0; r < RW; ++r) {
                                mma_bf16_16816(o[r][2 * (i + j)], w[r][ch][0], w[r][ch][1], w[r][ch][2], w[r][ch][3], b[j][0], b[j][1]);
                                mma_bf16_16816(o[r][2 * (i + j) + 1], w[r][ch][0], w[r][ch][1], w[r][ch][2], w[r][ch][3], b[j][2], b[j][3]);
                            }
                    }
                    continue;
                }
                const int left = len - (k0 + ch * 16);  // keys of the piece that exist
                if (left <= 0)
                    continue;
                // nothing behind the sequence's end takes part: not even as 0 times NaN
                const uint32_t in_lo = (2 * ti < left ? 0xFFFFu : 0u) | (2 * ti + 1 < left ? 0xFFFF0000u : 0u);
                const uint32_t in_hi = (2 * ti + 8 < left ? 0xFFFFu : 0u) | (2 * ti + 9 < left ? 0xFFFF0000u : 0u);
                uint32_t odd = 0;
#pragma unroll
                for (int i = 0; i < NC / 2; ++i) {
                    uint32_t b[4];
                    ldsm4_trans(b, at + (i >> 2) * half + v_row * 128 + ((((i & 3) * 2 + v_bit) ^ (v_row & 7)) << 4));
                    b[0] &= in_lo, b[1] &= in_hi, b[2] &= in_lo, b[3] &= in_hi;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t x = nonfinite2(b[j]);
                        odd |= x;
                        b[j] &= ~x;
                    }
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        mma_bf16_16816(o[r][2 * i], w[r][ch][0], w[r][ch][1], w[r][ch][2], w[r][ch][3], b[0], b[1]);
                        mma_bf16_16816(o[r][2 * i + 1], w[r][ch][0], w[r][ch][1], w[r][ch][2], w[r][ch][3], b[2], b[3]);
                    }
                }
                if (__any_sync(0xffffffffu, odd != 0)) {
                    // infinities and NaN among the values: they reach the rows that see their key alone
#pragma unroll 1
                    for (int k = 0; k < 16 && k < left; ++k) {
                        const int src = (lane & ~3) | ((k & 7) >> 1), bit = ch * 4 + (k >> 3) * 2 + (k & 1);
#pragma unroll
                        for (int r = 0; r < RW; ++r) {
                            const uint32_t p0 = __shfl_sync(0xffffffffu, k < 8 ? w[r][ch][0] : w[r][ch][2], src);
                            const uint32_t p1 = __shfl_sync(0xffffffffu, k < 8 ? w[r][ch][1] : w[r][ch][3], src);
                            const bool s0 = __shfl_sync(0xffffffffu, see[r][0], src) >> bit & 1, s1 = __shfl_sync(0xffffffffu, see[r][1], src) >> bit & 1;
                            const float w0 = k & 1 ? bf16hi_f32(p0) : bf16lo_f32(p0), w1 = k & 1 ? bf16hi_f32(p1) : bf16lo_f32(p1);
#pragma unroll
                            for (int i = 0; i < NC; ++i) {
                                uint32_t v;
                                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at + (i >> 3) * half + k * 128 + (((i & 7) ^ (k & 7)) << 4) + ti * 4) : "memory");
                                const uint32_t x = nonfinite2(v);
                                if (x & 0xFFFFu) {
                                    if (s0) o[r][i][0] += w0 * bf16lo_f32(v);
                                    if (s1) o[r][i][2] += w1 * bf16lo_f32(v);
                                }
                                if (x >> 16) {
                                    if (s0) o[r][i][1] += w0 * bf16hi_f32(v);
                                    if (s1) o[r][i][3] += w1 * bf16hi_f32(v);
                                }
                            }
                        }
                    }
                }
            }
            ++taken;
            __syncwarp();
            load();
        }

        // ---- the segment's end: the warps' parts of each row joined, some columns at a time
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[r][h] += __shfl_xor_sync(0xffffffffu, l[r][h], 1);
                l[r][h] += __shfl_xor_sync(0xffffffffu, l[r][h], 2);
                if (ti == 0)
                    *reinterpret_cast<float2*>(ml + (warp * ROWS + r * 16 + h * 8 + gi) * 2) = make_float2(m[r][h], l[r][h]);
            }
        named_bar_sync(1, kCtaThreads);
        float f[RW][2];
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < kWarps; ++k)
                    top = fmaxf(top, ml[(k * ROWS + r * 16 + h * 8 + gi) * 2]);
                f[r][h] = top == -INFINITY ? 1.f : attn_ex2(m[r][h] - top);
            }
        // a thread sums four columns of a row over the warps
        constexpr int kQuads = C::kCols / 4;
        const bool sums = threadIdx.x < ROWS * kQuads;
        const int sr = threadIdx.x / kQuads, sc = threadIdx.x % kQuads * 4;
        float top = -INFINITY, all = 0.f;
        if (sums) {
#pragma unroll
            for (int k = 0; k < kWarps; ++k)
                top = fmaxf(top, ml[(k * ROWS + sr) * 2]);
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int k = 0; k < kWarps; ++k)
                all = fmaf(attn_ex2(ml[(k * ROWS + sr) * 2] - ref), ml[(k * ROWS + sr) * 2 + 1], all);
        }
        const float inv = all == 0.f ? 0.f : 1.f / all;
        const bool whole = g.t0 == 0 && g.t1 == g.nt;
        float* part = p.parts + (int64_t)(g.t0 > 0 ? 2 * blockIdx.x : 2 * blockIdx.x + 1) * (ROWS * (HD + 2));
        const int row = g.rt * ROWS + sr;
        uint16_t* out = p.o + ((int64_t)(q.r0 + p.token_of(row)) * p.n_q + g.h * p.group + p.head_of(row)) * HD;
        if (sums && !whole && sc == 0 && row < n_rows)
            __stcg(reinterpret_cast<float2*>(part + ROWS * HD + 2 * sr), make_float2(top, all));
        auto finish = [&](int c0, const float* from) {
            if (!sums || row >= n_rows)
                return;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(from + (k * ROWS + sr) * C::kStride + sc);
                a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
            }
            if (whole)
                *reinterpret_cast<uint2*>(out + c0 + sc) = bf16x4(make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv));
            else
                __stcg(reinterpret_cast<float4*>(part + ((c0 + sc) / 4 * ROWS + sr) * 4), a);
        };
        // behind the CTA's last tile the rings are free and take all columns at once: one barrier in the place
        // of two of each kCols
        const bool last = u >= u1;
        constexpr int kRound = kWarps * ROWS * C::kStride;  // floats
        static_assert(HD / C::kCols * kRound * 4 <= kWarps * NS * C::kSlotBytes, "all columns in the rings");
        float* rings = reinterpret_cast<float*>(smem + C::ring(p.B));
#pragma unroll
        for (int c0 = 0; c0 < HD; c0 += C::kCols) {
            if (c0 > 0 && !last)
                named_bar_sync(1, kCtaThreads);  // the last columns have been read
            float* round = last ? rings + c0 / C::kCols * kRound : outbuf;
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                float* to = round + (warp * ROWS + r * 16 + gi) * C::kStride + ti * 2;
#pragma unroll
                for (int i = 0; i < C::kCols / 8; ++i) {
                    const float* v = o[r][c0 / 8 + i];
                    *reinterpret_cast<float2*>(to + i * 8) = make_float2(v[0] * f[r][0], v[1] * f[r][0]);
                    *reinterpret_cast<float2*>(to + 8 * C::kStride + i * 8) = make_float2(v[2] * f[r][1], v[3] * f[r][1]);
                }
            }
            if (!last) {
                named_bar_sync(1, kCtaThreads);
                finish(c0, round);
            }
        }
        if (last) {
            named_bar_sync(1, kCtaThreads);
#pragma unroll 2
            for (int c0 = 0; c0 < HD; c0 += C::kCols)
                finish(c0, rings + c0 / C::kCols * kRound);
        }
        if (threadIdx.x == 0)
            flags[2] = flags[0];
        named_bar_sync(1, kCtaThreads);  // the buffers may be written again; the part is written
        if (flags[2])                    // one answer for all warps
            break;
        if (!whole) {
            SplitItem& s = split[g.t0 > 0 ? 0 : 1];
            s = SplitItem{q, g.h, g.rt * ROWS, min(ROWS, n_rows - g.rt * ROWS), shares.cta_of(g.first), shares.cta_of(g.first + g.nt - 1)};
            if (threadIdx.x == 0)  // the barrier above and this release cover every thread's part
                part_written(p, s);
        }
    }
    for (int i = 0; i < 2; ++i)
        if (split[i].c0 <= split[i].c1)
            join_slice<ROWS, HD, kCtaThreads>(p, split[i], flags);
    // no copy may be in flight when the CTA leaves (after a wait that gave up)
    for (; taken < issued; ++taken)
        mbar_wait_bounded(&full[taken % NS], (taken / NS) & 1, p.limit_ns);
}

template <int HD, int RW>
cudaError_t launch(const AttnParams& p, const CUtensorMap& map, cudaStream_t stream)
{
    static_assert(Cfg<HD, RW>::smem(kMaxAttnSeqs) <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(tree_attn_warp_kernel<HD, RW>, (int)Cfg<HD, RW>::smem(kMaxAttnSeqs), done);
    if (e != cudaSuccess)
        return e;
    return launch_coop(tree_attn_warp_kernel<HD, RW>, dim3(device_sms()), dim3(kCtaThreads), Cfg<HD, RW>::smem(p.B), stream, p, map);
}

}  // namespace

int attn_warp_box(int head_dim, int page_size) { return head_dim == 256 ? 16 : page_size < 32 ? page_size : 32; }

cudaError_t launch_attn_warp(const AttnParams& p, int rows, const CUtensorMap& map, cudaStream_t stream)
{
    if (p.c.head_dim == 64)
        return rows == 16 ? launch<64, 1>(p, map, stream) : launch<64, 2>(p, map, stream);
    if (p.c.head_dim == 128)
        return rows == 16 ? launch<128, 1>(p, map, stream) : launch<128, 2>(p, map, stream);
    return launch<256, 1>(p, map, stream);
}

}  // namespace tfq
