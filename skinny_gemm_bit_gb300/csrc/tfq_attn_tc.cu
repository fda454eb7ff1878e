// Attention of many query rows: tcgen05 MMAs with scores, weights and output in tensor memory.
//
// More than some 32 query rows to a key/value head (a tree of drafts times the heads that share
// the keys) make enough arithmetic that the warp MMAs fall behind the cache's bytes. Here a CTA
// (one an SM) has a producer warp (TMA, a ring of K and V tiles), an MMA thread, and two groups
// of four softmax warps, a thread a query row, so that a row's maximum and sum need no shuffle:
//
//   S[w] = Q K^T          128 rows x KT keys, both operands in shared memory
//   p = 2^(S - m)         the row's thread, S and P in tensor memory (P over S, as bf16)
//   O[w] += P V           A from tensor memory, V as it lies in the cache (N-major)
//
// Each group has two score buffers: the scores of its next tile are formed while it works on this
// one's weights, so neither it nor the tensor cores wait for the other's latency. Trees of 64 rows
// by 8 heads to each of 4 key/value heads of 128, over 8 x 16,001 tokens: 125 us, 1080 TFLOP/s, against 206
// with one buffer and 128-key tiles, where a group spent 2600 of 6600 cycles a tile waiting. What
// is left is the softmax's own work and Q K^T at 64 keys, which reads 128 rows of queries from
// shared memory for each 64 of keys (some 67 cycles a 128 x 64 x 16 step). Up to 128 query rows (PAIR false) both
// groups have the same rows and every other tile, and their outputs are joined at the end; that is
// bound by the cache's bytes. Above (PAIR true) each group has 128 rows of its own and both read
// every tile, so a tile is fetched once for 256 rows. Tiles are 64 keys: two buffers of them a group
// and the output fill the tensor memory (4 * 64 + 2 * 128 columns).
//
// The reference m of a row moves only when its maximum has grown by more than 2^8: until then
// the weights stay below 256 and the sums are exact enough, and the output in tensor memory
// needs no rescaling; when it does, the group first waits for its last product with V.
#include "tfq_attn.cuh"

namespace tfq {
namespace {

constexpr int kTcThreads = 384;  // eight softmax warps, the producer, an MMA warp for each group, one idle
// registers: 168 a thread at launch; the last four warps give 96 of theirs to the softmax warps'
constexpr int kSoftRegs = 216, kOtherRegs = 72;
static_assert(kSoftRegs * 256 + kOtherRegs * 128 <= 168 * kTcThreads, "no more registers than the launch has");
constexpr int kSoftThreads = 256;
constexpr int kMaxSlots = 12;
constexpr int KT = 64;                            // keys of a tile
constexpr uint32_t kTmemCols = 512, kOCol = 256;  // S[w][buffer] at 128 w + 64 buffer, O[w] at 256 + 128 w
constexpr float kGrow = 8.f;

// offsets in shared memory
constexpr int kTcFull = 0, kTcEmpty = 128, kTcSFull = 256, kTcPReady = 288, kTcODone = 320, kTcQReady = 352, kTcOFull = 360, kTcFin = 368;
constexpr int kTcTmem = 384, kTcFlags = 400 /* [0] abort [2] abort as of a segment's end */, kTcOdd = 416;
constexpr int kTcMl = 1024;  // [2][128] (m, l)
constexpr int kTcSched = 3 * 1024;
static_assert(kMaxSlots * 8 <= 128, "slots");

template <int HD, bool PAIR>
struct TcCfg {
    static constexpr int ROWS = PAIR ? 256 : 128;
    static constexpr int kSlotBytes = KT * HD * 2;
    static constexpr int kQBytes = ROWS * HD * 2 < 32768 ? 32768 : ROWS * HD * 2;  // also the groups' exchange, 2 x 16 KB
    static constexpr size_t q_off(int B) { return (kTcSched + schedule_bytes(B) + 1023) / 1024 * 1024; }
    static constexpr int slots(int B)
    {
        const size_t n = (227 * 1024 - 1024 - q_off(B) - kQBytes) / kSlotBytes;
        return n < kMaxSlots ? (int)n : kMaxSlots;
    }
    static constexpr size_t smem(int B) { return 1024 + q_off(B) + kQBytes + (size_t)slots(B) * kSlotBytes; }
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Waits for the thread's loads; the operands keep the uses of r behind it.
__device__ __forceinline__ void tc_wait_ld(uint32_t* r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 columns of the thread's tensor-memory lane; the values are there after tc_wait_ld
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* a)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 :: "r"(addr), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7]),
                    "r"(a[8]), "r"(a[9]), "r"(a[10]), "r"(a[11]), "r"(a[12]), "r"(a[13]), "r"(a[14]), "r"(a[15]),
                    "r"(a[16]), "r"(a[17]), "r"(a[18]), "r"(a[19]), "r"(a[20]), "r"(a[21]), "r"(a[22]), "r"(a[23]),
                    "r"(a[24]), "r"(a[25]), "r"(a[26]), "r"(a[27]), "r"(a[28]), "r"(a[29]), "r"(a[30]), "r"(a[31])
                 : "memory");
}

// The MMA warp runs as a whole, so that descriptors stay in uniform registers (issued from a
// one-lane branch, an MMA took 80 cycles to hand over); `one` is true in the lane that issues.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}

__device__ __forceinline__ void tc_commit(uint64_t* bar, bool one)
{
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
                 " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)), "r"((int)one) : "memory");
}

// D (tensor memory) (+)= A B, A and B in shared memory / A in tensor memory
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, bool one)
{
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((int)add), "r"((int)one) : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, bool one)
{
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((int)add), "r"((int)one) : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: start, the step between blocks of 64
// elements along a contiguous N (lbo; unused for K-major), the step between groups of 8 rows (sbo)
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: fp32 accumulator, bf16 A (K-major) and B, M = 128
__host__ __device__ constexpr uint32_t instr_desc(int n, bool b_n_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(0), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ bool nonfinite16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

// Infinities and NaN among the block's values were taken out of the product with V: what they add
// to columns c0 .. c0 + 31 of a row that sees their tokens. Rare, so the scores are formed anew.
template <int HD>
__device__ __forceinline__ void add_odd(const AttnParams& p, const SeqRows& q, int head, int row, uint64_t odd, uint64_t mask,
                                        float sc, float sign, float ref, int c0, float (&acc)[32])
{
    const uint16_t* qr = p.q + (q.r0 + p.token_of(row)) * p.ldq + (int64_t)(head * p.group + row % p.group) * HD;
    for (odd &= mask; odd != 0; odd &= odd - 1) {
        const int tok = q.base + __ffsll((long long)odd) - 1;
        const int page = p.c.table[(int64_t)q.slot * p.c.max_pages + (tok >> p.c.page_shift)];
        if (page < 0 || page >= p.c.n_pages)
            continue;
        const int off = tok & (p.c.page_size - 1);
        const uint16_t* k = p.c.data + (p.c.row_of(p.layer, 0, page, head) + off) * HD;
        const uint16_t* v = p.c.data + (p.c.row_of(p.layer, 1, page, head) + off) * HD;
        float s = 0.f;
        for (int d = 0; d < HD; ++d)
            s = fmaf(__uint_as_float((uint32_t)qr[d] << 16), __uint_as_float((uint32_t)k[d] << 16), s);
        const float w = attn_ex2(fmaf(s * sign, sc, -ref));
#pragma unroll
        for (int d = 0; d < 32; ++d)
            if (nonfinite16(v[c0 + d]))
                acc[d] += w * __uint_as_float((uint32_t)v[c0 + d] << 16);
    }
}

template <int HD, bool PAIR>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map, uint32_t slots, int q_off)
{
    using C = TcCfg<HD, PAIR>;
    constexpr int ROWS = C::ROWS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kTcFull);
    uint64_t* empty = reinterpret_cast<uint64_t*>(smem + kTcEmpty);
    // [2 w + buffer]: scores there; weights there; the product with V done
    uint64_t* s_full = reinterpret_cast<uint64_t*>(smem + kTcSFull);
    uint64_t* p_ready = reinterpret_cast<uint64_t*>(smem + kTcPReady);
    uint64_t* o_done = reinterpret_cast<uint64_t*>(smem + kTcODone);
    uint64_t* q_ready = reinterpret_cast<uint64_t*>(smem + kTcQReady);
    uint64_t* o_full = reinterpret_cast<uint64_t*>(smem + kTcOFull);
    uint64_t* fin = reinterpret_cast<uint64_t*>(smem + kTcFin);
    volatile int* flags = reinterpret_cast<volatile int*>(smem + kTcFlags);
    unsigned* odd = reinterpret_cast<unsigned*>(smem + kTcOdd);
    float* ml = reinterpret_cast<float*>(smem + kTcMl);
    uint8_t* qbuf = smem + q_off;
    uint8_t* ring = qbuf + C::kQBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < slots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], PAIR ? 2 : 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&o_done[i], 1);
        }
        mbar_init(q_ready, 8);
        mbar_init(o_full, 2);
        mbar_init(fin, 2);
        flags[0] = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem + kTcTmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    Shares<ROWS, KT, 1, 0> shares(p, smem + kTcSched);
    tc_fence_before();
    shares.build();  // its barriers publish the tensor-memory address as well
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kTcTmem);
    const int u0 = shares.start_of(blockIdx.x), u1 = shares.start_of(blockIdx.x + 1);
    // Slots: one ring for both groups, or half of them for each. Every use of a slot is waited for, in
    // order, by each MMA warp that its ring serves: a wait can then not take the phase before last
    // for the one it is after.
    const uint32_t ring_slots = PAIR ? slots : slots / 2;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) {
            // ---- producer: a lane a box (64 columns of one page's rows of the tile); K then V of each tile
            const int box = min(p.c.page_size, KT), pieces = KT / box;
            const int z = lane / pieces, piece = lane % pieces;
            const bool active = lane < pieces * (HD / 64);
            uint32_t next_slot[2] = {0, 0}, pass[2] = {0, 0};
            bool gone = false;
            for (int u = u0; u < u1 && !gone;) {
                const Segment g = shares.segment(u, u1);
                u += g.units;
                const SeqRows& q = g.q;
                const int32_t* table = p.c.table + (int64_t)q.slot * p.c.max_pages;
                const int len = q.len();
                auto page_at = [&](int t) {
                    const int row = t * KT + piece * box;
                    return active && t < g.t1 && row < len ? __ldcg(table + (row >> p.c.page_shift)) : -1;
                };
                int page = page_at(g.t0);
                for (int t = g.t0; t < g.t1 && !gone; ++t) {
                    const int next = page_at(t + 1);
                    const int row = t * KT + piece * box;
                    const bool in = active && row < len, good = page >= 0 && page < p.c.n_pages;
                    if (in && !good)
                        record_status(p.status, TF_E_INVALID_ARG);
                    const int r = PAIR ? 0 : (t - g.t0) & 1;
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t slot = r * ring_slots + next_slot[r];
                        const bool ok = pass[r] == 0 || attn_wait(&empty[slot], (pass[r] - 1) & 1, flags, p.status, p.limit_ns);
                        if (!__all_sync(0xffffffffu, ok)) {
                            gone = true;
                            break;
                        }
                        if (lane == 0)
                            mbar_arrive_expect_tx(&full[slot], C::kSlotBytes);
                        __syncwarp();
                        if (active) {
                            const int y = in && good ? (int)p.c.row_of(p.layer, kv, page, g.h) + (row & (p.c.page_size - 1)) : p.total_rows;
                            tma_box(smem_u32(ring + (size_t)slot * C::kSlotBytes + z * KT * 128 + piece * box * 128), &map, y, z, &full[slot]);
                        }
                        if (++next_slot[r] == ring_slots) {
                            next_slot[r] = 0;
                            ++pass[r];
                        }
                    }
                    page = next;
                }
            }
            if (gone)  // no copy may be in flight when the CTA leaves: each slot's last one
                for (int r = 0; r < (PAIR ? 1 : 2); ++r)
                    for (uint32_t s = 0; s < ring_slots; ++s) {
                        const uint32_t uses = pass[r] + (s < next_slot[r] ? 1 : 0);
                        if (uses > 0)
                            mbar_wait_bounded(&full[r * ring_slots + s], (uses - 1) & 1, p.limit_ns);
                    }
        } else if (warp < 11) {
            // ---- an MMA warp: group w's scores and its products with V (one warp for both groups spent
            // 1340 cycles a step on its waits, one after the other, for 640 of MMAs)
            const int w = warp - 9;
            const bool one = elect_one();
            constexpr uint32_t kIdS = instr_desc(KT, false), kIdO = instr_desc(HD, true);
            const uint32_t first_slot = PAIR ? 0 : w * ring_slots;
            const uint32_t ra = smem_u32(ring) + first_slot * C::kSlotBytes;
            const uint64_t ad = smem_desc(smem_u32(qbuf) + (PAIR ? w * (128 * HD * 2) : 0), 16, 1024);
            full += first_slot;
            empty += first_slot;
            // the ring's slots of the next K and the next V tile: every second one
            uint32_t k_slot = 0, k_phase = 0, v_slot = 1, v_phase = 0, p_phase = 0 /* a bit a buffer */, seg = 0;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                return __all_sync(0xffffffffu, attn_wait(bar, parity, flags, p.status, p.limit_ns)) != 0;
            };
            auto forward = [&](uint32_t& slot, uint32_t& phase) {
                slot += 2;
                if (slot >= ring_slots) {
                    slot -= ring_slots;
                    phase ^= 1;
                }
            };
            auto scores = [&](int buf) {
                if (!wait(&full[k_slot], k_phase))
                    return false;
                const uint64_t bd = smem_desc(ra + k_slot * C::kSlotBytes, 16, 1024);
    #pragma unroll
                for (int ks = 0; ks < HD / 16; ++ks)  // 32 bytes on within 64 columns, then the next 64
                    tc_mma_ss(tmem + 64 * (2 * w + buf), ad + (((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4),
                              bd + (((ks >> 2) * (KT * 128) + (ks & 3) * 32) >> 4), kIdS, ks > 0, one);
                tc_commit(&s_full[2 * w + buf], one);
                tc_commit(&empty[k_slot], one);
                forward(k_slot, k_phase);
                return true;
            };
            bool ok = true;
            for (int u = u0; u < u1 && ok;) {
                const Segment g = shares.segment(u, u1);
                u += g.units;
                if (g.t0 == g.t1)
                    continue;
                const int n = PAIR ? g.t1 - g.t0 : (g.t1 - g.t0 + 1 - w) / 2;  // the group's tiles
                ok = wait(q_ready, seg & 1);
                if (!ok)
                    break;
                tc_fence_after();
                for (int k = 0; k < 2 && k < n && ok; ++k)
                    ok = scores(k);
                for (int k = 0; k < n && ok; ++k) {
                    const int buf = k & 1;
                    ok = wait(&p_ready[2 * w + buf], p_phase >> buf & 1) && wait(&full[v_slot], v_phase);
                    if (!ok)
                        break;
                    p_phase ^= 1u << buf;
                    tc_fence_after();
                    const uint64_t bd = smem_desc(ra + v_slot * C::kSlotBytes, KT * 128, 1024);
    #pragma unroll
                    for (int ks = 0; ks < KT / 16; ++ks)
                        tc_mma_ts(tmem + kOCol + 128 * w, tmem + 64 * (2 * w + buf) + 8 * ks, bd + (ks * 2048 >> 4), kIdO, k > 0 || ks > 0, one);
                    tc_commit(&o_done[2 * w + buf], one);
                    tc_commit(&empty[v_slot], one);
                    forward(v_slot, v_phase);
                    if (k + 2 < n)
                        ok = scores(buf);
                }
                if (ok)
                    tc_commit(o_full, one);
                ++seg;
            }
            // no MMA may be under way when the tensor memory is given back
            tc_commit(fin, one);
            mbar_wait_bounded(fin, 0, p.limit_ns);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ---- softmax: group w, a thread a row
        const int w = warp >> 2, wt = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_at = tmem + lanes + kOCol + 128 * w;
        const float sign = p.scale_log2 < 0.f ? -1.f : 1.f;  // a negative scale goes into Q
        const float sc = fmaxf(fabsf(p.scale_log2), 1e-37f);
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        uint32_t phase = 0 /* a bit a buffer */, seg = 0;
        SplitItem split[2];  // the item that the CTA continues, the one that it starts
        split[0].c0 = split[1].c0 = 1;
        split[0].c1 = split[1].c1 = 0;
        const uint32_t first_slot = PAIR ? 0 : w * ring_slots;
        uint32_t tiles = 0;  // the group's tiles so far
        for (int u = u0; u < u1;) {
            const Segment g = shares.segment(u, u1);
            u += g.units;
            if (g.t0 == g.t1)
                continue;
            const SeqRows& q = g.q;
            const int len = q.len(), n_rows = q.rows * p.group;
            // the item's queries, swizzled as the tiles are; a thread loads eight pieces before it stores one
            constexpr int kRowsAtOnce = kSoftThreads / (HD / 8);  // rows that the threads hold a piece each of
            const int qc = threadIdx.x % (HD / 8);
#pragma unroll 1
            for (int r0 = threadIdx.x / (HD / 8); r0 < ROWS; r0 += 8 * kRowsAtOnce) {
                uint4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = g.rt * ROWS + r0 + i * kRowsAtOnce;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (row < n_rows)
                        v[i] = __ldcg(reinterpret_cast<const uint4*>(p.q + (q.r0 + p.token_of(row)) * p.ldq +
                                                                     (int64_t)(g.h * p.group + p.head_of(row)) * HD + qc * 8));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = r0 + i * kRowsAtOnce;
                    *reinterpret_cast<uint4*>(qbuf + (r >> 7) * (128 * HD * 2) + (qc >> 3) * (128 * 128) + (r & 127) * 128 + (((qc & 7) ^ (r & 7)) << 4)) =
                        make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
                }
            }
            if (threadIdx.x == 0)
                odd[0] = odd[1] = 0;
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_ready);
            const int row = g.rt * ROWS + (PAIR ? w * 128 : 0) + wt;
            const bool valid = row < n_rows, busy = __any_sync(0xffffffffu, valid);
            uint64_t mask = 0;
            if (valid) {
                const int t = p.token_of(row);
                mask = block_mask(p, q, t);
            }
            float m = -INFINITY, l = 0.f;  // the reference, in score units, and the sum against it
            bool had = false, ok = true;
            int buf = 0;
            for (int t = g.t0 + (PAIR ? 0 : w); t < g.t1; t += PAIR ? 1 : 2, buf ^= 1) {
                ok = __all_sync(0xffffffffu, attn_wait(&s_full[2 * w + buf], phase >> buf & 1, flags, p.status, p.limit_ns));
                if (!ok)
                    break;
                const uint32_t s_at = tmem + lanes + 128 * w + 64 * buf;
                tc_fence_after();
                const int k0 = t * KT;
                const bool edge = k0 + KT > q.base;
                if (edge) {
                    // values behind the sequence's end become zeros, and infinities and NaN among the
                    // block's own are noted and taken out: a row that does not see them may not meet
                    // them, not even as 0 times NaN. (Of a pair each group does it: what the other has
                    // done it finds done, and its own product follows its own pass.)
                    const uint32_t pos = 2 * tiles + 1;
                    ok = __all_sync(0xffffffffu, attn_wait(&full[first_slot + pos % ring_slots], (pos / ring_slots) & 1, flags, p.status, p.limit_ns));
                    if (!ok)
                        break;
                    const int tok = k0 + wt % KT;
                    if (tok >= q.base) {
                        // two threads a row; each starts at a piece of its own, for the banks' sake
                        uint8_t* v = ring + (size_t)(first_slot + pos % ring_slots) * C::kSlotBytes + wt % KT * 128;
                        bool bad = false;
#pragma unroll 4
                        for (int c = wt / KT * (HD / 16); c < (wt / KT + 1) * (HD / 16); ++c) {
                            uint4* at = reinterpret_cast<uint4*>(v + (c >> 3) * (KT * 128) + ((c + wt) & 7) * 16);
                            uint32_t x[4];
                            *reinterpret_cast<uint4*>(x) = *at;
                            for (int j = 0; j < 4; ++j) {
                                if (tok >= len) {
                                    x[j] = 0;
                                    continue;
                                }
                                const bool lo = nonfinite16(x[j]), hi = nonfinite16(x[j] >> 16);
                                bad |= lo | hi;
                                x[j] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
                            }
                            *at = *reinterpret_cast<uint4*>(x);
                        }
                        if (bad)
                            atomicOr(&odd[(tok - q.base) >> 5], 1u << ((tok - q.base) & 31));
                    }
                    fence_async_smem();
                }
                if (busy) {
                    uint32_t s[KT];
                    auto read = [&]() {
                        tc_ld32(s_at, s);
                        tc_ld32(s_at + 32, s + 32);
                        tc_wait_ld(s);
                        tc_wait_ld(s + 32);
                        if (edge) {
                            const uint64_t see = tile_mask(mask, k0 - q.base);
#pragma unroll
                            for (int c = 0; c < KT; ++c)
                                s[c] = see >> c & 1 ? s[c] : 0xFF800000u;  // -inf
                        }
                    };
                    auto largest = [&]() {
                        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < KT; ++c)
                            x[c & 3] = fmaxf(x[c & 3], __uint_as_float(s[c]));
                        return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                    };
                    // the weights of the tile against m, in place of the scores, and their sum. Rounded to bf16
                    // they add 2^-8 of sum p |v| at most; 64-row trees over 16,001 tokens: 0.0023 of the output's
                    // norm against 64 bits, 0.0017 of it the output's own rounding
                    auto weigh = [&]() {
                        const float ref = m == -INFINITY ? 0.f : m * sc;
                        const float2 sc2 = make_float2(sc, sc), ref2 = make_float2(-ref, -ref);
                        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < KT; c += 2) {
                            float2 e = __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, ref2);
                            e.x = attn_ex2(e.x);
                            e.y = attn_ex2(e.y);
                            sum[c >> 1 & 1] = __fadd2_rn(sum[c >> 1 & 1], e);
                            s[c / 2] = f32x2_to_bf16x2(e.x, e.y);  // weights in V's type, as the product takes them: up to 2^-8 of each
                        }
                        const float2 both = __fadd2_rn(sum[0], sum[1]);
                        return both.x + both.y;
                    };
                    read();
                    const float top = largest();
                    if (!had)
                        m = top;
                    // the last reference serves nearly always, so the weights do not wait for the
                    // tile's maximum; when it has grown they are formed again
                    float added = weigh();
                    const bool grown = had && (top - m) * sc > kGrow;
                    if (__any_sync(0xffffffffu, grown)) {
                        // the last product with V: the other buffer's, whose phase has moved on since
                        ok = __all_sync(0xffffffffu, attn_wait(&o_done[2 * w + (buf ^ 1)], (phase >> (buf ^ 1) & 1) ^ 1, flags, p.status, p.limit_ns));
                        tc_fence_after();
                        const float f = grown ? attn_ex2((m - top) * sc) : 1.f;
                        if (grown)
                            m = top;
                        l *= f;
#pragma unroll 1
                        for (int c = 0; c < HD; c += 32) {
                            uint32_t o[32];
                            tc_ld32(o_at + c, o);
                            tc_wait_ld(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tc_st32(o_at + c, o);
                        }
                        read();
                        added = weigh();
                    }
                    l += added;
                    tc_st32(s_at, s);
                    tc_wait_st();
                }
                had = true;
                ++tiles;
                phase ^= 1u << buf;
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_ready[2 * w + buf]);
            }
            ok = ok && __all_sync(0xffffffffu, attn_wait(o_full, seg & 1, flags, p.status, p.limit_ns));
            tc_fence_after();

            // ---- the segment's end
            const bool whole = g.t0 == 0 && g.t1 == g.nt;
            float* part = p.parts + (int64_t)(g.t0 > 0 ? 2 * blockIdx.x : 2 * blockIdx.x + 1) * (ROWS * (HD + 2));
            const int prow = (PAIR ? w * 128 : 0) + wt;  // the row within the tile
            float mine = m == -INFINITY ? -INFINITY : m * sc, top = mine, all = l;
            if (!PAIR) {
                ml[(w * 128 + wt) * 2] = mine;
                ml[(w * 128 + wt) * 2 + 1] = l;
            }
            named_bar_sync(1, kSoftThreads);  // also: nobody reads Q or marks odd values any more
            if (!PAIR) {
                const float other = ml[((w ^ 1) * 128 + wt) * 2];
                top = fmaxf(mine, other);
                const float r = top == -INFINITY ? 0.f : top;
                all = l * attn_ex2(mine - r) + ml[((w ^ 1) * 128 + wt) * 2 + 1] * attn_ex2(other - r);
            }
            const float ref = top == -INFINITY ? 0.f : top, scale = PAIR ? 1.f : attn_ex2(mine - ref);
            const float inv = all == 0.f ? 0.f : 1.f / all;
            const uint64_t odd_bits = (uint64_t)odd[1] << 32 | odd[0];
            auto put = [&](float (&a)[32], int c0) {  // columns c0 .. c0 + 31 of the row, unscaled
                if (!valid)
                    return;
                if (odd_bits != 0)
                    add_odd<HD>(p, q, g.h, row, odd_bits, mask, sc, sign, ref, c0, a);
                if (whole) {
                    uint4* o = reinterpret_cast<uint4*>(p.o + ((int64_t)(q.r0 + p.token_of(row)) * p.n_q + g.h * p.group + p.head_of(row)) * HD + c0);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = make_uint4(f32x2_to_bf16x2(a[8 * i] * inv, a[8 * i + 1] * inv), f32x2_to_bf16x2(a[8 * i + 2] * inv, a[8 * i + 3] * inv),
                                          f32x2_to_bf16x2(a[8 * i + 4] * inv, a[8 * i + 5] * inv), f32x2_to_bf16x2(a[8 * i + 6] * inv, a[8 * i + 7] * inv));
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        __stcg(reinterpret_cast<float4*>(part + ((c0 / 4 + i) * ROWS + prow) * 4), make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]));
                    if (c0 == 0)
                        __stcg(reinterpret_cast<float2*>(part + ROWS * HD + 2 * prow), make_float2(top, all));
                }
            };
            auto load = [&](int c0, float (&a)[32]) {
                uint32_t o[32];
                if (had) {  // the output was never written otherwise
                    tc_ld32(o_at + c0, o);
                    tc_wait_ld(o);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    a[i] = had ? __uint_as_float(o[i]) * scale : 0.f;
            };
            if (PAIR) {
                if (busy)
#pragma unroll 1
                    for (int c0 = 0; c0 < HD; c0 += 32) {
                        float a[32];
                        load(c0, a);
                        put(a, c0);
                    }
            } else {
                // group 0 finishes the first half of the columns, group 1 the second; the other half
                // goes over in the Q buffer, 32 columns at a time
                float* give = reinterpret_cast<float*>(qbuf) + (w ^ 1) * (32 * 128);
                const float* take = reinterpret_cast<const float*>(qbuf) + w * (32 * 128);
#pragma unroll 1
                for (int c = 0; c < HD / 2; c += 32) {
                    float a[32];
                    load((w ^ 1) * (HD / 2) + c, a);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        give[i * 128 + wt] = a[i];
                    named_bar_sync(1, kSoftThreads);
                    load(w * (HD / 2) + c, a);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        a[i] += take[i * 128 + wt];
                    put(a, w * (HD / 2) + c);
                    named_bar_sync(1, kSoftThreads);
                }
            }
            if (threadIdx.x == 0)
                flags[2] = flags[0];
            tc_fence_before();                // the output has been read
            named_bar_sync(1, kSoftThreads);  // the Q buffer may be written again; the part is written
            if (flags[2])                     // one answer for all warps
                break;
            if (!whole) {
                SplitItem& s = split[g.t0 > 0 ? 0 : 1];
                s = SplitItem{q, g.h, g.rt * ROWS, min(ROWS, n_rows - g.rt * ROWS), shares.cta_of(g.first), shares.cta_of(g.first + g.nt - 1)};
                if (threadIdx.x == 0)  // the barrier above and this release cover every thread's part
                    part_written(p, s);
            }
            ++seg;
        }
        for (int i = 0; i < 2; ++i)
            if (split[i].c0 <= split[i].c1)
                join_slice<ROWS, HD, kSoftThreads>(p, split[i], flags, qbuf);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int HD, bool PAIR>
constexpr int kPartBytes = TcCfg<HD, PAIR>::ROWS * HD * 4;  // of a part's output

template <int HD, bool PAIR>
cudaError_t launch(const AttnParams& p, const CUtensorMap& map, cudaStream_t stream)
{
    using C = TcCfg<HD, PAIR>;
    // join_many: fewer parts than ROWS * HD / 4 / kSoftThreads + 1, and a slice's rounding for each
    static_assert(C::kQBytes + C::slots(kMaxAttnSeqs) * C::kSlotBytes >= kPartBytes<HD, PAIR> + (kPartBytes<HD, PAIR> / 16 / kSoftThreads + 1) * (kSoftThreads * 4 + 16),
                  "the queries' and the ring's memory takes a slice of the parts");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(tree_attn_tc_kernel<HD, PAIR>, 227 * 1024, done);
    if (e != cudaSuccess)
        return e;
    return launch_coop(tree_attn_tc_kernel<HD, PAIR>, dim3(device_sms()), dim3(kTcThreads), C::smem(p.B), stream, p, map,
                       (uint32_t)C::slots(p.B), (int)C::q_off(p.B));
}

}  // namespace

int attn_tc_box(int page_size) { return page_size < KT ? page_size : KT; }

cudaError_t launch_attn_tc(const AttnParams& p, int rows, const CUtensorMap& map, cudaStream_t stream)
{
    if (p.c.head_dim == 64)
        return rows == 128 ? launch<64, false>(p, map, stream) : launch<64, true>(p, map, stream);
    return rows == 128 ? launch<128, false>(p, map, stream) : launch<128, true>(p, map, stream);
}

}  // namespace tfq
