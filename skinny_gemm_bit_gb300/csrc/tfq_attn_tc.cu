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
//
// Prompts (CAUSAL) have a limit in the place of a mask, and an item's key tiles end with its last row's. Over a bf16 cache
// an item is 128 rows and each group works for itself (DUAL), with a producer warp, an MMA warp and half the ring of its
// own, as two CTAs would (the runtime places one CTA with tcgen05 on an SM): while one begins or ends an item the
// other computes. One prompt of 8191 rows, 16 / 8 heads of 128: 225 us, 1220 TFLOP/s (pairs of 256 rows 270); 24 packed ones
// of up to 2047 rows 213 us (293): 3000 items of nine tiles on average, whose beginnings and ends still cost some three
// tiles each. An item's queries come by TMA as soon as the scores of the one before are formed (loaded and stored by the
// softmax threads they took 8000 cycles an item: 250 and 268 us). Over 8 bits a pair shares its tiles, since each is
// converted but once then: 1500 rows behind 14,001 tokens, 32 / 4 heads, 375 us, 970 TFLOP/s; apart 452.
//
// Over a cache of 8 bits (E8) the TMA brings the tiles as they are into a ring of their own, and four more warps turn
// them into fp16 in the ring that the MMAs read (exactly: fp16 has every e4m3 value), so the MMAs and the
// rest stay as they are; Q and the weights are fp16 too. The blocks' scales enter the scores and the weights, as in
// tfq_attn_warp.cu: with the products' own constants for each 16 keys they cost nothing an element. The
// converting warps also zero what lies behind a sequence's end and take out NaN. The 64-row trees above take 161 us so,
// where bf16 takes 124: shared memory carries a tile once more in and out, and the conversions share the softmax's
// issue slots (144 us with zeros in their place). Q in tensor memory, for which head_dim 64 has room, gained nothing.
#include "tfq_attn.cuh"

namespace tfq {
namespace {

// eight softmax warps, the producer, an MMA warp for each group, one idle; 8 bits: and four converting warps
constexpr int tc_threads(bool e8) { return e8 ? 512 : 384; }
// registers: 168 a thread at launch; the last four warps give 96 of theirs to the softmax warps'. 8 bits: 128 a thread
constexpr int kOtherRegs = 72, kConvertRegs = 80;
constexpr int soft_regs(bool e8) { return e8 ? 176 : 216; }
static_assert(soft_regs(false) * 256 + kOtherRegs * 128 <= 168 * tc_threads(false), "no more registers than the launch has");
static_assert(soft_regs(true) * 256 + (kOtherRegs + kConvertRegs) * 128 <= 128 * tc_threads(true), "no more registers than the launch has");
constexpr int kSoftThreads = 256;
constexpr int kConvertThreads = 128;              // that convert a tile together
constexpr float kHead = 7.f;  // fp16 weights reach 2^(kGrow + kHead) = 2^15
constexpr int kMaxSlots = 12;
constexpr int KT = kTcTile;                       // keys of a tile
constexpr uint32_t kTmemCols = 512, kOCol = 256;  // S[w][buffer] at 128 w + 64 buffer, O[w] at 256 + 128 w
constexpr float kGrow = 8.f;

// offsets in shared memory
constexpr int kTcFull = 0, kTcEmpty = 128, kTcSFull = 256, kTcPReady = 288, kTcODone = 320, kTcQReady = 352, kTcOFull = 368, kTcFin = 480, kTcQFree = 496;
constexpr int kTcTmem = 384, kTcFlags = 400 /* [0] abort [2 + w] abort as of a segment's end */, kTcOdd = 416;
// tokens taken out of V, bits from the item's first: [groups][8] words (trees: 2); 8 bits: [items][8], as the
// converting warps may be some items ahead
constexpr int kTcOdd8 = 512, kOddItems = 8;
constexpr int kOddTokens = 256;  // behind them no row of the item sees a token
constexpr int kTcFull8 = 768, kTcEmpty8 = 832, kTcScaleFull = 896;  // 8 bits: the ring of codes; the rings' tiles' scales
constexpr int kTcMl = 1024;  // [2][128] (m, l)
constexpr int kTcSched = 3 * 1024;
// 8 bits: the rows' factors of the scores; by ring, the last 8 tiles' 3 x [4] of their blocks: 2^ks, log2 vs, 1 / vs; by slot
// of codes and box, the words with K's and V's scales and their places in them
constexpr int kMaxCodeSlots = 8, kScaleTiles = 8;
constexpr int kTcFactor = 3 * 1024, kTcScales = 4 * 1024, kTcWords = kTcScales + 2 * kScaleTiles * 48, kTcSched8 = 6 * 1024;
static_assert(kTcWords + kMaxCodeSlots * 48 <= kTcSched8, "scales");
static_assert(kMaxSlots * 8 <= 128 && kMaxCodeSlots * 8 <= 64 && kTcScaleFull + 2 * kScaleTiles * 8 <= kTcMl && kTcOdd + 64 <= kTcFin && kTcQFree + 16 <= kTcOdd8 && kTcOdd8 + kOddItems * 32 <= kTcFull8, "slots");

template <int HD, bool PAIR, bool E8, bool DUAL>
struct TcCfg {
    static_assert(!E8 || !DUAL, "groups apart would convert every tile twice");
    static constexpr int ROWS = PAIR ? 256 : 128;
    static constexpr int kSlotBytes = KT * HD * 2;
    static constexpr int kCodeBytes = KT * HD;  // 8 bits: of a tile of codes
    // also the groups' exchange, 2 x 16 KB
    static constexpr int kQBytes = (DUAL ? 2 : 1) * ROWS * HD * 2 < 32768 ? 32768 : (DUAL ? 2 : 1) * ROWS * HD * 2;
    static constexpr size_t q_off(int B) { return ((E8 ? kTcSched8 : kTcSched) + schedule_bytes(B) + 1023) / 1024 * 1024; }
    static constexpr int slots(int B)
    {
        const size_t n = (227 * 1024 - 1024 - q_off(B) - kQBytes - (E8 ? 4 * kCodeBytes : 0)) / kSlotBytes;
        return (int)(E8 && n >= 8 ? 8 : n < kMaxSlots ? n : kMaxSlots) / (DUAL ? 2 : 1) * (DUAL ? 2 : 1);
    }
    // an even number: K's tiles lie in the even ones
    static constexpr int code_slots(int B)
    {
        const size_t n = (227 * 1024 - 1024 - q_off(B) - kQBytes - (size_t)slots(B) * kSlotBytes) / kCodeBytes / 2 * 2;
        return !E8 ? 0 : n < kMaxCodeSlots ? (int)n : kMaxCodeSlots;
    }
    static constexpr size_t smem(int B) { return 1024 + q_off(B) + kQBytes + (size_t)slots(B) * kSlotBytes + (size_t)code_slots(B) * kCodeBytes; }
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
// Instruction descriptor: fp32 accumulator, bf16 (or fp16) A (K-major) and B, M = 128
__host__ __device__ constexpr uint32_t instr_desc(int n, bool b_n_major, bool f16)
{
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(0), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// A box {64 columns, 1, heads of a group, tokens} of the queries: the 128 rows of an item, as they lie in a tile.
__device__ __forceinline__ void tma_queries(uint32_t dst, const CUtensorMap* map, int half, int head, int token, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(map), "r"(0), "r"(half), "r"(head), "r"(token), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ bool nonfinite16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Infinities and NaN among the values from token `from` on were taken out of the product with V: what they add
// to columns c0 .. c0 + 31 of a row that sees their tokens. Rare, so the scores are formed anew.
template <int HD, bool E8>
__device__ __forceinline__ void add_odd(const AttnParams& p, const SeqRows& q, int head, int row, int from, uint64_t odd, uint64_t mask,
                                        float sc, float sign, float ref, int c0, float (&acc)[32])
{
    const uint16_t* qr = p.q + (q.r0 + p.token_of(row)) * p.ldq + (int64_t)(head * p.group + row % p.group) * HD;
    for (odd &= mask; odd != 0; odd &= odd - 1) {
        const int tok = from + __ffsll((long long)odd) - 1;
        const int page = p.c.table[(int64_t)q.slot * p.c.max_pages + (tok >> p.c.page_shift)];
        if (page < 0 || page >= p.c.n_pages)
            continue;
        const int off = tok & (p.c.page_size - 1);
        if constexpr (E8) {  // e4m3 has no infinities
            const uint8_t* codes = p.c.codes() + (p.c.row_of(p.layer, 1, page, head) + off) * HD + c0;
#pragma unroll
            for (int d = 0; d < 32; ++d)
                if ((codes[d] & 0x7F) == 0x7F)
                    acc[d] = NAN;
            continue;
        }
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

// The last key tile of an item, and the shares, by kind of call
template <int ROWS, bool CAUSAL>
struct SharesOf {
    using type = Shares<ROWS, KT, 1, 0>;
};
template <int ROWS>
struct SharesOf<ROWS, true> {
    using type = PromptShares<ROWS, KT, ROWS == 128 ? 2 : 1>;
};

template <int HD, bool PAIR, bool E8, bool CAUSAL>
__global__ void __launch_bounds__(tc_threads(E8), 1)
    tree_attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap map, const __grid_constant__ CUtensorMap q_map,
                        uint32_t slots, uint32_t code_slots, int q_off)
{
    constexpr bool DUAL = CAUSAL && !PAIR;  // the groups apart
    using C = TcCfg<HD, PAIR, E8, DUAL>;
    constexpr int ROWS = C::ROWS;
    constexpr bool ALT = !PAIR && !DUAL;  // the groups take every other tile of the same rows
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
    [[maybe_unused]] uint64_t* q_free = reinterpret_cast<uint64_t*>(smem + kTcQFree);  // groups apart: the item's scores are all formed
    volatile int* flags = reinterpret_cast<volatile int*>(smem + kTcFlags);
    unsigned* odd = reinterpret_cast<unsigned*>(smem + kTcOdd);
    float* ml = reinterpret_cast<float*>(smem + kTcMl);
    uint8_t* qbuf = smem + q_off;
    // Groups apart: each has its queries and ring in one piece, which at the end takes a slice of the parts
    constexpr int kOwnQ = DUAL ? C::kQBytes / 2 : C::kQBytes;
    const uint32_t own_bytes = kOwnQ + slots / 2 * C::kSlotBytes;
    uint8_t* ring = qbuf + kOwnQ;
    // 8 bits: the ring of codes and its barriers, and where the scales lie
    [[maybe_unused]] uint8_t* code_ring = ring + (size_t)slots * C::kSlotBytes;
    [[maybe_unused]] uint64_t* full8 = reinterpret_cast<uint64_t*>(smem + kTcFull8);
    [[maybe_unused]] uint64_t* empty8 = reinterpret_cast<uint64_t*>(smem + kTcEmpty8);
    // [ring][tile % 8]. A tile's K is converted when the products of tiles after the eighth before it are done, so nobody
    // reads that one's scales any more
    [[maybe_unused]] uint64_t* scale_full = reinterpret_cast<uint64_t*>(smem + kTcScaleFull);
    [[maybe_unused]] float* factor = reinterpret_cast<float*>(smem + kTcFactor);
    [[maybe_unused]] float* scales = reinterpret_cast<float*>(smem + kTcScales);
    [[maybe_unused]] uint32_t* words = reinterpret_cast<uint32_t*>(smem + kTcWords);
    [[maybe_unused]] unsigned* odd8 = reinterpret_cast<unsigned*>(smem + kTcOdd8);
    const int box = min(p.c.page_size, KT), pieces = KT / box;  // boxes of a tile
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < slots; ++i) {
            mbar_init(&full[i], E8 ? kConvertThreads / 32 : 1);
            mbar_init(&empty[i], PAIR ? 2 : 1);
        }
        for (uint32_t i = 0; E8 && i < code_slots; ++i) {
            // each box's lane, and again in K's slots where it has fetched scales
            mbar_init(&full8[i], 1 + pieces + (i & 1 ? 0 : pieces));
            mbar_init(&empty8[i], kConvertThreads / 32);
        }
        for (int i = 0; E8 && i < 2 * kScaleTiles; ++i)
            mbar_init(&scale_full[i], 1);
        for (int i = 0; E8 && i < kOddItems * 8; ++i)
            odd8[i] = 0;
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {  // of each group; else the first alone counts
            mbar_init(&q_ready[i], DUAL ? (p.q_boxes ? 1 : 4) : 8);
            mbar_init(&q_free[i], 1);
            mbar_init(&o_full[i], DUAL ? 1 : 2);
            mbar_init(&fin[i], DUAL ? 1 : 2);
        }
        flags[0] = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem + kTcTmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    typename SharesOf<ROWS, CAUSAL>::type shares(p, smem + (E8 ? kTcSched8 : kTcSched));
    tc_fence_before();
    shares.build();  // its barriers publish the tensor-memory address as well
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + kTcTmem);
    // Slots: one ring for both groups, or half of them for each. Every use of a slot is waited for, in
    // order, by each MMA warp that its ring serves: a wait can then not take the phase before last
    // for the one it is after.
    const uint32_t ring_slots = PAIR ? slots : slots / 2;
    // a CTA's units, or a group's
    auto cta_of_group = [&](int w) { return DUAL ? 2 * blockIdx.x + w : blockIdx.x; };
    const int cta_u0 = DUAL ? 0 : shares.start_of(blockIdx.x), cta_u1 = DUAL ? 0 : shares.start_of(blockIdx.x + 1);
    auto first_unit = [&](int w) { return DUAL ? shares.start_of(cta_of_group(w)) : cta_u0; };
    auto end_unit = [&](int w) { return DUAL ? shares.start_of(cta_of_group(w) + 1) : cta_u1; };
    // slots are counted over both groups' rings
    auto to_group = [&](int w) {
        if (!DUAL)
            return;
        qbuf += w * own_bytes;
        ring += w * (own_bytes - ring_slots * C::kSlotBytes);
    };
    // The first token that not every row of an item sees
    auto hidden_from = [&](const Segment& g) { return g.q.base + (CAUSAL ? p.token_of(g.rt * ROWS) : 0); };

    if (E8 && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
        // ---- codes to fp16: a thread 16 codes of a row. Eight lanes take the same piece of eight rows, so that
        // neither their reads nor their writes meet in a bank
        const int ct = threadIdx.x & (kConvertThreads - 1);
        const int r8 = ct & 7, c = (ct >> 3) % (HD / 16), first_row = (ct >> 3) / (HD / 16) * 8 + r8;
        constexpr int kStep = kConvertThreads / (HD / 16);  // rows that the threads take at once
        uint32_t next_slot[2] = {0, 0}, pass[2] = {0, 0}, tiles[2] = {0, 0}, from = 0, from_phase = 0, seg = 0;
        bool gone = false;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, attn_wait(bar, parity, flags, p.status, p.limit_ns)) != 0;
        };
        for (int u = cta_u0; u < cta_u1 && !gone;) {
            const Segment g = shares.segment(u, cta_u1);
            u += g.units;
            if (g.t0 == g.t1)
                continue;
            const int hidden = hidden_from(g), len = g.q.len();
            unsigned* odd_bits = odd8 + seg % kOddItems * 8;
            for (int t = g.t0; t < g.t1 && !gone; ++t) {
                const int r = PAIR ? 0 : (t - g.t0) & 1, k0 = t * KT;
                const bool edge = k0 + KT > hidden;
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t slot = r * ring_slots + next_slot[r];
                    if (!wait(&full8[from], from_phase)) {
                        gone = true;
                        break;
                    }
                    constexpr int kTimes = KT / kStep;
                    const uint8_t* in = code_ring + (size_t)from * C::kCodeBytes;
                    uint4 v[kTimes];  // all under way at once, and while the slot is waited for
#pragma unroll
                    for (int i = 0; i < kTimes; ++i) {
                        const int row = first_row + i * kStep;
                        v[i] = *reinterpret_cast<const uint4*>(in + (HD == 64 ? row * 64 + ((c ^ (row >> 1 & 3)) << 4) : row * 128 + ((c ^ (row & 7)) << 4)));
                    }
                    if (pass[r] > 0 && !wait(&empty[slot], (pass[r] - 1) & 1)) {
                        gone = true;
                        break;
                    }
                    if (kv == 0 && ct < 32) {  // the tile's scales
                        if (ct < KT / 16) {
                            const uint32_t* w = words + (from * 4 + ct * 16 / box) * 3;
                            const uint32_t within = ct * 16 % box / 2;
                            const int ks = min(max((int)(w[0] >> ((w[2] & 0xFFu) + within) & 0xFFu), 127 - 32), 127 + 32);
                            const int vs = min(max((int)(w[1] >> ((w[2] >> 8) + within) & 0xFFu), 127 - 32), 127 + 32);
                            float* to = scales + (r * kScaleTiles + tiles[r] % kScaleTiles) * 12 + ct;
                            to[0] = __uint_as_float((uint32_t)ks << 23);
                            to[4] = (float)(vs - 127);
                            to[8] = __uint_as_float((uint32_t)(254 - vs) << 23);
                        }
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(&scale_full[r * kScaleTiles + tiles[r] % kScaleTiles]);
                        ++tiles[r];
                    }
                    if (edge && kv == 1) {
#pragma unroll
                        for (int i = 0; i < kTimes; ++i) {
                            const int tok = k0 + first_row + i * kStep;
                            uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                            bool bad = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (tok >= len)
                                    w[k] = 0;
                                const uint32_t nan = __vcmpeq4(w[k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                                if (tok >= hidden) {
                                    bad |= nan != 0;
                                    w[k] &= ~nan;
                                }
                            }
                            if (bad && tok - hidden < kOddTokens)
                                atomicOr(&odd_bits[(tok - hidden) >> 5], 1u << ((tok - hidden) & 31));
                            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    uint8_t* out = ring + (size_t)slot * C::kSlotBytes + (c >> 2) * (KT * 128) + first_row * 128;
#pragma unroll
                    for (int i = 0; i < kTimes; ++i) {  // kStep is a multiple of 8: the same swizzle every time
                        uint4 lo, hi;
                        e4m3x4_to_f16x2(v[i].x, lo.x, lo.y);
                        e4m3x4_to_f16x2(v[i].y, lo.z, lo.w);
                        e4m3x4_to_f16x2(v[i].z, hi.x, hi.y);
                        e4m3x4_to_f16x2(v[i].w, hi.z, hi.w);
                        *reinterpret_cast<uint4*>(out + i * (kStep * 128) + (((2 * c & 7) ^ r8) << 4)) = lo;
                        *reinterpret_cast<uint4*>(out + i * (kStep * 128) + (((2 * c & 7) + 1 ^ r8) << 4)) = hi;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&full[slot]);
                        mbar_arrive(&empty8[from]);
                    }
                    if (++next_slot[r] == ring_slots) {
                        next_slot[r] = 0;
                        ++pass[r];
                    }
                    if (++from == code_slots) {
                        from = 0;
                        from_phase ^= 1;
                    }
                }
            }
            ++seg;
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8 || (DUAL && warp == 11)) {
            // ---- producer: a lane a box (64 columns of one page's rows of the tile); K then V of each tile
            const int w = DUAL && warp == 11 ? 1 : 0, u0 = first_unit(w), u1 = end_unit(w);
            to_group(w);
            const int z = lane / pieces, piece = lane % pieces;
            const bool active = lane < pieces * (E8 ? 1 : HD / 64);
            uint32_t next_slot[2] = {0, 0}, pass[2] = {0, 0};
            [[maybe_unused]] uint32_t items = 0;
            bool gone = false;
            for (int u = u0; u < u1 && !gone;) {
                const Segment g = shares.segment(u, u1);
                u += g.units;
                const SeqRows& q = g.q;
                if (DUAL && p.q_boxes && g.t0 < g.t1) {
                    // the item's queries, while the group is still busy with the end of the one before
                    if (items > 0 && !__all_sync(0xffffffffu, attn_wait(&q_free[w], (items - 1) & 1, flags, p.status, p.limit_ns))) {
                        gone = true;
                        break;
                    }
                    ++items;
                    if (lane == 0)
                        mbar_arrive_expect_tx(&q_ready[w], 128 * HD * 2);
                    __syncwarp();
                    if (lane < HD / 64)
                        tma_queries(smem_u32(qbuf + lane * (128 * 128)), &q_map, lane, g.h * p.group, q.r0 + p.token_of(g.rt * 128), &q_ready[w]);
                }
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
                    const int r = DUAL ? w : PAIR || E8 ? 0 : (t - g.t0) & 1;
                    for (int kv = 0; kv < 2; ++kv) {
                        if constexpr (E8) {
                            const uint32_t slot = next_slot[0];
                            const bool ok = pass[0] == 0 || attn_wait(&empty8[slot], (pass[0] - 1) & 1, flags, p.status, p.limit_ns);
                            if (!__all_sync(0xffffffffu, ok)) {
                                gone = true;
                                break;
                            }
                            if (lane == 0)
                                mbar_arrive_expect_tx(&full8[slot], C::kCodeBytes);
                            __syncwarp();
                            if (active) {
                                const bool there = in && good;
                                const int y = there ? (int)p.c.row_of(p.layer, kv, page, g.h) + (row & (p.c.page_size - 1)) : p.total_rows;
                                tma_box(smem_u32(code_ring + (size_t)slot * C::kCodeBytes + piece * box * HD), &map, y, 0, &full8[slot]);
                                if (kv == 0) {
                                    // the tile's scales, as the aligned words that hold them
                                    uint32_t* w = words + (slot * 4 + piece) * 3;
                                    if (there) {
                                        const int64_t k = y >> 4, v = k + (((int64_t)p.c.n_pages * p.c.n_kv) << (p.c.page_shift - 4));
                                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(w)), "l"(p.c.scales + (k & ~3ll)) : "memory");
                                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(w + 1)), "l"(p.c.scales + (v & ~3ll)) : "memory");
                                        w[2] = (uint32_t)(k & 3) * 8 | (uint32_t)(v & 3) * 8 << 8;
                                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full8[slot])) : "memory");
                                    } else {
                                        w[0] = w[1] = 0x7F7F7F7Fu;
                                        w[2] = 0;
                                        mbar_arrive(&full8[slot]);
                                    }
                                }
                                mbar_arrive(&full8[slot]);
                            }
                            if (++next_slot[0] == code_slots) {
                                next_slot[0] = 0;
                                ++pass[0];
                            }
                            continue;
                        }
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
            if (DUAL && p.q_boxes && items > 0)  // no copy may be in flight when the CTA leaves
                mbar_wait_bounded(&q_ready[w], (items - 1) & 1, p.limit_ns);
            if (gone)  // each slot's last one
                for (int r = 0; r < (PAIR || E8 ? 1 : 2); ++r)
                    for (uint32_t s = 0; s < (E8 ? code_slots : ring_slots); ++s) {
                        const uint32_t uses = pass[r] + (s < next_slot[r] ? 1 : 0);
                        if (uses > 0)
                            mbar_wait_bounded(E8 ? &full8[s] : &full[r * ring_slots + s], (uses - 1) & 1, p.limit_ns);
                    }
        } else if (warp < 11) {
            // ---- an MMA warp: group w's scores and its products with V (one warp for both groups spent
            // 1340 cycles a step on its waits, one after the other, for 640 of MMAs)
            const int w = warp - 9, u0 = first_unit(w), u1 = end_unit(w);
            to_group(w);
            const bool one = elect_one();
            constexpr uint32_t kIdS = instr_desc(KT, false, E8), kIdO = instr_desc(HD, true, E8);
            const uint32_t first_slot = PAIR ? 0 : w * ring_slots;
            const uint32_t ra = smem_u32(ring) + first_slot * C::kSlotBytes;
            const uint64_t ad = smem_desc(smem_u32(qbuf) + (PAIR ? w * (128 * HD * 2) : 0), 16, 1024);
            const int own = DUAL ? w : 0;
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
                const int n = !ALT ? g.t1 - g.t0 : (g.t1 - g.t0 + 1 - w) / 2;  // the group's tiles
                ok = wait(&q_ready[own], seg & 1);
                if (!ok)
                    break;
                tc_fence_after();
                for (int k = 0; k < 2 && k < n && ok; ++k)
                    ok = scores(k);
                if (DUAL && ok && n <= 2)
                    tc_commit(&q_free[w], one);
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
                    if (k + 2 < n) {
                        ok = scores(buf);
                        if (DUAL && ok && k + 3 == n)
                            tc_commit(&q_free[w], one);
                    }
                }
                if (ok)
                    tc_commit(&o_full[own], one);
                ++seg;
            }
            // no MMA may be under way when the tensor memory is given back
            tc_commit(&fin[own], one);
            mbar_wait_bounded(&fin[own], 0, p.limit_ns);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(soft_regs(E8)));
        // ---- softmax: group w, a thread a row
        const int w = warp >> 2, wt = threadIdx.x & 127, own = DUAL ? w : 0, u0 = first_unit(w), u1 = end_unit(w);
        // the threads that have items in common: both groups', or one's
        constexpr int kMates = DUAL ? 128 : kSoftThreads;
        const int mate = DUAL ? wt : threadIdx.x, bar = 1 + own, cta = cta_of_group(w);
        to_group(w);
        odd += own * 8;
        odd8 += own * kOddItems * 8;
        factor += own * 128;
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
        const bool wide = !PAIR && (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
        Segment upcoming{};
        if (DUAL && u0 < u1)
            upcoming = shares.segment(u0, u1);
        for (int u = u0; u < u1;) {
            const Segment g = DUAL ? upcoming : shares.segment(u, u1);
            u += g.units;
            if (g.t0 == g.t1) {
                if (DUAL && u < u1)
                    upcoming = shares.segment(u, u1);
                continue;
            }
            const SeqRows& q = g.q;
            const int len = q.len(), n_rows = q.rows * p.group;
            if (!E8 && mate < (CAUSAL ? 8 : 2))
                odd[mate] = 0;
            if (DUAL && p.q_boxes)
                named_bar_sync(bar, kMates);  // before anybody notes a token
            // the item's queries, swizzled as the tiles are; a thread loads eight pieces before it stores one
            if (!DUAL || !p.q_boxes) {
                constexpr int kRowsAtOnce = kMates / (HD / 8);  // rows that the threads hold a piece each of
                const int qc = mate % (HD / 8);
#pragma unroll 1
                for (int r0 = mate / (HD / 8); r0 < ROWS; r0 += 8 * kRowsAtOnce) {
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
                        if constexpr (E8) {
                            // fp16, the row's largest value moved to 2^14 .. 2^15 by a power of two (tfq_attn_warp.cu)
                            uint32_t top = __vmaxu2(__vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu), __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
                            top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
                            for (int o = HD / 16; o > 0; o >>= 1)
                                top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                            const int up = min(127 + 14 - (int)(top >> 7), 60);
                            const float f = __uint_as_float((uint32_t)(127 + up) << 23);
                            auto pair = [&](uint32_t x) { return f32x2_to_f16x2(bf16lo_f32(x) * f, bf16hi_f32(x) * f); };
                            v[i] = make_uint4(pair(v[i].x), pair(v[i].y), pair(v[i].z), pair(v[i].w));
                            if (qc == 0)
                                factor[r] = sc * __uint_as_float((uint32_t)(127 - up) << 23);
                        }
                        *reinterpret_cast<uint4*>(qbuf + (r >> 7) * (128 * HD * 2) + (qc >> 3) * (128 * 128) + (r & 127) * 128 + (((qc & 7) ^ (r & 7)) << 4)) =
                            make_uint4(v[i].x ^ flip, v[i].y ^ flip, v[i].z ^ flip, v[i].w ^ flip);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&q_ready[own]);
            }
            const int row = g.rt * ROWS + (PAIR ? w * 128 : 0) + wt;
            const bool valid = row < n_rows, busy = __any_sync(0xffffffffu, valid);
            const int hidden = hidden_from(g);
            uint64_t mask = 0;
            [[maybe_unused]] int sees = 0;  // causal: tokens that the row sees
            if (valid) {
                const int t = p.token_of(row);
                if constexpr (CAUSAL)
                    sees = q.base + t + 1;
                else
                    mask = block_mask(p, q, t);
            }
            // causal: the row's view of 64 tokens from `at` on
            auto view = [&](int at) -> uint64_t { return sees - at >= 64 ? ~0ull : sees - at <= 0 ? 0ull : ~0ull >> (64 - (sees - at)); };
            float m = -INFINITY, l = 0.f;  // the reference, in score units (8 bits: times its factor), and the sum against it
            [[maybe_unused]] float row_factor = 0.f;
            if constexpr (E8) {
                named_bar_sync(bar, kMates);  // the rows' factors are there
                row_factor = factor[(PAIR ? w * 128 : 0) + wt];
            }
            bool had = false, ok = true;
            int buf = 0;
            for (int t = g.t0 + (ALT ? w : 0); t < g.t1; t += ALT ? 2 : 1, buf ^= 1) {
                ok = __all_sync(0xffffffffu, attn_wait(&s_full[2 * w + buf], phase >> buf & 1, flags, p.status, p.limit_ns));
                if (!ok)
                    break;
                const uint32_t s_at = tmem + lanes + 128 * w + 64 * buf;
                tc_fence_after();
                const int k0 = t * KT;
                const bool edge = k0 + KT > hidden;
                [[maybe_unused]] const float* blocks = nullptr;
                if constexpr (E8) {
                    // the converting warps see to V, and have left the tile's scales
                    const int at = (PAIR ? 0 : w) * kScaleTiles + tiles % kScaleTiles;
                    ok = __all_sync(0xffffffffu, attn_wait(&scale_full[at], (tiles / kScaleTiles) & 1, flags, p.status, p.limit_ns));
                    if (!ok)
                        break;
                    blocks = scales + at * 12;
                } else if (edge) {
                    // values behind the sequence's end become zeros, and infinities and NaN among the
                    // block's own are noted and taken out: a row that does not see them may not meet
                    // them, not even as 0 times NaN. (Of a pair each group does it: what the other has
                    // done it finds done, and its own product follows its own pass.)
                    const uint32_t pos = 2 * tiles + 1;
                    ok = __all_sync(0xffffffffu, attn_wait(&full[first_slot + pos % ring_slots], (pos / ring_slots) & 1, flags, p.status, p.limit_ns));
                    if (!ok)
                        break;
                    const int tok = k0 + wt % KT;
                    if (tok >= hidden) {
                        // two threads a row; each starts at a piece of its own, for the banks' sake. Rows are
                        // rarely written: an exponent of all ones, or nothing else, carries into the bit above it
                        uint8_t* v = ring + (size_t)(first_slot + pos % ring_slots) * C::kSlotBytes + wt % KT * 128;
                        auto at = [&](int i) { return reinterpret_cast<uint4*>(v + ((wt / KT * (HD / 16) + i) >> 3) * (KT * 128) + ((wt / KT * (HD / 16) + i + wt) & 7) * 16); };
                        bool bad = false;
                        auto clean = [&](int i) {
                            uint32_t x[4];
                            *reinterpret_cast<uint4*>(x) = *at(i);
                            for (int j = 0; j < 4; ++j) {
                                if (tok >= len) {
                                    x[j] = 0;
                                    continue;
                                }
                                const bool lo = nonfinite16(x[j]), hi = nonfinite16(x[j] >> 16);
                                bad |= lo | hi;
                                x[j] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
                            }
                            *at(i) = *reinterpret_cast<uint4*>(x);
                        };
                        uint32_t sum = 0;
#pragma unroll
                        for (int i = 0; !PAIR && i < HD / 16; ++i) {
                            const uint4 x = *at(i);
                            sum |= (x.x & 0x7F807F80u) + 0x00800080u | (x.y & 0x7F807F80u) + 0x00800080u;
                            sum |= (x.z & 0x7F807F80u) + 0x00800080u | (x.w & 0x7F807F80u) + 0x00800080u;
                        }
                        if (PAIR) {  // each makes its own product safe
#pragma unroll 4
                            for (int i = 0; i < HD / 16; ++i)
                                clean(i);
                        } else if (tok >= len || (sum & 0x80008000u) != 0) {
#pragma unroll 1
                            for (int i = 0; i < HD / 16; ++i)
                                clean(i);
                            fence_async_smem();
                        }
                        if (bad && tok - hidden < kOddTokens)
                            atomicOr(&odd[(tok - hidden) >> 5], 1u << ((tok - hidden) & 31));
                    }
                    if (PAIR)
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
                            const uint64_t see = CAUSAL ? view(k0) : tile_mask(mask, k0 - q.base);
#pragma unroll
                            for (int c = 0; c < KT; ++c)
                                s[c] = see >> c & 1 ? s[c] : 0xFF800000u;  // -inf
                        }
                    };
                    [[maybe_unused]] float ks[4], lvs[4];  // 8 bits: factors of the blocks' scores, log2 of their V scales
                    if constexpr (E8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            ks[i] = fmaxf(row_factor * blocks[i], 1.2e-38f);  // not 0, which -inf times would be NaN
                            lvs[i] = blocks[4 + i];
                        }
                    }
                    auto largest = [&]() {
                        if constexpr (E8) {
                            float x = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float y[2] = {-INFINITY, -INFINITY};
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    y[c & 1] = fmaxf(y[c & 1], __uint_as_float(s[16 * i + c]));
                                x = fmaxf(x, fmaf(fmaxf(y[0], y[1]), ks[i], lvs[i]));
                            }
                            return x;
                        }
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
                        if constexpr (E8) {  // fp16: 2^-11 of each, or 2^-32 of the row's reference (2^7) below 2^-21 of it
                            const float ref = (m == -INFINITY ? 0.f : m) - kHead;
                            float added = 0.f;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 k2 = make_float2(ks[i], ks[i]), off = make_float2(lvs[i] - ref, lvs[i] - ref);
                                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                                for (int c = 16 * i; c < 16 * i + 16; c += 2) {
                                    float2 e = __ffma2_rn(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), k2, off);
                                    e.x = attn_ex2(e.x);
                                    e.y = attn_ex2(e.y);
                                    sum = __fadd2_rn(sum, e);
                                    s[c / 2] = f32x2_to_f16x2(e.x, e.y);
                                }
                                added = fmaf(sum.x + sum.y, blocks[8 + i], added);
                            }
                            return added;
                        }
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
                    const float units = E8 ? 1.f : sc;
                    const bool grown = had && (top - m) * units > kGrow;
                    if (__any_sync(0xffffffffu, grown)) {
                        // the last product with V: the other buffer's, whose phase has moved on since
                        ok = __all_sync(0xffffffffu, attn_wait(&o_done[2 * w + (buf ^ 1)], (phase >> (buf ^ 1) & 1) ^ 1, flags, p.status, p.limit_ns));
                        tc_fence_after();
                        const float f = grown ? attn_ex2((m - top) * units) : 1.f;
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
            if (DUAL && u < u1)  // while the last product with V is under way
                upcoming = shares.segment(u, u1);
            ok = ok && __all_sync(0xffffffffu, attn_wait(&o_full[own], seg & 1, flags, p.status, p.limit_ns));
            tc_fence_after();

            // ---- the segment's end
            const bool whole = g.t0 == 0 && g.t1 == g.nt;
            float* part = p.parts + (int64_t)(g.t0 > 0 ? 2 * cta : 2 * cta + 1) * (ROWS * (HD + 2));
            const int prow = (PAIR ? w * 128 : 0) + wt;  // the row within the tile
            float mine = m == -INFINITY ? -INFINITY : E8 ? m : m * sc, top = mine, all = l;
            if (ALT) {
                ml[(w * 128 + wt) * 2] = mine;
                ml[(w * 128 + wt) * 2 + 1] = l;
            }
            named_bar_sync(bar, kMates);  // also: nobody reads Q or marks odd values any more
            if (ALT) {
                const float other = ml[((w ^ 1) * 128 + wt) * 2];
                top = fmaxf(mine, other);
                const float r = top == -INFINITY ? 0.f : top;
                all = l * attn_ex2(mine - r) + ml[((w ^ 1) * 128 + wt) * 2 + 1] * attn_ex2(other - r);
            }
            const float ref = top == -INFINITY ? 0.f : top, scale = ALT ? attn_ex2(mine - ref) : 1.f;
            const float inv = all == 0.f ? 0.f : 1.f / all;
            [[maybe_unused]] const unsigned* odd_words = E8 ? odd8 + seg % kOddItems * 8 : odd;
            auto odd_bits = [&](int i) { return (uint64_t)odd_words[2 * i + 1] << 32 | odd_words[2 * i]; };  // tokens hidden + 64 i ..
            bool any_odd = odd_bits(0) != 0;
            for (int i = 1; CAUSAL && i < 4; ++i)
                any_odd |= odd_bits(i) != 0;
            auto put = [&](float (&a)[32], int c0) {  // columns c0 .. c0 + 31 of the row, unscaled
                if (!valid)
                    return;
                if (any_odd)
                    for (int i = 0; i < (CAUSAL ? 4 : 1); ++i)
                        add_odd<HD, E8>(p, q, g.h, row, hidden + 64 * i, odd_bits(i), CAUSAL ? view(hidden + 64 * i) : mask, sc, sign, ref, c0, a);
                if (whole) {
                    uint16_t* o = p.o + ((int64_t)(q.r0 + p.token_of(row)) * p.n_q + g.h * p.group + p.head_of(row)) * HD + c0;
                    uint32_t x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        x[i] = f32x2_to_bf16x2(a[2 * i] * inv, a[2 * i + 1] * inv);
                    if (wide) {  // a sector a store
#pragma unroll
                        for (int i = 0; i < 16; i += 8)
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + 2 * i), "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]),
                                         "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
                                         : "memory");
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            reinterpret_cast<uint4*>(o)[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    }
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
            if (!ALT) {
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
            if (mate == 0)
                flags[2 + own] = flags[0];
            tc_fence_before();            // the output has been read
            named_bar_sync(bar, kMates);  // the Q buffer may be written again; the part is written
            if (flags[2 + own])           // one answer for all warps
                break;
            if (E8 && mate < 8)           // for the item kOddItems on, whose tiles wait for those in between
                odd8[seg % kOddItems * 8 + mate] = 0;
            if (!whole) {
                SplitItem& s = split[g.t0 > 0 ? 0 : 1];
                s = SplitItem{q, g.h, g.rt * ROWS, min(ROWS, n_rows - g.rt * ROWS), shares.cta_of(g.first), shares.cta_of(g.first + g.nt - 1)};
                if (mate == 0)  // the barrier above and this release cover every thread's part
                    part_written(p, s);
            }
            ++seg;
        }
        for (int i = 0; i < 2; ++i)
            if (split[i].c0 <= split[i].c1)
                join_slice<ROWS, HD, kMates>(p, split[i], flags, qbuf, mate, cta, bar);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int HD, bool PAIR, bool E8, bool CAUSAL>
cudaError_t launch(const AttnParams& p, const CUtensorMap& map, const CUtensorMap& q_map, cudaStream_t stream)
{
    constexpr bool DUAL = CAUSAL && !PAIR;
    using C = TcCfg<HD, PAIR, E8, DUAL>;
    // join_many: fewer parts than ROWS * HD / 4 / threads + 1, and a slice's rounding for each
    constexpr int kPartBytes = C::ROWS * HD * 4, kThreads = DUAL ? 128 : kSoftThreads;  // of a part's output; that join it
    static_assert((C::smem(kMaxAttnSeqs) - 1024 - C::q_off(kMaxAttnSeqs)) / (DUAL ? 2 : 1) >= kPartBytes + (kPartBytes / 16 / kThreads + 1) * (kThreads * 4 + 16),
                  "the queries' and the rings' memory takes a slice of the parts");
    static_assert(C::slots(kMaxAttnSeqs) >= (PAIR ? 3 : 6) && (!E8 || C::code_slots(kMaxAttnSeqs) >= 4), "rings");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(tree_attn_tc_kernel<HD, PAIR, E8, CAUSAL>, 227 * 1024, done);
    if (e != cudaSuccess)
        return e;
    return launch_coop(tree_attn_tc_kernel<HD, PAIR, E8, CAUSAL>, dim3(device_sms()), dim3(tc_threads(E8)), C::smem(p.B), stream, p, map, q_map,
                       (uint32_t)C::slots(p.B), (uint32_t)C::code_slots(p.B), (int)C::q_off(p.B));
}

template <int HD, bool E8>
cudaError_t launch_any(const AttnParams& p, int rows, bool causal, const CUtensorMap& map, const CUtensorMap& q_map, cudaStream_t stream)
{
    if (causal)
        return launch<HD, E8, E8, true>(p, map, q_map, stream);  // 8 bits: a pair
    return rows == 128 ? launch<HD, false, E8, false>(p, map, q_map, stream) : launch<HD, true, E8, false>(p, map, q_map, stream);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnParams& p, int rows, bool causal, const CUtensorMap& map, const CUtensorMap& q_map, cudaStream_t stream)
{
    if (p.c.code == TF_KV_E4M3)
        return p.c.head_dim == 64 ? launch_any<64, true>(p, rows, causal, map, q_map, stream) : launch_any<128, true>(p, rows, causal, map, q_map, stream);
    return p.c.head_dim == 64 ? launch_any<64, false>(p, rows, causal, map, q_map, stream) : launch_any<128, false>(p, rows, causal, map, q_map, stream);
}

}  // namespace tfq
