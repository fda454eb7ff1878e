// Norm, rotation and store into a cache of 8 bits: the pass of tfq_rope.cu, with a scale for each block of 16 rows of a
// page and head.
//
//   scale = 2^e, e the least with max |x| <= 448 2^e over the block's rows of the call (and not below what the
//   block has, unless its first row is among them);  code = e4m3(x / scale)
//
// A block's scale hangs on all rows that the call stores to it, so those are one CTA's: it takes the rows from one
// block's first row of the call to another's (some 16 of a prompt's), a warp a row, and the warps meet once for each set
// of key or value heads, with their rows' largest values in shared memory; what is to be stored stays in registers
// in fp32 until then. Every element is read once and written once (q 2 + 2 bytes, k and v 2 + 1). The scales are powers
// of two: the division, and the raising of a scale that the block has, are exact but for e4m3's subnormals, and an
// attention adds exponents to its scores.
//
// 8191 rows of 16 + 2 * 8 heads of 128: 29.8 us, 3.9 TB/s of reads and writes, three quarters of the issue slots: what a row
// costs before its first head (some 3 us for each part that its heads are dealt into) and the meetings at half of the sets
// bound it (without norm and rotation 28.1; the pass into a bf16 cache 24.8). One warp to 16 rows of a head, which needs no meeting but 128 registers for
// the values, took 46 us where this took 31; a pair of warps 35; CTAs that take equal runs of sets of heads in the place
// of halves of them 31.0. One row 3.5 us, 64 rows of 64 sequences 5.1: there one or two of the
// 16 warps have a row. With four warps a CTA those 64 rows took 4.2, and a prompt more.
#include "tfq_rope.cuh"

namespace tfq {
namespace {

constexpr int kRows8 = 16, kThreads8 = kRows8 * 32;  // rows of a CTA at once, a warp each: a block's, or several blocks' of few rows
constexpr int kLeast = 127 - 32, kMost = 127 + 32;  // scale bytes

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // |e| <= 64

// The least scale byte with most <= 448 * scale (most >= 0, finite), within bounds: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_byte(float most)
{
    const uint32_t b = __float_as_uint(most);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, kLeast), kMost);
}

// Sine and cosine of hi + lo / 2^32 units of 2^-32 turn within some 2^-23 of their own values: a code lies on the other
// side of a rounding's border about as often as one from fp32 angles of a 64-bit cosine. The nearest quarter turn is taken
// off exactly; what is left is x + rest, x the nearest fp32 number, and within pi / 4 the Taylor polynomials end below
// x^10 / 11! and x^12 / 12!. A CTA makes each angle once for all its heads, so this costs little.
__device__ __forceinline__ void turn_sincos_near(uint32_t hi, uint32_t lo, float& sn, float& cs)
{
    constexpr float kUnit = 1.4629180792671596e-9f, kUnitRest = (float)(1.4629180792671596e-9 - (double)kUnit);  // 2 pi / 2^32
    const uint32_t quarter = (hi + 0x20000000u) >> 30;
    const int32_t v = (int32_t)(hi - (quarter << 30));
    const float a = (float)v, b = fmaf((float)lo, 0x1p-32f, (float)(v - (int32_t)a));
    const float x = a * kUnit, rest = fmaf(a, kUnit, -x) + fmaf(a, kUnitRest, b * kUnit);
    const float y = x * x;
    float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
    const float c0 = c;
    c = fmaf(-rest, s, c);
    s = fmaf(rest, c0, s);
    const bool odd = quarter & 1;
    sn = __uint_as_float(__float_as_uint(odd ? c : s) ^ (quarter & 2) << 30);
    cs = __uint_as_float(__float_as_uint(odd ? s : c) ^ (quarter + 1 & 2) << 30);
}

// Apart: packed they are no faster, and take more registers
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)); }

__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4])
{
    f[0] = make_float2(bf16lo_f32(v.x), bf16hi_f32(v.x)), f[1] = make_float2(bf16lo_f32(v.y), bf16hi_f32(v.y));
    f[2] = make_float2(bf16lo_f32(v.z), bf16hi_f32(v.z)), f[3] = make_float2(bf16lo_f32(v.w), bf16hi_f32(v.w));
}
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4], float by)
{
    const float2 s = make_float2(by, by);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 t = mul2(f[k], s);
        w[k] = f32x2_to_bf16x2(t.x, t.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint2 codes8(const float2 (&f)[4], float by)
{
    const float2 s = make_float2(by, by);
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 t = mul2(f[k], s);
        c[k] = f32x2_to_e4m3x2(t.x, t.y);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// LANES lanes take a head (head_dim / 16), a warp HEADS = 32 / LANES heads of its row at once.
template <int LANES>
__global__ void __launch_bounds__(kThreads8, 2) qk_norm_rope8_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int HD = LANES * 16, HEADS = 32 / LANES, OWN = 8 / HEADS;
    __shared__ float tops[2][kRows8][HEADS];  // each row's largest value of the heads at hand, and of those before
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane % LANES, sub = lane / LANES;
    const int part = blockIdx.x % (unsigned)p.parts;
    const int64_t g0 = (int64_t)(blockIdx.x / (unsigned)p.parts) * p.step;
    // the lane's chunks of 8 elements: both ends of its eight rotated pairs, as in tfq_rope.cu
    const bool rot = j < p.rot16;
    const int c0 = rot ? j : 2 * (j - p.rot16) + 2 * p.rot16;
    const int c1 = rot ? j + p.rot16 : c0 + 1;
    uint2 f[OWN];
    if (rot) {
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
            const int i = sub * OWN + k, idx = p.interleaved ? (i < 4 ? c0 * 4 + i : c1 * 4 + i - 4) : j * 8 + i;
            f[k] = __ldg(reinterpret_cast<const uint2*>(p.turns + idx));
        }
    }
    // the norms' weights in fp32, as the lanes take them: unpacked once and not for every head (8191 rows 30.9 us)
    __shared__ float4 gammas[2][4][LANES];
    uint4 ga = {}, gb = {};
    const uint4* gamma = reinterpret_cast<const uint4*>(warp == 0 ? p.q_gamma : warp == 1 ? p.k_gamma : nullptr);
    if (gamma != nullptr && lane < LANES) {
        ga = __ldg(gamma + c0);
        gb = __ldg(gamma + c1);
    }
    pdl_wait();
    pdl_launch_dependents();

    // rows that begin a block's run of the call; the CTA's rows are those from the first at or behind g0 to the first
    // at or behind g0 + step. A run has 16 rows at most, so both lie within 32 rows.
    const int32_t mine = g0 + lane < p.M ? p.slots[g0 + lane] : -1;  // a row's slot a lane, and its position
    const int32_t my_pos = g0 + lane < p.M ? p.positions[g0 + lane] : 0;
    const int32_t prior = g0 + lane >= 32 ? p.slots[g0 - 32 + lane] : -1;  // the 32 rows before g0 (8191 rows 29.6 us without)
    unsigned first;
    {
        int32_t before = __shfl_up_sync(0xffffffffu, mine, 1);
        if (lane == 0)
            before = g0 > 0 ? p.slots[g0 - 1] : -1;
        first = __ballot_sync(0xffffffffu, g0 + lane >= p.M || mine < 0 || before < 0 || mine >> 4 != before >> 4 || mine <= before);
    }
    if (warp < 2 && lane < LANES) {
        float2 g[4];
        unpack8(ga, g);
        gammas[warp][0][lane] = make_float4(g[0].x, g[0].y, g[1].x, g[1].y);
        gammas[warp][1][lane] = make_float4(g[2].x, g[2].y, g[3].x, g[3].y);
        unpack8(gb, g);
        gammas[warp][2][lane] = make_float4(g[0].x, g[0].y, g[1].x, g[1].y);
        gammas[warp][3][lane] = make_float4(g[2].x, g[2].y, g[3].x, g[3].y);
    }
    const unsigned ours = first & ((1u << p.step) - 1), later = first >> p.step;  // step <= 16
    if (ours == 0)
        return;
    const int begin = __ffs((int)ours) - 1, end = (int)min((int64_t)(later ? p.step + __ffs((int)later) - 1 : 32), p.M - g0);
    const int n_kv = p.c.n_kv, heads = p.n_q + 2 * n_kv;
    int buf = 0;
    for (int s = begin, e; s < end; s = e) {
        // up to 16 rows, whole runs
        e = end;
        if (end - s > kRows8) {
            const unsigned ends = (first >> s) & 0x1FFFEu;  // bits 1 .. 16: runs that begin behind s
            e = ends ? s + 31 - __clz((int)ends) : s + kRows8;
        }
        const int at = s + warp;  // the warp's row, from g0
        const bool row_in = at < e;
        const int64_t m = g0 + (row_in ? at : s);
        const uint4* row = reinterpret_cast<const uint4*>(p.qkv + m * p.ld) + sub * (HD / 8);
        uint4 na = {}, nb = {};
        auto fetch = [&](int h0) {
            if (row_in && h0 + sub < heads) {
                na = __ldcg(row + h0 * (HD / 8) + c0);
                nb = __ldcg(row + h0 * (HD / 8) + c1);
            }
        };
        fetch(part * HEADS);
        float cs[8], sn[8];
        {
            float mine_c[OWN] = {}, mine_s[OWN] = {};
            const uint32_t pos = (uint32_t)__shfl_sync(0xffffffffu, my_pos, at & 31);
            if (rot) {
                const uint32_t neg = (int32_t)pos < 0 ? 0xFFFFFFFFu : 0u;
#pragma unroll
                for (int k = 0; k < OWN; ++k)
                    turn_sincos_near(__umulhi(pos, f[k].x) + pos * f[k].y + neg * f[k].x, pos * f[k].x, mine_s[k], mine_c[k]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sn[i] = __shfl_sync(0xffffffffu, mine_s[i % OWN], i / OWN * LANES + j);
                cs[i] = __shfl_sync(0xffffffffu, mine_c[i % OWN], i / OWN * LANES + j);
            }
        }
        int32_t slot = __shfl_sync(0xffffffffu, mine, at & 31);
        // the row's run: rows lo .. hi, from s; and which rows of its block those are
        const unsigned runs = first >> s;
        const int r = row_in ? warp : 0, lo = 31 - __clz((int)(runs & (2u << r) - 1));
        // a run of its block's among the 32 rows before the row's own: two would race for the scale, so this one is refused
        const int32_t other = lane < s + lo ? mine : prior;
        const bool again = __any_sync(0xffffffffu, (uint32_t)(other ^ slot) < 16u);
        const bool bad = row_in && slot >= 0 && (again || slot >= (int64_t)p.c.n_pages << p.c.page_shift);
        if (bad && part == 0 && lane == 0)
            record_status(p.status, TF_E_INVALID_ARG);
        const bool store = row_in && slot >= 0 && !bad;
        if (!store)
            slot = 0;
        const unsigned behind = runs >> (r + 1);
        const int hi = min(e - s, behind ? r + __ffs((int)behind) : e - s);
        const unsigned stored = __reduce_or_sync(0xffffffffu, lane - s >= lo && lane - s < hi ? 1u << (mine & 15) : 0u);
        const bool anew = stored & 1;
        if (s == begin)
            __syncthreads();  // the norms' weights are there
        const int place = store ? (slot >> p.c.page_shift) * n_kv * p.c.page_size + (slot & (p.c.page_size - 1)) : -1;  // fewer than 2^31 rows
#pragma unroll 1
        for (int h0 = part * HEADS; h0 < heads; h0 += p.parts * HEADS) {
            const int h = h0 + sub;
            const bool is_q = h < p.n_q, is_k = !is_q && h < p.n_q + n_kv, live = row_in && h < heads;
            // the pool's row, and its block's scale before the call
            const int at_row = is_q ? 0 : place + ((p.layer * 2 + (is_k ? 0 : 1)) * p.c.n_pages * n_kv + h - p.n_q - (is_k ? 0 : n_kv)) * p.c.page_size;
            const bool stores = place >= 0 && live && !is_q;
            const int was = stores && !anew ? p.c.scales[at_row >> 4] : 0;
            float2 x[4], y[4];
            unpack8(na, x);
            unpack8(nb, y);
            fetch(h0 + p.parts * HEADS);
            float inv = 1.f;
            const bool norm = (is_q ? p.q_gamma : is_k ? p.k_gamma : nullptr) != nullptr;
            if (h0 < p.n_q + n_kv) {  // else the warp has values alone
                float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    ss = fma2(x[k], x[k], fma2(y[k], y[k], ss));
                float sum = ss.x + ss.y;
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (norm) {
                    const float mean = sum * (1.f / HD) + p.eps, near = rsqrtf(mean);
                    inv = fmaf(near * 0.5f, fmaf(-mean * near, near, 1.f), near);  // a Newton step: the last bit counts too
                    if (!(mean < INFINITY)) {  // rare: as in a cache of bf16, finite values give 0 and infinite ones NaN
                        inv = 1.f;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            x[k] = mul2(x[k], make_float2(near, near)), y[k] = mul2(y[k], make_float2(near, near));
                    }
                    const float4(*g)[LANES] = gammas[is_q ? 0 : 1];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float4 a = g[k][j], b = g[2 + k][j];
                        x[2 * k] = mul2(x[2 * k], make_float2(a.x, a.y)), x[2 * k + 1] = mul2(x[2 * k + 1], make_float2(a.z, a.w));
                        y[2 * k] = mul2(y[2 * k], make_float2(b.x, b.y)), y[2 * k + 1] = mul2(y[2 * k + 1], make_float2(b.z, b.w));
                    }
                }
                if (rot && (is_q || is_k)) {
                    if (p.interleaved) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 u = x[k], w = y[k];
                            x[k] = make_float2(u.x * cs[k] - u.y * sn[k], u.y * cs[k] + u.x * sn[k]);
                            y[k] = make_float2(w.x * cs[4 + k] - w.y * sn[4 + k], w.y * cs[4 + k] + w.x * sn[4 + k]);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 u = x[k], c2 = make_float2(cs[2 * k], cs[2 * k + 1]), s2 = make_float2(sn[2 * k], sn[2 * k + 1]);
                            x[k] = fma2(y[k], make_float2(-s2.x, -s2.y), mul2(u, c2));
                            y[k] = fma2(y[k], c2, mul2(u, s2));
                        }
                    }
                }
            }
            if (is_q && live) {
                uint4* o = reinterpret_cast<uint4*>(p.q + (m * p.n_q + h) * HD);
                o[c0] = pack8(x, inv);
                o[c1] = pack8(y, inv);
            }
            if (h0 + HEADS <= p.n_q)
                continue;
            // the row's largest finite value of the head, then the run's
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                top = fmaxf(fmaxf(fmaxf(top, fabsf(x[k].x)), fmaxf(fabsf(x[k].y), fabsf(y[k].x))), fabsf(y[k].y));
            top *= inv;
            if (!(top < INFINITY)) {  // rare
                top = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float v[4] = {fabsf(x[k].x) * inv, fabsf(x[k].y) * inv, fabsf(y[k].x) * inv, fabsf(y[k].y) * inv};
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        top = fmaxf(top, v[z] < INFINITY ? v[z] : 0.f);
                }
            }
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (j == 0)
                tops[buf][warp][sub] = top;
            __syncthreads();  // also: every row's warp has read the scales
            top = 0.f;
#pragma unroll
            for (int k = 0; k < kRows8 / LANES; ++k)
                if (k * LANES + j >= lo && k * LANES + j < hi)
                    top = fmaxf(top, tops[buf][k * LANES + j][sub]);
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            buf ^= 1;
            const int had = min(max(was, kLeast), kMost), need = scale_byte(top), now = anew ? need : max(had, need);
            if (stores) {
                const float by = pow2(127 - now) * inv;
                uint2* o = reinterpret_cast<uint2*>(p.c.codes() + (int64_t)at_row * HD);
                o[c0] = codes8(x, by);
                o[c1] = codes8(y, by);
                if (r == lo && j == 0)
                    p.c.scales[at_row >> 4] = (uint8_t)now;
            }
            // rare: the scale of a block that holds other rows has grown
            unsigned todo = __ballot_sync(0xffffffffu, stores && r == lo && !anew && now > had && j == 0);
            while (todo != 0) {
                const int src = __ffs((int)todo) - 1;
                todo &= todo - 1;
                uint2* block = reinterpret_cast<uint2*>(p.c.codes() + (int64_t)(__shfl_sync(0xffffffffu, at_row, src) & ~15) * HD);
                const float by = pow2(__shfl_sync(0xffffffffu, had - now, src));
                for (int k = lane; k < 16 * HD / 8; k += 32) {
                    if (stored >> (k / (HD / 8)) & 1)
                        continue;
                    const uint2 v = block[k];
                    const uint32_t w[4] = {e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.y), e4m3x2_to_f16x2(v.y >> 16)};
                    float2 t[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        t[z] = __half22float2(*reinterpret_cast<const __half2*>(&w[z]));
                    block[k] = codes8(t, by);
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope8(const RopeParams& given, bool pdl, cudaStream_t stream)
{
    RopeParams p = given;
    const int per_warp = 512 / p.c.head_dim, most_parts = (p.n_q + 2 * p.c.n_kv + per_warp - 1) / per_warp;
    const int64_t want = (int64_t)device_sms() * 2;
    // few rows: a CTA begins at fewer of them, and its heads are spread over as many CTAs as run at once, twice over:
    // 8191 rows 29.8 us in two parts; 0.5 more in one, 6 in four
    p.step = kRows8;
    while (p.step > 1 && (p.M + p.step / 2 - 1) / (p.step / 2) * most_parts <= want)
        p.step /= 2;
    const int64_t groups = (p.M + p.step - 1) / p.step;
    p.parts = 1;
    while (p.parts < most_parts && groups * p.parts < 2 * want)
        p.parts *= 2;
    if (p.parts > most_parts)
        p.parts = most_parts;
    const unsigned grid = (unsigned)(groups * p.parts);
    if (p.c.head_dim == 64)
        return launch_pdl(qk_norm_rope8_kernel<4>, dim3(grid), dim3(kThreads8), 0, stream, pdl, p);
    if (p.c.head_dim == 128)
        return launch_pdl(qk_norm_rope8_kernel<8>, dim3(grid), dim3(kThreads8), 0, stream, pdl, p);
    return launch_pdl(qk_norm_rope8_kernel<16>, dim3(grid), dim3(kThreads8), 0, stream, pdl, p);
}

}  // namespace tfq
