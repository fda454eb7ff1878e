// Norm, rotation and store into a cache of 8 bits: the pass of tfq_rope.cu, with a scale for each block of 16 rows of a
// page and head.
//
//   scale = 2^e, e the least with max |x| <= 448 2^e over the block's rows of the call (and not below what the
//   block has, unless its first row is among them);  code = e4m3(x / scale)
//
// A block's scale hangs on all rows that the call stores to it, so those are one CTA's: it takes the rows from one
// block's first row of the call to another's (some 16 of a prompt's), a pair of warps one head of them, whose values stay
// in registers in fp32 until the block's maximum is known: every element is read once and written once
// (q 2 + 2 bytes, k and v 2 + 1). The scales are powers of two: the division and the raising of a scale that the
// block has are exact but for e4m3's subnormals, and an attention adds exponents to its scores. A CTA's
// angles are made once, in shared memory, by all its warps.
#include "tfq_rope.cuh"

namespace tfq {
namespace {

constexpr int kThreads8 = 128, kPairs = kThreads8 / 64;
constexpr int kRows8 = 16;  // rows that a pair of warps holds at once: a block's, or several blocks' of few rows
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
        const float2 t = __fmul2_rn(f[k], s);
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
        const float2 t = __fmul2_rn(f[k], s);
        c[k] = f32x2_to_e4m3x2(t.x, t.y);
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// LANES lanes take a row of a head (head_dim / 16), a warp 32 / LANES rows at once.
template <int LANES>
__global__ void __launch_bounds__(kThreads8, LANES == 16 ? 2 : 4) qk_norm_rope8_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int HD = LANES * 16, RPW = 32 / LANES, IT = kRows8 / 2 / RPW;
    // cosines and sines of two of a lane's eight angles, lanes side by side, rows apart: no two lanes meet in a bank
    __shared__ float4 angle[kRows8][4 * LANES + LANES / 2];
    __shared__ int32_t slots[kRows8], places[kRows8];  // places: the pool row of head 0, layer 0's keys
    __shared__ float most[2][kPairs][kRows8];  // each row's largest, of a pair's head and the one before
    const int lane = threadIdx.x & 31, pair = threadIdx.x >> 6, half = threadIdx.x >> 5 & 1, j = lane % LANES;
    const int sub = half * (kRows8 / 2) + lane / LANES;  // the warp's rows are sub + i * RPW
    const int part = blockIdx.x % (unsigned)p.parts;
    const int64_t g0 = (int64_t)(blockIdx.x / (unsigned)p.parts) * p.step;
    const bool rot = j < p.rot16;
    const int c0 = rot ? j : 2 * (j - p.rot16) + 2 * p.rot16;
    const int c1 = rot ? j + p.rot16 : c0 + 1;
    const int n_kv = p.c.n_kv, heads = p.n_q + 2 * n_kv, pairs = p.rot16 * 8;
    const int64_t n_slots = (int64_t)p.c.n_pages << p.c.page_shift;
    pdl_wait();
    pdl_launch_dependents();

    // rows that begin a block's run of the call; the CTA's rows are those from the first at or behind g0 to the first
    // at or behind g0 + step. A run has 16 rows at most, so both lie within 32 rows.
    unsigned first;
    {
        const int64_t m = g0 + lane;
        const int32_t mine = m < p.M ? p.slots[m] : -1;
        int32_t before = __shfl_up_sync(0xffffffffu, mine, 1);
        if (lane == 0)
            before = m > 0 ? p.slots[m - 1] : -1;
        first = __ballot_sync(0xffffffffu, m >= p.M || mine < 0 || before < 0 || mine >> 4 != before >> 4 || mine <= before);
    }
    const unsigned ours = first & ((1u << p.step) - 1), later = first >> p.step;  // step <= 16
    if (ours == 0)
        return;
    const int begin = __ffs((int)ours) - 1, end = (int)min((int64_t)(later ? p.step + __ffs((int)later) - 1 : 32), p.M - g0);

    for (int s = begin, e; s < end; s = e) {
        // up to 16 rows, whole runs
        e = end;
        if (end - s > kRows8) {
            const unsigned ends = (first >> s) & 0x1FFFEu;  // bits 1 .. 16: runs that begin behind s
            e = ends ? s + 31 - __clz((int)ends) : s + kRows8;
        }
        const int n = e - s;
        const int64_t m0 = g0 + s;
        const unsigned runs = first >> s;
        if (s != begin)
            __syncthreads();  // the last rows' angles have been read
        uint4 a[IT], b[IT];
        auto fetch = [&](int h) {
            if (h >= heads)
                return;
            const uint4* row = reinterpret_cast<const uint4*>(p.qkv + (m0 + sub) * p.ld + (int64_t)h * HD);
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                if (i * RPW + sub < n) {
                    a[i] = __ldcg(row + c0);
                    b[i] = __ldcg(row + c1);
                }
                row = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(row) + RPW * p.ld);
            }
        };
        int h = part * kPairs + pair, buf = 0;
        fetch(h);
        if (const int k = threadIdx.x & ((1 << p.pair_shift) - 1); k < pairs) {
            const uint2 f = __ldg(reinterpret_cast<const uint2*>(p.turns + k));
            // the lane that turns the pair, and which of its eight it is there
            const int chunk = k >> 2, of = p.interleaved ? (chunk < p.rot16 ? chunk : chunk - p.rot16) : k >> 3;
            const int nth = p.interleaved ? (k & 3) + (chunk < p.rot16 ? 0 : 4) : k & 7;
            for (int r = threadIdx.x >> p.pair_shift; r < n; r += kThreads8 >> p.pair_shift) {
                const uint32_t pos = (uint32_t)p.positions[m0 + r], neg = (int32_t)pos < 0 ? 0xFFFFFFFFu : 0u;
                float sn, cs;
                turn_sincos_near(__umulhi(pos, f.x) + pos * f.y + neg * f.x, pos * f.x, sn, cs);
                float* to = reinterpret_cast<float*>(&angle[r][(nth >> 1) * LANES + of]) + (nth & 1);
                to[0] = cs;
                to[2] = sn;
            }
        }
        if (threadIdx.x < n) {
            int32_t slot = p.slots[m0 + threadIdx.x];
            if (slot >= n_slots) {
                record_status(p.status, TF_E_INVALID_ARG);
                slot = -1;
            }
            slots[threadIdx.x] = slot;
            places[threadIdx.x] = slot + (slot >> p.c.page_shift) * (n_kv - 1) * p.c.page_size;  // fewer than 2^31 rows
        }
        __syncthreads();
        const bool one = (runs & ((2u << (n - 1)) - 1)) == 1;  // all rows are one block's
        for (int next; h < heads; h = next) {
            next = h + p.parts * kPairs;
            const bool is_q = h < p.n_q, is_k = !is_q && h < p.n_q + n_kv;
            const uint4* gamma = reinterpret_cast<const uint4*>(is_q ? p.q_gamma : is_k ? p.k_gamma : nullptr);
            const int hk = is_q ? 0 : h - p.n_q - (is_k ? 0 : n_kv);
            // the head's rows of the pool: this and a row's place
            const int pool = ((p.layer * 2 + (is_q || is_k ? 0 : 1)) * p.c.n_pages * n_kv + hk) * p.c.page_size;
            int old[IT];  // the blocks' scales before the call
            if (!is_q) {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int r = one ? 0 : i * RPW + sub;
                    old[i] = r < n && slots[r] >= 0 && (i == 0 || !one) ? p.c.scales[(pool + places[r]) >> 4] : 0;
                }
            }
            float2 x[IT][4], y[IT][4];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                unpack8(a[i], x[i]);
                unpack8(b[i], y[i]);
            }
            fetch(next);  // the next head's rows are under way while this one's are worked on
            float inv[IT];  // of the rows' norms: they join at the end, as the rotation is linear
#pragma unroll
            for (int i = 0; i < IT; ++i)
                inv[i] = 1.f;
            if (gamma != nullptr) {
                float2 g[8];
                unpack8(__ldg(gamma + c0), *reinterpret_cast<float2(*)[4]>(g));
                unpack8(__ldg(gamma + c1), *reinterpret_cast<float2(*)[4]>(g + 4));
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    if (half * (kRows8 / 2) + i * RPW >= n)
                        break;
                    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        ss = __ffma2_rn(x[i][k], x[i][k], __ffma2_rn(y[i][k], y[i][k], ss));
                        x[i][k] = __fmul2_rn(x[i][k], g[k]);
                        y[i][k] = __fmul2_rn(y[i][k], g[4 + k]);
                    }
                    float sum = ss.x + ss.y;
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    inv[i] = __frsqrt_rn(sum * (1.f / HD) + p.eps);
                }
            }
            if (rot && (is_q || is_k)) {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int r = i * RPW + sub;
                    if (r >= n)
                        break;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // the lane's angles 2 k and 2 k + 1
                        const float4 t = angle[r][k * LANES + j];
                        const float2 cs = make_float2(t.x, t.y), sn = make_float2(t.z, t.w), no = make_float2(-t.z, -t.w);
                        if (p.interleaved) {
                            float2* v = k < 2 ? &x[i][2 * k] : &y[i][2 * k - 4];
                            const float2 u = make_float2(v[0].x, v[1].x), w = make_float2(v[0].y, v[1].y);
                            const float2 nu = __ffma2_rn(u, cs, __fmul2_rn(w, no)), nw = __ffma2_rn(w, cs, __fmul2_rn(u, sn));
                            v[0] = make_float2(nu.x, nw.x);
                            v[1] = make_float2(nu.y, nw.y);
                        } else {
                            const float2 u = x[i][k];
                            x[i][k] = __ffma2_rn(u, cs, __fmul2_rn(y[i][k], no));
                            y[i][k] = __ffma2_rn(y[i][k], cs, __fmul2_rn(u, sn));
                        }
                    }
                }
            }
            if (is_q) {
                uint4* o = reinterpret_cast<uint4*>(p.q + ((m0 + sub) * p.n_q + h) * HD);
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    if (i * RPW + sub < n) {
                        o[c0] = pack8(x[i], inv[i]);
                        o[c1] = pack8(y[i], inv[i]);
                    }
                    o += (int64_t)RPW * p.n_q * (HD / 8);
                }
                continue;
            }
            // the rows' largest finite values, and of each row's run
            float row_top[IT];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    top = fmaxf(fmaxf(fmaxf(top, fabsf(x[i][k].x)), fmaxf(fabsf(x[i][k].y), fabsf(y[i][k].x))), fabsf(y[i][k].y));
                top *= inv[i];
                if (!(top < INFINITY)) {  // rare
                    top = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float v[4] = {fabsf(x[i][k].x) * inv[i], fabsf(x[i][k].y) * inv[i], fabsf(y[i][k].x) * inv[i], fabsf(y[i][k].y) * inv[i]};
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            top = fmaxf(top, v[z] < INFINITY ? v[z] : 0.f);
                    }
                }
                row_top[i] = i * RPW + sub < n ? top : 0.f;
            }
            if (one) {
                float top = row_top[0];
#pragma unroll
                for (int i = 1; i < IT; ++i)
                    top = fmaxf(top, row_top[i]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (lane == 0)
                    most[buf][pair][half] = top;
            } else {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    float top = row_top[i];
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    if (j == 0)
                        most[buf][pair][i * RPW + sub] = top;
                }
            }
            named_bar_sync(1 + pair, 64);  // also: both warps have read the scales
            const float* tops = most[buf][pair];
            buf ^= 1;
            if (one) {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    row_top[i] = fmaxf(tops[0], tops[1]);
                    old[i] = old[0];
                }
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                if (half * (kRows8 / 2) + i * RPW >= n)
                    break;
                const int r = i * RPW + sub;
                const bool store = r < n && slots[r] >= 0;
                int lo = 0, hi = n;  // the row's run
                if (!one && r < n) {
                    lo = 31 - __clz((int)(runs & (2u << r) - 1));
                    const unsigned behind = runs >> (r + 1);
                    hi = min(n, behind ? r + __ffs((int)behind) : n);
                    float top = 0.f;
                    for (int k = lo; k < hi; ++k)
                        top = fmaxf(top, tops[k]);
                    row_top[i] = top;
                }
                const bool anew = (slots[lo] & 15) == 0;
                const int had = min(max(old[i], kLeast), kMost), need = scale_byte(row_top[i]), now = anew ? need : max(had, need);
                const int row = store ? pool + places[r] : 0;
                if (store) {
                    const float f = pow2(127 - now) * inv[i];
                    uint2* o = reinterpret_cast<uint2*>(p.c.codes() + (int64_t)row * HD);
                    o[c0] = codes8(x[i], f);
                    o[c1] = codes8(y[i], f);
                    if (r == lo && j == 0)
                        p.c.scales[row >> 4] = (uint8_t)now;
                }
                // rare: the scale of a block that holds other rows has grown
                const bool grown = store && r == lo && !anew && now > had;
                unsigned todo = __ballot_sync(0xffffffffu, grown && j == 0);
                while (todo != 0) {
                    const int src = __ffs((int)todo) - 1;
                    todo &= todo - 1;
                    const int r_lo = __shfl_sync(0xffffffffu, lo, src), r_hi = __shfl_sync(0xffffffffu, hi, src);
                    const int64_t at = __shfl_sync(0xffffffffu, row, src) & ~15;
                    const float f = pow2(__shfl_sync(0xffffffffu, had - now, src));
                    unsigned stored = 0;  // the block's rows that the call stores
                    for (int k = r_lo; k < r_hi; ++k)
                        stored |= 1u << (slots[k] & 15);
                    uint2* block = reinterpret_cast<uint2*>(p.c.codes() + at * HD);
                    for (int k = lane; k < 16 * HD / 8; k += 32) {
                        if (stored >> (k / (HD / 8)) & 1)
                            continue;
                        const uint2 v = block[k];
                        const uint32_t w[4] = {e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.y), e4m3x2_to_f16x2(v.y >> 16)};
                        float2 t[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            t[z] = __half22float2(*reinterpret_cast<const __half2*>(&w[z]));
                        block[k] = codes8(t, f);
                    }
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_rope8(const RopeParams& given, bool pdl, cudaStream_t stream)
{
    RopeParams p = given;
    const int heads = p.n_q + 2 * p.c.n_kv, most_parts = (heads + kPairs - 1) / kPairs;
    const int64_t want = (int64_t)device_sms() * 2;
    // few rows: a CTA begins at every row, or every few, and its heads are spread over as many CTAs as fill the GPU
    p.step = kRows8;
    while (p.step > 1 && (p.M + p.step - 1) / p.step * most_parts < want)
        p.step /= 2;
    const int64_t groups = (p.M + p.step - 1) / p.step;
    p.pair_shift = 3;
    while (8 * p.rot16 > 1 << p.pair_shift)
        ++p.pair_shift;
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
