// Norm, rotation and store into a cache of 8 bits: the pass of tfq_rope.cu, with a scale for each block of 16 rows of a
// page and head.
//
//   scale = 2^e, e the least with max |x| <= 448 2^e over the block's rows of the call (and not below what the
//   block has, unless its first row is among them);  code = e4m3(x / scale)
//
// A block's scale hangs on all rows that the call stores to it, so those are one warp's: a CTA takes the rows from one
// block's first row of the call to another's (some 16 of a prompt's), a warp one head of them, whose values stay in
// registers in fp32 until the block's maximum is known: every element is read once and written once
// (q 2 + 2 bytes, k and v 2 + 1). The scales are powers of two: the division and the raising of a scale that the
// block has are exact but for e4m3's subnormals, and an attention adds exponents to its scores. A CTA's
// angles are made once, in shared memory, by all its warps.
#include "tfq_rope.cuh"

namespace tfq {
namespace {

constexpr int kThreads8 = 256, kWarps8 = kThreads8 / 32;
constexpr int kRows8 = 16;  // rows that a warp holds at once: a block's, or several blocks' of few rows
constexpr int kLeast = 127 - 32, kMost = 127 + 32;  // scale bytes

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) { return f32x2_to_e4m3x2(a, b) | f32x2_to_e4m3x2(c, d) << 16; }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // |e| <= 64

// The least scale byte with most <= 448 * scale (most >= 0, finite), within bounds: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_byte(float most)
{
    const uint32_t b = __float_as_uint(most);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, kLeast), kMost);
}

// LANES lanes take a row of a head (head_dim / 16), a warp 32 / LANES rows at once.
template <int LANES>
__global__ void __launch_bounds__(kThreads8, LANES == 16 ? 1 : 2) qk_norm_rope8_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int HD = LANES * 16, RPW = 32 / LANES, IT = kRows8 / RPW;
    __shared__ float2 angle[kRows8][HD / 2];  // cosine, sine
    __shared__ int32_t slots[kRows8];
    __shared__ float most[kWarps8][kRows8];   // each row's largest, of a warp's head
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane % LANES, sub = lane / LANES;
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
            e = s + 31 - __clz((int)ends);
            if (ends == 0)
                e = s + kRows8;
        }
        const int n = e - s;
        const int64_t m0 = g0 + s;
        const unsigned runs = first >> s;
        if (s != begin)
            __syncthreads();  // the last rows' angles have been read
        uint4 a[IT], b[IT];
        int was[IT];
        auto fetch = [&](int h) {
            if (h >= heads)
                return;
            const bool kv = h >= p.n_q;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int r = i * RPW + sub;
                was[i] = 0;
                if (r < n) {
                    const uint4* row = reinterpret_cast<const uint4*>(p.qkv + (m0 + r) * p.ld + (int64_t)h * HD);
                    a[i] = __ldcg(row + c0);
                    b[i] = __ldcg(row + c1);
                }
            }
            if (kv) {
                const int hk = h - p.n_q, v = hk >= n_kv;
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int r = i * RPW + sub;
                    const int32_t slot = r < n ? p.slots[m0 + r] : -1;
                    if (slot >= 0 && slot < n_slots)
                        was[i] = p.c.scales[(p.c.row_of(p.layer, v, slot >> p.c.page_shift, hk - v * n_kv) + (slot & (p.c.page_size - 1))) >> 4];
                }
            }
        };
        int h = part * kWarps8 + warp;
        fetch(h);
        for (int i = threadIdx.x; i < n * pairs; i += kThreads8) {
            const int r = i / pairs, k = i - r * pairs;
            const uint2 f = __ldg(reinterpret_cast<const uint2*>(p.turns + k));
            const uint32_t pos = (uint32_t)p.positions[m0 + r], neg = (int32_t)pos < 0 ? 0xFFFFFFFFu : 0u;
            float sn, cs;
            turn_sincos(__umulhi(pos, f.x) + pos * f.y + neg * f.x, pos * f.x, sn, cs);
            angle[r][k] = make_float2(cs, sn);
        }
        if (threadIdx.x < n) {
            int32_t slot = p.slots[m0 + threadIdx.x];
            if (slot >= n_slots) {
                record_status(p.status, TF_E_INVALID_ARG);
                slot = -1;
            }
            slots[threadIdx.x] = slot;
        }
        __syncthreads();
        for (; h < heads; h += p.parts * kWarps8) {
            const bool is_q = h < p.n_q, is_k = !is_q && h < p.n_q + n_kv;
            const uint4* gamma = reinterpret_cast<const uint4*>(is_q ? p.q_gamma : is_k ? p.k_gamma : nullptr);
            const int hk = is_q ? 0 : h - p.n_q - (is_k ? 0 : n_kv);
            float x[IT][8], y[IT][8];
            float g0v[8], g1v[8];
            if (gamma != nullptr) {
                unpack8(__ldg(gamma + c0), g0v);
                unpack8(__ldg(gamma + c1), g1v);
            }
            int old[IT];
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                if (i * RPW >= n)
                    break;
                const int r = i * RPW + sub;
                unpack8(a[i], x[i]);
                unpack8(b[i], y[i]);
                old[i] = was[i];
                if (gamma != nullptr) {
                    float ss = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        ss = fmaf(x[i][k], x[i][k], fmaf(y[i][k], y[i][k], ss));
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1)
                        ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const float rs = rsqrtf(ss * (1.f / HD) + p.eps);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        x[i][k] = x[i][k] * rs * g0v[k];
                        y[i][k] = y[i][k] * rs * g1v[k];
                    }
                }
                if (rot && (is_q || is_k) && r < n) {
                    if (p.interleaved) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 t = angle[r][c0 * 4 + k], w = angle[r][c1 * 4 + k];
                            const float u = x[i][2 * k] * t.x - x[i][2 * k + 1] * t.y;
                            x[i][2 * k + 1] = x[i][2 * k + 1] * t.x + x[i][2 * k] * t.y;
                            x[i][2 * k] = u;
                            const float z = y[i][2 * k] * w.x - y[i][2 * k + 1] * w.y;
                            y[i][2 * k + 1] = y[i][2 * k + 1] * w.x + y[i][2 * k] * w.y;
                            y[i][2 * k] = z;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 t = angle[r][j * 8 + k];
                            const float u = x[i][k] * t.x - y[i][k] * t.y;
                            y[i][k] = y[i][k] * t.x + x[i][k] * t.y;
                            x[i][k] = u;
                        }
                    }
                }
            }
            fetch(h + p.parts * kWarps8);  // the next head's rows are under way while this one's are stored
            if (is_q) {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int r = i * RPW + sub;
                    if (r < n) {
                        uint4* o = reinterpret_cast<uint4*>(p.q + ((m0 + r) * p.n_q + h) * HD);
                        o[c0] = pack8(x[i]);
                        o[c1] = pack8(y[i]);
                    }
                }
                continue;
            }
            // each row's largest finite value
            __syncwarp();
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                if (i * RPW >= n)
                    break;
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float u = fabsf(x[i][k]), w = fabsf(y[i][k]);
                    top = fmaxf(top, fmaxf(u < INFINITY ? u : 0.f, w < INFINITY ? w : 0.f));
                }
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (j == 0)
                    most[warp][i * RPW + sub] = top;
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                if (i * RPW >= n)
                    break;
                const int r = i * RPW + sub;
                const int32_t slot = r < n ? slots[r] : -1;
                const bool store = slot >= 0;
                // the row's run: rows lo .. hi
                const int lo = r < n ? 31 - __clz((int)(runs & (2u << r) - 1)) : 0;
                const unsigned behind = r < n ? runs >> (r + 1) : 1;
                const int hi = min(n, behind ? r + __ffs((int)behind) : n);
                float top = 0.f;
                if (store)
                    for (int k = lo; k < hi; ++k)
                        top = fmaxf(top, most[warp][k]);
                const bool anew = store && (slots[lo] & 15) == 0;
                const int had = min(max(old[i], kLeast), kMost), need = scale_byte(top), now = anew ? need : max(had, need);
                const int page = store ? slot >> p.c.page_shift : 0, off = slot & (p.c.page_size - 1);
                const int64_t row = p.c.row_of(p.layer, is_k ? 0 : 1, page, hk) + off;
                if (store) {
                    const float f = pow2(127 - now);
                    uint2* o = reinterpret_cast<uint2*>(p.c.codes() + row * HD);
                    o[c0] = make_uint2(e4m3x4(x[i][0] * f, x[i][1] * f, x[i][2] * f, x[i][3] * f),
                                       e4m3x4(x[i][4] * f, x[i][5] * f, x[i][6] * f, x[i][7] * f));
                    o[c1] = make_uint2(e4m3x4(y[i][0] * f, y[i][1] * f, y[i][2] * f, y[i][3] * f),
                                       e4m3x4(y[i][4] * f, y[i][5] * f, y[i][6] * f, y[i][7] * f));
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
                    const int64_t at = __shfl_sync(0xffffffffu, row, src) & ~(int64_t)15;
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
                        uint32_t c[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[z]));
                            c[z] = f32x2_to_e4m3x2(t.x * f, t.y * f);
                        }
                        block[k] = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
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
    const int heads = p.n_q + 2 * p.c.n_kv, most_parts = (heads + kWarps8 - 1) / kWarps8;
    const int64_t want = (int64_t)device_sms() * 2;
    // few rows: a CTA begins at every row, or every few, and its heads are spread over as many CTAs as fill the GPU
    p.step = kRows8;
    while (p.step > 1 && (p.M + p.step - 1) / p.step * most_parts < want)
        p.step /= 2;
    const int64_t groups = (p.M + p.step - 1) / p.step;
    p.parts = 1;
    while (p.parts < most_parts && groups * p.parts < 4 * want)
        ++p.parts;
    const unsigned grid = (unsigned)(groups * p.parts);
    if (p.c.head_dim == 64)
        return launch_pdl(qk_norm_rope8_kernel<4>, dim3(grid), dim3(kThreads8), 0, stream, pdl, p);
    if (p.c.head_dim == 128)
        return launch_pdl(qk_norm_rope8_kernel<8>, dim3(grid), dim3(kThreads8), 0, stream, pdl, p);
    return launch_pdl(qk_norm_rope8_kernel<16>, dim3(grid), dim3(kThreads8), 0, stream, pdl, p);
}

}  // namespace tfq
