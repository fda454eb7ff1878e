// Norms of queries and keys for each head, the position rotation, and the store of keys and
// values to the paged cache, in one pass over the rows of a qkv projection.
//
//   q, k heads: x * rsqrt(mean(x^2) + eps) * gamma, then (a, b) -> (a cos - b sin, b cos + a sin)
//   v heads:    as they are
//
// Bound by memory: every element is read once and written once (2 + 2 bytes; a row of 16 + 2 * 8
// heads of 128 moves 16 KB), for about six multiply-adds. A lane holds two 16-byte chunks of
// one head, chosen so that both ends of each rotated pair are its own: head_dim / 16 lanes take
// a head (8 at 128, so a warp takes 4 heads at once), the sum of squares is a butterfly over
// those lanes, and the eight angles a lane needs are made once a row, by the warp's lanes together, and used
// for all its heads.
//
// 8191 such rows: 24.0 us, 5.6 TB/s of reads and writes (each row's loads run one set of heads ahead of the
// arithmetic); 8 rows: 2.3 us, of which a launch is most.
#include <cmath>

#include "tfq_rope.cuh"

namespace tfq {
namespace {

constexpr int kRopeThreads = 128;

// LANES lanes take a head (head_dim / 16); a warp takes HEADS = 32 / LANES heads at once.
// Seven blocks an SM: 72 registers a thread hold everything (8191 rows 24.0 us). With every lane making its eight
// angles itself: 24.7 with seven, 26.5 with eight (spills), 27.1 with six (fewer loads in flight).
template <int LANES>
__global__ void __launch_bounds__(kRopeThreads, 7) qk_norm_rope_kernel(const __grid_constant__ RopeParams p)
{
    constexpr int HD = LANES * 16, HEADS = 32 / LANES, OWN = 8 / HEADS;
    const int lane = threadIdx.x & 31, j = lane % LANES, sub = lane / LANES;
    const unsigned wid = blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const int64_t m = wid / (unsigned)p.parts;
    const int part = (int)(wid % (unsigned)p.parts);
    // the lane's chunks of 8 elements: j and j + rot16 hold the pairs (i, i + rot_dim / 2);
    // lanes behind the rotated part take the rest two by two
    const bool rot = j < p.rot16;
    const int c0 = rot ? j : 2 * (j - p.rot16) + 2 * p.rot16;
    const int c1 = rot ? j + p.rot16 : c0 + 1;
    // what the previous kernel did not write: gammas and frequencies (two registers a frequency). The lanes
    // of the warp's heads need the same eight angles: each makes OWN of them
    uint2 f[OWN];
    if (rot) {
#pragma unroll
        for (int k = 0; k < OWN; ++k) {
            const int i = sub * OWN + k, idx = p.interleaved ? (i < 4 ? c0 * 4 + i : c1 * 4 + i - 4) : j * 8 + i;
            f[k] = __ldg(reinterpret_cast<const uint2*>(p.turns + idx));
        }
    }
    pdl_wait();
    pdl_launch_dependents();
    if (m >= p.M)
        return;
    const int n_kv = p.c.n_kv, heads = p.n_q + 2 * n_kv;
    const uint4* row = reinterpret_cast<const uint4*>(p.qkv + m * p.ld) + sub * (HD / 8);
    // the next heads' chunks are under way while one set is worked on, the first while the angles are made
    uint4 na = {}, nb = {};
    auto fetch = [&](int h0) {
        if (h0 + sub < heads) {
            na = __ldcg(row + h0 * (HD / 8) + c0);
            nb = __ldcg(row + h0 * (HD / 8) + c1);
        }
    };
    fetch(part * HEADS);
    const int32_t slot = p.slots[m];
    // angle = position * turns modulo one turn, exact in 64 bits. Its sine and cosine keep their digits however
    // small they are: slow pairs turn by 1e-6 a token, where the fast functions' absolute error of 2^-21 is half
    // of the sine (9 % off at one token). A lane's share of them and sixteen shuffles take no longer than eight
    // fast ones: 8191 rows 24.0 us, 24.3 with those; CUDA's sincospif, all eight by every lane 25.7.
    float cs[8], sn[8];
    {
        float mine_c[OWN] = {}, mine_s[OWN] = {};
        if (rot) {
            const uint32_t pos = (uint32_t)p.positions[m];
            const uint32_t neg = (int32_t)pos < 0 ? 0xFFFFFFFFu : 0u;  // the sign of the 64-bit position
#pragma unroll
            for (int k = 0; k < OWN; ++k) {
                // (sign-extended position) * turns modulo 2^64
                const uint32_t hi = __umulhi(pos, f[k].x) + pos * f[k].y + neg * f[k].x, lo = pos * f[k].x;
                turn_sincos(hi, lo, mine_s[k], mine_c[k]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sn[i] = __shfl_sync(0xffffffffu, mine_s[i % OWN], i / OWN * LANES + j);
            cs[i] = __shfl_sync(0xffffffffu, mine_c[i % OWN], i / OWN * LANES + j);
        }
    }
    const bool bad = slot >= 0 && slot >= (int64_t)p.c.n_pages * p.c.page_size;
    if (bad && part == 0 && lane == 0)
        record_status(p.status, TF_E_INVALID_ARG);
    const bool store = slot >= 0 && !bad;
    const int page = store ? slot >> p.c.page_shift : 0, off = slot & (p.c.page_size - 1);
#pragma unroll 1
    for (int h0 = part * HEADS; h0 < heads; h0 += p.parts * HEADS) {
        const int h = h0 + sub;
        const bool live = h < heads;
        uint4 a = na, b = nb;
        fetch(h0 + p.parts * HEADS);
        const bool is_q = h < p.n_q, is_k = !is_q && h < p.n_q + n_kv;
        const uint4* gamma = reinterpret_cast<const uint4*>(is_q ? p.q_gamma : is_k ? p.k_gamma : nullptr);
        const bool norm = gamma != nullptr;
        if (h0 < p.n_q + n_kv) {  // else the warp has values alone
            float x[8], y[8];
            unpack8(a, x);
            unpack8(b, y);
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (norm) {
                const float r = rsqrtf(ss * (1.f / HD) + p.eps);
                float g0[8], g1[8];
                unpack8(__ldg(gamma + c0), g0);
                unpack8(__ldg(gamma + c1), g1);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = x[i] * r * g0[i];
                    y[i] = y[i] * r * g1[i];
                }
            }
            if (rot && (is_q || is_k)) {
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float u = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
                        x[2 * i + 1] = x[2 * i + 1] * cs[i] + x[2 * i] * sn[i];
                        x[2 * i] = u;
                        const float w = y[2 * i] * cs[4 + i] - y[2 * i + 1] * sn[4 + i];
                        y[2 * i + 1] = y[2 * i + 1] * cs[4 + i] + y[2 * i] * sn[4 + i];
                        y[2 * i] = w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float u = x[i] * cs[i] - y[i] * sn[i];
                        y[i] = y[i] * cs[i] + x[i] * sn[i];
                        x[i] = u;
                    }
                }
            }
            if (norm || (rot && (is_q || is_k))) {
                a = pack8(x);
                b = pack8(y);
            }
        }
        if (!live)
            continue;
        if (is_q) {
            uint4* o = reinterpret_cast<uint4*>(p.q + (m * p.n_q + h) * HD);
            o[c0] = a;
            o[c1] = b;
        } else if (store) {
            uint4* o = reinterpret_cast<uint4*>(
                p.c.data + (p.c.row_of(p.layer, is_k ? 0 : 1, page, h - p.n_q - (is_k ? 0 : n_kv)) + off) * HD);
            o[c0] = a;
            o[c1] = b;
        }
    }
}

}  // namespace
}  // namespace tfq

using namespace tfq;

extern "C" {

int tf_rope_turns(const double* inv_freq, int64_t n, uint64_t* turns)
{
    if (n < 0 || (n > 0 && (inv_freq == nullptr || turns == nullptr)))
        return report_error(TF_E_INVALID_ARG, "tf_rope_turns: NULL pointer or negative count");
    const double two_pi = 6.283185307179586;
    for (int64_t i = 0; i < n; ++i)
        if (!(std::fabs(inv_freq[i]) < two_pi))
            return report_error(TF_E_INVALID_ARG, "tf_rope_turns: inv_freq[%lld] is not within (-2 pi, 2 pi)", (long long)i);
    for (int64_t i = 0; i < n; ++i) {
        const double t = std::fabs(inv_freq[i]) / two_pi;  // below 1
        // 2^64 t without a double past 2^64: the top 53 bits as an integer, then shifted
        const uint64_t u = (uint64_t)std::ldexp(t, 63) << 1 | ((uint64_t)(std::ldexp(t, 64) - 2.0 * std::floor(std::ldexp(t, 63))) & 1);
        turns[i] = inv_freq[i] < 0 ? 0 - u : u;
    }
    return TF_OK;
}

int tf_qk_norm_rope_run(const uint16_t* qkv, int64_t ld, int64_t M, int n_q, const uint16_t* q_gamma,
                        const uint16_t* k_gamma, float eps, const int32_t* positions, const uint64_t* turns,
                        int rot_dim, int interleaved, uint16_t* q, const tf_kvcache* c, int layer,
                        const int32_t* slots, void* ws, size_t ws_bytes, unsigned flags, void* stream)
{
    const char* name = "tf_qk_norm_rope_run";
    RopeParams p{};
    int rc = check_cache(c, name, &p.c);
    if (rc || (rc = check_ws(ws, ws_bytes, 256, name)))
        return rc;
    if (qkv == nullptr || q == nullptr || slots == nullptr || positions == nullptr)
        return report_error(TF_E_INVALID_ARG, "%s: NULL pointer", name);
    if (n_q < 1 || n_q > 1024 || M < 1 || M >= ((int64_t)1 << 31) / 64)
        return report_error(TF_E_UNSUPPORTED_SHAPE, "%s: need 1 <= n_q <= 1024 and 1 <= M < 2^31 / 64", name);
    if (layer < 0 || layer >= p.c.n_layers)
        return report_error(TF_E_INVALID_ARG, "%s: layer %d outside the cache's %d", name, layer, p.c.n_layers);
    if (rot_dim < 0 || rot_dim > p.c.head_dim || rot_dim % 16 != 0)
        return report_error(TF_E_UNSUPPORTED_SHAPE, "%s: rot_dim must be a multiple of 16 within [0, head_dim]", name);
    if (rot_dim > 0 && (turns == nullptr || !is_aligned(turns, 8)))
        return report_error(TF_E_INVALID_ARG, "%s: turns NULL or misaligned", name);
    if (!is_aligned(qkv, 16) || !is_aligned(q, 16) || ld % 8 != 0 || ld < (int64_t)(n_q + 2 * p.c.n_kv) * p.c.head_dim)
        return report_error(TF_E_INVALID_ARG,
                            "%s: qkv and q must be 16-byte aligned, ld a multiple of 8 and >= (n_q + 2 n_kv) * head_dim",
                            name);
    if (rows_overlap(qkv, ld, (int64_t)(n_q + 2 * p.c.n_kv) * p.c.head_dim, q, (int64_t)n_q * p.c.head_dim,
                     (int64_t)n_q * p.c.head_dim, M))
        return report_error(TF_E_INVALID_ARG, "%s: q overlaps qkv", name);
    if (in_cache(p.c, q, (int64_t)n_q * p.c.head_dim, (int64_t)n_q * p.c.head_dim, M) ||
        in_cache(p.c, qkv, ld, (int64_t)(n_q + 2 * p.c.n_kv) * p.c.head_dim, M))
        return report_error(TF_E_INVALID_ARG, "%s: q or qkv overlaps the cache", name);
    if ((q_gamma != nullptr && !is_aligned(q_gamma, 16)) || (k_gamma != nullptr && !is_aligned(k_gamma, 16)) || !(eps >= 0.f))
        return report_error(TF_E_INVALID_ARG, "%s: gammas must be 16-byte aligned and eps >= 0", name);
    const size_t row = (size_t)p.c.head_dim * 2, rows = (size_t)M * 4;
    const MemRange ranges[] = {{q, M * n_q * row}, {positions, rows}, {slots, rows}, {rot_dim > 0 ? turns : nullptr, (size_t)rot_dim * 4},
                               {q_gamma, row}, {k_gamma, row}};
    if (outputs_overlap(ranges, 1, 6))
        return report_error(TF_E_INVALID_ARG, "%s: q overlaps another argument", name);
    p.qkv = qkv;
    p.ld = ld;
    p.M = M;
    p.n_q = n_q;
    p.q_gamma = q_gamma;
    p.k_gamma = k_gamma;
    p.eps = eps;
    p.positions = positions;
    p.turns = turns;
    p.rot16 = rot_dim / 16;
    p.interleaved = interleaved != 0;
    p.q = q;
    p.layer = layer;
    p.slots = slots;
    p.status = static_cast<int*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool pdl = (flags & TF_RUN_PDL) != 0;
    cudaError_t e;
    if (p.c.code == TF_KV_E4M3) {
        e = launch_rope8(p, pdl, s);
        return e == cudaSuccess ? TF_OK : report_error(TF_E_CUDA, "%s: %s", name, cudaGetErrorString(e));
    }
    // few rows: a row's heads spread over as many warps as it takes to fill the GPU. 16 warps an SM:
    // 2048 rows of 32 heads 7.6 us; 7.8 with 8, 8.4 with 32, 10.2 with 64; 512 rows 3.8 to 4.2 with any.
    const int per_warp = 512 / p.c.head_dim, groups = (n_q + 2 * p.c.n_kv + per_warp - 1) / per_warp;
    const int64_t want = (int64_t)device_sms() * 16;
    p.parts = 1;
    while (p.parts < groups && M * p.parts < want)
        p.parts *= 2;
    if (p.parts > groups)
        p.parts = groups;
    const unsigned grid = (unsigned)((M * p.parts + kRopeThreads / 32 - 1) / (kRopeThreads / 32));
    if (p.c.head_dim == 64)
        e = launch_pdl(qk_norm_rope_kernel<4>, dim3(grid), dim3(kRopeThreads), 0, s, pdl, p);
    else if (p.c.head_dim == 128)
        e = launch_pdl(qk_norm_rope_kernel<8>, dim3(grid), dim3(kRopeThreads), 0, s, pdl, p);
    else
        e = launch_pdl(qk_norm_rope_kernel<16>, dim3(grid), dim3(kRopeThreads), 0, s, pdl, p);
    return e == cudaSuccess ? TF_OK : report_error(TF_E_CUDA, "%s: %s", name, cudaGetErrorString(e));
}

}  // extern "C"
