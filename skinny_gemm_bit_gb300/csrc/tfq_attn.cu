// Attention of drafted rows (one token, a chain, a tree) over the paged cache.
//
//   o = sum_j softmax_j(scale q . k_j) v_j over the tokens a row sees: every token before its
//   sequence's block, and of the block those whose bits are set in the row's mask
//
// One warp takes one query head of one row: 32 keys at a time, a key a lane, with the
// running maximum and sum of the softmax; then the lanes hold the output's columns.
#include <cmath>

#include "tfq_cache.h"
#include "tfq_ptx.cuh"

namespace tfq {
namespace {

struct AttnParams {
    const uint16_t* q;
    int64_t ldq, M;
    int n_q, group;  // query heads, query heads of a key/value head
    CacheView c;
    int layer;
    const int32_t *seqs, *q_start;
    int B, max_rows;
    const uint64_t* masks;
    float scale_log2;  // scale * log2(e)
    uint16_t* o;
    int* status;
};

// Sequence b of the call: its rows and tokens, or why it has none.
struct SeqRows {
    int slot, r0, rows, base;  // rows r0 .. r0 + rows of q; tokens base .. base + rows of the slot
    bool rows_ok, ok;          // the rows lie within the call; and the rest holds too
};

__device__ __forceinline__ SeqRows seq_rows(const AttnParams& p, int b)
{
    SeqRows s;
    s.slot = p.seqs[b];
    s.r0 = p.q_start[b];
    const int r1 = p.q_start[b + 1];
    s.rows_ok = s.r0 >= 0 && s.r0 <= r1 && r1 <= p.M;
    s.rows = s.rows_ok ? r1 - s.r0 : 0;
    s.ok = s.rows_ok && s.rows <= p.max_rows && s.slot >= 0 && s.slot < p.c.n_seqs;
    s.base = 0;
    if (s.ok) {
        const int len = p.c.len[s.slot];
        s.base = len - s.rows;
        s.ok = s.base >= 0 && len <= (int64_t)p.c.max_pages << p.c.page_shift;
    }
    return s;
}

__global__ void __launch_bounds__(128) tree_attn_simple_kernel(const __grid_constant__ AttnParams p)
{
    __shared__ float qs[4][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SeqRows s = seq_rows(p, blockIdx.z);
    const int h = blockIdx.x * 4 + warp, hd = p.c.head_dim;
    pdl_wait();
    if (!s.ok && threadIdx.x == 0 && blockIdx.x == 0)
        record_status(p.status, TF_E_INVALID_ARG);
    if (h >= p.n_q)
        return;
    for (int i = blockIdx.y; i < s.rows; i += gridDim.y) {
        const int64_t m = s.r0 + i;
        for (int d = lane; d < hd; d += 32)
            qs[warp][d] = __uint_as_float((uint32_t)p.q[m * p.ldq + h * hd + d] << 16) * p.scale_log2;
        __syncwarp();
        float mx = -INFINITY, sum = 0.f, acc[8] = {};
        const uint64_t mask = p.masks == nullptr ? ~0ull >> (63 - i % 64) : p.masks[m];
        const int len = s.ok ? s.base + s.rows : 0;
        for (int k0 = 0; k0 < len; k0 += 32) {
            const int j = k0 + lane;
            const bool see = j < s.base || (j < len && (mask >> (j - s.base) & 1));
            float x = -INFINITY;
            int page = 0;
            if (see) {
                page = p.c.table[(int64_t)s.slot * p.c.max_pages + (j >> p.c.page_shift)];
                const bool good = page >= 0 && page < p.c.n_pages;
                x = 0.f;
                if (good) {
                    const uint16_t* k = p.c.data + (p.c.row_of(p.layer, 0, page, h / p.group) + (j & (p.c.page_size - 1))) * hd;
                    for (int d = 0; d < hd; ++d)
                        x = fmaf(qs[warp][d], __uint_as_float((uint32_t)k[d] << 16), x);
                } else {
                    record_status(p.status, TF_E_INVALID_ARG);
                    page = -1;
                }
            }
            float t = x;
            for (int o = 16; o > 0; o >>= 1)
                t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            const float now = fmaxf(mx, t), ref = now == -INFINITY ? 0.f : now;
            const float keep = exp2f(mx - ref), w = see ? exp2f(x - ref) : 0.f;
            mx = now;
            float ws = w;
            for (int o = 16; o > 0; o >>= 1)
                ws += __shfl_xor_sync(0xffffffffu, ws, o);
            sum = sum * keep + ws;
            for (int d = 0; d < 8; ++d)
                acc[d] *= keep;
            const unsigned seen = __ballot_sync(0xffffffffu, see);
            for (int l = 0; l < 32; ++l) {
                const float wl = __shfl_sync(0xffffffffu, w, l);
                const int pl = __shfl_sync(0xffffffffu, page, l);
                if (!(seen >> l & 1) || pl < 0)
                    continue;
                const uint16_t* v = p.c.data + (p.c.row_of(p.layer, 1, pl, h / p.group) + ((k0 + l) & (p.c.page_size - 1))) * hd;
                for (int d = 0; d < hd / 32; ++d)
                    acc[d] = fmaf(wl, __uint_as_float((uint32_t)v[d * 32 + lane] << 16), acc[d]);
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        for (int d = 0; d < hd / 32; ++d) {
            const __nv_bfloat16 r = __float2bfloat16_rn(acc[d] * inv);
            p.o[(m * p.n_q + h) * hd + d * 32 + lane] = *reinterpret_cast<const uint16_t*>(&r);
        }
        __syncwarp();
    }
}

}  // namespace
}  // namespace tfq

using namespace tfq;

extern "C" {

size_t tf_tree_attn_workspace_bytes(const tf_kvcache* c, int n_q, int64_t B, int max_rows)
{
    const char* name = "tf_tree_attn_workspace_bytes";
    CacheView v;
    if (check_cache(c, name, &v))
        return 0;
    if (n_q < 1 || n_q % v.n_kv != 0 || n_q / v.n_kv > 64 || B < 1 || B > 1024 || max_rows < 1 || max_rows > kMaxDraftRows) {
        report_error(TF_E_UNSUPPORTED_SHAPE, "%s: n_q, B or max_rows out of range", name);
        return 0;
    }
    return 256;
}

int tf_tree_attn_run(const uint16_t* q, int64_t ldq, int64_t M, int n_q, const tf_kvcache* c, int layer,
                     const int32_t* seqs, const int32_t* q_start, int64_t B, int max_rows, const uint64_t* masks,
                     float scale, uint16_t* o, void* ws, size_t ws_bytes, unsigned flags, void* stream)
{
    const char* name = "tf_tree_attn_run";
    AttnParams p{};
    int rc = check_cache(c, name, &p.c);
    if (rc)
        return rc;
    if (q == nullptr || o == nullptr || seqs == nullptr || q_start == nullptr)
        return report_error(TF_E_INVALID_ARG, "%s: NULL pointer", name);
    if (n_q < 1 || n_q % p.c.n_kv != 0 || n_q / p.c.n_kv > 64)
        return report_error(TF_E_UNSUPPORTED_SHAPE, "%s: n_q must be a multiple of n_kv, at most 64 query heads to one", name);
    if (B < 1 || B > 1024 || M < 1 || M > INT32_MAX / 1024 || max_rows < 1 || max_rows > kMaxDraftRows)
        return report_error(TF_E_UNSUPPORTED_SHAPE, "%s: need 1 <= B <= 1024, 1 <= M < 2^21 and 1 <= max_rows <= %d", name,
                            kMaxDraftRows);
    if (layer < 0 || layer >= p.c.n_layers)
        return report_error(TF_E_INVALID_ARG, "%s: layer %d outside the cache's %d", name, layer, p.c.n_layers);
    if (!is_aligned(q, 16) || !is_aligned(o, 16) || ldq % 8 != 0 || ldq < (int64_t)n_q * p.c.head_dim)
        return report_error(TF_E_INVALID_ARG, "%s: q and o must be 16-byte aligned, ldq a multiple of 8 and >= n_q * head_dim",
                            name);
    if (!std::isfinite(scale))
        return report_error(TF_E_INVALID_ARG, "%s: scale must be finite", name);
    if ((rc = check_ws(ws, ws_bytes, tf_tree_attn_workspace_bytes(c, n_q, B, max_rows), name)))
        return rc;
    p.q = q;
    p.ldq = ldq;
    p.M = M;
    p.n_q = n_q;
    p.group = n_q / p.c.n_kv;
    p.layer = layer;
    p.seqs = seqs;
    p.q_start = q_start;
    p.B = (int)B;
    p.max_rows = max_rows;
    p.masks = masks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.o = o;
    p.status = static_cast<int*>(ws);
    const cudaError_t e = launch_pdl(tree_attn_simple_kernel, dim3((n_q + 3) / 4, max_rows, (unsigned)B), dim3(128), 0,
                                     static_cast<cudaStream_t>(stream), (flags & TF_RUN_PDL) != 0, p);
    return e == cudaSuccess ? TF_OK : report_error(TF_E_CUDA, "%s: %s", name, cudaGetErrorString(e));
}

}  // extern "C"
