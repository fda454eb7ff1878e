// Attention of drafted rows (one token, a chain, a tree) over the paged cache: the entry point.
//
//   o = sum_j softmax_j(scale q . k_j) v_j over the tokens a row sees: every token before its
//   sequence's block, and of the block those whose bits are set in the row's mask
#include <cmath>

#include "tfq_attn.cuh"

namespace tfq {
namespace {

// Query rows of an item, and with them the kernel: up to 32 the warp MMAs, above the tensor-memory
// MMAs (which need the output of two row groups in tensor memory: head_dim up to 128). 8 key/value
// heads of 128, in us, warp and tensor-memory MMAs: 32 rows over 64 x 8192 tokens in pages of 16 329 and
// 417, over one sequence of 32,768 35 and 41, over 8 x 4096 43 and 49; 8 rows over 4097 11.6 and 18.9; 40 rows
// (two items of the warps') over 64 x 8192 633 and 342, over 32,768 64 and 38.
int attn_rows(int max_rows, int group, int head_dim)
{
    const int r = max_rows * group;
    if (head_dim > 128 || r <= 16)
        return 16;
    if (r <= 32)
        return 32;
    return r <= 128 ? 128 : 256;
}

// A segment's own cost in key tiles of its kernel, by which the CTAs' shares are measured. With more
// items than CTAs it is what evens out those that get several short ones (28 of the warp kernel's 32-key
// tiles: 64 ragged sequences 176 us, 183 with 16, 199 with 8, side by side); with fewer, what a CTA gets should
// still be a tile a warp (one token over 4097: 12.0 us with 16, 13.4 with 24).
int attn_over(int rows, int64_t items)
{
    if (rows > 32)  // 64-key tiles: 64-row trees over 16,001 tokens 131 us, 134 with 32, 135 with 8, side by side
        return 20;
    return items > device_sms() ? 28 : 16;
}

struct AttnLayout {
    size_t counters, parts, total;
};

AttnLayout attn_layout(int head_dim, int rows)
{
    AttnLayout L{};
    L.counters = 256;
    L.parts = L.counters + ((size_t)device_sms() * 2 * sizeof(unsigned) + 255) / 256 * 256;
    L.total = L.parts + (size_t)2 * device_sms() * rows * (head_dim + 2) * sizeof(float);  // two parts a CTA
    return L;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder; nullptr where there is no driver.
EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return (EncodeTiled) nullptr;
        }
        return (EncodeTiled)f;
    }();
    return fn;
}

// The pool as {64 columns, rows, head_dim / 64}: a box is `rows` rows of `halves` times 64 columns
// (128 bytes a row, swizzled), one 64 after the other.
bool encode_rows(const CacheView& c, int total_rows, int rows, int halves, CUtensorMap* map)
{
    const EncodeTiled fn = encode_tiled();
    if (fn == nullptr)
        return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)total_rows, (cuuint64_t)c.head_dim / 64};
    const cuuint64_t strides[2] = {(cuuint64_t)c.head_dim * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)rows, (cuuint32_t)halves}, one[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c.data, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    return attn_layout(v.head_dim, attn_rows(max_rows, n_q / v.n_kv, v.head_dim)).total;
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
    if (rows_overlap(q, ldq, (int64_t)n_q * p.c.head_dim, o, (int64_t)n_q * p.c.head_dim, (int64_t)n_q * p.c.head_dim, M))
        return report_error(TF_E_INVALID_ARG, "%s: o overlaps q", name);
    if (in_cache(p.c, o, (int64_t)n_q * p.c.head_dim, (int64_t)n_q * p.c.head_dim, M))
        return report_error(TF_E_INVALID_ARG, "%s: o overlaps the cache", name);
    const MemRange ranges[] = {{o, (size_t)M * n_q * p.c.head_dim * 2}, {seqs, (size_t)B * 4}, {q_start, (size_t)(B + 1) * 4},
                               {masks, (size_t)M * 8}};
    if (outputs_overlap(ranges, 1, 4))
        return report_error(TF_E_INVALID_ARG, "%s: o overlaps another argument", name);
    if (!std::isfinite(scale))
        return report_error(TF_E_INVALID_ARG, "%s: scale must be finite", name);
    if ((rc = check_ws(ws, ws_bytes, tf_tree_attn_workspace_bytes(c, n_q, B, max_rows), name)))
        return rc;
    p.q = q;
    p.ldq = ldq;
    p.M = M;
    p.n_q = n_q;
    p.group = n_q / p.c.n_kv;
    p.group_inv = ((1u << 20) + p.group - 1) / p.group;
    p.layer = layer;
    p.seqs = seqs;
    p.q_start = q_start;
    p.B = (int)B;
    p.max_rows = max_rows;
    p.masks = masks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.o = o;
    p.status = static_cast<int*>(ws);
    (void)flags;  // the launch is cooperative, which excludes a programmatic dependent one
    p.total_rows = (int)p.c.row_of(p.c.n_layers, 0, 0, 0);
    p.limit_ns = kDefaultWaitLimitNs;
    const int rows = attn_rows(max_rows, p.group, p.c.head_dim);
    const int64_t items = B * p.c.n_kv * ((max_rows * p.group + rows - 1) / rows);
    p.over = attn_over(rows, items);
    p.few = items <= device_sms() && B <= 256;
    const AttnLayout L = attn_layout(p.c.head_dim, rows);
    p.counters = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + L.counters);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + L.parts);
    CUtensorMap map;
    const bool tc = rows > 64;
    if (!encode_rows(p.c, p.total_rows, tc ? attn_tc_box(p.c.page_size) : attn_warp_box(p.c.head_dim, p.c.page_size),
                     tc ? 1 : p.c.head_dim / 64, &map))
        return report_error(TF_E_CUDA, "%s: the cache's tensor map could not be made", name);
    const cudaError_t e = (tc ? launch_attn_tc : launch_attn_warp)(p, rows, map, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? TF_OK : report_error(TF_E_CUDA, "%s: %s", name, cudaGetErrorString(e));
}

}  // extern "C"
