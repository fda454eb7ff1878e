// The K/V cache as its kernels see it, and the checks its entry points share.
#pragma once

#include <atomic>

#include "tfq_internal.h"

namespace tfq {

constexpr int kMaxSeqs = 1024;
constexpr int kMaxDraftRows = TF_MAX_DRAFT_ROWS;

// Passed by value. Row r of page p of head h (K: kv = 0, V: 1) of a layer starts at element
//   ((((layer * 2 + kv) * n_pages + p) * n_kv + h) * page_size + r) * head_dim   (64 bits)
// Of an 8-bit cache `data` holds bytes, and pool row i (row_of + r) belongs to the block with scale byte i / 16.
struct CacheView {
    uint16_t* data;
    int32_t *len, *refs, *table;
    int n_layers, n_kv, head_dim, page_size, page_shift;
    int n_seqs, n_pages, max_pages;
    int code;         // TF_KV_*
    uint8_t* scales;  // of an 8-bit cache
    __host__ __device__ uint8_t* codes() const { return reinterpret_cast<uint8_t*>(data); }
    __host__ __device__ int elem_bytes() const { return code == TF_KV_E4M3 ? 1 : 2; }

    __host__ __device__ int64_t row_of(int layer, int kv, int page, int head) const
    {
        return (((int64_t)(layer * 2 + kv) * n_pages + page) * n_kv + head) * page_size;
    }
};

// Validate a descriptor filled by tf_kvcache_init; fills `v` (tfq_kvcache.cu).
int check_cache(const tf_kvcache* c, const char* name, CacheView* v);
// ws at least `need` bytes, 256-byte aligned
int check_ws(const void* ws, size_t ws_bytes, size_t need, const char* name);

inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Whether rows x cols elements of 2 bytes at a (leading dimension lda) and at b share memory.
inline bool rows_overlap(const void* a, int64_t lda, int64_t cols_a, const void* b, int64_t ldb, int64_t cols_b, int64_t rows)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + (uintptr_t)((rows - 1) * ldb + cols_b) * 2 && b0 < a0 + (uintptr_t)((rows - 1) * lda + cols_a) * 2;
}

struct MemRange {
    const void* p;
    size_t bytes;
};

inline bool overlap(const MemRange& a, const MemRange& b)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p != nullptr && b.p != nullptr && a.bytes != 0 && b.bytes != 0 && x < y + b.bytes && y < x + a.bytes;
}

// Whether one of the first n_out (the outputs) shares memory with another of the n.
inline bool outputs_overlap(const MemRange* r, int n_out, int n)
{
    for (int i = 0; i < n_out; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlap(r[i], r[j]))
                return true;
    return false;
}

// Whether a range, or rows x cols elements of 2 bytes (leading dimension ld), shares memory with the cache's data or book.
inline bool in_cache(const CacheView& c, const MemRange& r)
{
    return overlap(r, MemRange{c.data, (size_t)c.row_of(c.n_layers, 0, 0, 0) * c.head_dim * c.elem_bytes()}) ||
           overlap(r, MemRange{c.scales, (size_t)c.row_of(c.n_layers, 0, 0, 0) / TF_KV_BLOCK}) ||
           overlap(r, MemRange{c.len, (c.n_seqs + (size_t)c.n_pages + (size_t)c.n_seqs * c.max_pages) * 4});
}
inline bool in_cache(const CacheView& c, const void* a, int64_t ld, int64_t cols, int64_t rows)
{
    return in_cache(c, MemRange{a, (size_t)((rows - 1) * ld + cols) * 2});
}

// Launch with (or without) programmatic dependent launch on the previous kernel.
template <class... KArgs, class... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
                       Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Raise a kernel's dynamic shared-memory limit, once for each device. `done` is the kernel's own.
template <class Kernel>
cudaError_t allow_smem(Kernel* kernel, int bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit != 0 && (done.load(std::memory_order_relaxed) & bit))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// The four E4M3 bytes of v as two fp16 pairs, bytes 0 and 1 in r0.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t v, uint32_t& r0, uint32_t& r1)
{
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}" : "=r"(r0), "=r"(r1) : "r"(v));
}

// lo and hi as E4M3, rounded to nearest even, +-448 where larger (bits 0-7 and 8-15).
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void record_status(int* status, int code) { atomicCAS(status, 0, code); }

}  // namespace tfq
