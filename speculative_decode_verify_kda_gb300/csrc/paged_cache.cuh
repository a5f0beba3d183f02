// paged_cache.cuh -- what the kernels over a paged cache share: the sessions' lengths and
// rows, where a token lies, which keys a row sees, and the checks of the entry points.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "kda_internal.h"

namespace kda {
namespace pages {

constexpr int SMS = 152;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct Cache {
    uint16_t *k, *v;
    const int *table, *lens;
    long long page_stride, head_stride, slot_stride;
    int B, Hkv, D, shift, pages, cols;  // page = 1 << shift
    __host__ __device__ long long capacity() const { return static_cast<long long>(cols) << shift; }
};

// Which keys a row at position p sees: j <= p and (window == 0 or p - j < window or j < sinks).
struct Seen {
    int window, sinks;
};

__device__ __forceinline__ void raise(int *status, int bits)
{
    if (status)
        atomicOr(status, bits);
}

// A session's tokens n and rows t of this call.  False, with the status bits in `bad`, for a
// session that is left untouched; also (with no bits) for one without rows.
__device__ __forceinline__ bool session(const Cache &c, const int *t_rows, int T, int b, int &n, int &t, int &bad)
{
    n = c.lens[b];
    t = t_rows ? t_rows[b] : T;
    bad = 0;
    if (t < 0 || t > T)
        bad = KDA_ST_BADKEEP;
    else if (n < 0 || n + static_cast<long long>(t) > c.capacity())
        bad = KDA_ST_BADLEN;
    if (bad)
        t = 0;
    return t > 0;
}

// Offset of token j of session b in k and v for kv head h, or -1 for a bad page.
__device__ __forceinline__ long long token_at(const Cache &c, const int *table_row, int h, int j)
{
    const int id = table_row[j >> c.shift];
    if (id < 0 || id >= c.pages)
        return -1;
    return id * c.page_stride + h * c.head_stride + (j & ((1 << c.shift) - 1)) * c.slot_stride;
}

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The checks that every entry point over a cache makes (KDA_OK or KDA_EINVAL).
inline int check_cache(const kda_cache *c, Cache *out)
{
    if (!c)
        return fail(KDA_EINVAL, "cache must not be NULL");
    if (c->B < 0 || c->Hkv < 1 || (c->D != 64 && c->D != 128))
        return fail(KDA_EINVAL, "a cache needs B >= 0, Hkv >= 1 and D of 64 or 128");
    if (c->dtype != KDA_BF16 && c->dtype != KDA_F16)
        return fail(KDA_EINVAL, "a cache holds KDA_BF16 or KDA_F16");
    int shift = 3;
    while (shift < 10 && (1 << shift) != c->page)
        ++shift;
    if ((1 << shift) != c->page)
        return fail(KDA_EINVAL, "page must be a power of two in 8..1024, got " + std::to_string(c->page));
    if (c->pages < 1 || c->table_cols < 1 || static_cast<long long>(c->table_cols) * c->page > KDA_CACHE_MAX)
        return fail(KDA_EINVAL, "a cache needs pages >= 1 and 1 <= table_cols * page <= KDA_CACHE_MAX");
    for (long long s : {c->page_stride, c->head_stride, c->slot_stride})
        if (s < c->D || s % 8 || s >= (1ll << 38))
            return fail(KDA_EINVAL, "cache strides must be multiples of 8 elements, of D at least");
    if (c->Hkv > 65535)
        return fail(KDA_EINVAL, "Hkv must be at most 65535");
    if (c->B > 0 && (!c->k || !c->v || !c->table || !c->lens))
        return fail(KDA_EINVAL, "the cache's k, v, table and lens must not be NULL");
    if (!aligned16(c->k) || !aligned16(c->v))
        return fail(KDA_EINVAL, "the cache's k and v must be 16-byte aligned");
    if (!aligned4(c->table) || !aligned4(c->lens))
        return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    *out = Cache{static_cast<uint16_t *>(c->k), static_cast<uint16_t *>(c->v), c->table, c->lens, c->page_stride,
                 c->head_stride, c->slot_stride, c->B, c->Hkv, c->D, shift, c->pages, c->table_cols};
    return KDA_OK;
}

// Rows [B][T][width] with ld elements from row to row.
inline int check_rows(const Cache &c, const void *rows, int T, long long width, long long ld, const char *name)
{
    if (T < 0 || static_cast<long long>(c.B) * T > 0x7fffffffll)
        return fail(KDA_EINVAL, "T must be >= 0 and B * T fit in 32 bits");
    if (c.B == 0 || T == 0)
        return KDA_OK;
    if (!rows || !aligned16(rows))
        return fail(KDA_EINVAL, std::string(name) + " must not be NULL and must be 16-byte aligned");
    if (ld < width || ld % 8 || ld >= (1ll << 38))
        return fail(KDA_EINVAL, std::string(name) + ": ld must be a multiple of 8, of a row's elements at least");
    return KDA_OK;
}

inline int check_query(const Cache &c, int Hq, int window, int sinks, float scale)
{
    if (Hq < c.Hkv || Hq % c.Hkv || Hq / c.Hkv > KDA_GROUP_MAX)
        return fail(KDA_EINVAL, "Hq must be 1..128 times Hkv");
    if (window < 0 || sinks < 0)
        return fail(KDA_EINVAL, "window and sinks must be >= 0");
    if (!(scale >= KDA_SCALE_MIN && scale <= KDA_SCALE_MAX))
        return fail(KDA_EINVAL, "scale must lie in KDA_SCALE_MIN..KDA_SCALE_MAX");
    return KDA_OK;
}

// One launch that may begin while the kernel before it ends (it waits for that kernel's results
// itself) and that is given its arguments as they are.
template <class... A>
int launch(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream, const char *what,
           const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
    return check_launch(what);
}

// After the wait everything that the stream's earlier kernels wrote is visible; the next kernel
// may begin its own prologue.
__device__ __forceinline__ void after_previous()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace pages
}  // namespace kda
