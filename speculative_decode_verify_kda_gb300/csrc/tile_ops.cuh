// tile_ops.cuh -- the pieces of a pipeline on the fifth-generation tensor cores: barriers in
// shared memory with bounded waits, tensor copies, descriptors, products and tensor memory.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>

#include "kda_internal.h"

namespace kda {
namespace tiles {

constexpr uint64_t WAIT_NS = 1000000000ull;  // a wait gives up after one second

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// What a CTA does when a wait runs out: `gave_up` is set, every later wait returns at once, and
// the threads walk to the end of the kernel without results (no thread leaves a barrier short);
// there the status is raised and what the CTA had to compute becomes NaN.  The loop is short: it
// stands in the code wherever a warp waits.
__device__ __forceinline__ bool bar_wait_long(volatile int *gave_up, uint32_t bar, uint32_t parity, bool keep_on)
{
    const uint64_t t0 = now_ns();
    while (!bar_try(bar, parity)) {
        if (*gave_up && !keep_on)
            return false;
        if (now_ns() - t0 > WAIT_NS) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

// What `gave_up` starts with.  The tests' own build stops every n-th CTA so, as if its first wait had run out.
__device__ __forceinline__ int stopped()
{
#ifdef KDA_STOP_EVERY
    return blockIdx.x % KDA_STOP_EVERY == 0;
#else
    return 0;
#endif
}

// A warp's wait for the phase of `bar` with `parity`, for a second at most; the warp goes on
// together.  False (in every lane) when a lane gave up.
__device__ __forceinline__ bool warp_wait(volatile int *gave_up, uint32_t bar, uint32_t parity)
{
    if (__all_sync(0xffffffffu, bar_try(bar, parity)))
        return true;
    const bool ok = bar_wait_long(gave_up, bar, parity, false);
    return __all_sync(0xffffffffu, ok);
}

// One lane of a warp that is together.  Products, copies and their barriers are issued by
// `if (elect())` from values that are the same in every lane: so they stay in uniform registers
// (eight products issue in 206 cycles so, in 418 from inside `if (lane == 0)`).
__device__ __forceinline__ bool elect()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Ordinary writes to shared memory before this are seen by copies and products after it.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void copy_3d(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

__device__ __forceinline__ void copy_4d(uint32_t dst, const CUtensorMap *m, int x, int y, int z, int u, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(bar) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// ---- tensor memory ------------------------------------------------------------------
template <int COLS>
__device__ __forceinline__ void tmem_alloc(uint32_t dst)  // a whole warp; the address goes to shared memory
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

template <int COLS>
__device__ __forceinline__ void tmem_free(uint32_t addr)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "n"(COLS) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define KDA_OUT8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), \
                       "=r"(a[i + 6]), "=r"(a[i + 7])
#define KDA_IN8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), \
                      "r"(a[i + 6]), "r"(a[i + 7])

// 32 columns of this thread's lane (a warp reads the 32 lanes of its quarter).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : KDA_OUT8(r, 0), KDA_OUT8(r, 8), KDA_OUT8(r, 16), KDA_OUT8(r, 24) : "r"(addr));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(addr), KDA_IN8(r, 0), KDA_IN8(r, 8), KDA_IN8(r, 16), KDA_IN8(r, 24) : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16};"
                 ::"r"(addr), KDA_IN8(r, 0), KDA_IN8(r, 8) : "memory");
}

// ---- products -----------------------------------------------------------------------
// A tile in shared memory is rows of 128 bytes in groups of eight with the 128-byte swizzle, as
// a tensor copy writes it.  `group` bytes lie between groups of eight rows; `block` bytes between
// blocks of 64 elements along the rows where those are the product's M or N.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t block, uint32_t group)
{
    return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | static_cast<uint64_t>(block >> 4) << 16 |
           static_cast<uint64_t>(group >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// M x N products of 16-bit operands with f32 sums; b_rows: B's rows are the summed index.
__host__ __device__ constexpr uint32_t product_desc(bool bf16, int M, int N, bool b_rows)
{
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_rows ? 1u << 16 : 0u) | static_cast<uint32_t>(N >> 3) << 17 |
           static_cast<uint32_t>(M >> 4) << 24;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d), "l"(a), "l"(b), "r"(desc), "r"(static_cast<uint32_t>(add)) : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(desc), "r"(static_cast<uint32_t>(add)) : "memory");
}

// `bar` is arrived at once when this thread's products so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// ---- small arithmetic -----------------------------------------------------------------
__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));  // at most 2 ulp off; -inf gives 0
    return r;
}

// 32 bytes of a row: one store where they are aligned to their size.  (A thread a row touches a
// cache line a store; with 16 bytes a store the results took twice as many turns.)
__device__ __forceinline__ void store8(void *to, const uint32_t *x, bool wide)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), KDA_IN8(x, 0) : "memory");
    } else {
        static_cast<uint4 *>(to)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        static_cast<uint4 *>(to)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack(float lo, float hi)
{
    uint32_t r;
    if (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// a pair of 16-bit values times 0 plus another: NaN where a value is not finite or the other is NaN
template <bool BF16>
__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t sum)
{
    uint32_t r;
    if (BF16)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(sum));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(sum));
    return r;
}

template <bool BF16>
__device__ __forceinline__ bool is_nan2(uint32_t x)
{
    constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
    return (x & 0x7fffu) > E || (x >> 16 & 0x7fffu) > E;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));  // a NaN is passed over
    return r;
}

// Two f32 in one instruction.
struct Two {
    uint64_t x;
};

__device__ __forceinline__ Two two(uint32_t lo, uint32_t hi)
{
    Two r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.x) : "r"(lo), "r"(hi));
    return r;
}

__device__ __forceinline__ Two two(float lo, float hi) { return two(__float_as_uint(lo), __float_as_uint(hi)); }

__device__ __forceinline__ float2 apart(Two a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.x));
    return r;
}

__device__ __forceinline__ Two add2(Two a, Two b)
{
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.x) : "l"(a.x), "l"(b.x));
    return r;
}

__device__ __forceinline__ Two mul2(Two a, Two b)
{
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.x) : "l"(a.x), "l"(b.x));
    return r;
}

__device__ __forceinline__ Two fma2(Two a, Two b, Two c)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.x) : "l"(a.x), "l"(b.x), "l"(c.x));
    return r;
}

// ---- host ---------------------------------------------------------------------------
using EncodeTiled = PFN_cuTensorMapEncodeTiled_v12000;

inline EncodeTiled lookup_encode()
{
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    return reinterpret_cast<EncodeTiled>(f);
}

// Tensor map of 16-bit elements: dims and box innermost first, strides in bytes from the second
// dimension on, boxes 64 elements wide with the 128-byte swizzle.
inline int encode_map(CUtensorMap *m, bool bf16, int rank, const void *base, const cuuint64_t *dims,
                      const cuuint64_t *strides, const cuuint32_t *box)
{
    static const EncodeTiled encode = lookup_encode();
    if (!encode)
        return fail(KDA_ECUDA, "cuTensorMapEncodeTiled is not available from the CUDA driver");
    const cuuint32_t one[4] = {1, 1, 1, 1};
    const CUresult r = encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                              static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, box, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(KDA_ECUDA, "cuTensorMapEncodeTiled failed with CUresult " + std::to_string(static_cast<int>(r)));
    return KDA_OK;
}

}  // namespace tiles
}  // namespace kda
