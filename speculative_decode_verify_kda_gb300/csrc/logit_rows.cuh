// logit_rows.cuh -- what the row reductions over logits share (spec_logprobs.cu,
// spec_distill.cu): element access, the order of (value, id) and sums over a CTA.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "kda_internal.h"

namespace kda {
namespace rows {

constexpr int THREADS = 256;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

template <bool BF16>
__device__ __forceinline__ float element(const void *p, long long i)
{
    if (BF16)
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
    return static_cast<const float *>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void put(void *p, long long i, float x)
{
    if (BF16) {
        uint16_t b;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(x));
        static_cast<uint16_t *>(p)[i] = b;
    } else {
        static_cast<float *>(p)[i] = x;
    }
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Whole numbers in the order of the floats; the two zeros are one value.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float from_ordered(uint32_t o)
{
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

// Alternatives are ordered by (value descending, id ascending): a larger key comes
// first.  0 is below every finite logit's key and stands for "none".
__device__ __forceinline__ unsigned long long key_of(float x, int id)
{
    return (static_cast<unsigned long long>(ordered(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}

__device__ __forceinline__ int key_id(unsigned long long key)
{
    return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
}

// Reductions over the CTA's THREADS threads; `buf` holds one value a warp and may be
// used again after the call.
template <class T, class Op>
__device__ __forceinline__ T block_reduce(T v, Op op, T *buf)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w)
        v = op(v, buf[w]);
    return v;
}

// Argument checks that every entry point over logits makes (KDA_OK or KDA_EINVAL).
inline int check_logits(const void *logits, int dtype, int N, int V, long long ld, float temperature)
{
    if (N < 0)
        return fail(KDA_EINVAL, "N must be >= 0");
    if (V < 1)
        return fail(KDA_EINVAL, "V must be >= 1");
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return fail(KDA_EINVAL, "logit_dtype must be KDA_F32 or KDA_BF16");
    if (ld < V)
        return fail(KDA_EINVAL, "ld must be >= V, got " + std::to_string(ld));
    if (!(temperature >= KDA_TEMPERATURE_MIN && temperature <= KDA_TEMPERATURE_MAX))
        return fail(KDA_EINVAL, "temperature must lie in 1e-4..1e4");
    if (N > 0 && !logits)
        return fail(KDA_EINVAL, "logits must not be NULL");
    if (reinterpret_cast<uintptr_t>(logits) % (dtype == KDA_BF16 ? 2 : 4))
        return fail(KDA_EINVAL, "logits must be aligned to their element");
    return KDA_OK;
}

// An output of logit gradients: present, aligned, and either the logits themselves (the
// same rows) or apart from them.
inline int check_grad(const void *logits, const void *grad, int dtype, int N, int V, long long ld, long long ldg)
{
    const uintptr_t es = dtype == KDA_BF16 ? 2 : 4;
    const uintptr_t x = reinterpret_cast<uintptr_t>(logits), g = reinterpret_cast<uintptr_t>(grad);
    if (N > 0 && !grad)
        return fail(KDA_EINVAL, "dlogits must not be NULL");
    if (ldg < V)
        return fail(KDA_EINVAL, "ldg must be >= V, got " + std::to_string(ldg));
    if (g % es)
        return fail(KDA_EINVAL, "dlogits must be aligned to their element");
    if (N > 0 && !(x == g && ld == ldg)) {
        const uintptr_t xe = x + es * (static_cast<uintptr_t>(N - 1) * ld + V);
        const uintptr_t ge = g + es * (static_cast<uintptr_t>(N - 1) * ldg + V);
        if (x < ge && g < xe)
            return fail(KDA_EINVAL, "dlogits must be the logits themselves (same ld) or not overlap them");
    }
    return KDA_OK;
}

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace rows
}  // namespace kda
