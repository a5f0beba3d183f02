// logit_rows.cuh -- what the row reductions over logits share (spec_logprobs.cu,
// spec_distill.cu).
//
// A row is read in 16-byte vectors and belongs to one CTA or to a cluster of CTAs, each
// of which takes a run of the row's vectors.  They pass through shared memory ahead of their
// use (Run); a thread works on a few of them at a time, in registers (Tile).
//
// The sums are taken relative to a logit of the warp's own (Running), and a warp's triple
// (maximum, sum of weights, weighted sum of exponents) joins the others' once, through the
// shared memory of the CTA or of every CTA of the cluster: one barrier between reading a row
// and knowing its statistics.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <string>
#include <type_traits>

#include "kda_internal.h"

namespace kda {
namespace rows {

namespace cg = cooperative_groups;

constexpr int SMS = 152;           // of a GB300
constexpr int MAX_CL = 8;          // CTAs of a cluster (the portable size)
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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));  // at most 2 ulp off; -inf gives 0
    return r;
}

// Two f32 operations in one instruction.
struct F2 {
    unsigned long long b;
};
__device__ __forceinline__ F2 f2(float lo, float hi)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.b) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 split(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.b));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(b.b), "l"(c.b));
    return r;
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

__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float warp_max_nan(float x)
{
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The value of rank r (0 the largest) among the warp's 32.
template <class T>
__device__ __forceinline__ T warp_rank(T x, int r)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
        for (int j = k >> 1; j; j >>= 1) {  // a bitonic network, descending over the lanes
            const T y = __shfl_xor_sync(0xffffffffu, x, j);
            const bool up = ((lane & k) == 0) == ((lane & j) == 0);
            x = up == (x > y) ? x : y;
        }
    }
    return __shfl_sync(0xffffffffu, x, r);
}

// ---------------------------------------------------------------------------
// A row in 16-byte vectors
// ---------------------------------------------------------------------------
// The vector at p whose first element has the place `first` in a row of V: the elements
// outside of the row are -inf and not read.
template <bool BF16>
__device__ __noinline__ uint4 edge_vector(const char *p, int first, int V)
{
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (BF16) {
            const volatile uint16_t *x = reinterpret_cast<const volatile uint16_t *>(p) + 2 * k;
            const int e = first + 2 * k;
            const uint32_t lo = e >= 0 && e < V ? x[0] : 0xff80u, hi = e + 1 >= 0 && e + 1 < V ? x[1] : 0xff80u;
            w[k] = lo | (hi << 16);
        } else {
            const int e = first + k;
            w[k] = e >= 0 && e < V ? reinterpret_cast<const volatile uint32_t *>(p)[k] : 0xff800000u;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The vector's elements, the first of which has the place `first` in a row of V, one by one to
// p; those outside of the row are left out.
template <bool BF16>
__device__ __noinline__ void store_elements(char *p, int first, int V, uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < (BF16 ? 8 : 4); ++k) {
        if (first + k < 0 || first + k >= V)
            continue;
        if (BF16)
            reinterpret_cast<uint16_t *>(p)[k] = static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1)));
        else
            reinterpret_cast<uint32_t *>(p)[k] = w[k];
    }
}

template <bool BF16>
struct RowPtr {
    static constexpr int PER = BF16 ? 8 : 4;  // elements of a vector
    static constexpr int ES = BF16 ? 2 : 4;
    static constexpr uint32_t MASKED = BF16 ? 0xff80ff80u : 0xff800000u;  // -inf

    char *base;   // the row's address rounded down to a vector
    int skip;     // elements of the first vector that precede the row
    int V, nvec;  // elements and vectors of the row
    int full0, full1;  // the vectors [full0, full1) lie wholly inside the row

    __device__ __forceinline__ RowPtr(const void *p, long long first, int V_) : V(V_)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(first) * ES;
        skip = static_cast<int>(at & 15u) / ES;
        base = reinterpret_cast<char *>(at & ~static_cast<uintptr_t>(15));
        nvec = (skip + V + PER - 1) / PER;
        full0 = skip > 0;
        full1 = (skip + V) / PER;
    }
    __device__ __forceinline__ bool full(int i) const { return i >= full0 && i < full1; }
    __device__ __forceinline__ int first_id(int i) const { return i * PER - skip; }

    // A vector that lies wholly inside the row.  No ordinary load may take this one's place:
    // the logits may be overwritten later in the same kernel.
    __device__ __forceinline__ uint4 load(int i) const
    {
        uint4 v;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(base + 16ll * i));
        return v;
    }
    __device__ __forceinline__ uint4 load_edge(int i) const { return edge_vector<BF16>(base + 16ll * i, first_id(i), V); }
    __device__ __forceinline__ float at(int id) const
    {
        const char *p = base + (static_cast<long long>(skip) + id) * ES;
        if (BF16)
            return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const volatile uint16_t *>(p)) << 16);
        return *reinterpret_cast<const volatile float *>(p);
    }
    __device__ __forceinline__ void set(int id, float x) const
    {
        put<BF16>(base, static_cast<long long>(skip) + id, x);
    }
    __device__ __forceinline__ void store(int i, uint4 v) const
    {
        *reinterpret_cast<uint4 *>(base + 16ll * i) = v;
    }
    // Vector i of `src` (which starts at another place in its vector, or crosses an end of the
    // row) into this row.
    __device__ __forceinline__ void store_edge(const RowPtr &src, int i, uint4 v) const
    {
        const int e = src.first_id(i);
        store_elements<BF16>(base + (static_cast<long long>(skip) + e) * ES, e, V, v);
    }
};

// The vectors first, first + step, ... below `end` of a row in registers, masked past the end.
template <bool BF16, int VPT>
struct Tile {
    uint4 v[VPT];

    __device__ __forceinline__ void load(const RowPtr<BF16> &row, int first, int step, int end)
    {
        constexpr uint32_t M = RowPtr<BF16>::MASKED;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = first + j * step;
            v[j] = make_uint4(M, M, M, M);
            if (i < end && row.full(i))
                v[j] = row.load(i);
        }
        if (row.full0 > 0)
            load_edge(row, 0, first, step, end);
        if (row.full1 < row.nvec && (row.full0 == 0 || row.nvec > 1))
            load_edge(row, row.nvec - 1, first, step, end);
    }
    // Vector i, which crosses an end of the row, if it is one of the thread's.
    __device__ __forceinline__ void load_edge(const RowPtr<BF16> &row, int i, int first, int step, int end)
    {
        const int j0 = (i - first) / step;
        if (i < first || i >= end || j0 >= VPT || first + j0 * step != i)
            return;
        const uint4 u = row.load_edge(i);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (j == j0)
                v[j] = u;
    }

    // f(pair of neighbouring elements) for every pair; with a floor: elements below it raised.
    template <class F>
    __device__ __forceinline__ void each(F f) const
    {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            each_of(v[j], f);
    }
    template <class F>
    __device__ __forceinline__ void each_above(uint32_t floor, F f) const
    {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (BF16)
                    asm("max.bf16x2 %0, %0, %1;" : "+r"(w[k]) : "r"(floor));
                else
                    w[k] = __float_as_uint(fmaxf(__uint_as_float(w[k]), __uint_as_float(floor)));
            }
            each_of(make_uint4(w[0], w[1], w[2], w[3]), f);
        }
    }
    template <class F>
    static __device__ __forceinline__ void each_of(const uint4 &u, F f)
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if (BF16) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                f(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
        } else {
            f(__uint_as_float(w[0]), __uint_as_float(w[1]));
            f(__uint_as_float(w[2]), __uint_as_float(w[3]));
        }
    }

    // The largest element of the vectors [J0, J1), or a NaN.
    template <int J0 = 0, int J1 = VPT>
    __device__ __forceinline__ float max_of() const
    {
        if (BF16) {
            uint32_t m = max_nan_bf16x2(max_nan_bf16x2(v[J0].x, v[J0].y), max_nan_bf16x2(v[J0].z, v[J0].w));
#pragma unroll
            for (int j = J0 + 1; j < J1; ++j)
                m = max_nan_bf16x2(m, max_nan_bf16x2(max_nan_bf16x2(v[j].x, v[j].y), max_nan_bf16x2(v[j].z, v[j].w)));
            return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
        }
        float m = -INFINITY;
#pragma unroll
        for (int j = J0; j < J1; ++j)
            each_of(v[j], [&](float p, float q) { m = max_nan(m, max_nan(p, q)); });
        return m;
    }
};

// f(pair) of every pair of a tile of `src` into the same elements of `out`, or zeros.
template <bool BF16, int VPT, class F>
__device__ __forceinline__ void store_tile(const Tile<BF16, VPT> &t, const RowPtr<BF16> &src,
                                           const RowPtr<BF16> &out, int first, int step, int end, bool zero, F f)
{
    const bool even = src.skip == out.skip;  // vector for vector
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = first + j * step;
        if (i >= end)
            break;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (!zero) {
            int k = 0;
            t.each_of(t.v[j], [&](float p, float q) {
                const float2 d = split(f(p, q));
                if (BF16) {
                    w[k++] = pack_bf16(d.x, d.y);
                } else {
                    w[k++] = __float_as_uint(d.x);
                    w[k++] = __float_as_uint(d.y);
                }
            });
        }
        const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
        if (even && src.full(i))
            out.store(i, v);
        else
            out.store_edge(src, i, v);
    }
}

// What a warp hands to the others: its maximum, its sums without the maximum's own term (whose
// weight is 1), and a value of its largest ones.
struct __align__(16) Part {
    float m, S, E;
    uint32_t key;
};


// The same for a tile whose vectors, STEP apart, all lie in the row and go to whole vectors at p.
template <int STEP, bool BF16, int VPT, class F>
__device__ __forceinline__ void store_whole(const Tile<BF16, VPT> &t, uint4 *p, F f)
{
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        uint32_t w[4];
        int k = 0;
        t.each_of(t.v[j], [&](float x, float y) {
            const float2 d = split(f(x, y));
            if (BF16) {
                w[k++] = pack_bf16(d.x, d.y);
            } else {
                w[k++] = __float_as_uint(d.x);
                w[k++] = __float_as_uint(d.y);
            }
        });
        p[j * STEP] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Logits to exponents of two.
struct Scale {
    float c;       // log2(e) / temperature
    float margin;  // 16 / c
    float inv;     // 1 / temperature
};

// Sums of a warp's share of a row relative to a logit `at`, in units of exp2: c =
// log2(e) / tau, d = (x - at) c, S = sum 2^d, E = sum d 2^d; the sums are the lane's.
//
// `at` is the warp's largest logit so far or one at most 2^16 times less likely, so it
// rarely moves after the first tile.  A term costs one multiply-add, x c - ref with ref =
// at c rounded: what the rounding left out is the same for every term and is put back by
// settle().  From |at| c = 2^30 on it could be more than an exponent holds; two different
// f32 logits are then 2^6 apart in units of exp2, so that nothing but the largest ones
// counts, and a smaller c with |at| c = 2^30 gives just that.
template <bool ENTROPY>
struct Running {
    static constexpr float FAR = 1073741824.0f;
    float at = -INFINITY, limit = -INFINITY;  // a maximum above `limit` moves `at`
    float c = 0.0f, ref = 0.0f;
    F2 s = F2{0}, e = F2{0};

    // The sums relative to `top`; z.c is the row's.
    __device__ __forceinline__ void settle(float top, Scale z, float &S, float &E) const
    {
        const float2 s2 = split(s), e2 = split(e);
        // a term's exponent was (x - at) c + left
        const float left = fmaf(at, c, -ref), d = fmaxf((at - top) * z.c - left, -1e4f), w = ex2(d);
        S = (s2.x + s2.y) * w;
        E = c == z.c ? (e2.x + e2.y) * w + S * d : 0.0f;  // (among equal logits d = 0)
    }

    template <bool BF16, int N>
    __device__ __forceinline__ void add(const Tile<BF16, N> &t, float tile_max, Scale z)
    {
        if (__any_sync(0xffffffffu, !(tile_max <= limit))) {
            const float top = max_nan(at, warp_max_nan(tile_max));
            float S = 0.0f, E = 0.0f;
            if (at != -INFINITY)
                settle(top, z, S, E);
            s = f2(S, 0.0f);
            e = f2(E, 0.0f);
            at = top;
            limit = top + z.margin;
            c = fabsf(top * z.c) < FAR ? z.c : FAR / fabsf(top);
            ref = top * c;
        }
        if (at == -INFINITY)  // nothing but masked tokens so far
            return;
        // a tile's sums are formed apart: a long row's are then sums of sums
        const F2 cc = f2(c, c), neg = f2(-ref, -ref);
        F2 ts = f2(0.0f, 0.0f), te = ts;
        if (ENTROPY) {
            // a masked token's term of the entropy is 0, not 0 times -inf: its logit is raised
            // to -1e30 (0xf149 as bf16), where its weight is 0 as well, unless that is among
            // the largest ones
            const bool raise = c == z.c;
            const uint32_t floor = BF16 ? (raise ? 0xf149f149u : 0xff80ff80u) : (raise ? 0xf149f2cau : 0xff800000u);
            t.each_above(floor, [&](float p, float q) {
                const F2 d = fma2(f2(p, q), cc, neg);
                const float2 u = split(d);
                const F2 w = f2(ex2(u.x), ex2(u.y));
                ts = ts + w;
                te = fma2(w, d, te);
            });
            e = e + te;
        } else {
            t.each([&](float p, float q) {
                const float2 u = split(fma2(f2(p, q), cc, neg));
                ts = ts + f2(ex2(u.x), ex2(u.y));
            });
        }
        s = s + ts;
    }

    // The warp's part, from the lanes' largest logits.  The largest one's own term is 1 and its
    // exponent 0: what was added for it is taken back out of its lane's sums (it was formed by the
    // same operations), so that in a row where one token has nearly everything the others'
    // share is not lost in the rounding of that one exponential.
    __device__ __forceinline__ Part part(float most, Scale z, uint32_t key) const
    {
        const float top = warp_max_nan(most);
        float S = 0.0f, E = 0.0f;
        if (top != -INFINITY) {
            const float2 s2 = split(s), e2 = split(e);
            const float own = fmaf(top, c, -ref), w_own = ex2(own);
            const unsigned lanes = __ballot_sync(0xffffffffu, most == top);
            const bool here = lanes && (threadIdx.x & 31) == __ffs(lanes) - 1;
            const float left = fmaf(at, c, -ref), d = (at - top) * z.c - left, w = ex2(d);
            S = (here ? fmaxf(s2.x + s2.y - w_own, 0.0f) : s2.x + s2.y) * w;
            E = c == z.c ? (here ? fmaf(-w_own, own, e2.x + e2.y) : e2.x + e2.y) * w + S * d : 0.0f;
        }
        return Part{top, warp_sum(S), ENTROPY ? warp_sum(E) : 0.0f, key};
    }
};

struct Stats {
    float m, lnS, entropy;  // NaN for a row with a NaN or +inf, (-inf, -inf, 0) for an empty one
    __device__ __forceinline__ bool bad() const { return m != m; }
    __device__ __forceinline__ bool empty() const { return m == -INFINITY; }
};

// The row's statistics from its parts (every lane of the calling warp gets them).  The order
// of the sums is fixed by the parts' places.
__device__ __forceinline__ Stats join(const Part *parts, int n, float c)
{
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
#pragma unroll 1
    for (int p = lane; p < n; p += 32)
        m = max_nan(m, parts[p].m);
    m = warp_max_nan(m);
    if (m == -INFINITY)
        return Stats{m, m, 0.0f};
    if (!(m < INFINITY))
        return Stats{NAN, NAN, NAN};
    // S = 1 + R: one part that holds the row's maximum gives the 1
    int first = n;
#pragma unroll 1
    for (int p = lane; p < n; p += 32)
        if (first == n && parts[p].m == m)
            first = p;
    first = __reduce_min_sync(0xffffffffu, first);
    float R = 0.0f, E = 0.0f;
#pragma unroll 1
    for (int p = lane; p < n; p += 32) {
        const Part q = parts[p];
        const float d = fmaxf((q.m - m) * c, -1e4f), w = ex2(d);
        const float one = q.m != -INFINITY && p != first ? 1.0f : 0.0f;
        R += (q.S + one) * w;
        E += (q.E + (q.S + one) * d) * w;
    }
    R = warp_sum(R);
    E = warp_sum(E);
    const float lnS = log1pf(R);
    return Stats{m, lnS, fmaxf(lnS - LN2 * __fdividef(E, 1.0f + R), 0.0f)};
}

// ln p of a logit, inv = 1 / temperature.  The difference is formed of the halves, which are
// exact (but for subnormals): between logits at both ends of the range it would pass it, and
// the quotient by a temperature above 1 need not.
__device__ __forceinline__ float log_prob(float x, const Stats &st, float inv)
{
    return (0.5f * x - 0.5f * st.m) * (2.0f * inv) - st.lnS;
}

// The CTA's place: its row, its run of the row's vectors, and its cluster.
struct Place {
    long long row;
    int rank, cl, shift, warps;  // cl = 2^shift
    __device__ __forceinline__ Place(int cl_, int threads)
        : cl(cl_), shift((cl_ > 1) + (cl_ > 2) + (cl_ > 4)), warps(threads >> 5)
    {
        row = blockIdx.x >> shift;
        rank = blockIdx.x & (cl - 1);
    }
    __device__ __forceinline__ int begin(int nvec) const { return rank * per(nvec); }
    __device__ __forceinline__ int end(int nvec) const { return min(nvec, (rank + 1) * per(nvec)); }
    __device__ __forceinline__ int per(int nvec) const { return (nvec + cl - 1) >> shift; }
    // started() ... wait(): every CTA of the cluster runs from here on, so its shared memory may
    // be written.  arrive() ... wait(): what a CTA wrote before is seen by all after.
    __device__ __forceinline__ void started() const
    {
        if (cl > 1)
            asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    }
    __device__ __forceinline__ void arrive() const
    {
        if (cl > 1)
            asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    }
    __device__ __forceinline__ void wait() const
    {
        if (cl > 1)
            asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    }
    // Barrier over the CTAs that share the row.
    __device__ __forceinline__ void sync() const
    {
        if (cl > 1) {
            arrive();
            wait();
        } else {
            __syncthreads();
        }
    }
    template <class T>
    __device__ __forceinline__ T *in_cta(T *shared, int r) const
    {
        return cl > 1 ? cg::this_cluster().map_shared_rank(shared, r) : shared;
    }
    // The warp's part into every CTA of the row (call by all lanes with the same part).
    __device__ __forceinline__ void hand_out(Part *parts, const Part &p) const
    {
        const int lane = threadIdx.x & 31;
        if (lane < cl)
            in_cta(parts, lane)[rank * warps + (threadIdx.x >> 5)] = p;
    }
    __device__ __forceinline__ int parts() const { return cl * warps; }
};

// ---------------------------------------------------------------------------
// A run of vectors through shared memory
// ---------------------------------------------------------------------------
// Each of T threads copies the vectors that it will use into slots of its own in shared
// memory, groups of VT vectors ahead of their use (cp.async): nothing has to be waited for
// but the thread's own copies, and a vector that crosses an end of the row is read element
// by element by the thread that uses it.  (A row per CTA, several CTAs an SM: CTAs that stay
// and take row after row through such slots measured slower, 364 against 170 us for the step
// on 8192 bf16 rows of 32768: what is done once a row costs more than a CTA's start.)

// Waits until at most `pending` of the thread's newest groups of copies are under way.
__device__ __forceinline__ void copies_done(int pending)
{
    switch (pending) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

template <bool BF16, int T, int VT>
struct Run {
    static constexpr int GROUP = T * VT;
    using TileT = Tile<BF16, VT>;

    const RowPtr<BF16> row;
    int begin, end, groups;
    int whole0, whole1;  // the groups [whole0, whole1) lie wholly in the row and the run
    uint4 *slots;        // this thread's: slot s, vector v at [s GROUP + v T]

    __device__ __forceinline__ Run(const RowPtr<BF16> &row_, const Place &at, uint4 *shared)
        : Run(row_, at.begin(row_.nvec), at.end(row_.nvec), shared)
    {
    }
    __device__ __forceinline__ Run(const RowPtr<BF16> &row_, int begin_, int end_, uint4 *shared)
        : row(row_), begin(begin_), end(end_), slots(shared + threadIdx.x)
    {
        groups = max(1, (end - begin + GROUP - 1) / GROUP);
        whole0 = begin < row.full0;
        whole1 = max(0, min(row.full1, end) - begin) / GROUP;
    }
    __device__ __forceinline__ bool whole(int g) const { return g >= whole0 && g < whole1; }
    // The thread's first vector of group g.
    __device__ __forceinline__ int vector(int g) const { return begin + g * GROUP + static_cast<int>(threadIdx.x); }

    static __device__ __forceinline__ void copy(uint32_t to, const char *from)
    {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    }
    // Starts the copies of group g into slot s (past the last group: an empty group of copies).
    __device__ __forceinline__ void start(int g, int s) const
    {
        if (g < groups) {
            uint4 *to = slots + s * GROUP;
            const int i0 = vector(g);
            const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(to));
            const char *src = row.base + 16ll * i0;
            if (whole(g)) {
#pragma unroll
                for (int v = 0; v < VT; ++v)
                    copy(dst + v * T * 16, src + v * T * 16);
            } else {
#pragma unroll 1
                for (int v = 0; v < VT; ++v) {
                    const int i = i0 + v * T;
                    if (i >= end)
                        break;
                    if (row.full(i))
                        copy(dst + v * T * 16, src + v * T * 16);
                    else  // the one or two vectors of a row that cross its ends
                        to[v * T] = row.load_edge(i);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // The vectors of group g from slot s.
    __device__ __forceinline__ void get(TileT &t, int g, int s) const
    {
        constexpr uint32_t M = RowPtr<BF16>::MASKED;
        const uint4 *from = slots + s * GROUP;
        if (whole(g)) {
#pragma unroll
            for (int v = 0; v < VT; ++v)
                t.v[v] = from[v * T];
        } else {
            const int i0 = vector(g);
#pragma unroll
            for (int v = 0; v < VT; ++v)
                t.v[v] = i0 + v * T < end ? from[v * T] : make_uint4(M, M, M, M);
        }
    }
    // f(tile, g, s) for every group, through SLOTS slots s that are used again and again; keep: not
    // before f is done with the slot.
    template <int SLOTS, class F>
    __device__ __forceinline__ void each(bool keep, F f) const
    {
        static_assert(SLOTS <= 4, "copies_done waits for up to three groups");
#pragma unroll 1
        for (int g = 0; g < SLOTS; ++g)
            start(g, g);
        int s = 0;
#pragma unroll 1
        for (int g = 0; g < groups; ++g) {
            TileT t;
            copies_done(SLOTS - 1);
            get(t, g, s);
            const bool early = whole(g) && !keep;
            if (early)
                start(g + SLOTS, s);
            f(t, g, s);
            if (!early)
                start(g + SLOTS, s);
            s = s + 1 == SLOTS ? 0 : s + 1;
        }
    }
    // value(pair) of every pair of group g, whose tile is t and which is in slot s, into the
    // same elements of `out`.  Only whole groups whose rows start alike within a vector are
    // stored from the tile: then the slot is not looked at.
    template <class F>
    __device__ __forceinline__ void put(const TileT &t, int g, int s, const RowPtr<BF16> &out, F value) const
    {
        const int i0 = vector(g);
        if (row.skip == out.skip && whole(g)) {
            store_whole<T>(t, reinterpret_cast<uint4 *>(out.base) + i0, value);
            return;
        }
#pragma unroll 1
        for (int v = 0; v < VT; ++v) {
            const int i = i0 + v * T;
            if (i >= end)
                break;
            Tile<BF16, 1> one;
            one.v[0] = slots[s * GROUP + v * T];
            store_tile(one, row, out, i, T, end, false, value);
        }
    }
    // Zeros into the run's elements of `out`.
    __device__ __forceinline__ void clear(const RowPtr<BF16> &out) const
    {
        Tile<BF16, 1> none;
#pragma unroll 1
        for (int i = begin + static_cast<int>(threadIdx.x); i < end; i += T)
            store_tile(none, row, out, i, T, end, true, [](float, float) { return F2{0}; });
    }
};

// Allows a kernel its launch with `bytes` of dynamic shared memory: `most`, the same number at
// every call, since calls of other host threads may lie between this one and its launch.
template <class A>
inline int allow_shared(void (*kernel)(A), size_t bytes, size_t most)
{
    if (bytes <= 24 * 1024)  // with what the kernels hold besides, less than what needs no leave
        return KDA_OK;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string("shared memory: ") + cudaGetErrorString(e));
    return KDA_OK;
}

// Vectors that the longest of N rows may touch.
inline long long vectors_of(const void *p, int V, long long ld, int bf16)
{
    const long long per = bf16 ? 8 : 4;
    const bool even = (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % per == 0;
    return (V + per - 1) / per + (even ? 0 : 1);
}

// A pass that needs nothing of the rest of a row: CTAs of T threads, each with a run of up to
// RUN_GROUPS groups of PIECE_VT vectors a thread, which pass through PIECE_SLOTS slots.  Runs of
// 2 / 4 / 8 / 16 groups took 87 / 79 / 81 / 88 us for the gradient of 1024 f32 rows of 65537.
constexpr int PIECE_VT = 4, PIECE_SLOTS = 3;
constexpr size_t piece_shared(int threads) { return static_cast<size_t>(PIECE_SLOTS) * PIECE_VT * threads * 16; }

struct Pieces {
    int threads, per, runs;  // per: vectors of a run
    size_t shared;
};

inline Pieces pieces_of(long long nvec)
{
    constexpr int RUN_GROUPS = 4;
    const int threads = nvec <= 32 * PIECE_VT ? 32 : nvec <= 128 * PIECE_VT ? 128 : 256;
    const int group = threads * PIECE_VT, per = group * RUN_GROUPS;
    const long long groups = (nvec + group - 1) / group;
    return Pieces{threads, per, static_cast<int>((nvec + per - 1) / per),
                  static_cast<size_t>(groups < PIECE_SLOTS ? groups : PIECE_SLOTS) * group * 16};
}

// f with the threads of a CTA as a constant.
template <class F>
inline int with_threads(int threads, F f)
{
    switch (threads) {
    case 32: return f(std::integral_constant<int, 32>());
    case 128: return f(std::integral_constant<int, 128>());
    default: return f(std::integral_constant<int, 256>());
    }
}

// Launches kernel(args) with `cl` CTAs a cluster, as a programmatic dependent of the launch
// before it.
template <class A>
inline int launch_rows(void (*kernel)(A), const A &args, long long blocks, int threads, int cl, size_t smem,
                       cudaStream_t stream, const char *what)
{
    if (blocks > 0x7fffffffll)
        return fail(KDA_EINVAL, "too many rows for one launch");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cl);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cl > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args);
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
    return check_launch(what);
}

// Argument checks that every entry point over logits makes (KDA_OK or KDA_EINVAL).
inline int check_logits(const void *logits, int dtype, int N, int V, long long ld, float temperature)
{
    if (N < 0)
        return fail(KDA_EINVAL, "N must be >= 0");
    if (V < 1 || V > KDA_ROW_MAX)
        return fail(KDA_EINVAL, "V must lie in 1..2^30");
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
