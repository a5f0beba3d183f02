// spec_cache.cu -- what enters and leaves a paged cache: spec_cache_append writes a round's keys
// and values behind the committed tokens, spec_cache_evict cuts sessions to a budget by mass.
#include "paged_cache.cuh"

namespace kda {
namespace {

using namespace pages;

// ---- append -------------------------------------------------------------------------
// A copy of B T rows of Hkv D elements: nothing but memory.  A CTA takes a few rows, a thread
// 16 bytes of k and of v at a time.
constexpr int APPEND_T = 256;

struct Append {
    Cache c;
    const uint16_t *k, *v;
    long long ld_k, ld_v;
    int T, rows, per;  // B * T rows, `per` of them a CTA
    const int *t_rows;
    int *status;
};

__global__ void __launch_bounds__(APPEND_T) cache_append_kernel(const Append a)
{
    after_previous();
    const int vecs = a.c.Hkv * a.c.D / 8, dv = a.c.D / 8;
    const int first = blockIdx.x * a.per, count = min(a.per, a.rows - first);
    for (int i = threadIdx.x; i < count * vecs; i += APPEND_T) {
        const int r = i / vecs, x = i - r * vecs, h = x / dv;
        const int b = (first + r) / a.T, t = first + r - b * a.T;
        int n, tb, bad;
        if (!session(a.c, a.t_rows, a.T, b, n, tb, bad)) {
            if (bad && t == 0 && x == 0)
                raise(a.status, bad);
            continue;
        }
        if (t >= tb)
            continue;
        const long long at = token_at(a.c, a.c.table + static_cast<long long>(b) * a.c.cols, h, n + t);
        if (at < 0) {
            raise(a.status, KDA_ST_BADPAGE);
            continue;
        }
        const long long row = first + r;
        const uint4 k = *reinterpret_cast<const uint4 *>(a.k + row * a.ld_k + x * 8ll);
        const uint4 v = *reinterpret_cast<const uint4 *>(a.v + row * a.ld_v + x * 8ll);
        *reinterpret_cast<uint4 *>(a.c.k + at + (x - h * dv) * 8) = k;
        *reinterpret_cast<uint4 *>(a.c.v + at + (x - h * dv) * 8) = v;
    }
}

// ---- evict --------------------------------------------------------------------------
// First launch, a CTA for a (session, kv head): the masses between the first `sinks` and the
// last `recent` tokens as whole numbers in the order of the floats; three passes of 11, 11 and
// 10 bits count digits (a histogram in shared memory) to find the smallest kept number and how
// many of its equals are kept; a last pass gives the kept positions their places in order.
// Second launch: the kept keys and values move.
constexpr int SELECT_T = 1024, BINS = 2048;

struct Evict {
    Cache c;
    const float *mass;
    float *mass_out;
    long long ld, ld_out;
    int budget, recent, sinks, dst_cols;
    const int *dst;  // the pages that receive the tokens
    int *kept, *lens_out, *status;
};

// Rising with the float, the two zeros equal, a NaN below every number.
__device__ __forceinline__ uint32_t rank_of(float x)
{
    if (x != x)
        return 0;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum over the CTA of the values of threads before this one; `total` over all.
__device__ int scan_before(int x, int *part, int &total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d)
            s += y;
    }
    __syncthreads();
    if (lane == 31)
        part[w] = s;
    __syncthreads();
    const int mine = part[lane];  // SELECT_T / 32 = 32 warps
    int p = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, p, d);
        if (lane >= d)
            p += y;
    }
    total = __shfl_sync(0xffffffffu, p, 31);
    return s - x + __shfl_sync(0xffffffffu, p - mine, w);
}

__global__ void __launch_bounds__(SELECT_T) evict_select_kernel(const Evict a)
{
    __shared__ int hist[BINS], part[32], found[2];
    after_previous();
    const int tid = threadIdx.x, b = blockIdx.x / a.c.Hkv;
    const float *mass = a.mass + blockIdx.x * a.ld;
    float *mass_out = a.mass_out ? a.mass_out + blockIdx.x * a.ld_out : nullptr;
    int *kept = a.kept + static_cast<long long>(blockIdx.x) * a.budget;
    int n = a.c.lens[b];
    if (n < 0 || n > a.c.capacity()) {
        if (tid == 0)
            raise(a.status, KDA_ST_BADLEN);
        n = 0;
    }
    const int low = a.sinks, high = n - a.recent;  // chosen by mass: low <= j < high
    uint32_t edge = 0;                             // kept: rank > edge, and `ties` of rank == edge
    int ties = 0;
    if (n > a.budget) {
        int need = a.budget - a.sinks - a.recent;
        uint32_t mask = 0;
        if (need == 0)
            edge = 0xffffffffu;
#pragma unroll 1
        for (int pass = 0; pass < 3 && need > 0; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass < 2 ? 11 : 10;
            for (int i = tid; i < BINS; i += SELECT_T)
                hist[i] = 0;
            __syncthreads();
            for (int j = low + tid; j < high; j += SELECT_T) {
                const uint32_t r = rank_of(mass[j]);
                if ((r & mask) == edge)
                    atomicAdd(&hist[(r >> shift) & ((1 << bits) - 1)], 1);
            }
            __syncthreads();
            // thread i holds the bins 2i and 2i + 1 from the top
            const int top = (1 << bits) - 1 - 2 * tid;
            const int x = top >= 0 ? hist[top] : 0, y = top >= 1 ? hist[top - 1] : 0;
            int total;
            const int before = scan_before(x + y, part, total);
            if (before < need && before + x + y >= need) {
                const bool second = before + x < need;
                found[0] = top - second;
                found[1] = need - before - (second ? x : 0);
            }
            __syncthreads();
            edge |= static_cast<uint32_t>(found[0]) << shift;
            mask |= ((1u << bits) - 1) << shift;
            need = found[1];
            __syncthreads();
        }
        ties = need;
    }
    int done = 0, tied = 0;  // kept, and equal to the edge, among the positions before
    for (int j0 = 0; j0 < n; j0 += SELECT_T) {
        const int j = j0 + tid;
        const float m = j < n ? mass[j] : 0.0f;
        bool sure = j < n && (n <= a.budget || j < low || j >= high), tie = false;
        if (j < n && !sure) {
            const uint32_t r = rank_of(m);
            sure = r > edge;
            tie = r == edge && ties > 0;
        }
        int total;
        const int before = scan_before((sure ? 1 : 0) | (tie ? 1 << 16 : 0), part, total);
        const int ties_before = tied + (before >> 16);
        if (sure || (tie && ties_before < ties)) {
            const int place = done + (before & 0xffff) + min(ties_before, ties) - min(tied, ties);
            kept[place] = j;
            if (mass_out)
                mass_out[place] = m;  // at or before j: everything there has been read
        }
        const int all = tied + (total >> 16);
        done += (total & 0xffff) + min(all, ties) - min(tied, ties);
        tied = all;
    }
    for (int i = done + tid; i < a.budget; i += SELECT_T)
        kept[i] = -1;
}

// A CTA takes 64 bytes of every kept row of k or v of one (session, kv head) in rising order:
// a row moves to a place at or before its own, so what a step writes was read by it or before.
constexpr int MOVE_T = 256, MOVE_ROWS = MOVE_T / 4;

__global__ void __launch_bounds__(MOVE_T) evict_move_kernel(const Evict a)
{
    after_previous();
    const int slices = a.c.D / 32, part = blockIdx.y;
    const int b = blockIdx.x / a.c.Hkv, h = blockIdx.x - b * a.c.Hkv;
    const int *kept = a.kept + static_cast<long long>(blockIdx.x) * a.budget;
    const int *from = a.c.table + static_cast<long long>(b) * a.c.cols;
    const int *to = a.dst + static_cast<long long>(b) * a.dst_cols;
    uint16_t *x = (part < slices ? a.c.k : a.c.v) + (part % slices) * 32 + (threadIdx.x & 3) * 8;
    if (h == 0 && part == 0 && threadIdx.x == 0) {
        const int n = a.c.lens[b];  // lens_out may be lens: read and written here alone
        if (n >= 0 && n <= a.c.capacity())
            a.lens_out[b] = min(n, a.budget);
    }
    for (int i0 = 0; i0 < a.budget; i0 += MOVE_ROWS) {
        const int i = i0 + (threadIdx.x >> 2);
        const int j = i < a.budget ? kept[i] : -1;
        long long dst = -1;
        uint4 w;
        if (j >= 0) {
            const long long src = token_at(a.c, from, h, j);
            dst = token_at(a.c, to, h, i);
            if (src < 0 || dst < 0)
                raise(a.status, KDA_ST_BADPAGE);
            w = src < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(x + src);
        }
        __syncthreads();
        if (dst >= 0)
            *reinterpret_cast<uint4 *>(x + dst) = w;
    }
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int spec_cache_append(const kda_cache *cache, const void *k_rows, const void *v_rows, int T, long long ld_k,
                                 long long ld_v, const int *t_rows, int *dev_status, cudaStream_t stream)
{
    Append a{};
    if (int rc = pages::check_cache(cache, &a.c))
        return rc;
    const long long width = static_cast<long long>(a.c.Hkv) * a.c.D;
    if (int rc = pages::check_rows(a.c, k_rows, T, width, ld_k, "k_rows"))
        return rc;
    if (int rc = pages::check_rows(a.c, v_rows, T, width, ld_v, "v_rows"))
        return rc;
    if (!pages::aligned4(t_rows) || !pages::aligned4(dev_status))
        return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    if (a.c.B == 0 || T == 0)
        return ok();
    a.k = static_cast<const uint16_t *>(k_rows);
    a.v = static_cast<const uint16_t *>(v_rows);
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.T = T;
    a.rows = a.c.B * T;
    a.per = static_cast<int>(std::max(1ll, APPEND_T / (width / 8)));
    a.t_rows = t_rows;
    a.status = dev_status;
    return pages::launch(cache_append_kernel, dim3((a.rows - 1) / a.per + 1), APPEND_T, 0, stream,
                         "cache_append_kernel", a);
}

extern "C" int spec_cache_evict(const kda_cache *cache, const float *mass, long long ld_mass, int budget, int recent,
                                int sinks, const int *dst_table, int dst_cols, int *kept, float *mass_out,
                                long long ld_mass_out, int *lens_out, int *dev_status, cudaStream_t stream)
{
    Evict a{};
    if (int rc = pages::check_cache(cache, &a.c))
        return rc;
    const long long capacity = a.c.capacity();
    if (budget < 1 || budget > capacity)
        return fail(KDA_EINVAL, "budget must lie in 1..table_cols * page, got " + std::to_string(budget));
    if (recent < 0 || sinks < 0 || static_cast<long long>(recent) + sinks > budget)
        return fail(KDA_EINVAL, "recent and sinks must be >= 0 and leave the budget room");
    if (dst_table && (dst_cols < 1 || (static_cast<long long>(dst_cols) << a.c.shift) < budget))
        return fail(KDA_EINVAL, "dst_cols * page must be at least the budget");
    if (ld_mass < capacity || ld_mass >= (1ll << 40))
        return fail(KDA_EINVAL, "ld_mass must be at least table_cols * page");
    if (mass_out && (ld_mass_out < budget || ld_mass_out >= (1ll << 40)))
        return fail(KDA_EINVAL, "ld_mass_out must be at least the budget");
    if (static_cast<long long>(a.c.B) * a.c.Hkv > 0x7fffffffll)
        return fail(KDA_EINVAL, "B * Hkv must fit in 32 bits");
    if (a.c.B == 0)
        return ok();
    if (!mass || !kept || !lens_out)
        return fail(KDA_EINVAL, "mass, kept and lens_out must not be NULL");
    for (const void *p : {static_cast<const void *>(mass), static_cast<const void *>(dst_table),
                          static_cast<const void *>(kept), static_cast<const void *>(mass_out),
                          static_cast<const void *>(lens_out), static_cast<const void *>(dev_status)})
        if (!pages::aligned4(p))
            return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    if (mass_out) {
        const long long heads = static_cast<long long>(a.c.B) * a.c.Hkv;
        const uintptr_t m = reinterpret_cast<uintptr_t>(mass), o = reinterpret_cast<uintptr_t>(mass_out);
        const uintptr_t m_end = m + 4 * ((heads - 1) * ld_mass + capacity);
        const uintptr_t o_end = o + 4 * ((heads - 1) * ld_mass_out + budget);
        if (!(m == o && ld_mass == ld_mass_out) && m < o_end && o < m_end)
            return fail(KDA_EINVAL, "mass_out must be mass itself or lie apart from it");
    }
    a.mass = mass;
    a.mass_out = mass_out;
    a.ld = ld_mass;
    a.ld_out = ld_mass_out;
    a.budget = budget;
    a.recent = recent;
    a.sinks = sinks;
    a.dst = dst_table ? dst_table : a.c.table;
    a.dst_cols = dst_table ? dst_cols : a.c.cols;
    a.kept = kept;
    a.lens_out = lens_out;
    a.status = dev_status;
    const unsigned heads = static_cast<unsigned>(a.c.B) * a.c.Hkv;
    if (int rc = pages::launch(evict_select_kernel, dim3(heads), SELECT_T, 0, stream, "evict_select_kernel", a))
        return rc;
    return pages::launch(evict_move_kernel, dim3(heads, 2 * a.c.D / 32), MOVE_T, 0, stream, "evict_move_kernel", a);
}
