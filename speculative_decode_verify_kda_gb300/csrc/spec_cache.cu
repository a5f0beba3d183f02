// spec_cache.cu -- what enters and leaves a paged cache: spec_cache_append writes a round's keys
// and values behind the committed tokens, spec_cache_evict cuts sessions to a budget by mass.
#include <cooperative_groups.h>

#include "paged_cache.cuh"

namespace kda {
namespace {

using namespace pages;

// ---- append -------------------------------------------------------------------------
// A copy of B T rows of Hkv D elements: nothing but memory.  A CTA takes a few rows, a thread
// 16 bytes of k and of v at a time.  A verify round's rows take a launch (3.0 us), 8192 rows of 8
// heads 12.7 us (5.3 TB/s).
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
// First launch, a cluster of one or eight CTAs for a (session, kv head): the masses between the
// first `sinks` and the last `recent` tokens as whole numbers in the order of the floats; three
// passes of 11, 11 and 10 bits count digits (a histogram in each CTA's shared memory) and find the
// smallest kept number and how many of its equals are kept: a warp reads the cluster's sums of 64
// bins, then the 64 bins that hold the digit.  Every warp has a run of positions: one pass counts
// what it keeps, one gives the kept positions their places.  The numbers are read once and stay
// in shared memory (8 heads of 131072 tokens took 74 us for 50 when every pass read them again); more than
// 393 thousand tokens of a head do not fit and are read again, from the caches, by every pass.  With
// REGISTERS up to HELD numbers a lane stay in those: better where heads fill the SMs (64 heads of 8192
// tokens 31.3 us for 35.5), worse for a few, whose time is that of the code (8 heads of 2048 tokens 12.5 us for
// 10.9, of 8192 16.4 for 15.0).
// Second launch: the kept keys, values and masses move.  Bound by the chain of passes and barriers for a
// few heads (8 heads of 32768 tokens to 4096: 25 us, 5 of them for the bytes), by the move's bytes for many
// (256 heads of up to 8000 tokens to 2000: 105 us, the bytes 79).
constexpr int SELECT_T = 512, SELECT_W = SELECT_T / 32, BINS = 2048, HELD = 16;
constexpr int STORED = 96 * 32;  // numbers of a warp in shared memory

struct Evict {
    Cache c;
    const float *mass;
    float *mass_out;
    long long ld, ld_out;
    int budget, recent, sinks, dst_cols;
    const int *dst;  // the pages that receive the tokens
    int *kept, *lens_out, *status;
    int room;  // numbers that a warp has room for in shared memory
};

// Rising with the float, the two zeros equal, a NaN below every number.
__device__ __forceinline__ uint32_t rank_of(float x)
{
    if (x != x)
        return 0;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <int CL>
__device__ __forceinline__ void meet()
{
    if constexpr (CL > 1)
        cooperative_groups::this_cluster().sync();
    else
        __syncthreads();
}

// CTA r's copy of a word of shared memory.
template <int CL>
__device__ __forceinline__ int of_cta(int *x, int r)
{
    if constexpr (CL > 1)
        return *cooperative_groups::this_cluster().map_shared_rank(x, r);
    else
        return *x;
}

// Sum over the lanes before this one; `total` over all.
__device__ __forceinline__ int lanes_before(int x, int &total)
{
    int s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if ((threadIdx.x & 31) >= d)
            s += y;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    return s - x;
}

template <int CL, bool REGISTERS>
__global__ void __launch_bounds__(SELECT_T) evict_select_kernel(const Evict a)
{
    extern __shared__ uint32_t stored[];
    __shared__ int hist[BINS], group[BINS / 64], found[2], sums[2], part[2][SELECT_W];
    after_previous();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x % CL, head = blockIdx.x / CL, b = head / a.c.Hkv;
    const float *mass = a.mass + head * a.ld;
    int *kept = a.kept + static_cast<long long>(head) * a.budget;
    int n = a.c.lens[b];
    if (n < 0 || n > a.c.capacity()) {
        if (tid == 0)
            raise(a.status, KDA_ST_BADLEN);
        n = 0;
    }
    const int low = a.sinks, high = n - a.recent;  // chosen by mass: low <= j < high
    const bool choose = n > a.budget;
    // this CTA's positions, and this warp's
    const int cta_run = (n + CL - 1) / CL, begin = min(n, cta * cta_run), end = min(n, begin + cta_run);
    const int warp_run = ((end - begin + SELECT_W - 1) / SELECT_W + 31) / 32 * 32;
    const int from = min(end, begin + warp * warp_run), to = min(end, from + warp_run);
    auto number = [&](int j) { return choose && j < to && j >= low && j < high ? rank_of(mass[j]) : 0; };
    const bool held = REGISTERS && warp_run <= 32 * HELD;
    uint32_t own[HELD];
#pragma unroll
    for (int e = 0; e < HELD; ++e)
        own[e] = held && from + 32 * e < to ? number(from + 32 * e + lane) : 0;
    const bool kept_near = !held && warp_run <= a.room;
    uint32_t *near = stored + warp * a.room + lane;
    if (kept_near)
#pragma unroll 8
        for (int j0 = from; j0 < to; j0 += 32)
            near[j0 - from] = number(j0 + lane);
    // f(position, number) for 32 positions at a time
    auto each = [&](auto f) {
        if (held) {
#pragma unroll
            for (int e = 0; e < HELD; ++e)
                if (from + 32 * e < to)
                    f(from + 32 * e + lane, own[e]);
        } else if (kept_near) {
#pragma unroll 4
            for (int j0 = from; j0 < to; j0 += 32)
                f(j0 + lane, near[j0 - from]);
        } else {
#pragma unroll 4
            for (int j0 = from; j0 < to; j0 += 32)
                f(j0 + lane, number(j0 + lane));
        }
    };
    uint32_t edge = 0;  // kept: a number above it, and `ties` equal to it
    int ties = 0;
    if (choose) {
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
            each([&](int j, uint32_t r) {
                const bool in = j < to && j >= low && j < high && (r & mask) == edge;
                const int bin = in ? static_cast<int>(r >> shift) & ((1 << bits) - 1) : -1;
                const int first = __shfl_sync(0xffffffffu, bin, 0);
                if (__all_sync(0xffffffffu, bin == first)) {  // equal masses: one addition for all
                    if (lane == 0 && in)
                        atomicAdd(&hist[bin], 32);
                } else if (in) {
                    atomicAdd(&hist[bin], 1);
                }
            });
            __syncthreads();
            for (int i = warp; i < BINS / 64; i += SELECT_W) {
                int total;
                lanes_before(hist[64 * i + lane] + hist[64 * i + 32 + lane], total);
                if (lane == 0)
                    group[i] = total;
            }
            meet<CL>();
            if (warp == 0) {
                // lane i: the groups, then the pairs of bins, from the top
                int x = 0, total;
#pragma unroll
                for (int c = 0; c < CL; ++c)
                    x += of_cta<CL>(&group[BINS / 64 - 1 - lane], c);
                int before = lanes_before(x, total);
                const uint32_t at = __ballot_sync(0xffffffffu, before < need && before + x >= need);
                const int g = __ffs(at) - 1, rest = need - __shfl_sync(0xffffffffu, before, g);
                const int top = 64 * (BINS / 64 - g) - 1 - 2 * lane;
                int y = 0;
                x = 0;
#pragma unroll
                for (int c = 0; c < CL; ++c) {
                    x += of_cta<CL>(&hist[top], c);
                    y += of_cta<CL>(&hist[top - 1], c);
                }
                before = lanes_before(x + y, total);
                if (before < rest && before + x + y >= rest) {
                    const bool second = before + x < rest;
                    found[0] = top - second;
                    found[1] = rest - before - (second ? x : 0);
                }
            }
            meet<CL>();  // and the histograms have been read
            edge |= static_cast<uint32_t>(found[0]) << shift;
            mask |= ((1u << bits) - 1) << shift;
            need = found[1];
        }
        ties = need;
    }
    auto look = [&](int j, uint32_t r, bool &sure, bool &tie) {
        sure = j < to && (!choose || j < low || j >= high || r > edge);
        tie = j < to && !sure && r == edge && ties > 0;
    };
    int sures = 0, equals = 0;
    each([&](int j, uint32_t r) {
        bool sure, tie;
        look(j, r, sure, tie);
        sures += __popc(__ballot_sync(0xffffffffu, sure));
        equals += __popc(__ballot_sync(0xffffffffu, tie));
    });
    if (lane == 0) {
        part[0][warp] = sures;
        part[1][warp] = equals;
    }
    __syncthreads();
    // before this warp: in the warps and CTAs before it
    int cta_sures, cta_equals;
    int sure_before = lanes_before(lane < SELECT_W ? part[0][lane] : 0, cta_sures);
    int tie_before = lanes_before(lane < SELECT_W ? part[1][lane] : 0, cta_equals);
    sure_before = __shfl_sync(0xffffffffu, sure_before, warp);
    tie_before = __shfl_sync(0xffffffffu, tie_before, warp);
    int all_sures = cta_sures, all_equals = cta_equals;
    if constexpr (CL > 1) {
        if (tid == 0) {
            sums[0] = cta_sures;
            sums[1] = cta_equals;
        }
        meet<CL>();
        all_sures = all_equals = 0;
#pragma unroll
        for (int c = 0; c < CL; ++c) {
            const int s = of_cta<CL>(&sums[0], c), t = of_cta<CL>(&sums[1], c);
            if (c < cta) {
                sure_before += s;
                tie_before += t;
            }
            all_sures += s;
            all_equals += t;
        }
    }
    each([&](int j, uint32_t r) {
        bool sure, tie;
        look(j, r, sure, tie);
        const uint32_t s = __ballot_sync(0xffffffffu, sure), t = __ballot_sync(0xffffffffu, tie);
        const uint32_t below = (1u << lane) - 1;
        const int t_before = tie_before + __popc(t & below);
        if (sure || (tie && t_before < ties))
            kept[sure_before + __popc(s & below) + min(t_before, ties)] = j;
        sure_before += __popc(s);
        tie_before += __popc(t);
    });
    for (int i = all_sures + min(all_equals, ties) + cta * SELECT_T + tid; i < a.budget; i += CL * SELECT_T)
        kept[i] = -1;
    if constexpr (CL > 1)
        meet<CL>();  // no CTA ends while another may read its sums
}

// The move.  Into other pages, rows are independent: a CTA takes 64 kept rows of a (session, kv
// head), D / 8 threads a row, each 16 bytes of k and of v at a time.  In place, a CTA takes 64
// bytes of every kept row of k or v in rising order, STEP rows at a time: a row moves to a place at
// or before its own, so what a step writes has been read by it or by a step before.  The masses go the
// same way as one more part.
constexpr int MOVE_T = 256, DEEP = 8, MOVE_ROWS = 64;

__device__ __forceinline__ void move_masses(const Evict &a, int head, const int *kept)
{
    const float *from = a.mass + head * a.ld;
    float *to = a.mass_out + head * a.ld_out;
    for (int i0 = 0; i0 < a.budget; i0 += MOVE_T * DEEP) {
        float m[DEEP];
        int place[DEEP];
#pragma unroll
        for (int e = 0; e < DEEP; ++e) {
            const int i = i0 + e * MOVE_T + threadIdx.x, j = i < a.budget ? kept[i] : -1;
            place[e] = j >= 0 ? i : -1;
            m[e] = j >= 0 ? from[j] : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < DEEP; ++e)
            if (place[e] >= 0)
                to[place[e]] = m[e];
    }
}

__device__ __forceinline__ void new_length(const Evict &a, int b)
{
    const int n = a.c.lens[b];  // lens_out may be lens: read and written by one thread
    if (n >= 0 && n <= a.c.capacity())
        a.lens_out[b] = min(n, a.budget);
}

template <int D>
__global__ void __launch_bounds__(MOVE_T) evict_move_kernel(const Evict a, int chunks)
{
    after_previous();
    const int head = blockIdx.x / chunks, chunk = blockIdx.x - head * chunks;
    const int b = head / a.c.Hkv, h = head - b * a.c.Hkv;
    const int *kept = a.kept + static_cast<long long>(head) * a.budget;
    if (chunk == chunks - 1) {
        if (h == 0 && threadIdx.x == 0)
            new_length(a, b);
        if (a.mass_out)
            move_masses(a, head, kept);
        return;
    }
    constexpr int V = D / 8, R = MOVE_T / V, E = MOVE_ROWS / R;  // threads a row, rows at a time, times
    const int *from = a.c.table + static_cast<long long>(b) * a.c.cols;
    const int *to = a.dst + static_cast<long long>(b) * a.dst_cols;
    const int x = (threadIdx.x % V) * 8;
    long long src[E], dst[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = chunk * MOVE_ROWS + e * R + threadIdx.x / V, j = i < a.budget ? kept[i] : -1;
        src[e] = j >= 0 ? token_at(a.c, from, h, j) : 0;
        dst[e] = j >= 0 ? token_at(a.c, to, h, i) : -1;
        if (j >= 0 && (src[e] < 0 || dst[e] < 0))
            raise(a.status, KDA_ST_BADPAGE);
    }
    uint4 k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        k[e] = v[e] = make_uint4(0, 0, 0, 0);
        if (src[e] >= 0 && dst[e] >= 0) {
            k[e] = *reinterpret_cast<const uint4 *>(a.c.k + src[e] + x);
            v[e] = *reinterpret_cast<const uint4 *>(a.c.v + src[e] + x);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (dst[e] >= 0) {
            *reinterpret_cast<uint4 *>(a.c.k + dst[e] + x) = k[e];
            *reinterpret_cast<uint4 *>(a.c.v + dst[e] + x) = v[e];
        }
}

__global__ void __launch_bounds__(MOVE_T) evict_in_place_kernel(const Evict a)
{
    after_previous();
    const int slices = a.c.D / 32, part = blockIdx.y, head = blockIdx.x;
    const int b = head / a.c.Hkv, h = head - b * a.c.Hkv;
    const int *kept = a.kept + static_cast<long long>(head) * a.budget;
    if (part == 2 * slices) {
        if (h == 0 && threadIdx.x == 0)
            new_length(a, b);
        if (a.mass_out)
            move_masses(a, head, kept);
        return;
    }
    const int *table = a.c.table + static_cast<long long>(b) * a.c.cols;
    uint16_t *x = (part < slices ? a.c.k : a.c.v) + (part % slices) * 32 + (threadIdx.x & 3) * 8;
    constexpr int R = MOVE_T / 4, STEP = R * DEEP;
    int j[DEEP];
    auto look = [&](int i0) {
#pragma unroll
        for (int e = 0; e < DEEP; ++e) {
            const int i = i0 + e * R + (threadIdx.x >> 2);
            j[e] = i < a.budget ? kept[i] : -1;
        }
    };
    look(0);
    for (int i0 = 0; i0 < a.budget; i0 += STEP) {
        uint4 w[DEEP];
        long long dst[DEEP];
#pragma unroll
        for (int e = 0; e < DEEP; ++e) {
            const int i = i0 + e * R + (threadIdx.x >> 2);
            dst[e] = -1;
            if (j[e] >= 0 && j[e] != i) {
                const long long src = token_at(a.c, table, h, j[e]);
                dst[e] = token_at(a.c, table, h, i);
                if (src < 0 || dst[e] < 0)
                    raise(a.status, KDA_ST_BADPAGE);
                w[e] = src < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(x + src);
            }
        }
        look(i0 + STEP);
        __syncthreads();
#pragma unroll
        for (int e = 0; e < DEEP; ++e)
            if (dst[e] >= 0)
                *reinterpret_cast<uint4 *>(x + dst[e]) = w[e];
    }
}

template <int CL, bool REGISTERS>
int select(Evict a, unsigned heads, cudaStream_t stream)
{
    // room for each warp's run at full length, unless registers hold that
    const long long cta_run = (a.c.capacity() + CL - 1) / CL;
    const long long warp_run = ((cta_run + SELECT_W - 1) / SELECT_W + 31) / 32 * 32;
    cudaLaunchConfig_t cfg{};
    if (!REGISTERS || warp_run > 32 * HELD) {
        a.room = static_cast<int>(std::min(warp_run, static_cast<long long>(STORED)));
        cfg.dynamicSmemBytes = sizeof(uint32_t) * a.room * SELECT_W;
        const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<CL, REGISTERS>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(sizeof(uint32_t)) * STORED * SELECT_W);
        if (e != cudaSuccess)
            return fail(KDA_ECUDA, std::string("evict_select_kernel shared memory: ") + cudaGetErrorString(e));
    }
    cfg.gridDim = dim3(heads * CL);
    cfg.blockDim = dim3(SELECT_T);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CL;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel<CL, REGISTERS>, a);
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string("evict_select_kernel launch: ") + cudaGetErrorString(e));
    return check_launch("evict_select_kernel");
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
    const int chunks = (budget + MOVE_ROWS - 1) / MOVE_ROWS + 1;  // of a head, with other pages
    if (dst_table && static_cast<long long>(a.c.B) * a.c.Hkv * chunks > 0x7fffffffll)
        return fail(KDA_EINVAL, "too many rows for one launch");
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
    // Eight CTAs a head while the device has room for them and a head has work for them, and where one
    // CTA could not hold its numbers.  One against eight, us (budget 1024, in a CUDA graph): 8 heads of 4096
    // tokens 13.6 and 14.1, of 8192 18.5 and 14.8, of 32768 48 and 19; 64 heads of 8192 31 and 39, of
    // 16384 48 and 43, of 32768 70 and 51; 128 heads of 32768 87 and 105, of 65536 239 and 140.
    const bool few = heads <= pages::SMS / 4;
    const bool wide = capacity > (few ? 4096 : heads <= pages::SMS / 2 ? 16384 : SELECT_W * STORED);
    if (int rc = few ? (wide ? select<8, false>(a, heads, stream) : select<1, false>(a, heads, stream))
                     : (wide ? select<8, true>(a, heads, stream) : select<1, true>(a, heads, stream)))
        return rc;
    if (!dst_table)
        return pages::launch(evict_in_place_kernel, dim3(heads, 2 * a.c.D / 32 + 1), MOVE_T, 0, stream,
                             "evict_in_place_kernel", a);
    return pages::launch(a.c.D == 128 ? evict_move_kernel<128> : evict_move_kernel<64>, dim3(heads * chunks), MOVE_T, 0,
                         stream, "evict_move_kernel", a, chunks);
}
