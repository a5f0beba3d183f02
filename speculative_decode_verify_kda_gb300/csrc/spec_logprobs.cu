// spec_logprobs.cu -- log-probabilities of given tokens with entropy and top
// alternatives, and their gradient (sm_103a).
//
// For a row x with m = max x, d = (x - m) / temperature, S = sum exp d and s = ln S:
//   ln p = d - s,  H = s - (1/S) sum d exp d,
//   d x_i = (1/temperature) [ g (1{i = t} - p_i) - h p_i (ln p_i + H) ]
// for g = dL/d log p_t and h = dL/dH.
//
// A row is read once for its maximum and sums.  The top alternatives come from the threads'
// maxima, which the sums need anyway: what K of those reach is a threshold that K logits at
// least reach, and for logits in no particular order not many more.  The few that do go to
// a list in shared memory, and counting how many of the list precede an entry gives its
// place.  Where more reach the threshold than the list holds (many equal logits), it is
// taken again with a logit's place in the row as a part of its value; where that too leaves
// more, the alternatives are found one after the other.  All three give the same answer.
#include <algorithm>
#include <cfloat>

#include "logit_rows.cuh"

namespace kda {
namespace {

using namespace rows;
using Key = unsigned long long;

constexpr int CLUSTER = 8, CLUSTER_T = 256;  // CTAs of a row and their threads where rows are few
constexpr int CLUSTER_LIST = 2048;           // candidates that a row's list holds there

struct Score {
    const void *x;
    long long ld, N;
    int V, K;
    int r, w;  // the threshold is what w of the warps' r-th largest maxima reach
    const int *tokens;
    Scale z;
    float *logprob, *entropy, *stats, *top_logprobs;
    int *top_ids, *status;
};

constexpr int MAX_PARTS = CLUSTER * CLUSTER_T / 32;

// The list of a row's candidates and what finds its threshold.
template <int CAP>
struct Candidates {
    Part parts[MAX_PARTS];
    Key bound;
    int count;
    __align__(16) Key list[CAP];
};

// The w-th largest (from 1) of n keys, by all threads of the CTA.
__device__ __forceinline__ Key rank_of(const Key *keys, int n, int w, Key *out)
{
    if (n <= 32) {
        const int lane = threadIdx.x & 31;
        return warp_rank<Key>(lane < n ? keys[lane] : 0, w - 1);
    }
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const Key mine = keys[i];
        int before = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j)
            before += keys[j] > mine || (keys[j] == mine && j < i);
        if (before == w - 1)
            *out = mine;
    }
    __syncthreads();
    return *out;
}

// The largest number with 16 low zero bits that at least K of the warp's 32 N values reach (0
// if fewer than K are above 0): two bits a step.  Called by whole warps.
template <int N>
__device__ __forceinline__ uint32_t reached(const uint32_t (&v)[N], int K)
{
    static_assert(32 * N < 1024, "three counts share a word");
    uint32_t t = 0;
#pragma unroll 1
    for (int at = 30; at >= 16; at -= 2) {
        const uint32_t t1 = t | 1u << at, t2 = t | 2u << at, t3 = t | 3u << at;
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            n += (v[i] >= t1 ? 1u : 0u) + (v[i] >= t2 ? 1u << 10 : 0u) + (v[i] >= t3 ? 1u << 20 : 0u);
        n = __reduce_add_sync(0xffffffffu, n);
        const uint32_t k = K;
        t = (n >> 20) >= k ? t3 : (n >> 10 & 1023u) >= k ? t2 : (n & 1023u) >= k ? t1 : t;
    }
    return t;
}

template <int CAP>
__device__ __forceinline__ void append(int *count, Key *list, Key key)
{
    const int at = atomicAdd(count, 1);
    if (at < CAP)
        list[at] = key;
}

// The logits of a vector that reach `least`; id is the first one's.
template <bool BF16, int CAP>
__device__ __noinline__ void append_reaching(int *count, Key *list, uint4 u, int id, float least)
{
    Tile<BF16, 1>::each_of(u, [&](float p, float q) {
        if (p >= least && p > -INFINITY)
            append<CAP>(count, list, key_of(p, id));
        if (q >= least && q > -INFINITY)
            append<CAP>(count, list, key_of(q, id + 1));
        id += 2;
    });
}

// Calls f with the key of every logit above -inf of the CTA's share, read again.
template <bool BF16, class F>
__device__ __forceinline__ void each_key(const RowPtr<BF16> &row, int first, int step, int end, F f)
{
#pragma unroll 1
    for (int i = first; i < end; i += step) {
        int id = row.first_id(i);
        Tile<BF16, 1>::each_of(row.full(i) ? row.load(i) : row.load_edge(i), [&](float p, float q) {
            if (p > -INFINITY)
                f(key_of(p, id));
            if (q > -INFINITY)
                f(key_of(q, id + 1));
            id += 2;
        });
    }
}

// Second try at the list, for a row with many equal logits: the lanes' largest keys (value,
// then place) of the row read again, and the threshold from those, which min(K, 32) lanes of
// ceil(K / 32) warps reach.
template <bool BF16, int CAP>
__device__ __noinline__ void list_by_key(int K, RowPtr<BF16> row, Place at, Candidates<CAP> &sh)
{
    const int first = at.begin(row.nvec) + threadIdx.x, end = at.end(row.nvec), lane = threadIdx.x & 31;
    Key best = 0;
    each_key(row, first, blockDim.x, end, [&](Key k) { best = k > best ? k : best; });
    __syncwarp();
    best = warp_rank<Key>(best, min(K, 32) - 1);
    Key *keys = reinterpret_cast<Key *>(sh.parts);
    at.sync();  // the parts and the count have been read by every CTA
    if (lane < at.cl)
        at.in_cta(keys, lane)[at.rank * at.warps + (threadIdx.x >> 5)] = best;
    if (threadIdx.x == 0)
        sh.count = 0;
    at.sync();
    const int n = at.parts(), w = (K + 31) / 32;
    const Key bound = w <= n ? rank_of(keys, n, w, &sh.bound) : 0;
    int *count = at.in_cta(&sh.count, 0);
    Key *list = at.in_cta(sh.list, 0);
    each_key(row, first, blockDim.x, end, [&](Key k) {
        if (k >= bound)
            append<CAP>(count, list, k);
    });
    at.sync();
}

// Last resort, by the first CTA alone: the alternatives one after the other, each the largest
// key below the last one.
template <bool BF16, int CAP>
__device__ __noinline__ void list_by_rounds(int K, RowPtr<BF16> row, Candidates<CAP> &sh)
{
    Key *best_of = reinterpret_cast<Key *>(sh.parts), last = ~0ull;
    int n = 0;
#pragma unroll 1
    for (; n < K && last; ++n) {
        Key best = 0;
        each_key(row, threadIdx.x, blockDim.x, row.nvec, [&](Key k) { best = k < last && k > best ? k : best; });
        __syncwarp();
        best = warp_rank<Key>(best, 0);
        __syncthreads();
        if ((threadIdx.x & 31) == 0)
            best_of[threadIdx.x >> 5] = best;
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < (blockDim.x >> 5); ++i)
            best = best_of[i] > best ? best_of[i] : best;
        last = best;
        if (threadIdx.x == 0)
            sh.list[n] = best;
    }
    __syncthreads();
    if (threadIdx.x == 0)
        sh.count = n;
    __syncthreads();
}

// The row's results that are not alternatives, by one thread.
template <bool BF16>
__device__ __forceinline__ void write_scores(const Score &a, long long n, const RowPtr<BF16> &row, const Stats &st)
{
    float lp = 0.0f;
    if (a.tokens) {
        const int token = a.tokens[n];
        if (token >= a.V && a.status)
            atomicOr(a.status, KDA_ST_BADTOKEN);
        if (token >= 0 && token < a.V)
            lp = st.bad() ? NAN : st.empty() ? -INFINITY : log_prob(row.at(token), st, a.z.inv);
    }
    if (a.logprob)
        a.logprob[n] = lp;
    if (a.entropy)
        a.entropy[n] = st.entropy;
    if (a.stats) {
        a.stats[2 * n] = st.m;
        a.stats[2 * n + 1] = st.lnS;
    }
    if (st.bad() && a.status)
        atomicOr(a.status, KDA_ST_NAN);
}

// The alternatives from the row's list, by all threads of a CTA.
__device__ __forceinline__ void write_top(const Score &a, long long n, const Stats &st, const Key *list, int found)
{
    const long long o = n * a.K;
#pragma unroll 1
    for (int i = threadIdx.x; i < found; i += blockDim.x) {
        const Key key = list[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < found; ++j)
            place += list[j] > key;
        if (place < a.K) {
            a.top_ids[o + place] = key_id(key);
            a.top_logprobs[o + place] = log_prob(from_ordered(static_cast<uint32_t>(key >> 32)), st, a.z.inv);
        }
    }
#pragma unroll 1
    for (int k = found + threadIdx.x; k < a.K; k += blockDim.x) {
        a.top_ids[o + k] = -1;
        a.top_logprobs[o + k] = st.bad() ? NAN : -INFINITY;
    }
}

// For few long rows: a cluster of CTAs a row, which holds it in registers.  Each warp orders its
// lanes' maxima and names the r-th largest; what w of those reach, with r w >= K, is reached
// by r lanes' maxima of w warps.  One barrier of the cluster lies between reading the row and
// knowing its statistics and the threshold, one more before the first CTA orders the list.
template <bool BF16, int VPT>
__global__ void __launch_bounds__(CLUSTER_T) logprobs_cluster_kernel(const Score a)
{
    __shared__ Candidates<CLUSTER_LIST> sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Place at(CLUSTER, CLUSTER_T);
    const int tid = threadIdx.x;
    if (tid == 0)
        sh.count = 0;
    at.started();
    const RowPtr<BF16> row(a.x, at.row * a.ld, a.V);
    const int begin = at.begin(row.nvec), end = at.end(row.nvec), step = CLUSTER_T, round = step * VPT;
    Tile<BF16, VPT> t;
    Running<true> run;
    float most = -INFINITY;
    int b = begin;
#pragma unroll 1
    do {
        t.load(row, b + tid, step, end);
        const float m = t.max_of();
        most = max_nan(most, m);
        run.add(t, m, a.z);
        b += round;
    } while (b < end);
    const uint32_t mine = most > -INFINITY ? ordered(most) : 0u;
    const uint32_t named = a.K > 0 ? warp_rank<uint32_t>(mine, a.r - 1) : 0u;
    const Part part = run.part(most, a.z, named);
    at.wait();
    at.hand_out(sh.parts, part);
    at.sync();
    const int n = at.parts();
    const Stats st = join(sh.parts, n, a.z.c);
    if (at.rank == 0 && tid == 0)
        write_scores(a, at.row, row, st);
    if (a.K == 0)
        return;
    if (!st.bad() && !st.empty()) {
        uint32_t v[MAX_PARTS / 32];
#pragma unroll
        for (int i = 0; i < MAX_PARTS / 32; ++i)
            v[i] = 32 * i + (tid & 31) < n ? sh.parts[32 * i + (tid & 31)].key : 0u;
        const uint32_t bound = reached(v, a.w);
        if (mine && mine >= bound) {
            const float least = bound ? from_ordered(bound) : -INFINITY;
            int *count = at.in_cta(&sh.count, 0);
            Key *list = at.in_cta(sh.list, 0);
            b = begin;
#pragma unroll 1
            do {
                if (round < end - begin)  // of several rounds the registers hold the last one alone
                    t.load(row, b + tid, step, end);
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    Tile<BF16, 1> one;
                    one.v[0] = t.v[j];
                    if (one.max_of() >= least)
                        append_reaching<BF16, CLUSTER_LIST>(count, list, t.v[j], row.first_id(b + tid + j * step),
                                                            least);
                }
                b += round;
            } while (b < end);
        }
    }
    at.sync();
    int found = *at.in_cta(&sh.count, 0);
    if (found > CLUSTER_LIST) {  // the same for every CTA of the row
        list_by_key(a.K, row, at, sh);
        found = *at.in_cta(&sh.count, 0);
    }
    at.arrive();  // the first CTA's shared memory has been read by the others
    if (at.rank == 0) {
        if (found > CLUSTER_LIST) {
            list_by_rounds(a.K, row, sh);
            found = sh.count;
        }
        write_top(a, at.row, st, sh.list, found);
    }
    at.wait();
}

// One CTA a row, which passes through shared memory ahead of its use.  A thread keeps the
// maxima of up to SPANS equal spans of its share of the row, half a group or a multiple.  The
// threshold is the K-th largest of the threads' maxima, to 16 bits; the spans that reach it
// are read again, through L2, to fill the list.  4096 bf16 rows of 131072 take 153 us without
// alternatives (7.0 TB/s: the reads bound it), 166 with 20 and 185 with 64: a CTA that looks
// for alternatives reads nothing ahead, and what it reads again is 5 % more (to 32 bytes a
// vector).  Two slots, not three or four: four CTAs an SM hide more than deeper slots do
// (three slots and CTAs 195 us, 512 threads and two CTAs 219).
constexpr int ROW_VT = 4, ROW_SLOTS = 2, SPANS = 16, WORK = 1024;

template <int T>
struct RowShared {
    static constexpr int LIST = T == 256 ? 1024 : 512;
    Candidates<LIST> top;
    uint32_t bound, most[T];
    float lnS;
    int works;
    uint16_t work[WORK];
    uint16_t span[SPANS][T];  // the upper halves of the maxima's ordered() values
};

// Leaves those of the list that reach what K of it reach, by a whole CTA of T threads.
template <int T, int LIST>
__device__ __noinline__ int thin_list(int K, Key *list, int *count, uint32_t *bound)
{
    const int found = *count;
    if (threadIdx.x < 32) {
        uint32_t v[LIST / 32];
#pragma unroll
        for (int i = 0; i < LIST / 32; ++i) {
            const int k = 32 * i + threadIdx.x;
            v[i] = k < found ? static_cast<uint32_t>(list[k] >> 32) : 0u;
        }
        uint32_t t = 0;
#pragma unroll 1
        for (int at = 31; at >= 0; --at) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < LIST / 32; ++i)
                n += v[i] >= (t | 1u << at);
            if (__reduce_add_sync(0xffffffffu, n) >= K)
                t |= 1u << at;
        }
        if (threadIdx.x == 0)
            *bound = t;
    }
    Key mine[LIST / T];
#pragma unroll
    for (int i = 0; i < LIST / T; ++i) {
        const int k = T * i + threadIdx.x;
        mine[i] = k < found ? list[k] : 0;
    }
    __syncthreads();
    const Key least = static_cast<Key>(*bound) << 32;
    if (threadIdx.x == 0)
        *count = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < LIST / T; ++i)
        if (mine[i] && mine[i] >= least)
            append<LIST>(count, list, mine[i]);
    __syncthreads();
    return *count;
}

template <bool BF16, int T>
__global__ void __launch_bounds__(T, T >= 128 ? 1024 / T : 12) logprobs_row_kernel(const Score a)
{
    constexpr int WARPS = T / 32, VT = ROW_VT, HALF = VT / 2, LIST = RowShared<T>::LIST;
    extern __shared__ uint4 slots[];
    __shared__ RowShared<T> sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0)
        sh.top.count = sh.works = 0;
    const Place at(1, T);
    const long long n = at.row;
    const RowPtr<BF16> row(a.x, n * a.ld, a.V);
    using R = Run<BF16, T, VT>;
    const R run(row, at, slots);
    const int each = (2 * run.groups + SPANS - 1) / SPANS;  // halves of a group in a span
    Running<true> sums;
    float most = -INFINITY, top = -INFINITY;
    int span = 0, left = each;
    auto half = [&](float m) {
        top = max_nan(top, m);
        if (--left == 0) {
            sh.span[span++][tid] = ordered(top) >> 16;  // read by this thread alone
            most = max_nan(most, top);
            top = -INFINITY;
            left = each;
        }
    };
    run.template each<ROW_SLOTS>(false, [&](const typename R::TileT &t, int, int) {
        const float m0 = t.template max_of<0, HALF>(), m1 = t.template max_of<HALF, VT>();
        sums.add(t, max_nan(m0, m1), a.z);
        half(m0);
        half(m1);
    });
    if (left != each) {
        sh.span[span++][tid] = ordered(top) >> 16;
        most = max_nan(most, top);
    }
    const uint32_t mine = most > -INFINITY ? ordered(most) : 0u;
    const Part part = sums.part(most, a.z, 0u);
    if (lane == 0)
        sh.top.parts[warp] = part;
    sh.most[tid] = mine;
    __syncthreads();
    if (warp == WARPS - 1) {
        const Stats st = join(sh.top.parts, WARPS, a.z.c);
        if (lane == 0) {
            write_scores(a, n, row, st);
            sh.lnS = st.lnS;
        }
    }
    if (a.K == 0)
        return;
    if (warp == 0) {
        uint32_t v[T / 32];
#pragma unroll
        for (int i = 0; i < T / 32; ++i)
            v[i] = sh.most[32 * i + lane];
        const uint32_t bound = reached(v, a.K);
        if (lane == 0)
            sh.bound = bound;
    }
    const float m = warp_max_nan(sh.top.parts[lane % WARPS].m);
    __syncthreads();
    const bool plain = m > -INFINITY && m < INFINITY;
    const uint32_t bound = sh.bound;
    const float least = bound ? from_ordered(bound) : -INFINITY;
    if (plain && mine && mine >= bound) {
        const uint32_t need = max(bound, ordered(-FLT_MAX)) >> 16;  // (the bound's lower half is 0)
#pragma unroll 4
        for (int s = 0; s < span; ++s) {
            if (sh.span[s][tid] >= need) {
                const int i = atomicAdd(&sh.works, 1);
                if (i < WORK)
                    sh.work[i] = static_cast<uint16_t>(s * T + tid);
            }
        }
    }
    __syncthreads();
    int found = 0;
    if (plain) {
        const int works = sh.works, vectors = each * HALF;
        if (works <= WORK) {
            const int lanes = vectors == 2 ? 1 : 2;  // 2^lanes threads a span
#pragma unroll 1
            for (int i = tid >> lanes; i < works; i += T >> lanes) {
                const int item = sh.work[i], first = item / T * vectors, owner = item % T;
#pragma unroll 1
                for (int v = tid & ((1 << lanes) - 1); v < vectors; v += 1 << lanes) {
                    const int vec = (first + v) * T + owner;
                    if (vec >= row.nvec)
                        break;
                    append_reaching<BF16, LIST>(&sh.top.count, sh.top.list,
                                                row.full(vec) ? row.load(vec) : row.load_edge(vec),
                                                row.first_id(vec), least);
                }
            }
        }
        __syncthreads();
        found = works <= WORK ? sh.top.count : LIST + 1;
        if (found > LIST) {
            list_by_key(a.K, row, at, sh.top);
            found = sh.top.count;
            if (found > LIST) {
                list_by_rounds(a.K, row, sh.top);
                found = sh.top.count;
            }
        }
        if (found > 2 * a.K + 64)  // (a short row, whose vectors are hardly more than K)
            found = thin_list<T, LIST>(a.K, sh.top.list, &sh.top.count, &sh.bound);
    }
    write_top(a, n, Stats{m < INFINITY ? m : NAN, sh.lnS, 0.0f}, sh.top.list, found);
}

struct ScoreGrad {
    const void *x;
    void *dx;
    long long ld, ldg;
    int V, per, runs;  // vectors of a run, runs of a row
    const int *tokens;
    const float *stats, *entropy, *g, *h;
    Scale z;
};

// A row is cut into runs that need nothing of one another: read, weighted, written.  With
// u = (x - m) c - s log2(e), p = 2^u and
//   d x_i = p (A + B u) + [i = t] g / tau,  A = -(g + h H) / tau, B = -h ln 2 / tau.
template <bool BF16, int T>
__global__ void __launch_bounds__(T) logprobs_backward_kernel(const ScoreGrad a)
{
    extern __shared__ uint4 slots[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = blockIdx.x / a.runs;
    const int begin = static_cast<int>(blockIdx.x % a.runs) * a.per, tid = threadIdx.x;
    const RowPtr<BF16> row(a.x, n * a.ld, a.V), out(a.dx, n * a.ldg, a.V);
    using R = Run<BF16, T, PIECE_VT>;
    const R run(row, begin, min(row.nvec, begin + a.per), slots);
    const int t = a.tokens ? a.tokens[n] : -1;
    const bool has = t >= 0 && t < a.V;
    const float g = a.g && has ? a.g[n] : 0.0f, h = a.h ? a.h[n] : 0.0f;
    const float m = a.stats[2 * n], off = -a.stats[2 * n + 1] * LOG2E;
    if (m == -INFINITY || (g == 0.0f && h == 0.0f)) {
        run.clear(out);
        return;
    }
    const float A = -(g + (h != 0.0f ? h * a.entropy[n] : 0.0f)) * a.z.inv, B = -h * LN2 * a.z.inv;
    const int at = has ? (row.skip + t) / row.PER : -1;
    const bool mine = at >= run.begin && at < run.end;  // the same for the whole CTA
    const float x_token = mine && tid == 0 ? row.at(t) : 0.0f;
    const F2 neg = f2(-m, -m), cc = f2(a.z.c, a.z.c), oo = f2(off, off), AA = f2(A, A), BB = f2(B, B);
    run.template each<PIECE_SLOTS>(row.skip != out.skip, [&](const typename R::TileT &x, int k, int s) {
        if (k == 0 && mine)
            __syncthreads();  // the token's logit is read before its gradient may replace it
        run.put(x, k, s, out, [&](float p, float q) {
            const float2 v = split(fma2(f2(p, q) + neg, cc, oo));
            const F2 w = f2(ex2(v.x), ex2(v.y));
            return w * fma2(BB, f2(fmaxf(v.x, -1e4f), fmaxf(v.y, -1e4f)), AA);
        });
    });
    if (mine) {
        __syncthreads();  // after the element's ordinary value
        if (tid == 0) {
            const float u = fmaf(x_token - m, a.z.c, off);
            out.set(t, ex2(u) * fmaf(B, fmaxf(u, -1e4f), A) + g * a.z.inv);
        }
    }
}

template <int T>
int launch_row(const Score &a, bool bf16, long long nvec, cudaStream_t stream)
{
    const size_t most = static_cast<size_t>(ROW_SLOTS) * ROW_VT * T * 16;
    const size_t smem = std::min(most, static_cast<size_t>((nvec + T - 1) / T) * T * 16);
    auto *kernel = bf16 ? logprobs_row_kernel<true, T> : logprobs_row_kernel<false, T>;
    if (int rc = allow_shared(kernel, smem, most))
        return rc;
    return launch_rows(kernel, a, a.N, T, 1, smem, stream, "logprobs_row_kernel");
}

template <int VPT>
int launch_cluster(Score a, bool bf16, cudaStream_t stream)
{
    // r lanes of w warps make the threshold: about two thirds of the warps, so that one warp of
    // small logits does not lower it
    constexpr int WARPS = CLUSTER * CLUSTER_T / 32;
    a.r = std::max(1, std::min(32, (5 * a.K + 3 * WARPS - 1) / (3 * WARPS)));
    a.w = (a.K + a.r - 1) / a.r;
    return launch_rows(bf16 ? logprobs_cluster_kernel<true, VPT> : logprobs_cluster_kernel<false, VPT>, a,
                       a.N * CLUSTER, CLUSTER_T, CLUSTER, 0, stream, "logprobs_cluster_kernel");
}

// Which kernel, and how many threads a row.  us on GB300, K = 20 unless said otherwise:
//   bf16 rows of logits          eight CTAs a row   one CTA of 256 threads
//     1 / 8 / 16 / 32 of  32768   4.7 / 5.4 / 5.6 / 7.0    5.7 / 6.1 / 6.2 / 6.2
//     1 / 8 / 16 / 32 of 131072   5.7 / 6.3 / 6.9 / 8.5   11.5 / 11.6 / 11.5 / 11.6
//     1 of 8192 / 16384           4.9 / 4.8                4.4 / 4.9
//   8000 bf16 rows of 1000 / 5000 / 9000 logits: 32 threads 28 / 44 / 52, 64: 28 / 39 / 49, 128: 37 / 48 /
//     59, 256: 64 / 75 / 89; 1000 of 17000: 64 threads 16.3, 128 12.8, 256 16.8; 2000 f32 of 32768: 128
//     threads 47, 256 51; 4096 of 131072 (K = 64): 128 threads 205, 256 182.
// The threshold comes from the threads' maxima, so there are at least 2 K threads.
int launch_scores(const Score &a, bool bf16, long long nvec, cudaStream_t stream)
{
    if ((a.N * CLUSTER <= SMS && nvec >= 3072) || (a.N * CLUSTER <= 2 * SMS && nvec >= 8192)) {
        const long long per = (nvec + CLUSTER - 1) / CLUSTER;
        return per <= 2 * CLUSTER_T   ? launch_cluster<2>(a, bf16, stream)
               : per <= 4 * CLUSTER_T ? launch_cluster<4>(a, bf16, stream)
                                      : launch_cluster<8>(a, bf16, stream);
    }
    const bool full = a.N > 2 * SMS;
    if (nvec <= (full ? 160 : 32) && a.K <= 16)
        return launch_row<32>(a, bf16, nvec, stream);
    if (nvec <= (full ? 1536 : 96) && a.K <= 32)
        return launch_row<64>(a, bf16, nvec, stream);
    if (nvec <= (full ? 8192 : 512) && a.K <= 64)
        return launch_row<128>(a, bf16, nvec, stream);
    return launch_row<256>(a, bf16, nvec, stream);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int spec_logprobs(const void *logits, int logit_dtype, int N, int V, long long ld, const int *tokens, int K,
                             float temperature, float *logprob, float *entropy, float *stats, int *top_ids,
                             float *top_logprobs, int *dev_status, cudaStream_t stream)
{
    if (int rc = rows::check_logits(logits, logit_dtype, N, V, ld, temperature))
        return rc;
    if (K < 0 || K > KDA_TOPK_MAX)
        return fail(KDA_EINVAL, "K must lie in 0..128, got " + std::to_string(K));
    if (N == 0)
        return ok();
    if (K > 0 && (!top_ids || !top_logprobs))
        return fail(KDA_EINVAL, "top_ids and top_logprobs must not be NULL when K > 0");
    if (logprob && !tokens)
        return fail(KDA_EINVAL, "logprob needs tokens");
    for (const void *p : {static_cast<const void *>(tokens), static_cast<const void *>(logprob),
                          static_cast<const void *>(entropy), static_cast<const void *>(stats),
                          static_cast<const void *>(top_ids), static_cast<const void *>(top_logprobs),
                          static_cast<const void *>(dev_status)})
        if (!rows::aligned4(p))
            return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    Score a{};
    a.x = logits;
    a.ld = ld;
    a.N = N;
    a.V = V;
    a.K = K;
    a.tokens = tokens;
    a.z = Scale{LOG2E / temperature, 16.0f * LN2 * temperature, 1.0f / temperature};
    a.logprob = logprob;
    a.entropy = entropy;
    a.stats = stats;
    a.top_logprobs = top_logprobs;
    a.top_ids = top_ids;
    a.status = dev_status;
    const bool bf16 = logit_dtype == KDA_BF16;
    return launch_scores(a, bf16, vectors_of(logits, V, ld, bf16), stream);
}

extern "C" int spec_logprobs_backward(const void *logits, int logit_dtype, int N, int V, long long ld,
                                      const int *tokens, const float *stats, const float *entropy,
                                      const float *grad_logprob, const float *grad_entropy, float temperature,
                                      void *dlogits, long long ldg, cudaStream_t stream)
{
    if (int rc = rows::check_logits(logits, logit_dtype, N, V, ld, temperature))
        return rc;
    if (int rc = rows::check_grad(logits, dlogits, logit_dtype, N, V, ld, ldg))
        return rc;
    if (N == 0)
        return ok();
    if (!stats)
        return fail(KDA_EINVAL, "stats must not be NULL");
    if (!grad_logprob && !grad_entropy)
        return fail(KDA_EINVAL, "grad_logprob and grad_entropy must not both be NULL");
    if (grad_logprob && !tokens)
        return fail(KDA_EINVAL, "grad_logprob needs tokens");
    if (grad_entropy && !entropy)
        return fail(KDA_EINVAL, "grad_entropy needs entropy");
    for (const void *p : {static_cast<const void *>(tokens), static_cast<const void *>(stats),
                          static_cast<const void *>(entropy), static_cast<const void *>(grad_logprob),
                          static_cast<const void *>(grad_entropy)})
        if (!rows::aligned4(p))
            return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    const bool bf16 = logit_dtype == KDA_BF16;
    const rows::Pieces cut = rows::pieces_of(rows::vectors_of(logits, V, ld, bf16));
    const ScoreGrad a{logits, dlogits, ld, ldg, V, cut.per, cut.runs, tokens, stats, entropy, grad_logprob,
                      grad_entropy, Scale{rows::LOG2E / temperature, 0.0f, 1.0f / temperature}};
    return rows::with_threads(cut.threads, [&](auto threads) {
        constexpr int T = decltype(threads)::value;
        auto *kernel = bf16 ? logprobs_backward_kernel<true, T> : logprobs_backward_kernel<false, T>;
        if (int rc = rows::allow_shared(kernel, cut.shared, rows::piece_shared(T)))
            return rc;
        return rows::launch_rows(kernel, a, static_cast<long long>(N) * cut.runs, T, 1, cut.shared, stream,
                                 "logprobs_backward_kernel");
    });
}
