// spec_logprobs.cu -- log-probabilities of given tokens with entropy and top
// alternatives, and their gradient (sm_103a).
//
// For a row x with m = max x, d = (x - m) / temperature, S = sum exp d and s = ln S:
//   ln p = d - s,  H = s - (1/S) sum d exp d,
//   d x_i = (1/temperature) [ g (1{i = t} - p_i) - h p_i (ln p_i + H) ]
// for g = dL/d log p_t and h = dL/dH.
//
// logprobs_kernel: a row stays in the registers of its CTA or cluster (logit_rows.cuh), so
// it is read once.  The top alternatives come out of the same registers: from the
// threads' maxima, which the sums need anyway, a threshold is taken that at least K
// logits reach, the few that reach it go to a list in the first CTA's shared memory, and
// counting how many of the list precede an entry gives its place.
//
// The threshold: each warp orders its lanes' maxima and names the r-th largest; the w-th
// largest of those, with r w >= K, is reached by r lanes' maxima of w warps, that is by K
// logits at least.  For logits in no particular order about K of them reach it.  Where
// more than the list holds do (many equal logits), the threshold is taken again with a
// logit's place in the row as a part of its value; where that too leaves more, the first
// CTA finds the alternatives one after the other.  All three give the same answer.
#include <algorithm>

#include "logit_rows.cuh"

namespace kda {
namespace {

using namespace rows;
using Key = unsigned long long;

constexpr int LIST = 2048;         // candidates that a row's list holds
constexpr int LONG_LIST = 512;     // (of the kernel for long rows)

struct Score {
    const void *x;
    long long ld, N;
    int V, K, cl;
    int r, w;  // the threshold is the w-th largest of the warps' r-th largest maxima
    const int *tokens;
    float tau;
    Scale z;
    float *logprob, *entropy, *stats, *top_logprobs;
    int *top_ids, *status;
};

constexpr int MAX_PARTS = MAX_CL * (MAX_THREADS / 32);

// The list of a row's candidates and what finds its threshold.
template <int CAP>
struct Candidates {
    Part parts[MAX_PARTS];
    Key bound;
    int count;
    __align__(16) Key list[CAP];
};

// The w-th largest (from 1) of n values, by all threads of the CTA.
template <class T, class Get>
__device__ __forceinline__ T rank_of(Get get, int n, int w, Key *out)
{
    if (n <= 32) {
        const int lane = threadIdx.x & 31;
        return warp_rank<T>(lane < n ? get(lane) : T(0), w - 1);
    }
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const T mine = get(i);
        int before = 0;
        for (int j = 0; j < n; ++j) {
            const T other = get(j);
            before += other > mine || (other == mine && j < i);
        }
        if (before == w - 1)
            *out = mine;
    }
    __syncthreads();
    return static_cast<T>(*out);
}

template <int CAP>
__device__ __forceinline__ void append(int *count, Key *list, Key key)
{
    const int at = atomicAdd(count, 1);
    if (at < CAP)
        list[at] = key;
}

// Calls f with the key of every logit above -inf of the CTA's share, read again.
template <bool BF16, class F>
__device__ __forceinline__ void each_key(const RowPtr<BF16> &row, int first, int step, int end, F f)
{
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
    const Key bound = w <= n ? rank_of<Key>([&](int i) { return keys[i]; }, n, w, &sh.bound) : 0;
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
    for (; n < K && last; ++n) {
        Key best = 0;
        each_key(row, threadIdx.x, blockDim.x, row.nvec, [&](Key k) { best = k < last && k > best ? k : best; });
        __syncwarp();
        best = warp_rank<Key>(best, 0);
        __syncthreads();
        if ((threadIdx.x & 31) == 0)
            best_of[threadIdx.x >> 5] = best;
        __syncthreads();
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
            lp = st.bad() ? NAN : st.empty() ? -INFINITY : (row.at(token) - st.m) / a.tau - st.lnS;
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
__device__ __forceinline__ void write_top(const Score &a, long long n, float m, float lnS, const Key *list, int found)
{
    const long long o = n * a.K;
    for (int i = threadIdx.x; i < found; i += blockDim.x) {
        const Key key = list[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < found; ++j)
            place += list[j] > key;
        if (place < a.K) {
            a.top_ids[o + place] = key_id(key);
            a.top_logprobs[o + place] = (from_ordered(static_cast<uint32_t>(key >> 32)) - m) / a.tau - lnS;
        }
    }
    for (int k = found + threadIdx.x; k < a.K; k += blockDim.x) {
        a.top_ids[o + k] = -1;
        a.top_logprobs[o + k] = m != m ? NAN : -INFINITY;
    }
}

template <bool BF16, int VPT>
__global__ void __launch_bounds__(MAX_THREADS, 3) logprobs_kernel(const Score a)
{
    __shared__ Candidates<LIST> sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Place at(a.cl, blockDim.x);
    const int tid = threadIdx.x;
    if (tid == 0)
        sh.count = 0;
    at.arrive();
    const RowPtr<BF16> row(a.x, at.row * a.ld, a.V);
    const int begin = at.begin(row.nvec), end = at.end(row.nvec), step = blockDim.x, round = step * VPT;
    Tile<BF16, VPT> t;
    Running<true> run;
    float most = -INFINITY;
    int b = begin;
    do {
        t.load(row, b + tid, step, end);
        const float m = t.max_of();
        most = max_nan(most, m);
        run.add(t, m, a.z);
        b += round;
    } while (b < end);
    const uint32_t mine = most > -INFINITY ? ordered(most) : 0u;
    const uint32_t named = a.K > 0 ? warp_rank<uint32_t>(mine, a.r - 1) : 0u;
    const Part part = run.part(most, a.z.c, named);
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
        const uint32_t bound =
            a.w <= n ? rank_of<uint32_t>([&](int i) { return sh.parts[i].key; }, n, a.w, &sh.bound) : 0u;
        if (mine && mine >= bound) {
            const float least = bound ? from_ordered(bound) : -INFINITY;
            int *count = at.in_cta(&sh.count, 0);
            Key *list = at.in_cta(sh.list, 0);
            b = begin;
            do {
                if (round < end - begin)  // of several rounds the registers hold the last one alone
                    t.load(row, b + tid, step, end);
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    int id = row.first_id(b + tid + j * step);
                    t.each_of(t.v[j], [&](float p, float q) {
                        if (p >= least && p > -INFINITY)
                            append<LIST>(count, list, key_of(p, id));
                        if (q >= least && q > -INFINITY)
                            append<LIST>(count, list, key_of(q, id + 1));
                        id += 2;
                    });
                }
                b += round;
            } while (b < end);
        }
    }
    at.sync();
    int found = *at.in_cta(&sh.count, 0);
    if (found > LIST) {  // the same for every CTA of the row
        list_by_key(a.K, row, at, sh);
        found = *at.in_cta(&sh.count, 0);
    }
    at.arrive();  // the first CTA's shared memory has been read by the others
    if (at.rank == 0) {
        if (found > LIST) {
            list_by_rounds(a.K, row, sh);
            found = sh.count;
        }
        write_top(a, at.row, st.m, st.lnS, sh.list, found);
    }
    at.wait();
}

// For many long rows: one CTA a row, which passes through shared memory ahead of its use.  A
// thread keeps the maxima of up to SPANS equal spans of its share of the row, half a group or
// a multiple; the spans that reach the threshold are read again, through L2, to fill the list.
constexpr int LONG_T = 256, LONG_VT = 4, LONG_SLOTS = 3, HALF = LONG_VT / 2;
constexpr int LONG_WARPS = LONG_T / 32, SPANS = 16, WORK = 1024;

struct LongShared {
    Candidates<LONG_LIST> top;
    float lnS;
    int works;
    uint16_t work[WORK];
    float span[SPANS][LONG_T];
};

template <bool BF16>
__global__ void __launch_bounds__(LONG_T, 4) logprobs_long_kernel(const Score a)
{
    extern __shared__ uint4 slots[];
    __shared__ LongShared sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0)
        sh.top.count = sh.works = 0;
    const Place at(1, LONG_T);
    const long long n = at.row;
    const RowPtr<BF16> row(a.x, n * a.ld, a.V);
    using R = Run<BF16, LONG_T, LONG_VT>;
    const R run(row, at, slots);
    const int each = (2 * run.groups + SPANS - 1) / SPANS;  // halves of a group in a span
    Running<true> sums;
    float most = -INFINITY, top = -INFINITY;
    int span = 0, left = each;
    auto half = [&](float m) {
        top = max_nan(top, m);
        if (--left == 0) {
            sh.span[span++][tid] = top;  // read by this thread alone
            most = max_nan(most, top);
            top = -INFINITY;
            left = each;
        }
    };
    run.template each<LONG_SLOTS>([&](const typename R::TileT &t, int) {
        const float m0 = t.template max_of<0, HALF>(), m1 = t.template max_of<HALF, LONG_VT>();
        sums.add(t, max_nan(m0, m1), a.z);
        half(m0);
        half(m1);
    });
    if (left != each) {
        sh.span[span++][tid] = top;
        most = max_nan(most, top);
    }
    const uint32_t mine = most > -INFINITY ? ordered(most) : 0u;
    const uint32_t named = a.K > 0 ? warp_rank<uint32_t>(mine, a.r - 1) : 0u;
    const Part part = sums.part(most, a.z.c, named);
    if (lane == 0)
        sh.top.parts[warp] = part;
    __syncthreads();
    if (warp == LONG_WARPS - 1) {
        const Stats st = join(sh.top.parts, LONG_WARPS, a.z.c);
        if (lane == 0) {
            write_scores(a, n, row, st);
            sh.lnS = st.lnS;  // read by the others after the next barrier
        }
    }
    if (a.K == 0)
        return;
    const Part mate = sh.top.parts[lane % LONG_WARPS];
    const float m = warp_max_nan(mate.m);
    const bool plain = m > -INFINITY && m < INFINITY;
    float least = -INFINITY;
    if (plain) {
        const uint32_t bound = warp_rank<uint32_t, LONG_WARPS>(mate.key, a.w - 1);
        if (bound)
            least = from_ordered(bound);
        if (mine && mine >= bound) {
            for (int s = 0; s < span; ++s) {
                const float v = sh.span[s][tid];
                if (v >= least && v > -INFINITY) {
                    const int i = atomicAdd(&sh.works, 1);
                    if (i < WORK)
                        sh.work[i] = static_cast<uint16_t>(s * LONG_T + tid);
                }
            }
        }
    }
    __syncthreads();
    int found = 0;
    if (plain) {
        const int works = sh.works;
        if (works <= WORK) {
            // HALF threads a span, each with one vector of every half group
            for (int i = tid / HALF; i < works; i += LONG_T / HALF) {
                const int item = sh.work[i], first = item / LONG_T * each, owner = item % LONG_T;
                for (int h = first; h < first + each; ++h) {
                    const int vec = (h * HALF + tid % HALF) * LONG_T + owner;
                    if (vec >= row.nvec)
                        break;
                    int id = row.first_id(vec);
                    Tile<BF16, 1>::each_of(row.full(vec) ? row.load(vec) : row.load_edge(vec), [&](float p, float q) {
                        if (max(p, q) >= least) {
                            if (p >= least && p > -INFINITY)
                                append<LONG_LIST>(&sh.top.count, sh.top.list, key_of(p, id));
                            if (q >= least && q > -INFINITY)
                                append<LONG_LIST>(&sh.top.count, sh.top.list, key_of(q, id + 1));
                        }
                        id += 2;
                    });
                }
            }
        }
        __syncthreads();
        found = works <= WORK ? sh.top.count : LONG_LIST + 1;
        if (found > LONG_LIST) {
            list_by_key(a.K, row, at, sh.top);
            found = sh.top.count;
            if (found > LONG_LIST) {
                list_by_rounds(a.K, row, sh.top);
                found = sh.top.count;
            }
        }
    }
    write_top(a, n, m < INFINITY ? m : NAN, sh.lnS, sh.top.list, found);
}

struct ScoreGrad {
    const void *x;
    void *dx;
    long long ld, ldg;
    int V, per, runs;  // vectors of a run, runs of a row
    const int *tokens;
    const float *stats, *entropy, *g, *h;
    float tau, c;
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
        for (int k = 0; k < run.groups; ++k)
            run.put(typename R::TileT(), k, out, true, [](float, float) { return F2{0}; });
        return;
    }
    const float A = -(g + (h != 0.0f ? h * a.entropy[n] : 0.0f)) / a.tau, B = -h * LN2 / a.tau;
    const int at = (row.skip + t) / row.PER;
    const bool mine = has && at >= run.begin && at < run.end;  // the same for the whole CTA
    float at_token = 0.0f;
    if (mine) {
        if (tid == 0) {
            const float u = fmaf(row.at(t) - m, a.c, off);
            at_token = ex2(u) * fmaf(B, fmaxf(u, -1e4f), A) + g / a.tau;
        }
        __syncthreads();  // the token's logit is read before its gradient may replace it
    }
    const F2 neg = f2(-m, -m), cc = f2(a.c, a.c), oo = f2(off, off), AA = f2(A, A), BB = f2(B, B);
    run.template each<PIECE_SLOTS>([&](const typename R::TileT &x, int k) {
        run.put(x, k, out, false, [&](float p, float q) {
            const float2 v = split(fma2(f2(p, q) + neg, cc, oo));
            const F2 w = f2(ex2(v.x), ex2(v.y));
            return w * fma2(BB, f2(fmaxf(v.x, -1e4f), fmaxf(v.y, -1e4f)), AA);
        });
    });
    if (mine) {
        __syncthreads();  // after the element's ordinary value
        if (tid == 0)
            out.set(t, at_token);
    }
}

// Many rows, each of more than a tile a thread.
bool is_long(long long N, long long nvec) { return N > 152 && nvec > MAX_THREADS * MAX_VPT / 2; }

template <bool BF16>
int launch_long(const Score &a, cudaStream_t stream)
{
    constexpr size_t smem = static_cast<size_t>(LONG_SLOTS) * LONG_VT * LONG_T * 16;
    if (int rc = allow_shared(logprobs_long_kernel<BF16>, smem))
        return rc;
    return launch_rows(logprobs_long_kernel<BF16>, a, a.N, LONG_T, 1, smem, stream, "logprobs_long_kernel");
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
    const bool bf16 = logit_dtype == KDA_BF16;
    const long long nvec = rows::vectors_of(logits, V, ld, bf16);
    Score a{logits, ld, N, V, K, 1, 1, 1, tokens, temperature,
            Scale{rows::LOG2E / temperature, 16.0f * rows::LN2 * temperature}, logprob, entropy, stats,
            top_logprobs, top_ids, dev_status};
    // r lanes of w warps make the threshold: about two thirds of the warps, so that one warp of
    // small logits does not lower it
    auto threshold = [&](int warps) {
        a.r = std::max(1, std::min(32, (5 * K + 3 * warps - 1) / (3 * warps)));
        a.w = (K + a.r - 1) / a.r;
    };
    if (is_long(N, nvec)) {
        threshold(LONG_WARPS);
        return bf16 ? launch_long<true>(a, stream) : launch_long<false>(a, stream);
    }
    const Shape sh = rows::shape_of(N, nvec);
    a.cl = sh.cl;
    threshold(sh.cl * sh.threads / 32);
    return rows::with_vpt(sh.vpt, [&](auto vpt) {
        constexpr int VPT = decltype(vpt)::value;
        return rows::launch_rows(bf16 ? logprobs_kernel<true, VPT> : logprobs_kernel<false, VPT>, a,
                                 static_cast<long long>(N) * sh.cl, sh.threads, sh.cl, 0, stream, "logprobs_kernel");
    });
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
                      grad_entropy, temperature, rows::LOG2E / temperature};
    return rows::with_threads(cut.threads, [&](auto threads) {
        constexpr int T = decltype(threads)::value;
        auto *kernel = bf16 ? logprobs_backward_kernel<true, T> : logprobs_backward_kernel<false, T>;
        if (int rc = rows::allow_shared(kernel, cut.shared))
            return rc;
        return rows::launch_rows(kernel, a, static_cast<long long>(N) * cut.runs, T, 1, cut.shared, stream,
                                 "logprobs_backward_kernel");
    });
}
