// spec_distill.cu -- distillation from a teacher's top entries: loss, gradient, and
// both in one call (sm_103a).
//
// A row has K teacher entries (id_k, v_k).  With m = max x of the student's row x,
// d = (x - m) / tau, s = ln sum exp d and ln p = d - s:
//   q_k  = exp(v_k / tau) / sum_j exp(v_j / tau)   (KDA_TEACHER_LOGITS), or
//   q_k  = exp(v_k)                                (KDA_TEACHER_LOGPROBS),
//   loss = w tau^2 sum_k q_k (ln q_k - ln p_{id_k}),
//   d x_i = g w tau (Q p_i - sum_{k: id_k = i} q_k),  Q = sum_k q_k.
// tau^2 keeps the gradient's size when tau changes (d ln p / d x has a factor 1 / tau).
//
// distill_kernel: a row stays in the registers of its CTA or cluster (logit_rows.cuh)
// between the sum and the gradient, so loss and gradient together read the logits once.
// The gradient is written as g w tau Q p for every element; after that, the CTA that
// holds a teacher's entry writes that element again with its q taken off.
#include <algorithm>
#include <cfloat>

#include "logit_rows.cuh"

namespace kda {
namespace {

using namespace rows;

struct Distill {
    const void *x;
    void *dx;
    long long ld, ldg, N;
    int V, K;
    int cl;         // CTAs of a row
    int per, runs;  // the gradient alone: vectors of a run, runs of a row
    const int *ids;
    const void *values;
    int value_bf16, value_logprobs;
    const float *weight, *g, *stats_in;
    float tau;
    Scale z;
    float *loss, *stats_out;
    int *status;
};

constexpr int EACH = KDA_TOPK_MAX / 32;  // entries of a lane

// The teacher's entries of a row.
struct __align__(16) Entries {
    int id[KDA_TOPK_MAX];    // -1: no entry, or one whose id an earlier entry has
    float off[KDA_TOPK_MAX]; // sum of the q of the entries with this id
    float q[KDA_TOPK_MAX];   // probability
    float lnq[KDA_TOPK_MAX];
    float x[KDA_TOPK_MAX];   // the student's logit, where it was asked for
    float Q;                 // sum of q: 1 for renormalised entries, 0 without any, NaN for a NaN
};

// One warp reads a row's entries in three steps, so that the latencies of the loads can be
// spent on something else: ids and values, the student's logits at the ids, the
// probabilities.
template <bool BF16>
struct Reader {
    int id[EACH];
    float v[EACH], x[EACH];

    __device__ __forceinline__ void load(const Distill &a, long long n)
    {
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int k = (threadIdx.x & 31) + 32 * i;
            id[i] = -1;
            v[i] = -INFINITY;
            if (k < a.K) {
                const long long o = n * a.K + k;
                id[i] = a.ids[o];
                v[i] = a.value_bf16 ? element<true>(a.values, o) : element<false>(a.values, o);
            }
        }
    }
    // The logits of ids in [lo, hi).
    __device__ __forceinline__ void gather(const Distill &a, const RowPtr<BF16> &row, int lo, int hi)
    {
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            if (id[i] >= a.V && a.status)
                atomicOr(a.status, KDA_ST_BADTOKEN);
            if (id[i] < 0 || id[i] >= a.V) {
                id[i] = -1;
                v[i] = -INFINITY;
            }
            x[i] = id[i] >= lo && id[i] < hi ? row.at(id[i]) : 0.0f;
        }
    }
    __device__ __forceinline__ void finish(const Distill &a, Entries &t)
    {
        const int lane = threadIdx.x & 31;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            if (!a.value_logprobs)
                v[i] /= a.tau;
            top = max_nan(top, v[i]);
        }
        top = warp_max_nan(top);
        const bool none = top == -INFINITY;
        const float ref = none || a.value_logprobs ? 0.0f : top;
        float e[EACH], Q = 0.0f;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            e[i] = expf(v[i] - ref);
            Q += e[i];
        }
        Q = warp_sum(Q);
        if (!(top < INFINITY))
            Q = NAN;
        const bool whole = !a.value_logprobs && !none;  // to be renormalised
        const float lnsum = whole ? logf(Q) : 0.0f;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const float q = whole ? e[i] / Q : e[i];
            t.id[lane + 32 * i] = id[i];
            t.off[lane + 32 * i] = q;
            t.q[lane + 32 * i] = q;
            t.lnq[lane + 32 * i] = v[i] - ref - lnsum;
            t.x[lane + 32 * i] = x[i];
        }
        if (lane == 0)
            t.Q = whole && Q == Q ? 1.0f : Q;
        __syncwarp();
        // an id listed twice: its first entry takes every q off
        int same[EACH] = {};
        const int4 *ids = reinterpret_cast<const int4 *>(t.id);
        for (int j = 0; j < (a.K + 3) / 4; ++j) {
            const int4 o = ids[j];
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                if (32 * i < a.K)
                    same[i] += (o.x == id[i]) + (o.y == id[i]) + (o.z == id[i]) + (o.w == id[i]);
        }
        bool twice = false;
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            twice |= id[i] >= 0 && same[i] > 1;
        if (__any_sync(0xffffffffu, twice)) {
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const int k = lane + 32 * i;
                if (id[i] >= 0 && same[i] > 1) {
                    float q = 0.0f;
                    for (int j = 0; j < a.K; ++j) {
                        if (t.id[j] == id[i]) {
                            if (j < k) {
                                id[i] = -1;
                                break;
                            }
                            q += t.q[j];
                        }
                    }
                    t.off[k] = q;
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                t.id[lane + 32 * i] = id[i];
        }
    }
};

// Loss and statistics of a row, by one warp.
__device__ __forceinline__ void write_loss(const Distill &a, long long n, float w, const Stats &st, const Entries &t)
{
    const int lane = threadIdx.x & 31;
    float kl = 0.0f, most = -INFINITY;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int k = lane + 32 * i;
        if (t.q[k] != 0.0f) {
            const float lp = st.empty() ? -INFINITY : (t.x[k] - st.m) / a.tau - st.lnS;
            const float term = t.q[k] * (t.lnq[k] - lp);
            kl += term;
            most = max_nan(most, term);
        }
    }
    kl = warp_sum(kl);
    most = warp_max_nan(most);
    if (kl == INFINITY && most < INFINITY)  // finite terms, rounded past the range
        kl = FLT_MAX;
    if (lane == 0) {
        a.loss[n] = t.Q == 0.0f ? 0.0f : kl * (a.tau * a.tau) * w;
        if (a.stats_out) {
            a.stats_out[2 * n] = st.m;
            a.stats_out[2 * n + 1] = st.lnS;
        }
        if ((st.bad() || t.Q != t.Q) && a.status)
            atomicOr(a.status, KDA_ST_NAN);
    }
}

// d x of the entries whose ids lie in [lo, hi), over what store_tile wrote there, by threads
// `who` of `many`.
template <bool BF16>
__device__ __forceinline__ void take_off(const Distill &a, const Entries &t, const RowPtr<BF16> &out, int lo, int hi,
                                         float m, float off, float scale, int who, int many)
{
    for (int k = who; k < a.K; k += many) {
        const int id = t.id[k];
        if (id >= lo && id < hi)
            out.set(id, scale * (t.Q * ex2(fmaf(t.x[k] - m, a.z.c, off)) - t.off[k]));
    }
}

// scale Q p of a pair.
__device__ __forceinline__ F2 weighted(float p, float q, float m, float c, float off, float sq)
{
    const float2 u = split(fma2(f2(p, q) + f2(-m, -m), f2(c, c), f2(off, off)));
    return f2(ex2(u.x), ex2(u.y)) * f2(sq, sq);
}

template <bool BF16, int VPT, bool GRAD>
__global__ void __launch_bounds__(MAX_THREADS, 3) distill_kernel(const Distill a)
{
    __shared__ Part parts[MAX_CL * (MAX_THREADS / 32)];
    __shared__ Entries t;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Place at(a.cl, blockDim.x);
    const int tid = threadIdx.x, step = blockDim.x, round = step * VPT;
    const long long n = at.row;
    const RowPtr<BF16> row(a.x, n * a.ld, a.V), out(GRAD ? a.dx : nullptr, GRAD ? n * a.ldg : 0, a.V);
    const int begin = at.begin(row.nvec), end = at.end(row.nvec);
    const float w = a.weight ? a.weight[n] : 1.0f;
    const float scale = GRAD ? w * a.tau * (a.g ? a.g[n] : 1.0f) : 0.0f;
    Tile<BF16, VPT> tile;
    if (w == 0.0f) {  // a row that takes no part is not read
        if (at.rank == 0 && tid == 0) {
            a.loss[n] = 0.0f;
            if (a.stats_out)
                a.stats_out[2 * n] = a.stats_out[2 * n + 1] = 0.0f;
        }
        if (GRAD)
            for (int b = begin; b < end; b += round)
                store_tile(tile, row, out, b + tid, step, end, true, [](float, float) { return F2{0}; });
        return;
    }
    at.arrive();
    // the ids of the CTA's run; the first CTA reads every entry's logit for the loss
    const int lo = max(0, row.first_id(begin)), hi = min(a.V, row.first_id(end));
    Running<false> run;
    float most = -INFINITY;
    int b = begin;
    do {
        tile.load(row, b + tid, step, end);
        if (b == begin && tid < 32) {
            Reader<BF16> r;
            r.load(a, n);
            r.gather(a, row, at.rank ? lo : 0, at.rank ? hi : a.V);
            r.finish(a, t);
        }
        const float m = tile.max_of();
        most = max_nan(most, m);
        run.add(tile, m, a.z);
        b += round;
    } while (b < end);
    const Part part = run.part(most, a.z.c, 0u);
    at.wait();
    at.hand_out(parts, part);
    at.sync();
    const Stats st = join(parts, at.parts(), a.z.c);
    if (at.rank == 0 && tid < 32)
        write_loss(a, n, w, st, t);
    if (GRAD) {
        const bool zero = st.empty() || t.Q == 0.0f || scale == 0.0f;
        const float off = -st.lnS * LOG2E, m = st.m, sq = scale * t.Q;
        b = begin;
        do {
            if (round < end - begin && !zero)  // of several rounds the registers hold the last one alone
                tile.load(row, b + tid, step, end);
            store_tile(tile, row, out, b + tid, step, end, zero,
                       [&](float p, float q) { return weighted(p, q, m, a.z.c, off, sq); });
            b += round;
        } while (b < end);
        if (!zero) {
            __syncthreads();
            take_off(a, t, out, lo, hi, m, off, scale, tid, step);
        }
    }
}

// For many long rows.  T threads pass their CTA's run of the row through shared memory; one
// more warp reads the teacher's entries meanwhile and writes the loss.  With a gradient the
// run stays in shared memory between the sum and the gradient where it fits (HELD); where
// it does not, and without a gradient, it passes through a few slots, for the gradient once
// more, out of L2.
constexpr int LONG_T = 256, LONG_VT = 4, LONG_SLOTS = 3, LONG_GROUP = LONG_T * LONG_VT;

template <bool BF16, bool GRAD, bool HELD>
__global__ void __launch_bounds__(LONG_T + 32, 4) distill_long_kernel(const Distill a)
{
    extern __shared__ uint4 slots[];
    __shared__ Part parts[MAX_CL * (LONG_T / 32)];
    __shared__ Entries t;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Place at(a.cl, LONG_T);
    const int tid = threadIdx.x;
    const bool reader = tid >= LONG_T;
    const long long n = at.row;
    const RowPtr<BF16> row(a.x, n * a.ld, a.V), out(GRAD ? a.dx : nullptr, GRAD ? n * a.ldg : 0, a.V);
    using R = Run<BF16, LONG_T, LONG_VT>;
    const R run(row, at, slots);
    const float w = a.weight ? a.weight[n] : 1.0f, g = GRAD && a.g ? a.g[n] : 1.0f;
    if (w == 0.0f) {  // a row that takes no part is not read
        if (at.rank == 0 && tid == LONG_T) {
            a.loss[n] = 0.0f;
            if (a.stats_out)
                a.stats_out[2 * n] = a.stats_out[2 * n + 1] = 0.0f;
        }
        if (GRAD && !reader)
            for (int k = 0; k < run.groups; ++k)
                run.put(typename R::TileT(), k, out, true, [](float, float) { return F2{0}; });
        return;
    }
    at.arrive();
    const float scale = GRAD ? w * a.tau * g : 0.0f;
    const int lo = max(0, row.first_id(run.begin)), hi = min(a.V, row.first_id(run.end));
    if (reader) {
        Reader<BF16> r;
        r.load(a, n);
        // the first CTA reads every entry's logit for the loss
        r.gather(a, row, at.rank ? lo : 0, at.rank ? hi : a.V);
        r.finish(a, t);
        at.wait();
    } else {
        Running<false> sums;
        float most = -INFINITY;
        auto add = [&](const typename R::TileT &x) {
            const float m = x.max_of();
            most = max_nan(most, m);
            sums.add(x, m, a.z);
        };
        if (HELD) {
            for (int k = 0; k < run.groups; ++k)
                run.start(k, k);
            for (int k = 0; k < run.groups; ++k) {
                typename R::TileT x;
                copies_done(min(3, run.groups - 1 - k));
                run.get(x, k, k);
                add(x);
            }
        } else {
            run.template each<LONG_SLOTS>([&](const typename R::TileT &x, int) { add(x); });
        }
        const Part part = sums.part(most, a.z.c, 0u);
        at.wait();
        at.hand_out(parts, part);
    }
    at.sync();
    if (!GRAD && !reader)
        return;
    const Stats st = join(parts, at.parts(), a.z.c);
    const bool zero = st.empty() || t.Q == 0.0f || scale == 0.0f;
    const float off = -st.lnS * LOG2E, m = st.m, sq = scale * t.Q;
    if (reader) {
        if (at.rank == 0)
            write_loss(a, n, w, st, t);
    } else {
        auto value = [&](float p, float q) { return weighted(p, q, m, a.z.c, off, sq); };
        if (HELD) {
            for (int k = 0; k < run.groups; ++k) {
                typename R::TileT x;
                run.get(x, k, k);
                run.put(x, k, out, zero, value);
            }
        } else {
            run.template each<LONG_SLOTS>(
                [&](const typename R::TileT &x, int k) { run.put(x, k, out, zero, value); });
        }
    }
    if (GRAD) {
        __syncthreads();
        if (!zero)
            take_off(a, t, out, lo, hi, m, off, scale, tid, LONG_T + 32);
    }
}

// The gradient alone.  A row is cut into runs that need nothing of one another; a run passes
// through shared memory while one more warp reads the entries.
template <bool BF16, int T>
__global__ void __launch_bounds__(T + 32) distill_backward_kernel(const Distill a)
{
    extern __shared__ uint4 slots[];
    __shared__ Entries t;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = blockIdx.x / a.runs;
    const int begin = static_cast<int>(blockIdx.x % a.runs) * a.per, tid = threadIdx.x;
    const RowPtr<BF16> row(a.x, n * a.ld, a.V), out(a.dx, n * a.ldg, a.V);
    using R = Run<BF16, T, PIECE_VT>;
    const R run(row, begin, min(row.nvec, begin + a.per), slots);
    const int lo = max(0, row.first_id(run.begin)), hi = min(a.V, row.first_id(run.end));
    const float w = a.weight ? a.weight[n] : 1.0f, g = a.g ? a.g[n] : 1.0f;
    const float m = a.stats_in[2 * n], off = -a.stats_in[2 * n + 1] * LOG2E;
    const float scale = w == 0.0f ? 0.0f : w * a.tau * g;
    const bool out_of_it = m == -INFINITY || scale == 0.0f;  // the row is not read
    auto meet = [] { asm volatile("barrier.sync 1, %0;" ::"n"(T + 32) : "memory"); };
    if (tid >= T) {
        if (out_of_it)
            return;
        Reader<BF16> r;
        r.load(a, n);
        r.gather(a, row, lo, hi);
        r.finish(a, t);
        meet();  // the entries are there, and the logits at them have been read
    } else if (out_of_it) {
        for (int k = 0; k < run.groups; ++k)
            run.put(typename R::TileT(), k, out, true, [](float, float) { return F2{0}; });
        return;
    } else {
        float sq = 0.0f;
        bool zero = false;
        run.template each<PIECE_SLOTS>([&](const typename R::TileT &x, int k) {
            if (k == 0) {
                meet();
                zero = t.Q == 0.0f;
                sq = scale * t.Q;
            }
            run.put(x, k, out, zero, [&](float p, float q) { return weighted(p, q, m, a.z.c, off, sq); });
        });
    }
    meet();  // the gradient is written, the corrections come over it
    if (t.Q != 0.0f)
        take_off(a, t, out, lo, hi, m, off, scale, tid, T + 32);
}

int check_teacher(const kda_teacher *t, int N)
{
    if (!t)
        return fail(KDA_EINVAL, "teacher must not be NULL");
    if (t->K < 1 || t->K > KDA_TOPK_MAX)
        return fail(KDA_EINVAL, "teacher K must lie in 1..128, got " + std::to_string(t->K));
    if (t->value_dtype != KDA_F32 && t->value_dtype != KDA_BF16)
        return fail(KDA_EINVAL, "teacher value_dtype must be KDA_F32 or KDA_BF16");
    if (t->kind != KDA_TEACHER_LOGITS && t->kind != KDA_TEACHER_LOGPROBS)
        return fail(KDA_EINVAL, "teacher kind must be KDA_TEACHER_LOGITS or KDA_TEACHER_LOGPROBS");
    if (N > 0 && (!t->ids || !t->values))
        return fail(KDA_EINVAL, "teacher ids and values must not be NULL");
    const uintptr_t es = t->value_dtype == KDA_BF16 ? 2 : 4;
    if (!aligned4(t->ids) || !aligned4(t->weight) || reinterpret_cast<uintptr_t>(t->values) % es)
        return fail(KDA_EINVAL, "teacher arrays must be aligned to their element");
    return KDA_OK;
}

// Many rows, each of more than a tile a thread.
bool is_long(long long N, long long nvec) { return N > 152 && nvec > MAX_THREADS * MAX_VPT / 2; }

template <bool BF16, bool GRAD, bool HELD>
int launch_long(const Distill &a, size_t smem, cudaStream_t stream)
{
    auto *kernel = distill_long_kernel<BF16, GRAD, HELD>;
    if (int rc = allow_shared(kernel, smem))
        return rc;
    return launch_rows(kernel, a, a.N * a.cl, LONG_T + 32, a.cl, smem, stream, "distill_long_kernel");
}

template <bool BF16, bool GRAD>
int launch_long(Distill a, long long nvec, cudaStream_t stream)
{
    constexpr size_t group = static_cast<size_t>(LONG_GROUP) * 16;
    a.cl = 1;
    if (GRAD) {
        constexpr long long HELD_GROUPS = 65536 / group;  // three CTAs an SM
        while (a.cl < MAX_CL && nvec > a.cl * HELD_GROUPS * LONG_GROUP)
            a.cl *= 2;
        const long long groups = ((nvec + a.cl - 1) / a.cl + LONG_GROUP - 1) / LONG_GROUP;
        if (groups * group <= 200 * 1024)
            return launch_long<BF16, true, true>(a, groups * group, stream);
        a.cl = 1;
    }
    return launch_long<BF16, GRAD, false>(a, LONG_SLOTS * group, stream);
}

template <bool GRAD>
int launch(Distill a, int dtype, cudaStream_t stream)
{
    const bool bf16 = dtype == KDA_BF16;
    const long long nvec = vectors_of(a.x, a.V, a.ld, bf16);
    if (is_long(a.N, nvec))
        return bf16 ? launch_long<true, GRAD>(a, nvec, stream) : launch_long<false, GRAD>(a, nvec, stream);
    const Shape sh = shape_of(a.N, nvec);
    a.cl = sh.cl;
    return with_vpt(sh.vpt, [&](auto vpt) {
        constexpr int VPT = decltype(vpt)::value;
        return launch_rows(bf16 ? distill_kernel<true, VPT, GRAD> : distill_kernel<false, VPT, GRAD>, a,
                           a.N * sh.cl, sh.threads, sh.cl, 0, stream, "distill_kernel");
    });
}

int launch_backward(Distill a, int dtype, cudaStream_t stream)
{
    const bool bf16 = dtype == KDA_BF16;
    const long long nvec = vectors_of(a.x, a.V, a.ld, bf16);
    const Pieces cut = pieces_of(nvec);
    a.per = cut.per;
    a.runs = cut.runs;
    return with_threads(cut.threads, [&](auto threads) {
        constexpr int T = decltype(threads)::value;
        auto *kernel = bf16 ? distill_backward_kernel<true, T> : distill_backward_kernel<false, T>;
        if (int rc = allow_shared(kernel, cut.shared))
            return rc;
        return launch_rows(kernel, a, a.N * cut.runs, T + 32, 1, cut.shared, stream, "distill_backward_kernel");
    });
}

Distill params(const void *x, void *dx, long long ld, long long ldg, int N, int V, const kda_teacher &t, float tau,
               const float *g, const float *stats_in, float *loss, float *stats_out, int *status)
{
    Distill a{};
    a.x = x;
    a.dx = dx;
    a.ld = ld;
    a.ldg = ldg;
    a.N = N;
    a.V = V;
    a.K = t.K;
    a.ids = t.ids;
    a.values = t.values;
    a.value_bf16 = t.value_dtype == KDA_BF16;
    a.value_logprobs = t.kind == KDA_TEACHER_LOGPROBS;
    a.weight = t.weight;
    a.g = g;
    a.stats_in = stats_in;
    a.tau = tau;
    a.z = Scale{LOG2E / tau, 16.0f * LN2 * tau};
    a.loss = loss;
    a.stats_out = stats_out;
    a.status = status;
    return a;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int spec_distill(const void *logits, int logit_dtype, int N, int V, long long ld,
                            const kda_teacher *teacher, float temperature, float *loss, float *stats, int *dev_status,
                            cudaStream_t stream)
{
    if (int rc = check_logits(logits, logit_dtype, N, V, ld, temperature))
        return rc;
    if (int rc = check_teacher(teacher, N))
        return rc;
    if (N == 0)
        return ok();
    if (!loss)
        return fail(KDA_EINVAL, "loss must not be NULL");
    if (!aligned4(loss) || !aligned4(stats) || !aligned4(dev_status))
        return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    return launch<false>(params(logits, nullptr, ld, 0, N, V, *teacher, temperature, nullptr, nullptr, loss, stats,
                                      dev_status), logit_dtype, stream);
}

extern "C" int spec_distill_backward(const void *logits, int logit_dtype, int N, int V, long long ld,
                                     const kda_teacher *teacher, float temperature, const float *stats,
                                     const float *grad_loss, void *dlogits, long long ldg, int *dev_status,
                                     cudaStream_t stream)
{
    if (int rc = check_logits(logits, logit_dtype, N, V, ld, temperature))
        return rc;
    if (int rc = check_teacher(teacher, N))
        return rc;
    if (int rc = check_grad(logits, dlogits, logit_dtype, N, V, ld, ldg))
        return rc;
    if (N == 0)
        return ok();
    if (!stats)
        return fail(KDA_EINVAL, "stats must not be NULL");
    if (!aligned4(stats) || !aligned4(grad_loss) || !aligned4(dev_status))
        return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    return launch_backward(params(logits, dlogits, ld, ldg, N, V, *teacher, temperature, grad_loss, stats, nullptr,
                                      nullptr, dev_status), logit_dtype, stream);
}

extern "C" int spec_distill_step(const void *logits, int logit_dtype, int N, int V, long long ld,
                                 const kda_teacher *teacher, float temperature, const float *grad_loss, float *loss,
                                 float *stats, void *dlogits, long long ldg, int *dev_status, cudaStream_t stream)
{
    if (int rc = check_logits(logits, logit_dtype, N, V, ld, temperature))
        return rc;
    if (int rc = check_teacher(teacher, N))
        return rc;
    if (int rc = check_grad(logits, dlogits, logit_dtype, N, V, ld, ldg))
        return rc;
    if (N == 0)
        return ok();
    if (!loss)
        return fail(KDA_EINVAL, "loss must not be NULL");
    if (!aligned4(grad_loss) || !aligned4(loss) || !aligned4(stats) || !aligned4(dev_status))
        return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    return launch<true>(params(logits, dlogits, ld, ldg, N, V, *teacher, temperature, grad_loss, nullptr, loss, stats,
                                     dev_status), logit_dtype, stream);
}
