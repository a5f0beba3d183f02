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
// The gradient is written as g w tau Q p for every element; after that, the CTA that holds a
// teacher's entry writes that element again with its q taken off.
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

// One warp reads a row's entries in steps, so that the latencies of the loads can be spent on
// something else: load() ids and values, gather() the student's logits at the ids, finish()
// the probabilities, keep() those logits, once() ids listed twice.  gather() comes before and
// keep() after the barrier behind which the gradient may replace the logits.
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
        for (int i = 0; i < EACH; ++i)
            top = max_nan(top, v[i]);
        top = warp_max_nan(top);
        const bool none = top == -INFINITY;
        float e[EACH], Q = 0.0f;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            // the difference before the quotient: at a low temperature v / tau alone is large, and
            // its rounding would be q's, or past the range
            if (!a.value_logprobs && !none)
                v[i] = (v[i] - top) * a.z.inv;
            e[i] = 32 * i < a.K ? expf(v[i]) : 0.0f;
            Q += e[i];
        }
        Q = warp_sum(Q);
        if (!(top < INFINITY))
            Q = NAN;
        const bool whole = !a.value_logprobs && !none;  // to be renormalised
        const float lnsum = whole ? logf(Q) : 0.0f, part = 1.0f / Q;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const float q = whole ? e[i] * part : e[i];
            t.id[lane + 32 * i] = id[i];
            t.off[lane + 32 * i] = q;
            t.q[lane + 32 * i] = q;
            t.lnq[lane + 32 * i] = v[i] - lnsum;
        }
        if (lane == 0)
            t.Q = whole && Q == Q ? 1.0f : Q;
    }
    __device__ __forceinline__ void keep(Entries &t) const
    {
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            t.x[(threadIdx.x & 31) + 32 * i] = x[i];
        __syncwarp();
    }
    // An id listed twice: its first entry takes every q off.  Not needed before the gradient's
    // corrections, so it is done while the others write the gradient.
    __device__ __forceinline__ void once(const Distill &a, Entries &t)
    {
        const int lane = threadIdx.x & 31;
        int same[EACH] = {};
        const int4 *ids = reinterpret_cast<const int4 *>(t.id);
#pragma unroll 2
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
        if (!__any_sync(0xffffffffu, twice))
            return;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int k = lane + 32 * i;
            if (id[i] >= 0 && same[i] > 1) {
                float q = 0.0f;
#pragma unroll 1
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
};

// Loss and statistics of a row, by one warp.  The loss is formed as
//   w tau sum_k q_k (tau (ln q_k + s) - (x_k - m)),
// the sum 2^-40 times as large: no difference of finite logits, no quotient by tau and no sum of
// such terms then passes the range of f32, although the loss may (it is held at its end).
__device__ __forceinline__ void write_loss(const Distill &a, long long n, float w, const Stats &st, const Entries &t)
{
    constexpr float UP = 1099511627776.0f, DOWN = 1.0f / UP;  // 2^40
    const int lane = threadIdx.x & 31;
    const float tau = a.tau * DOWN, m = st.m * DOWN;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int k = lane + 32 * i;
        if (t.q[k] != 0.0f)  // (a masked logit's term is +inf)
            sum += st.empty() ? INFINITY : t.q[k] * fmaf(t.lnq[k] + st.lnS, tau, m - t.x[k] * DOWN);
    }
    sum = warp_sum(sum) * a.tau;
    // times w 2^40, the factor first that brings it towards 1
    float loss = fabsf(sum) >= UP ? sum * w * UP : sum * UP * w;
    if (fabsf(sum) <= FLT_MAX && fabsf(w) <= FLT_MAX)
        loss = fminf(fmaxf(loss, -FLT_MAX), FLT_MAX);
    if (lane == 0) {
        // (Q is NaN where a value is no number or +inf, whatever the sum has made of it)
        a.loss[n] = t.Q == 0.0f ? 0.0f : t.Q != t.Q ? t.Q : loss;
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
#pragma unroll 1
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

// Loss, or loss and gradient.  T threads pass their CTA's run of the row through shared memory;
// one more warp reads the teacher's entries meanwhile and writes the loss.  With a gradient the
// run stays in shared memory between the sum and the gradient where it fits (HELD); where
// it does not, and without a gradient, it passes through a few slots, for the gradient once
// more, out of L2.
constexpr int ROW_VT = 4, ROW_SLOTS = 3;

template <bool BF16, int T, bool GRAD, bool HELD>
__global__ void __launch_bounds__(T + 32, T == 256 ? 4 : T == 128 ? 6 : 8) distill_kernel(const Distill a)
{
    extern __shared__ uint4 slots[];
    __shared__ Part parts[MAX_CL * (T / 32)];
    __shared__ Entries t;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Place at(a.cl, T);
    const int tid = threadIdx.x;
    const bool reader = tid >= T;
    const long long n = at.row;
    const RowPtr<BF16> row(a.x, n * a.ld, a.V), out(GRAD ? a.dx : nullptr, GRAD ? n * a.ldg : 0, a.V);
    using R = Run<BF16, T, ROW_VT>;
    const R run(row, at, slots);
    const float w = a.weight ? a.weight[n] : 1.0f, g = GRAD && a.g ? a.g[n] : 1.0f;
    if (w == 0.0f) {  // a row that takes no part is not read
        if (at.rank == 0 && tid == T) {
            a.loss[n] = 0.0f;
            if (a.stats_out)
                a.stats_out[2 * n] = a.stats_out[2 * n + 1] = 0.0f;
        }
        if (GRAD && !reader)
            run.clear(out);
        return;
    }
    at.started();
    const float scale = GRAD ? w * a.tau * g : 0.0f;
    const int lo = max(0, row.first_id(run.begin)), hi = min(a.V, row.first_id(run.end));
    Reader<BF16> r;
    if (reader) {
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
#pragma unroll 1
            for (int k = 0; k < run.groups; ++k)
                run.start(k, k);
#pragma unroll 1
            for (int k = 0; k < run.groups; ++k) {
                typename R::TileT x;
                copies_done(min(3, run.groups - 1 - k));
                run.get(x, k, k);
                add(x);
            }
        } else {
            run.template each<ROW_SLOTS>(false, [&](const typename R::TileT &x, int, int) { add(x); });
        }
        const Part part = sums.part(most, a.z, 0u);
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
        r.keep(t);
        if (at.rank == 0)
            write_loss(a, n, w, st, t);
        if (GRAD)
            r.once(a, t);
    } else {
        auto value = [&](float p, float q) { return weighted(p, q, m, a.z.c, off, sq); };
        if (zero) {
            run.clear(out);
        } else if (HELD) {
#pragma unroll 1
            for (int k = 0; k < run.groups; ++k) {
                typename R::TileT x;
                run.get(x, k, k);
                run.put(x, k, k, out, value);
            }
        } else {
            run.template each<ROW_SLOTS>(row.skip != out.skip, [&](const typename R::TileT &x, int k, int s) {
                run.put(x, k, s, out, value);
            });
        }
    }
    if (GRAD) {
        __syncthreads();
        if (!zero)
            take_off(a, t, out, lo, hi, m, off, scale, tid, T + 32);
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
        meet();  // Q is there, and the logits at the ids have been read
        r.keep(t);
        r.once(a, t);
    } else if (out_of_it) {
        run.clear(out);
        return;
    } else {
        float sq = 0.0f;
        run.template each<PIECE_SLOTS>(row.skip != out.skip, [&](const typename R::TileT &x, int k, int s) {
            if (k == 0) {
                meet();
                sq = scale * t.Q;
            }
            if (t.Q != 0.0f)
                run.put(x, k, s, out, [&](float p, float q) { return weighted(p, q, m, a.z.c, off, sq); });
        });
        if (t.Q == 0.0f)
            run.clear(out);
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

// Vectors of a run with which an SM holds three CTAs, or two.
constexpr long long THREE = 4480, TWO = 6912;

template <int T, bool GRAD, bool HELD>
int launch_with(const Distill &a, bool bf16, long long per, cudaStream_t stream)
{
    constexpr size_t most = (HELD ? TWO : ROW_SLOTS * ROW_VT * T) * 16;
    const size_t smem = std::min(most, static_cast<size_t>(per) * 16);
    auto *kernel = bf16 ? distill_kernel<true, T, GRAD, HELD> : distill_kernel<false, T, GRAD, HELD>;
    if (int rc = allow_shared(kernel, smem, most))
        return rc;
    return launch_rows(kernel, a, a.N * a.cl, T + 32, a.cl, smem, stream, "distill_kernel");
}

// Threads by the vectors of a run: what is fixed for a warp weighs on short runs, so those of
// many rows get few warps (us for 8000 bf16 rows of 1000 / 5000 / 9000 / 17000 logits, 32
// threads: 15.6 / 36 / 61 / -, 64: 20.3 / 34.5 / 48 / -, 128: 31 / 43 / 56 / 82, 256: 44 / 59 /
// 70 / 94); where the GPU is not full a row's latency counts, and they get more (15 rows of
// 1001 f32: 64 threads 3.03, 128 2.83, 256 2.88).
template <bool GRAD, bool HELD>
int launch_held(const Distill &a, bool bf16, long long per, cudaStream_t stream)
{
    const bool full = a.N * a.cl > 2 * SMS;
    if (per <= (full ? 400 : 32))
        return launch_with<32, GRAD, HELD>(a, bf16, per, stream);
    if (per <= (full ? 1536 : 96))
        return launch_with<64, GRAD, HELD>(a, bf16, per, stream);
    if (per <= (full ? 2880 : 1024))
        return launch_with<128, GRAD, HELD>(a, bf16, per, stream);
    return launch_with<256, GRAD, HELD>(a, bf16, per, stream);
}

template <bool GRAD>
int launch(Distill a, int dtype, cudaStream_t stream)
{
    const bool bf16 = dtype == KDA_BF16;
    const long long nvec = vectors_of(a.x, a.V, a.ld, bf16);
    // With a gradient a run is held if an SM then has three CTAs (or two, where eight CTAs a row
    // cannot do better); beyond that a row is read twice by one CTA.  Held against read twice, us:
    // 4096 bf16 rows of 131072 (four CTAs a row) 340 against 456, 480 of 32768 14.4 against 17.2.
    a.cl = 1;
    bool held = GRAD;
    if (GRAD) {
        while (a.cl < MAX_CL && nvec > a.cl * THREE)
            a.cl *= 2;
        held = (nvec + a.cl - 1) / a.cl <= TWO;
        if (!held)
            a.cl = 1;
    }
    // Few rows: more CTAs a row while there are SMs to spare and a run keeps 512 vectors (us for 1
    // / 8 / 32 / 64 bf16 rows of 32768 logits: one CTA 4.96 / 4.97 / 4.99 / 4.99, two 4.28 / 4.38 /
    // 4.37 / 4.44, four 3.76 / 3.88 / 4.04 / 4.50, eight 3.62 / 3.82 / 4.21 / 5.47).
    while (a.cl < MAX_CL && a.N * a.cl * 2 <= SMS && nvec >= 1024ll * a.cl)
        a.cl *= 2;
    const long long per = (nvec + a.cl - 1) / a.cl;
    return held ? launch_held<GRAD, GRAD>(a, bf16, per, stream) : launch_held<GRAD, false>(a, bf16, per, stream);
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
        if (int rc = allow_shared(kernel, cut.shared, piece_shared(T)))
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
    a.z = Scale{LOG2E / tau, 16.0f * LN2 * tau, 1.0f / tau};
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
