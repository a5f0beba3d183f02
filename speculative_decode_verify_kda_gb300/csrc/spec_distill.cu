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
// One CTA a row; the row is read once for the maximum, once for the sum and once for
// the gradient.
#include <cfloat>

#include "logit_rows.cuh"

namespace kda {
namespace {

using namespace rows;

struct Distill {
    const void *x;
    void *dx;
    long long ld, ldg;
    int V, K;
    const int *ids;
    const void *values;
    int value_bf16, value_logprobs;
    const float *weight, *g, *stats_in;
    float tau, c;
    float *loss, *stats_out;
    int *status;
};

// The teacher's entries of the CTA's row.
struct Entries {
    int id[KDA_TOPK_MAX];     // -1: no entry
    float q[KDA_TOPK_MAX];    // probability
    float lnq[KDA_TOPK_MAX];
};

// Fills `t` and returns Q (1 for renormalised entries, 0 when there is none, NaN for a NaN
// among the values).  All threads call it; it ends with a barrier.
__device__ __forceinline__ float read_entries(const Distill &a, long long n, Entries &t, float *fbuf)
{
    const int k = threadIdx.x;
    int id = -1;
    float v = -INFINITY;
    if (k < a.K) {
        id = a.ids[n * a.K + k];
        if (id >= a.V) {
            if (a.status)
                atomicOr(a.status, KDA_ST_BADTOKEN);
            id = -1;
        }
        if (id >= 0) {
            v = a.value_bf16 ? element<true>(a.values, n * a.K + k) : element<false>(a.values, n * a.K + k);
            if (!a.value_logprobs)
                v /= a.tau;
        }
    }
    const float top = block_reduce(v, [](float p, float q) { return max_nan(p, q); }, fbuf);
    const bool none = top == -INFINITY;
    const float ref = none || a.value_logprobs ? 0.0f : top;
    const float e = none ? 0.0f : expf(v - ref);
    float Q = block_reduce(e, [](float p, float q) { return p + q; }, fbuf);
    if (!(top < INFINITY))
        Q = NAN;
    const float lnsum = a.value_logprobs || none ? 0.0f : logf(Q);
    if (k < KDA_TOPK_MAX) {
        t.id[k] = id;
        t.q[k] = a.value_logprobs ? e : none ? 0.0f : e / Q;
        t.lnq[k] = v - ref - lnsum;
    }
    __syncthreads();
    return none ? 0.0f : a.value_logprobs || Q != Q ? Q : 1.0f;
}

template <bool BF16, bool LOSS, bool GRAD>
__global__ void __launch_bounds__(THREADS) distill_kernel(const Distill a)
{
    __shared__ float fbuf[THREADS / 32];
    __shared__ Entries t;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = blockIdx.x, base = n * a.ld;
    const int V = a.V, tid = threadIdx.x;
    const float w = a.weight ? a.weight[n] : 1.0f;
    const float scale = GRAD ? w * a.tau * (a.g ? a.g[n] : 1.0f) : 0.0f;
    if (w == 0.0f || (!LOSS && scale == 0.0f)) {  // a row that takes no part is not read
        if (LOSS && tid == 0) {
            a.loss[n] = 0.0f;
            if (a.stats_out)
                a.stats_out[2 * n] = a.stats_out[2 * n + 1] = 0.0f;
        }
        if (GRAD)
            for (int i = tid; i < V; i += THREADS)
                put<BF16>(a.dx, n * a.ldg + i, 0.0f);
        return;
    }
    const float Q = read_entries(a, n, t, fbuf);
    float m, lnS;
    if (LOSS) {
        m = -INFINITY;
        for (int i = tid; i < V; i += THREADS)
            m = max_nan(m, element<BF16>(a.x, base + i));
        m = block_reduce(m, [](float p, float q) { return max_nan(p, q); }, fbuf);
        if (!(m < INFINITY))
            m = NAN;
        float S = 0.0f;
        if (m != -INFINITY)
            for (int i = tid; i < V; i += THREADS)
                S += exp2f((element<BF16>(a.x, base + i) - m) * a.c);
        lnS = logf(block_reduce(S, [](float p, float q) { return p + q; }, fbuf));
        float part = 0.0f;
        if (tid < a.K && t.id[tid] >= 0 && t.q[tid] != 0.0f) {
            const float x = element<BF16>(a.x, base + t.id[tid]);
            const float lp = m == -INFINITY ? -INFINITY : (x - m) / a.tau - lnS;
            part = t.q[tid] * (t.lnq[tid] - lp);
        }
        float kl = block_reduce(part, [](float p, float q) { return p + q; }, fbuf);
        const float most = block_reduce(part, [](float p, float q) { return max_nan(p, q); }, fbuf);
        if (kl == INFINITY && most < INFINITY)  // finite terms, rounded past the range
            kl = FLT_MAX;
        if (tid == 0) {
            a.loss[n] = Q == 0.0f ? 0.0f : kl * (a.tau * a.tau) * w;
            if (a.stats_out) {
                a.stats_out[2 * n] = m;
                a.stats_out[2 * n + 1] = lnS;
            }
            if ((m != m || Q != Q) && a.status)
                atomicOr(a.status, KDA_ST_NAN);
        }
    } else {
        m = a.stats_in[2 * n];
        lnS = a.stats_in[2 * n + 1];
    }
    if (!GRAD)
        return;
    // p = exp2(d log2(e) + off)
    const float off = -lnS * LOG2E;
    const bool zero = m == -INFINITY || Q == 0.0f || scale == 0.0f;
    float fix = 0.0f;
    bool first = false;
    if (tid < a.K && t.id[tid] >= 0 && !zero) {
        first = true;
        for (int j = 0; j < tid; ++j)
            first &= t.id[j] != t.id[tid];
        float q = 0.0f;
        for (int j = tid; j < a.K; ++j)
            q += t.id[j] == t.id[tid] ? t.q[j] : 0.0f;
        const float x = element<BF16>(a.x, base + t.id[tid]);
        fix = scale * (Q * exp2f(fmaf(x - m, a.c, off)) - q);
    }
    __syncthreads();  // the entries' logits are read before the gradient may replace them
    for (int i = tid; i < V; i += THREADS) {
        float d = 0.0f;
        if (!zero) {
            const float x = element<BF16>(a.x, base + i);
            d = scale * Q * exp2f(fmaf(x - m, a.c, off));
        }
        put<BF16>(a.dx, n * a.ldg + i, d);
    }
    __syncthreads();
    if (first)
        put<BF16>(a.dx, n * a.ldg + t.id[tid], fix);
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

template <bool LOSS, bool GRAD>
int launch(const Distill &a, int dtype, int N, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(N));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = dtype == KDA_BF16 ? cudaLaunchKernelEx(&cfg, distill_kernel<true, LOSS, GRAD>, a)
                                            : cudaLaunchKernelEx(&cfg, distill_kernel<false, LOSS, GRAD>, a);
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string("distill_kernel launch: ") + cudaGetErrorString(e));
    return check_launch("distill_kernel");
}

Distill params(const void *x, void *dx, long long ld, long long ldg, int V, const kda_teacher &t, float tau,
               const float *g, const float *stats_in, float *loss, float *stats_out, int *status)
{
    return Distill{x,     dx,    ld, ldg,    V,   t.K,           t.ids, t.values, t.value_dtype == KDA_BF16,
                   t.kind == KDA_TEACHER_LOGPROBS, t.weight, g,  stats_in, tau, LOG2E / tau, loss,  stats_out,  status};
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
    return launch<true, false>(params(logits, nullptr, ld, 0, V, *teacher, temperature, nullptr, nullptr, loss, stats,
                                      dev_status), logit_dtype, N, stream);
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
    return launch<false, true>(params(logits, dlogits, ld, ldg, V, *teacher, temperature, grad_loss, stats, nullptr,
                                      nullptr, dev_status), logit_dtype, N, stream);
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
    return launch<true, true>(params(logits, dlogits, ld, ldg, V, *teacher, temperature, grad_loss, nullptr, loss, stats,
                                     dev_status), logit_dtype, N, stream);
}
