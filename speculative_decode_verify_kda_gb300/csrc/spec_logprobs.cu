// spec_logprobs.cu -- log-probabilities of given tokens with entropy and top
// alternatives, and their gradient (sm_103a).
//
// For a row x with m = max x, d = (x - m) / temperature, S = sum exp d and s = ln S:
//   ln p = d - s,  H = s - (1/S) sum d exp d,
//   d x_i = (1/temperature) [ g (1{i = t} - p_i) - h p_i (ln p_i + H) ]
// for g = dL/d log p_t and h = dL/dH.
//
// One CTA a row.  The row is read once for the maximum, once for the two sums and
// once for each alternative (the largest key below the last one taken).
#include "logit_rows.cuh"

namespace kda {
namespace {

using namespace rows;
using Key = unsigned long long;

struct Score {
    const void *x;
    long long ld;
    int V, K;
    const int *tokens;
    float tau, c;  // c = log2(e) / tau
    float *logprob, *entropy, *stats, *top_logprobs;
    int *top_ids, *status;
};

template <bool BF16>
__global__ void __launch_bounds__(THREADS) logprobs_kernel(const Score a)
{
    __shared__ float fbuf[THREADS / 32];
    __shared__ Key kbuf[THREADS / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = blockIdx.x, base = n * a.ld;
    const int V = a.V, tid = threadIdx.x;
    float m = -INFINITY;
    for (int i = tid; i < V; i += THREADS)
        m = max_nan(m, element<BF16>(a.x, base + i));
    m = block_reduce(m, [](float p, float q) { return max_nan(p, q); }, fbuf);
    const bool bad = !(m < INFINITY), empty = m == -INFINITY;
    float S = 0.0f, E = 0.0f;
    if (!bad && !empty) {
        for (int i = tid; i < V; i += THREADS) {
            // below -1e4 (a masked token) the weight is 0 and so is its term of the entropy
            const float d = fmaxf((element<BF16>(a.x, base + i) - m) * a.c, -1e4f);
            const float e = exp2f(d);
            S += e;
            E += e * d;
        }
    }
    S = block_reduce(S, [](float p, float q) { return p + q; }, fbuf);
    E = block_reduce(E, [](float p, float q) { return p + q; }, fbuf);
    const float lnS = logf(S);
    const float none = bad ? NAN : -INFINITY;
    if (tid == 0) {
        float lp = 0.0f;
        if (a.tokens) {
            const int t = a.tokens[n];
            if (t >= V && a.status)
                atomicOr(a.status, KDA_ST_BADTOKEN);
            if (t >= 0 && t < V)
                lp = bad || empty ? none : (element<BF16>(a.x, base + t) - m) / a.tau - lnS;
        }
        if (a.logprob)
            a.logprob[n] = lp;
        if (a.entropy)
            a.entropy[n] = bad ? NAN : empty ? 0.0f : lnS - LN2 * E / S;
        if (a.stats) {
            a.stats[2 * n] = bad ? NAN : m;
            a.stats[2 * n + 1] = bad || empty ? none : lnS;
        }
        if (bad && a.status)
            atomicOr(a.status, KDA_ST_NAN);
    }
    Key last = ~0ull;
    for (int k = 0; k < a.K; ++k) {
        Key best = 0;
        if (!bad && !empty && last) {
            for (int i = tid; i < V; i += THREADS) {
                const float x = element<BF16>(a.x, base + i);
                const Key key = x > -INFINITY ? key_of(x, i) : 0;
                if (key < last && key > best)
                    best = key;
            }
        }
        best = block_reduce(best, [](Key p, Key q) { return p > q ? p : q; }, kbuf);
        last = best;
        if (tid == 0) {
            const long long o = n * a.K + k;
            a.top_ids[o] = best ? key_id(best) : -1;
            a.top_logprobs[o] = best ? (from_ordered(static_cast<uint32_t>(best >> 32)) - m) / a.tau - lnS : none;
        }
    }
}

struct ScoreGrad {
    const void *x;
    void *dx;
    long long ld, ldg;
    int V;
    const int *tokens;
    const float *stats, *entropy, *g, *h;
    float tau;
};

template <bool BF16>
__global__ void __launch_bounds__(THREADS) logprobs_backward_kernel(const ScoreGrad a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long n = blockIdx.x;
    const int t = a.tokens ? a.tokens[n] : -1;
    const bool has = t >= 0 && t < a.V;
    const float g = a.g && has ? a.g[n] : 0.0f, h = a.h ? a.h[n] : 0.0f;
    const float m = a.stats[2 * n], lnS = a.stats[2 * n + 1], H = a.h ? a.entropy[n] : 0.0f;
    const float inv = 1.0f / a.tau;
    for (int i = threadIdx.x; i < a.V; i += THREADS) {
        float d = 0.0f;
        if (m != -INFINITY && (g != 0.0f || h != 0.0f)) {
            const float lp = fmaf(element<BF16>(a.x, n * a.ld + i) - m, inv, -lnS);
            const float p = exp2f(lp * LOG2E);
            d = (i == t ? g : 0.0f) - p * (g + h * (fmaxf(lp, -1e4f) + H));
        }
        put<BF16>(a.dx, n * a.ldg + i, d * inv);
    }
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
    Score a{logits, ld, V, K, tokens, temperature, rows::LOG2E / temperature, logprob, entropy, stats, top_logprobs,
            top_ids, dev_status};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(N));
    cfg.blockDim = dim3(rows::THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = logit_dtype == KDA_BF16 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<true>, a)
                                                  : cudaLaunchKernelEx(&cfg, logprobs_kernel<false>, a);
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string("logprobs_kernel launch: ") + cudaGetErrorString(e));
    return check_launch("logprobs_kernel");
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
    ScoreGrad a{logits, dlogits, ld, ldg, V, tokens, stats, entropy, grad_logprob, grad_entropy, temperature};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(N));
    cfg.blockDim = dim3(rows::THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = logit_dtype == KDA_BF16 ? cudaLaunchKernelEx(&cfg, logprobs_backward_kernel<true>, a)
                                                  : cudaLaunchKernelEx(&cfg, logprobs_backward_kernel<false>, a);
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string("logprobs_backward_kernel launch: ") + cudaGetErrorString(e));
    return check_launch("logprobs_backward_kernel");
}
