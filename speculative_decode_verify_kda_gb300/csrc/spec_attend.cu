// spec_attend.cu -- attention of a call's rows over a paged cache.
#include "paged_cache.cuh"

namespace kda {
namespace {

using namespace pages;

struct Attend {
    Cache c;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    long long ld;
    int T, Hq, G;
    Seen seen;
    float scale;
    const int *t_rows;
    int *status;
};

template <bool BF16>
__device__ __forceinline__ float widen(uint16_t x)
{
    if (BF16)
        return __uint_as_float(static_cast<uint32_t>(x) << 16);
    return __half2float(__ushort_as_half(x));
}

template <bool BF16>
__device__ __forceinline__ uint16_t narrow(float x)
{
    return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// A warp for a row and head, one pass over the keys with the running maximum and sum.
template <bool BF16, int D>
__global__ void __launch_bounds__(128) attend_kernel(const Attend a)
{
    after_previous();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = blockIdx.x * 4ll + (threadIdx.x >> 5);
    if (w >= static_cast<long long>(a.c.B) * a.T * a.Hq)
        return;
    const int row = static_cast<int>(w / a.Hq), hq = static_cast<int>(w - static_cast<long long>(row) * a.Hq);
    const int b = row / a.T, t = row - b * a.T, h = hq / a.G;
    int n, tb, bad;
    session(a.c, a.t_rows, a.T, b, n, tb, bad);
    if (t >= tb) {
        if (bad && lane == 0)
            raise(a.status, bad);
        return;
    }
    float q[E], o[E] = {}, m = -INFINITY, l = 0.0f;
    for (int e = 0; e < E; ++e)
        q[e] = widen<BF16>(a.q[row * a.ld + hq * D + lane + 32 * e]) * (a.scale * LOG2E);
    const int p = n + t, *table = a.c.table + static_cast<long long>(b) * a.c.cols;
    for (int j = 0; j <= p; ++j) {
        if (a.seen.window && p - j >= a.seen.window && j >= a.seen.sinks) {
            j = p - a.seen.window;
            continue;
        }
        const long long at = token_at(a.c, table, h, j);
        if (at < 0 && lane == 0)
            raise(a.status, KDA_ST_BADPAGE);
        float s = 0.0f;
        for (int e = 0; e < E && at >= 0; ++e)
            s += q[e] * widen<BF16>(a.c.k[at + lane + 32 * e]);
        s = warp_sum(s);
        const float top = fmaxf(m, s), off = top == -INFINITY ? 0.0f : top, f = exp2f(m - off), x = exp2f(s - off);
        m = top;
        l = l * f + x;
        for (int e = 0; e < E; ++e)
            o[e] = o[e] * f + (at < 0 ? 0.0f : x * widen<BF16>(a.c.v[at + lane + 32 * e]));
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int e = 0; e < E; ++e)
        a.out[w * D + lane + 32 * e] = narrow<BF16>(o[e] * inv);
    if (a.lse && lane == 0)
        a.lse[w] = l == 0.0f ? -INFINITY : (m + log2f(l)) * LN2;
}

struct Mass {
    Attend a;
    const float *lse;
    float *mass;
    long long ld_mass;
};

// A warp for a key: the rows that see it one after another.
template <bool BF16, int D>
__global__ void __launch_bounds__(128) attend_mass_kernel(const Mass x)
{
    after_previous();
    constexpr int E = D / 32;
    const Attend &a = x.a;
    const int lane = threadIdx.x & 31, b = blockIdx.y / a.c.Hkv, h = blockIdx.y - b * a.c.Hkv;
    const int j = blockIdx.x * 4 + (threadIdx.x >> 5);
    int n, tb, bad;
    session(a.c, a.t_rows, a.T, b, n, tb, bad);
    if (bad && j == 0 && lane == 0)
        raise(a.status, bad);
    if (j >= n + tb || tb == 0)
        return;
    long long at = -2;
    float k[E], sum = 0.0f;
    for (int t = max(0, j - n); t < tb; ++t) {
        if (a.seen.window && n + t - j >= a.seen.window && j >= a.seen.sinks)
            break;
        if (at == -2) {
            at = token_at(a.c, a.c.table + static_cast<long long>(b) * a.c.cols, h, j);
            if (at < 0 && lane == 0)
                raise(a.status, KDA_ST_BADPAGE);
            for (int e = 0; e < E; ++e)
                k[e] = at < 0 ? 0.0f : widen<BF16>(a.c.k[at + lane + 32 * e]) * (a.scale * LOG2E);
        }
        const long long row = static_cast<long long>(b) * a.T + t;
        for (int g = 0; g < a.G; ++g) {
            const int hq = h * a.G + g;
            float s = 0.0f;
            for (int e = 0; e < E; ++e)
                s += k[e] * widen<BF16>(a.q[row * a.ld + hq * D + lane + 32 * e]);
            s = warp_sum(s);
            const float lse = x.lse[row * a.Hq + hq];
            sum += lse == -INFINITY ? 0.0f : exp2f(s - lse * LOG2E);
        }
    }
    float *to = x.mass + static_cast<long long>(blockIdx.y) * x.ld_mass + j;
    if (lane == 0 && (at != -2 || j >= n))
        *to = (j < n ? *to : 0.0f) + sum;
}

int check_attend(const kda_cache *cache, const void *q, int T, int Hq, long long ld_q, const int *t_rows, int window,
                 int sinks, float scale, int *dev_status, Attend *a)
{
    if (int rc = check_cache(cache, &a->c))
        return rc;
    if (int rc = check_query(a->c, Hq, window, sinks, scale))
        return rc;
    if (int rc = check_rows(a->c, q, T, static_cast<long long>(Hq) * a->c.D, ld_q, "q"))
        return rc;
    if (!aligned4(t_rows) || !aligned4(dev_status))
        return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    a->q = static_cast<const uint16_t *>(q);
    a->ld = ld_q;
    a->T = T;
    a->Hq = Hq;
    a->G = Hq / a->c.Hkv;
    a->seen = Seen{window, sinks};
    a->scale = scale;
    a->t_rows = t_rows;
    a->status = dev_status;
    return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t spec_attend_workspace_bytes(int, int, int, int, int) { return 16; }

extern "C" int spec_attend(const kda_cache *cache, const void *q, int T, int Hq, long long ld_q, const int *t_rows,
                           int window, int sinks, float scale, void *out, float *lse, int *dev_status, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream)
{
    Attend a{};
    if (int rc = check_attend(cache, q, T, Hq, ld_q, t_rows, window, sinks, scale, dev_status, &a))
        return rc;
    if (a.c.B == 0 || T == 0)
        return ok();
    if (!out || !aligned16(out) || !pages::aligned4(lse))
        return fail(KDA_EINVAL, "out must not be NULL and must be 16-byte aligned, lse 4-byte aligned");
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < spec_attend_workspace_bytes(a.c.B, T, Hq, a.c.Hkv, a.c.D))
        return fail(KDA_EINVAL, "workspace must hold spec_attend_workspace_bytes(...) bytes, 16-byte aligned");
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    const bool bf16 = cache->dtype == KDA_BF16;
    auto *kernel = a.c.D == 128 ? (bf16 ? attend_kernel<true, 128> : attend_kernel<false, 128>)
                                : (bf16 ? attend_kernel<true, 64> : attend_kernel<false, 64>);
    const long long blocks = (static_cast<long long>(a.c.B) * T * Hq + 3) / 4;
    if (blocks > 0x7fffffffll)
        return fail(KDA_EINVAL, "too many rows for one launch");
    return pages::launch(kernel, dim3(static_cast<unsigned>(blocks)), 128, 0, stream, "attend_kernel", a);
}

extern "C" int spec_attend_mass(const kda_cache *cache, const void *q, int T, int Hq, long long ld_q, const float *lse,
                                const int *t_rows, int window, int sinks, float scale, float *mass, long long ld_mass,
                                int *dev_status, cudaStream_t stream)
{
    Mass x{};
    if (int rc = check_attend(cache, q, T, Hq, ld_q, t_rows, window, sinks, scale, dev_status, &x.a))
        return rc;
    if (ld_mass < x.a.c.capacity() || ld_mass >= (1ll << 40))
        return fail(KDA_EINVAL, "ld_mass must be at least table_cols * page");
    if (x.a.c.B == 0 || T == 0)
        return ok();
    if (!lse || !mass || !pages::aligned4(lse) || !pages::aligned4(mass))
        return fail(KDA_EINVAL, "lse and mass must not be NULL and must be 4-byte aligned");
    x.lse = lse;
    x.mass = mass;
    x.ld_mass = ld_mass;
    const bool bf16 = cache->dtype == KDA_BF16;
    auto *kernel = x.a.c.D == 128 ? (bf16 ? attend_mass_kernel<true, 128> : attend_mass_kernel<false, 128>)
                                  : (bf16 ? attend_mass_kernel<true, 64> : attend_mass_kernel<false, 64>);
    return pages::launch(kernel, dim3(static_cast<unsigned>((x.a.c.capacity() + 3) / 4), x.a.c.B * x.a.c.Hkv), 128, 0,
                         stream, "attend_mass_kernel", x);
}
