// spec_attend_mass.cu -- what every key of a paged cache was worth to a call's rows.
#include "attend_common.cuh"

namespace kda {
namespace {

using namespace pages;

template <bool BF16>
__device__ __forceinline__ float widen(uint16_t x)
{
    if (BF16)
        return __uint_as_float(static_cast<uint32_t>(x) << 16);
    return __half2float(__ushort_as_half(x));
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
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

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int spec_attend_mass(const kda_cache *cache, const void *q, int T, int Hq, long long ld_q, const float *lse,
                                const int *t_rows, int window, int sinks, float scale, float *mass, long long ld_mass,
                                int *dev_status, cudaStream_t stream)
{
    Mass x{};
    if (int rc = pages::check_attend(cache, q, T, Hq, ld_q, t_rows, window, sinks, scale, dev_status, &x.a))
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
