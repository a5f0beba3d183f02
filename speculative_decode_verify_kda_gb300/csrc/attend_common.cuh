// attend_common.cuh -- the arguments that attention over a paged cache and its mass share.
#pragma once

#include "paged_cache.cuh"

namespace kda {
namespace pages {

struct Attend {
    Cache c;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    long long ld;
    int T, Hq, G;  // G = Hq / Hkv query heads read a kv head
    Seen seen;
    float scale;
    const int *t_rows;
    int *status;
};

inline int check_attend(const kda_cache *cache, const void *q, int T, int Hq, long long ld_q, const int *t_rows, int window,
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

}  // namespace pages
}  // namespace kda
