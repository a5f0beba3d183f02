// attend_common.cuh -- what attention over a paged cache and its mass share: arguments, tiles of
// rows and keys, which of them a unit of work sees, and how tiles are copied.
//
// The rows of a session that read one kv head (t rows of G query heads each) are packed into
// tiles of 128: row r of a tile is token r / G, head r % G.  Keys come in tiles of 128 too.
#pragma once

#include "paged_cache.cuh"
#include "tile_ops.cuh"

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

constexpr int KT = 128;  // keys of a tile, and rows of a tile

__host__ __device__ constexpr int tile_bytes(int D) { return KT * D * 2; }

// A call cut into units: TQ tokens of a session and a kv head.
struct Span {
    Attend a;
    int TT, TQ, nq;  // tokens of a tile, of a unit; units a session and kv head
    int box;         // keys of a copied box: a page, or 128 of a larger one
    float c;         // scale log2 e
};

// One session's unit: which rows, and which key tiles they see.
struct Unit {
    int b, n, t0, nt;     // tokens before the call, first row, rows
    int hi, lo;           // keys [lo, hi) and below `sinks` are seen by some row
    int near, far, count; // key tiles: [0, far) for the sinks, then from `near`
};

__device__ __forceinline__ Unit unit_of(const Span &w, int i)
{
    Unit u;
    u.b = i / w.nq;
    u.t0 = (i - u.b * w.nq) * w.TQ;
    int t, bad;
    session(w.a.c, w.a.t_rows, w.a.T, u.b, u.n, t, bad);
    u.nt = min(w.TQ, t - u.t0);
    u.count = u.hi = u.lo = u.near = u.far = 0;
    if (u.nt <= 0)
        return u;
    u.hi = u.n + u.t0 + u.nt;
    if (w.a.seen.window) {
        u.lo = max(0, u.n + u.t0 - w.a.seen.window + 1);
        u.near = u.lo / KT;
        u.far = min((min(w.a.seen.sinks, u.hi) + KT - 1) / KT, u.near);
    }
    u.count = u.far + (u.hi + KT - 1) / KT - u.near;
    return u;
}

// Keys that some row of the unit sees, and keys that every row sees.
__device__ __forceinline__ bool some_see(const Span &w, const Unit &u, int j)
{
    return j < u.hi && (j >= u.lo || j < w.a.seen.sinks);
}

__device__ __forceinline__ bool all_see(const Span &w, const Unit &u, int j)
{
    return j <= u.n + u.t0 &&
           (!w.a.seen.window || u.hi - 1 - j < w.a.seen.window || j < w.a.seen.sinks);
}

// Some key of the tile from j0 on is hidden from some row.
__device__ __forceinline__ bool is_edge(const Span &w, const Unit &u, int j0)
{
    return !all_see(w, u, j0) || !all_see(w, u, j0 + KT - 1) ||
           (w.a.seen.window && j0 < w.a.seen.sinks && j0 + KT > w.a.seen.sinks);
}

// The first key of a unit's i-th tile.
__device__ __forceinline__ int tile_key(const Unit &u, int i) { return (i < u.far ? i : u.near + i - u.far) * KT; }

// The bits 0 .. n - 1 of 32.
__device__ __forceinline__ uint32_t bits_below(int n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// A place in the ring of tiles and the parity of its turn.
template <int ST>
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step()
    {
        if (++stage == ST) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// A lane has a box of each tile of keys (up to 16 boxes): whether some row sees it, ...
__device__ __forceinline__ bool box_seen(const Span &w, const Unit &u, int j0)
{
    const int lane = threadIdx.x & 31, j = j0 + lane * w.box;
    return lane * w.box < KT && j < u.hi && (j + w.box > u.lo || j < w.a.seen.sinks);
}

// ... and the page that it lies in.
__device__ __forceinline__ int page_of(const Span &w, const Unit &u, int j0)
{
    const int j = j0 + (threadIdx.x & 31) * w.box;
    return box_seen(w, u, j0) ? w.a.c.table[static_cast<long long>(u.b) * w.a.c.cols + (j >> w.a.c.shift)] : 0;
}

// A warp copies the tile of keys (or values) from j0 on to shared memory, `id` being page_of(j0);
// boxes that no row sees are left out.  `bar` counts the bytes.  Each lane issues its own box: a
// loop of one lane over all boxes took twice as long where a tile has eight.
template <int D>
__device__ __forceinline__ void copy_tile(const Span &w, const Unit &u, int h, int j0, int id, const CUtensorMap *m,
                                          uint32_t dst, uint32_t bar)
{
    const int lane = threadIdx.x & 31;
    const bool want = box_seen(w, u, j0);
    const uint32_t all = __ballot_sync(0xffffffffu, want);
    if (lane == 0)
        tiles::bar_expect(bar, static_cast<uint32_t>(__popc(all)) * w.box * D * 2);
    __syncwarp();
    if (want) {
        if (id < 0 || id >= w.a.c.pages) {
            raise(w.a.status, KDA_ST_BADPAGE);
            id = w.a.c.pages;  // behind the last: zeros
        }
#pragma unroll
        for (int half = 0; half < D / 64; ++half)
            tiles::copy_4d(dst + lane * w.box * 128 + half * KT * 128, m, half * 64,
                           (j0 + lane * w.box) & ((1 << w.a.c.shift) - 1), h, id, bar);
    }
    __syncwarp();
}

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
    // a window that holds every token is none, and no more sinks than tokens: sums of positions fit
    a->seen = Seen{window >= a->c.capacity() ? 0 : window, static_cast<int>(std::min<long long>(sinks, a->c.capacity()))};
    a->scale = scale;
    a->t_rows = t_rows;
    a->status = dev_status;
    return KDA_OK;
}

// Units of TQ tokens.
inline void lay_out(Span *w, int TQ)
{
    w->TT = KT / w->a.G;
    w->TQ = TQ;
    w->nq = (w->a.T - 1) / TQ + 1;
    w->box = std::min(1 << w->a.c.shift, KT);
    w->c = w->a.scale * LOG2E;
}

// Tensor map of k or v [pages][Hkv][page][D]: boxes of a page's rows (128 at most), 64 elements wide.
inline int cache_map(CUtensorMap *m, const Span &w, const void *base, bool bf16)
{
    const Cache &c = w.a.c;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), 1ull << c.shift, static_cast<cuuint64_t>(c.Hkv),
                                static_cast<cuuint64_t>(c.pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.slot_stride) * 2,
                                   static_cast<cuuint64_t>(c.head_stride) * 2,
                                   static_cast<cuuint64_t>(c.page_stride) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(w.box), 1, 1};
    return tiles::encode_map(m, bf16, 4, base, dims, strides, box);
}

// Tensor map of the rows q [B T][Hq][D]: boxes of one kv head's query heads and a tile's tokens.
inline int query_map(CUtensorMap *m, const Span &w, bool bf16)
{
    const Attend &a = w.a;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.c.D), static_cast<cuuint64_t>(a.Hq),
                                static_cast<cuuint64_t>(a.c.B) * a.T};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.c.D) * 2, static_cast<cuuint64_t>(a.ld) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(w.TT)};
    return tiles::encode_map(m, bf16, 3, a.q, dims, strides, box);
}

}  // namespace pages
}  // namespace kda
