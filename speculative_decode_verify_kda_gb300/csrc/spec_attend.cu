// spec_attend.cu -- attention of a call's rows over a paged cache.
//
// The rows of a session that read one kv head (t rows of G query heads each) are packed into
// tiles of 128: row r of a tile is token r / G, head r % G.  A unit of work is one session, one
// kv head and one tile (or two) of rows against the key tiles of 128 that any of them sees; all
// units' key tiles in a row are cut into equal shares, one a CTA, whatever the sessions' lengths.
// A unit that lies within one share writes its result; the parts of the others go to the
// workspace with their maxima and sums and are joined by a second launch.
//
// A CTA is a pipeline: one warp copies key and value tiles page by page (tensor copies into a
// ring of shared memory), one thread issues the products S = Q K^T and O += P V (tcgen05, sums
// in tensor memory), and two groups of 128 threads turn S into P, a thread a row: running
// maximum and sum, exp2, 16-bit weights back into tensor memory over S.  With more than 128 rows
// (PAIR) the groups have a tile of rows each and share the key tiles; with fewer both have the
// same rows and take every other key tile, and their results are joined at the end.  While one
// group computes weights, the tensor cores work for the other.
#include "attend_common.cuh"
#include "tile_ops.cuh"

namespace kda {
namespace {

using namespace pages;
using namespace tiles;

constexpr int KT = 128;              // keys of a tile, and rows of a tile
constexpr int COPY_WARP = 8, MMA_WARP = 9;
constexpr int THREADS = 384;         // two groups of 128 and four warps more, two of them idle
// Registers are handed from the last four warps to the groups (a row of 128 scores is held in
// them): 256 x 216 + 128 x 72 = 384 x 168, what the launch has.
constexpr int GROUP_REGS = 216, OTHER_REGS = 72;
constexpr int SPARE = 2048;          // barriers and what the groups tell each other
// The running maximum that weights are taken against follows the true one only when it falls
// behind by more than this many powers of two: weights stay below 2^8, and the sums in tensor
// memory are seldom rescaled.
constexpr float LAG = 8.0f;

__host__ __device__ constexpr int tile_bytes(int D) { return KT * D * 2; }
__host__ __device__ constexpr int stages(int D) { return D == 128 ? 5 : 8; }
__host__ __device__ constexpr int shared_bytes(int D) { return 2 * tile_bytes(D) + stages(D) * tile_bytes(D) + SPARE + 1024; }

struct Walk {
    Attend a;
    int TT, TQ, nq;  // tokens of a tile, of a unit; units a session and kv head
    int box;         // rows of a copied box: a page, or 128 rows of a larger one
    float c;         // scale log2 e
    long long *plan;         // [P + 1]: tiles before each (session, unit), and a CTA's share
    float2 *stats;           // [2 grid][rows] maximum and sum of a part
    float *parts;            // [2 grid][rows][D] its sums
};

// One session's unit: which rows, and which key tiles they see.
struct Unit {
    int b, n, t0, nt;     // tokens before the call, first row, rows
    int hi, lo;           // keys [lo, hi) and below `sinks` are seen by some row
    int near, far, count; // key tiles: [0, far) for the sinks, then from `near`
};

__device__ __forceinline__ Unit unit_of(const Walk &w, int i)
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
__device__ __forceinline__ bool some_see(const Walk &w, const Unit &u, int j)
{
    return j < u.hi && (j >= u.lo || j < w.a.seen.sinks);
}

__device__ __forceinline__ bool all_see(const Walk &w, const Unit &u, int j)
{
    return j <= u.n + u.t0 &&
           (!w.a.seen.window || u.hi - 1 - j < w.a.seen.window || j < w.a.seen.sinks);
}

// A CTA's share of the tiles and where it begins.
struct Share {
    long long first, last;  // tiles
    long long pair, before; // the (session, unit) of `first`, and the tiles before that
};

// The runs of one unit's tiles after another within a share.
struct Runs {
    const Walk &w;
    long long left;      // tiles from this run on
    int pair, slot;
    Unit u;
    int h, off, todo;    // tiles off .. off + todo - 1 of the unit
    bool whole;          // all of them; else the parts go to `slot` of the workspace
    __device__ Runs(const Walk &w_, const Share &s)
        : w(w_), left(s.last - s.first), pair(static_cast<int>(s.pair)), slot(2 * blockIdx.x), todo(0)
    {
        if (left > 0) {
            u = unit_of(w, pair);
            h = static_cast<int>((s.first - s.before) / u.count);
            off = static_cast<int>(s.first - s.before - static_cast<long long>(u.count) * h);
        }
    }
    __device__ __forceinline__ bool next()
    {
        if (todo > 0) {
            left -= todo;
            off = 0;
            slot |= 1;
            ++h;
        }
        if (left <= 0)
            return false;
        if (h == w.a.c.Hkv) {
            h = 0;
            do
                u = unit_of(w, ++pair);
            while (u.count == 0);
        }
        todo = static_cast<int>(min(static_cast<long long>(u.count - off), left));
        whole = todo == u.count;
        return true;
    }
};

// Every CTA finds its share: the tiles of all units in the order (session, unit, kv head).
// CTA 0 leaves the tiles before each (session, unit) in the workspace.  `part`: 16 long longs.
__device__ Share share_of(const Walk &w, long long *part, Share *found)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long P = static_cast<long long>(w.a.c.B) * w.nq;
    auto tiles_of = [&](long long i) { return i < P ? static_cast<long long>(unit_of(w, static_cast<int>(i)).count) * w.a.c.Hkv : 0ll; };
    // over all: one chunk of THREADS units, or more
    long long mine = 0;
    for (long long i = tid; i < P; i += THREADS)
        mine += tiles_of(i);
#pragma unroll
    for (int d = 16; d; d >>= 1)
        mine += __shfl_xor_sync(0xffffffffu, mine, d);
    if (lane == 0)
        part[warp] = mine;
    if (tid == 0)
        *found = Share{0, 0, 0, 0};
    __syncthreads();
    long long total = 0;
    for (int i = 0; i < THREADS / 32; ++i)
        total += part[i];
    __syncthreads();
    const long long per = max(1ll, (total + gridDim.x - 1) / gridDim.x);
    const long long first = per * blockIdx.x, last = min(total, first + per);
    long long carry = 0;
    for (long long i0 = 0; i0 < P && (carry <= first || blockIdx.x == 0); i0 += THREADS) {
        const long long x = tiles_of(i0 + tid);
        long long s = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d)
                s += y;
        }
        if (lane == 31)
            part[warp] = s;
        __syncthreads();
        long long before = carry + s - x;
        for (int i = 0; i < THREADS / 32; ++i) {
            if (i < warp)
                before += part[i];
            carry += part[i];
        }
        if (first < last && before <= first && first < before + x)
            *found = Share{first, last, i0 + tid, before};
        if (blockIdx.x == 0 && i0 + tid < P)
            w.plan[i0 + tid] = before;
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0)
        w.plan[P] = per;
    __syncthreads();
    return *found;
}

// The place in the ring's order of a run's i-th value tile: key tiles run `lead` ahead.
__device__ __forceinline__ uint32_t value_at(int lead, int todo, int i) { return lead + i + min(i, todo - lead); }

template <int D, bool PAIR, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) attend_kernel(const __grid_constant__ Walk w,
                                                            const __grid_constant__ CUtensorMap map_q,
                                                            const __grid_constant__ CUtensorMap map_k,
                                                            const __grid_constant__ CUtensorMap map_v)
{
    constexpr int TILE = tile_bytes(D), HALF = KT * 128, HALVES = D / 64, ST = stages(D);
    constexpr int LEAD = PAIR ? 1 : 2;  // key tiles ahead of value tiles
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t q_at = base, ring = base + 2 * TILE, bars = ring + ST * TILE;
    // barriers
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (ST + s); };
    auto q_full = [&](int i) { return bars + 8u * (2 * ST + i); };
    auto q_empty = [&](int i) { return bars + 8u * (2 * ST + 2 + i); };
    auto s_full = [&](int g) { return bars + 8u * (2 * ST + 4 + g); };
    auto p_full = [&](int g) { return bars + 8u * (2 * ST + 6 + g); };
    auto o_full = [&](int g) { return bars + 8u * (2 * ST + 8 + g); };
    auto v_clean = [&](int i) { return bars + 8u * (2 * ST + 10 + i); };
    const uint32_t told = bars + 8u * (2 * ST + 14), joined = told + 8, drained = told + 16;
    // behind the barriers
    unsigned char *spare = raw + (bars - smem_addr(raw)) + 512;
    volatile int *gave_up = reinterpret_cast<volatile int *>(spare);
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(spare + 4);
    uint32_t *poison = reinterpret_cast<uint32_t *>(spare + 16);             // [2 groups][2][4]
    long long *part = reinterpret_cast<long long *>(spare + 128);            // [10]
    Share *found = reinterpret_cast<Share *>(spare + 256);
    float2 *other = reinterpret_cast<float2 *>(spare + 512);                 // [128]: the second group's statistics
    static_assert(8 * (2 * stages(64) + 17) <= 512 && 512 + 512 + 128 * 8 <= SPARE, "room behind the ring");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == MMA_WARP)
        tmem_alloc<512>(smem_addr(tmem_at));
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int g = 0; g < 2; ++g) {
            bar_init(q_full(g), 1);
            bar_init(q_empty(g), 1);
            bar_init(s_full(g), 1);
            bar_init(p_full(g), 4);
            bar_init(o_full(g), 1);
            bar_init(v_clean(2 * g), 4);
            bar_init(v_clean(2 * g + 1), 4);
        }
        bar_init(told, 4);
        bar_init(joined, 4);
        bar_init(drained, 1);
        *gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
        prefetch_map(&map_q);
        prefetch_map(&map_k);
        prefetch_map(&map_v);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_at;
    after_previous();
    if (blockIdx.x == 0 && w.a.status)  // sessions that are left untouched
        for (int b = tid; b < w.a.c.B; b += THREADS) {
            int n, t, bad;
            session(w.a.c, w.a.t_rows, w.a.T, b, n, t, bad);
            if (bad)
                raise(w.a.status, bad);
        }
    const Share share = share_of(w, part, found);
    const Watch watch{gave_up, w.a.status};
    Runs r(w, share);
    uint32_t seq = 0;  // tiles that passed through the ring before this run
    int nth = 0;       // runs before this one

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp == COPY_WARP) {
            auto tile_of = [&](const Runs &run, int i) {
                const int x = run.off + i;
                return x < run.u.far ? x : run.u.near + x - run.u.far;
            };
            const int boxes = KT / w.box, page = 1 << w.a.c.shift;
            auto load = [&](const Runs &run, const CUtensorMap *m, int i, uint32_t s) {
                const uint32_t st = s % ST;
                warp_wait(watch, empty(st), ((s / ST) & 1) ^ 1);
                if (__any_sync(0xffffffffu, *gave_up))
                    return;
                const int j0 = tile_of(run, i) * KT;
                const int j = j0 + lane * w.box;  // up to 16 boxes: one a lane
                int id = 0;
                const bool want = lane < boxes && j < run.u.hi && (j + w.box > run.u.lo || j < w.a.seen.sinks);
                if (want) {
                    id = w.a.c.table[static_cast<long long>(run.u.b) * w.a.c.cols + (j >> w.a.c.shift)];
                    if (id < 0 || id >= w.a.c.pages) {
                        raise(w.a.status, KDA_ST_BADPAGE);
                        id = w.a.c.pages;  // behind the last: zeros
                    }
                }
                const int count = __popc(__ballot_sync(0xffffffffu, want));
                if (lane == 0)
                    bar_expect(full(st), static_cast<uint32_t>(count) * w.box * D * 2);
                __syncwarp();
                if (want) {
                    const uint32_t dst = ring + st * TILE + lane * w.box * 128;
    #pragma unroll
                    for (int half = 0; half < HALVES; ++half)
                        copy_4d(dst + half * HALF, m, half * 64, j & (page - 1), run.h, id, full(st));
                }
            };
            auto load_q = [&](const Runs &run) {
                const int buf = PAIR ? 0 : nth & 1;
                warp_wait(watch, q_empty(buf), ((PAIR ? nth : nth >> 1) & 1) ^ 1);
                if (lane != 0 || *gave_up)
                    return;
                const int two = PAIR && run.u.nt > w.TT;
                bar_expect(q_full(buf), static_cast<uint32_t>(1 + two) * w.TT * w.a.G * D * 2);
                for (int i = 0; i <= two; ++i)
                    for (int half = 0; half < HALVES; ++half)
                        copy_3d(q_at + (PAIR ? i : buf) * TILE + half * HALF, &map_q, half * 64, run.h * w.a.G,
                                run.u.b * w.a.T + run.u.t0 + i * w.TT, q_full(buf));
            };
            while (r.next()) {
                const int lead = min(LEAD, r.todo);
                for (int i = 0; i < lead; ++i)
                    load(r, &map_k, i, seq + i);
                load_q(r);
                for (int i = 0; i < r.todo; ++i) {
                    const uint32_t s = seq + value_at(lead, r.todo, i);
                    load(r, &map_v, i, s);
                    if (i + LEAD < r.todo)
                        load(r, &map_k, i + LEAD, s + 1);
                }
                seq += 2 * r.todo;
                ++nth;
            }
            if (*gave_up && lane == 0) {  // copies in flight land before the CTA ends
                for (uint32_t s = seq > ST ? seq - ST : 0; s < seq; ++s)
                    bar_wait_long(watch, full(s % ST), (s / ST) & 1, true);
            }
        } else if (warp == MMA_WARP) {
        if (lane == 0) {
                constexpr uint32_t SCORES = product_desc(BF16, KT, KT, false), VALUES = product_desc(BF16, KT, D, true);
                uint32_t done[2] = {0, 0};
                auto stage_full = [&](uint32_t s) { bar_wait(watch, full(s % ST), (s / ST) & 1); };
                auto scores = [&](int g, uint32_t q, uint32_t s) {
                    const uint64_t a = tile_desc(q, 16, 1024), b = tile_desc(ring + (s % ST) * TILE, 16, 1024);
                    if (*gave_up)
                        return;
    #pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t step = (k / 4 * HALF + k % 4 * 32) >> 4;
                        mma_ss(tmem + g * KT, a + step, b + step, SCORES, k > 0);
                    }
                    mma_commit(s_full(g));
                };
                auto values = [&](int g, uint32_t s, bool add) {
                    const uint64_t b = tile_desc(ring + (s % ST) * TILE, HALF, 1024);
                    bar_wait(watch, p_full(g), done[g] & 1);
                    ++done[g];
                    fence_after();
                    if (*gave_up)
                        return;
    #pragma unroll
                    for (int k = 0; k < KT / 16; ++k)
                        mma_ts(tmem + 2 * KT + g * KT, tmem + g * KT + k * 8, b + (k * 16 * 128 >> 4), VALUES, add || k > 0);
                    mma_commit(o_full(g));
                };
                auto commit = [&](uint32_t bar) {
                    if (!*gave_up)
                        mma_commit(bar);
                };
                while (r.next()) {
                    const int lead = min(LEAD, r.todo), buf = PAIR ? 0 : nth & 1;
                    const int groups = PAIR ? (r.u.nt > w.TT ? 2 : 1) : 0;
                    const uint32_t q = q_at + (PAIR ? 0 : buf * TILE);
                    bar_wait(watch, q_full(buf), (PAIR ? nth : nth >> 1) & 1);
                    for (int i = 0; i < lead; ++i) {
                        stage_full(seq + i);
                        fence_after();
                        if (PAIR)
                            for (int g = 0; g < groups; ++g)
                                scores(g, q + g * TILE, seq + i);
                        else
                            scores(i, q, seq + i);
                        commit(empty((seq + i) % ST));
                    }
                    if (r.todo <= LEAD)
                        commit(q_empty(buf));
                    for (int i = 0; i < r.todo; ++i) {
                        const uint32_t sv = seq + value_at(lead, r.todo, i), sk = sv + 1;
                        const bool more = i + LEAD < r.todo;
                        stage_full(sv);
                        if (PAIR) {
                            for (int g = 0; g < groups; ++g) {
                                values(g, sv, i > 0);
                                if (more) {
                                    if (g == 0)
                                        stage_full(sk);
                                    scores(g, q + g * TILE, sk);
                                }
                            }
                        } else {
                            values(i & 1, sv, i > 1);
                        }
                        commit(empty(sv % ST));
                        if (more) {
                            if (!PAIR) {
                                stage_full(sk);
                                scores(i & 1, q, sk);
                            }
                            commit(empty(sk % ST));
                            if (i + LEAD == r.todo - 1)
                                commit(q_empty(buf));
                        }
                    }
                    seq += 2 * r.todo;
                    ++nth;
                }
                if (*gave_up) {  // products in flight end before the tensor memory is freed
                    mma_commit(drained);
                    bar_wait_long(watch, drained, 0, true);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(GROUP_REGS));
        const int g = warp >> 2, row = tid & 127;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);  // lane 32 (warp % 4)
        const uint32_t s_at = lanes + g * KT, o_at = lanes + 2 * KT + g * KT;
        const int rt = row / w.a.G, rg = row - rt * w.a.G;
        uint32_t done[2] = {0, 0}, cleaned = 0, joins = 0;
        while (r.next()) {
            const Unit &u = r.u;
            const int lead = min(LEAD, r.todo);
            const int t = (PAIR ? g * w.TT : 0) + rt;  // of the unit's rows
            const bool live = rt < w.TT && t < u.nt;
            const bool busy = __any_sync(0xffffffffu, live);
            const int p = u.n + u.t0 + t;
            const int p_low = w.a.seen.window ? max(0, p - w.a.seen.window + 1) : 0;
            const int tiles0 = PAIR ? r.todo : (r.todo + 1) / 2;
            const int tiles1 = PAIR ? (u.nt > w.TT ? r.todo : 0) : r.todo / 2;
            const int tiles = g == 0 ? tiles0 : tiles1;
            float m = -INFINITY, used = -INFINITY, l = 0.0f;
            bool spoiled = false;
            auto key_of = [&](int i) {
                const int y = r.off + i;
                return (y < u.far ? y : u.near + y - u.far) * KT;
            };
            // some key of the tile is hidden from some row
            auto is_edge = [&](int j0) {
                return !all_see(w, u, j0) || !all_see(w, u, j0 + KT - 1) ||
                       (w.a.seen.window && j0 < w.a.seen.sinks && j0 + KT > w.a.seen.sinks);
            };
            if (PAIR && tiles == 0)  // the first group cleans tiles without the second
                for (int i = 0; i < r.todo; ++i)
                    cleaned += is_edge(key_of(i));
            for (int x = 0; x < tiles; ++x) {
                const int i = PAIR ? x : 2 * x + g;
                const int j0 = key_of(i);
                const bool edge = is_edge(j0);
                warp_wait(watch, s_full(g), (done[g] + x) & 1);
                if (busy) {
                    fence_after();
                    uint32_t s[KT];
#pragma unroll
                    for (int k = 0; k < KT; k += 32)
                        tmem_ld32(s_at + k, s + k);
                    tmem_wait_ld();
                    if (edge) {
                        const int most = p - j0, low = p_low - j0, sinks = w.a.seen.sinks - j0;
#pragma unroll
                        for (int k = 0; k < KT; ++k)
                            if (k > most || (k < low && k >= sinks))
                                s[k] = 0xff800000u;
                    }
                    float top[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < KT; k += 2)
                        top[k / 2 & 3] = max3(top[k / 2 & 3], __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
                    m = fmaxf(max3(top[0], top[1], top[2]), top[3]);
                    if (x == 0) {
                        used = m;
                    } else if (__any_sync(0xffffffffu, (m - used) * w.c > LAG || (used == -INFINITY && m > used))) {
                        warp_wait(watch, o_full(g), (done[g] + x - 1) & 1);
                        fence_after();
                        const float f = m == used ? 1.0f : ex2((used - m) * w.c);
                        l *= f;
                        used = m;
#pragma unroll
                        for (int k = 0; k < D; k += 32) {
                            uint32_t o[32];
                            tmem_ld32(o_at + k, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(o_at + k, o);
                        }
                    }
                    const float off = used == -INFINITY ? 0.0f : used * w.c;
                    const Two cc = two(w.c, w.c), minus = two(-off, -off);
                    Two sum[2] = {two(0.0f, 0.0f), two(0.0f, 0.0f)};
#pragma unroll
                    for (int k = 0; k < KT; k += 64) {
                        uint32_t weights[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float2 z = apart(fma2(two(s[k + 2 * e], s[k + 2 * e + 1]), cc, minus));
                            const float p0 = ex2(z.x), p1 = ex2(z.y);
                            sum[e & 1] = add2(sum[e & 1], two(p0, p1));
                            weights[e] = pack<BF16>(p0, p1);
                        }
                        tmem_st32(s_at + k / 2, weights);
                    }
                    const float2 all = apart(add2(sum[0], sum[1]));
                    l += all.x + all.y;
                    tmem_wait_st();
                }
                if (edge) {
                    // Values of keys that no row sees become zeros (a weight of 0 times anything is
                    // then 0); of a key that only some rows see, values that are not finite do too,
                    // and the rows that see it are marked.
                    const uint32_t place = seq + value_at(lead, r.todo, i), st = place % ST;
                    const int who = PAIR ? 0 : g;
                    uint32_t *said = poison + (who * 2 + (cleaned & 1)) * 4;
                    if (g == who) {
                        warp_wait(watch, full(st), (place / ST) & 1);
                        const int j = j0 + row;
                        unsigned char *v = raw + (ring + st * TILE - smem_addr(raw)) + row * 128;
                        bool zero = !some_see(w, u, j), bad = false;
                        if (!zero && !all_see(w, u, j)) {
                            constexpr uint32_t E = BF16 ? 0x7f807f80u : 0x7c007c00u;
                            for (int k = 0; k < D / 8; ++k) {
                                const uint4 q = *reinterpret_cast<const uint4 *>(v + (k / 8) * HALF + ((k ^ row) & 7) * 16);
                                for (uint32_t e : {q.x, q.y, q.z, q.w})
                                    bad |= (e & E & 0xffffu) == (E & 0xffffu) || (e & E) >> 16 == E >> 16;
                            }
                            zero = bad;
                        }
                        if (zero)
                            for (int k = 0; k < D / 8; ++k)
                                *reinterpret_cast<uint4 *>(v + (k / 8) * HALF + ((k ^ row) & 7) * 16) = make_uint4(0, 0, 0, 0);
                        const uint32_t mask = __ballot_sync(0xffffffffu, bad);
                        if (lane == 0)
                            said[warp & 3] = mask;
                        fence_async();
                        __syncwarp();
                        if (lane == 0)
                            bar_arrive(v_clean(2 * who + (cleaned & 1)));
                    }
                    // two barriers in turn: the first group may be a tile ahead of the second
                    warp_wait(watch, v_clean(2 * who + (cleaned & 1)), (cleaned >> 1) & 1);
                    ++cleaned;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        for (uint32_t left = said[k]; left; left &= left - 1) {
                            const int j = j0 + 32 * k + __ffs(left) - 1;
                            spoiled |= j <= p && (j >= p_low || j < w.a.seen.sinks);
                        }
                }
                fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(p_full(g));
            }
            // the result of the run
            if (tiles > 0)
                warp_wait(watch, o_full(g), (done[g] + tiles - 1) & 1);
            done[0] += tiles0;
            done[1] += tiles1;
            fence_after();
            const bool join = !PAIR && tiles1 > 0;
            float f0 = 1.0f, f1 = 0.0f;
            if (join && g == 1) {
                other[row] = make_float2(used, spoiled ? -1.0f : l);
                fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(told);
            }
            if (join && g == 0) {
                warp_wait(watch, told, joins & 1);
                ++joins;
                fence_after();
                const float2 o = other[row];
                spoiled |= o.y < 0.0f;
                const float l1 = o.y < 0.0f ? 0.0f : o.y, both = fmaxf(used, o.x);
                if (both != -INFINITY) {
                    f0 = used == both ? 1.0f : ex2((used - both) * w.c);
                    f1 = o.x == both ? 1.0f : ex2((o.x - both) * w.c);
                }
                used = both;
                l = l * f0 + l1 * f1;
            }
            if (busy && (PAIR ? tiles > 0 : g == 0) && !__any_sync(0xffffffffu, *gave_up)) {
                const int hq = r.h * w.a.G + rg;
                const long long to = (static_cast<long long>(u.b) * w.a.T + u.t0 + t) * w.a.Hq + hq;
                const long long slot = static_cast<long long>(r.slot) * (PAIR ? 2 * KT : KT) + (PAIR ? g * KT : 0) + row;
                const float inv = r.whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
                f0 *= inv;
                f1 *= inv;
#pragma unroll
                for (int k = 0; k < D; k += 32) {
                    uint32_t o[32];
                    tmem_ld32(o_at + k, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
                    if (join) {
                        uint32_t o1[32];
                        tmem_ld32(o_at + KT + k, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
                    }
                    if (spoiled)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = 0x7fc00000u;
                    if (live && r.whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(w.a.out + to * D + k);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t x[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                x[z] = pack<BF16>(__uint_as_float(o[8 * e + 2 * z]), __uint_as_float(o[8 * e + 2 * z + 1]));
                            dst[e] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else if (live) {
                        uint4 *dst = reinterpret_cast<uint4 *>(w.parts + slot * D + k);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                    __syncwarp();
                }
                if (live && r.whole && w.a.lse)
                    w.a.lse[to] = l == 0.0f ? -INFINITY : (used * w.c + log2f(l)) * LN2;
                if (live && !r.whole)
                    w.stats[slot] = make_float2(used, l);
            }
            if (join) {  // the second group's sums and statistics have been read
                fence_before();
                __syncwarp();
                if (g == 0) {
                    if (lane == 0)
                        bar_arrive(joined);
                } else {
                    warp_wait(watch, joined, joins & 1);
                    ++joins;
                    fence_after();
                }
            }
            seq += 2 * r.todo;
            ++nth;
        }
    }
    fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        __syncwarp();
        tmem_free<512>(tmem);
    }
}

// The second launch: a warp a row and head joins the parts of a unit that was cut.
constexpr int JOIN_T = 256;

template <int D, bool BF16>
__global__ void __launch_bounds__(JOIN_T) attend_join_kernel(const __grid_constant__ Walk w, int rows_a_part)
{
    after_previous();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long items = static_cast<long long>(w.a.c.B) * w.a.T * w.a.Hq;
    const long long P = static_cast<long long>(w.a.c.B) * w.nq, per = w.plan[P];
    for (long long i = static_cast<long long>(blockIdx.x) * (JOIN_T / 32) + (threadIdx.x >> 5); i < items;
         i += static_cast<long long>(gridDim.x) * (JOIN_T / 32)) {
        const long long bt = i / w.a.Hq;
        const int hq = static_cast<int>(i - bt * w.a.Hq), b = static_cast<int>(bt / w.a.T);
        const int t = static_cast<int>(bt - static_cast<long long>(b) * w.a.T), h = hq / w.a.G;
        const int pair = b * w.nq + t / w.TQ;
        const Unit u = unit_of(w, pair);
        if (t - u.t0 >= u.nt)
            continue;
        const long long from = w.plan[pair] + static_cast<long long>(h) * u.count;
        const long long c0 = from / per, c1 = (from + u.count - 1) / per;
        if (c0 == c1)
            continue;
        const int tl = t - u.t0, row = tl / w.TT * KT + tl % w.TT * w.a.G + hq - h * w.a.G;
        auto slot = [&](long long c) { return (2 * c + (from > c * per ? 1 : 0)) * rows_a_part + row; };
        float top = -INFINITY;
        for (long long c = c0 + lane; c <= c1; c += 32)
            top = fmaxf(top, w.stats[slot(c)].x);
#pragma unroll
        for (int d = 16; d; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        float o[E] = {}, l = 0.0f;
        for (long long c = c0; c <= c1; ++c) {
            const float2 s = w.stats[slot(c)];
            const float f = s.x == top ? 1.0f : ex2((s.x - top) * w.c);
            const float *x = w.parts + slot(c) * D + lane * E;
            l += s.y * f;
            if (E == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(x);
                o[0] += v.x * f;
                o[1] += v.y * f;
                o[2 % E] += v.z * f;
                o[3 % E] += v.w * f;
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(x);
                o[0] += v.x * f;
                o[1] += v.y * f;
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint32_t *dst = reinterpret_cast<uint32_t *>(w.a.out + i * D + lane * E);
        dst[0] = pack<BF16>(o[0] * inv, o[1] * inv);
        if (E == 4)
            dst[1] = pack<BF16>(o[2 % E] * inv, o[3 % E] * inv);
        if (lane == 0 && w.a.lse)
            w.a.lse[i] = l == 0.0f ? -INFINITY : (top * w.c + log2f(l)) * LN2;
    }
}

// More than 128 rows of a session and kv head fill two tiles.
bool is_pair(int T, int G) { return static_cast<long long>(T) > KT / G; }

size_t plan_bytes(int B, int T, int G)
{
    const long long TQ = KT / G * (is_pair(T, G) ? 2 : 1);
    return (static_cast<size_t>(B) * ((T + TQ - 1) / TQ) * 8 + 8 + 15) / 16 * 16;
}

template <int D, bool PAIR, bool BF16>
int run(const Walk &w, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, unsigned grid,
        cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, PAIR, BF16>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, shared_bytes(D));
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string("attend_kernel shared memory: ") + cudaGetErrorString(e));
    if (int rc = launch(attend_kernel<D, PAIR, BF16>, dim3(grid), THREADS, shared_bytes(D), stream, "attend_kernel", w,
                        q, k, v))
        return rc;
    const long long items = static_cast<long long>(w.a.c.B) * w.a.T * w.a.Hq;
    const unsigned blocks = static_cast<unsigned>(std::min<long long>((items + JOIN_T / 32 - 1) / (JOIN_T / 32), 8 * SMS));
    return launch(attend_join_kernel<D, BF16>, dim3(blocks), JOIN_T, 0, stream, "attend_join_kernel", w,
                  PAIR ? 2 * KT : KT);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t spec_attend_workspace_bytes(int B, int T, int Hq, int Hkv, int D)
{
    if (B < 1 || T < 1 || Hkv < 1 || Hq < Hkv || Hq / Hkv > KDA_GROUP_MAX)
        return 16;
    const size_t rows = 2 * pages::SMS * (is_pair(T, Hq / Hkv) ? 2 * KT : KT);
    return plan_bytes(B, T, Hq / Hkv) + rows * (8 + 4 * static_cast<size_t>(D));
}

extern "C" int spec_attend(const kda_cache *cache, const void *q, int T, int Hq, long long ld_q, const int *t_rows,
                           int window, int sinks, float scale, void *out, float *lse, int *dev_status, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream)
{
    Walk w{};
    Attend &a = w.a;
    if (int rc = pages::check_attend(cache, q, T, Hq, ld_q, t_rows, window, sinks, scale, dev_status, &a))
        return rc;
    if (!pages::aligned4(lse))
        return fail(KDA_EINVAL, "4-byte arrays must be 4-byte aligned");
    if (a.c.B == 0 || T == 0)
        return ok();
    if (!out || !aligned16(out))
        return fail(KDA_EINVAL, "out must not be NULL and must be 16-byte aligned");
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < spec_attend_workspace_bytes(a.c.B, T, Hq, a.c.Hkv, a.c.D))
        return fail(KDA_EINVAL, "workspace must hold spec_attend_workspace_bytes(...) bytes, 16-byte aligned");
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    const bool bf16 = cache->dtype == KDA_BF16, pair = is_pair(T, a.G);
    const int D = a.c.D, page = cache->page;
    w.TT = KT / a.G;
    w.TQ = w.TT * (pair ? 2 : 1);
    w.nq = (T + w.TQ - 1) / w.TQ;
    w.box = std::min(page, KT);
    w.c = scale * pages::LOG2E;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    w.plan = reinterpret_cast<long long *>(ws);
    ws += plan_bytes(a.c.B, T, a.G);
    w.stats = reinterpret_cast<float2 *>(ws);
    w.parts = reinterpret_cast<float *>(ws + sizeof(float2) * 2 * pages::SMS * (pair ? 2 * KT : KT));

    CUtensorMap map_q, map_k, map_v;
    const cuuint64_t kv_dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(page),
                                   static_cast<cuuint64_t>(a.c.Hkv), static_cast<cuuint64_t>(a.c.pages)};
    const cuuint64_t kv_strides[3] = {static_cast<cuuint64_t>(a.c.slot_stride) * 2,
                                      static_cast<cuuint64_t>(a.c.head_stride) * 2,
                                      static_cast<cuuint64_t>(a.c.page_stride) * 2};
    const cuuint32_t kv_box[4] = {64, static_cast<cuuint32_t>(w.box), 1, 1};
    const cuuint64_t q_dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq),
                                  static_cast<cuuint64_t>(a.c.B) * T};
    const cuuint64_t q_strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(ld_q) * 2};
    const cuuint32_t q_box[3] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(w.TT)};
    if (int rc = tiles::encode_map(&map_k, bf16, 4, a.c.k, kv_dims, kv_strides, kv_box))
        return rc;
    if (int rc = tiles::encode_map(&map_v, bf16, 4, a.c.v, kv_dims, kv_strides, kv_box))
        return rc;
    if (int rc = tiles::encode_map(&map_q, bf16, 3, q, q_dims, q_strides, q_box))
        return rc;
    // as many CTAs as there can be tiles, one an SM at most
    const long long most = static_cast<long long>(a.c.B) * w.nq * a.c.Hkv * ((a.c.capacity() + KT - 1) / KT);
    const unsigned grid = static_cast<unsigned>(std::min<long long>(most, pages::SMS));
    auto go = [&](auto d, auto two) {
        return bf16 ? run<decltype(d)::value, decltype(two)::value, true>(w, map_q, map_k, map_v, grid, stream)
                    : run<decltype(d)::value, decltype(two)::value, false>(w, map_q, map_k, map_v, grid, stream);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (D == 128)
        return pair ? go(D128{}, std::true_type{}) : go(D128{}, std::false_type{});
    return pair ? go(D64{}, std::true_type{}) : go(D64{}, std::false_type{});
}
