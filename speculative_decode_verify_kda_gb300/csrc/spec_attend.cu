// spec_attend.cu -- attention of a call's rows over a paged cache.
//
// The rows of a session that read one kv head (t rows of G query heads each) are packed into
// tiles of 128: row r of a tile is token r / G, head r % G.  A unit of work is one session, one
// kv head and one tile (or two) of rows against the key tiles of 128 that any of them sees; all
// units' key tiles in a row are cut into equal shares, one a CTA, whatever the sessions' lengths.
// A unit that lies within one share writes its result; the parts of the others go to the
// workspace with their maxima and sums and are joined by a second launch.
//
// A CTA is a pipeline: two warps copy key and value tiles page by page (tensor copies into rings of
// shared memory), one issues the products S = Q K^T and O += P V (tcgen05, sums in tensor memory),
// one cleans the values of tiles that are not seen whole, and two groups of 128 threads turn S into
// P, a thread a row: running maximum and sum, exp2, 16-bit weights back into tensor memory over S.
// With more than 128 rows (PAIR) the groups have a tile of rows each and share the key tiles; with
// fewer both have the same rows and take every other key tile, and their results are joined at the
// end.  While one group computes weights, the tensor cores work for the other.
//
// Rounded to 16 bits: the weights (as an operand of the products must be) and the results.  Weights
// are taken against a maximum that is at most 2^8 too small, their sum is of the unrounded ones.
//
// Measured on GB300 (alone in a CUDA graph): a prompt's chunk of 2048 rows of 64 heads over 16384 keys 686
// us, 1.7 PFLOP/s (87 % of the measured product rate; 745 to 768 us, 78 to 80 %, among other calls); 32 sessions of 15 rows over up to 16384 keys
// 235 us, 6.4 TB/s; one row of 32 heads over 131072 keys 88 us, 6.1 TB/s.  A round of few keys is
// bound by a chain of latencies: lengths, table, keys, scores, weights, result, join (14 us for one
// row of 64 heads over 4096 keys).  Runs are short where windows are, and then the code of their ends
// and masks is fetched anew each time: loops there are kept short rather than unrolled.
#include "attend_common.cuh"

namespace kda {
namespace {

using namespace pages;
using namespace tiles;

constexpr int KEY_WARP = 8, VALUE_WARP = 9, MMA_WARP = 10, CLEAN_WARP = 11;
constexpr int THREADS = 384;         // two groups of 128 and four warps more
// Registers are handed from the last four warps to the groups (a row of 128 scores is held in
// them): 256 x 216 + 128 x 72 = 384 x 168, what the launch has.
constexpr int GROUP_REGS = 216, OTHER_REGS = 72;
// The running maximum that weights are taken against follows the true one only when it falls
// behind by more than this many powers of two: weights stay below 2^8, and the sums in tensor
// memory are seldom rescaled.
constexpr float LAG = 8.0f;
// f16 ends at 2^-24: its weights, and with them their sum, are held 2^7 times as large, up to 2^15, and one
// is off by 2^-32 of the largest at most.  (With 2^-25, the small weights of a long text behind a strong key
// were missing from the result and not from the sum.  A lag of 4 and 2^11 took 1 % longer for a prompt's
// chunk, 3 % for a window's; this takes no time.)
template <bool BF16>
constexpr float LIFT = BF16 ? 0.0f : 7.0f;

// Barriers and what the warps tell each other.
__host__ __device__ constexpr int spare_bytes(int D) { return D == 128 ? 3072 : 3200; }

// Tiles in shared memory: two of rows for two groups' rows, else one.
__host__ __device__ constexpr int row_tiles(bool pair) { return pair ? 2 : 1; }
__host__ __device__ constexpr int key_stages(int D, bool pair) { return D == 128 ? (pair ? 3 : 4) : 6; }
__host__ __device__ constexpr int value_stages(int D) { return D == 128 ? 2 : 4; }
__host__ __device__ constexpr int shared_bytes(int D, bool pair)
{
    return (row_tiles(pair) + key_stages(D, pair) + value_stages(D)) * tile_bytes(D) + spare_bytes(D);
}

// Keys of a run that only some rows see and whose values are not finite: bit j - (n + t0) of the
// first half for the call's own, bit j - lo of the second for those at the window's end.
struct Poison {
    uint32_t any, bits[16];
};
// Runs whose poison is held.  The cleaning of run c clears its place when tile c - 1 has a stage, that is
// when the products of a tile VS before it are through; in runs of one tile the group of the tile
// before that one may still be at its results: run c - 2 - VS.
__host__ __device__ constexpr int held_runs(int D) { return value_stages(D) + 3; }

struct Walk : Span {
    bool wide;               // out is 32-byte aligned
    struct Cut *cuts;        // [grid] the unit that is cut at a CTA's end
    float2 *stats;           // [2 grid][rows] maximum and sum of a part
    float *parts;            // [2 grid][rows][D] its sums
};

// A unit that begins as the last of CTA c's and goes on in the CTAs behind: its n parts lie in
// `slot`, 2 (c + 1), 2 (c + 2), ...  n = 0: none.
struct Cut {
    int n, slot, b, t0, nt, h, pad[2];
};

// The largest of 64 scores, in four strands.
__device__ __forceinline__ void highest(float (&top)[4], const uint32_t *s)
{
#pragma unroll
    for (int k = 0; k < 64; k += 2)
        top[k / 2 & 3] = max3(top[k / 2 & 3], __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
}

constexpr int RUNS = 16;  // records of the walk that are held
constexpr int BARS = 448; // bytes of barriers
// Record n is written when tile n - 1 has a stage: the products are at run n - 1 - KS at least, the
// slower group, in runs of one tile, at the results of the second before it.
static_assert(RUNS > 6 + 3, "a record is read before its place is taken");

// Where a CTA's share of the tiles begins.
struct Share {
    Unit u;
    int left, per;  // tiles of this share (0: none), of a full one
    int pair, h, off;
};

// The unit to look at behind unit i: a session's first one without rows is followed by others without,
// thousands where a session decodes beside another's prompt.
__device__ __forceinline__ int after(const Walk &w, const Unit &u, int i) { return u.count > 0 ? i + 1 : (u.b + 1) * w.nq; }

// The runs of one unit's tiles after another within a share.
struct alignas(8) Runs {
    Unit u;
    int left;            // tiles from this run on
    int pair, slot;
    int h, off, todo;    // tiles off .. off + todo - 1 of the unit
    bool whole;          // all of them; else the parts go to `slot` of the workspace
    __device__ explicit Runs(const Share &s)
        : u(s.u), left(s.left), pair(s.pair), slot(2 * blockIdx.x), h(s.h), off(s.off), todo(0), whole(false)
    {
    }
    __device__ __forceinline__ bool next(const Walk &w)
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
            do {
                pair = after(w, u, pair);
                u = unit_of(w, pair);
            } while (u.count == 0);
        }
        todo = min(u.count - off, left);
        whole = todo == u.count;
        return true;
    }
};

// Every CTA finds its share of the tiles of all units in the order (session, unit, kv head).
// `part`: a word a warp.
__device__ __forceinline__ void share_of(const Walk &w, int *part, Share *found)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = w.a.c.B * w.nq, each = (P - 1) / THREADS + 1;
    const int i0 = tid * each, i1 = min(P, i0 + each);
    Unit u;
    int mine = 0;
    for (int i = i0; i < i1; i = after(w, u, i)) {
        u = unit_of(w, i);
        mine += u.count * w.a.c.Hkv;
    }
    int s = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d)
            s += y;
    }
    if (lane == 31)
        part[warp] = s;
    if (tid == 0)
        found->left = 0;
    __syncthreads();
    int before = s - mine, total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i == warp)
            before += total;
        total += part[i];
    }
    const int per = (total + gridDim.x - 1) / gridDim.x;
    const int first = per * blockIdx.x, last = min(total, first + per);
    if (first < last && before <= first && first < before + mine) {
        int i = i1 - 1;
        if (each > 1)
            for (i = i0;; i = after(w, u, i)) {
                u = unit_of(w, i);
                if (first < before + u.count * w.a.c.Hkv)
                    break;
                before += u.count * w.a.c.Hkv;
            }
        const int h = (first - before) / u.count;
        *found = Share{u, last - first, per, i, h, first - before - h * u.count};
    }
    __syncthreads();
}

// A CTA that gave up: the rows that it had a part in become NaN, here and, where parts are joined, by its
// parts' statistics.  (By the groups' threads, which have the registers.)
template <int D, bool PAIR>
__device__ __noinline__ void spoil(const Walk &w, const Share &found)
{
    constexpr int ROWS = PAIR ? 2 * KT : KT, GROUPS = 256;
    const float nan = __int_as_float(0x7fffffff);
    for (int i = threadIdx.x; i < 2 * ROWS; i += GROUPS)
        w.stats[2 * blockIdx.x * ROWS + i] = make_float2(nan, nan);
    const int G = w.a.G, words = G * D / 2;
    for (Runs r(found); r.next(w);) {
        const long long row = (static_cast<long long>(r.u.b) * w.a.T + r.u.t0) * w.a.Hq + r.h * G;
        for (int i = threadIdx.x; i < r.u.nt * words; i += GROUPS)
            reinterpret_cast<uint32_t *>(w.a.out + (row + static_cast<long long>(i / words) * w.a.Hq) * D)[i % words] = 0x7fff7fffu;
        for (int i = threadIdx.x; w.a.lse && i < r.u.nt * G; i += GROUPS)
            w.a.lse[row + static_cast<long long>(i / G) * w.a.Hq + i % G] = nan;
    }
}

template <int D, bool PAIR, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) attend_kernel(const __grid_constant__ Walk w,
                                                            const __grid_constant__ CUtensorMap map_q,
                                                            const __grid_constant__ CUtensorMap map_k,
                                                            const __grid_constant__ CUtensorMap map_v)
{
    constexpr int TILE = tile_bytes(D), HALF = KT * 128, HALVES = D / 64, KS = key_stages(D, PAIR), VS = value_stages(D), ST = KS + VS;
    constexpr int LEAD = PAIR ? 1 : 2;  // key tiles ahead of value tiles
    extern __shared__ __align__(1024) unsigned char raw[];
    const uint32_t base = smem_addr(raw);
    const uint32_t q_at = base, ring = base + row_tiles(PAIR) * TILE, ring_v = ring + KS * TILE, bars = ring + ST * TILE;
    // barriers
    auto full = [&](int s) { return bars + 8u * s; };  // key stages, then value stages
    auto empty = [&](int s) { return bars + 8u * (ST + s); };
    auto more = [&](int i) { return bars + 8u * (2 * ST + i); };
    const uint32_t q_full = more(0), q_empty = more(1);
    auto s_full = [&](int g) { return more(4 + g); };
    auto p_half = [&](int g) { return more(6 + g); };  // the first 64 keys' weights
    auto p_full = [&](int g) { return more(8 + g); };
    auto o_full = [&](int g) { return more(10 + g); };
    const uint32_t drained = more(12), told = more(13), joined = more(14);
    auto v_clean = [&](int s) { return more(15 + s); };
    auto known = [&](int i) { return more(15 + VS + i); };  // a run of the walk
    // behind the barriers
    unsigned char *spare = raw + (bars - base) + BARS;
    volatile int *gave_up = reinterpret_cast<volatile int *>(spare);
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(spare + 4);
    int *part = reinterpret_cast<int *>(spare + 16);                         // [12]
    Share *found = reinterpret_cast<Share *>(spare + 64);
    float2 *other = reinterpret_cast<float2 *>(spare + 128);                 // [128]: the other group's statistics
    Runs *runs = reinterpret_cast<Runs *>(spare + 128 + 1024);               // [RUNS + 1]: the walk, the last the walker's
    Poison *poison = reinterpret_cast<Poison *>(runs + RUNS + 1);            // [HELD]
    constexpr int HELD = held_runs(D);
    static_assert(8 * (2 * ST + 15 + VS + RUNS) <= BARS && sizeof(Share) <= 64 && sizeof(Runs) == 64 &&
                      BARS + 128 + 1024 + (RUNS + 1) * sizeof(Runs) + HELD * sizeof(Poison) <= spare_bytes(D),
                  "room behind the ring");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == MMA_WARP)
        tmem_alloc<512>(smem_addr(tmem_at));
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int g = 0; g < 2; ++g) {
            bar_init(s_full(g), 1);
            bar_init(p_half(g), 4);
            bar_init(p_full(g), 4);
            bar_init(o_full(g), 1);
        }
        for (int s = 0; s < VS; ++s)
            bar_init(v_clean(s), 1);
        for (int i = 0; i < RUNS; ++i)
            bar_init(known(i), 1);
        bar_init(q_full, 1);
        bar_init(q_empty, 1);
        bar_init(drained, 1);
        bar_init(told, 4);
        bar_init(joined, 4);
        *gave_up = stopped();
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
    share_of(w, part, found);
    uint32_t seq = 0;   // tiles before this run
    int nth = 0;        // runs before this one
    bool dead = false;  // a wait gave up: nothing more is issued

    // The key warp walks, the others follow its records: short code, and no wait for lengths between
    // two runs (each warp's own walk took the prompt's chunk 699 us for 686, a window's 77 for 75).
    const Runs *r = runs;
    auto next_run = [&] {
        r = runs + nth % RUNS;
        return warp_wait(gave_up, known(nth % RUNS), nth / RUNS & 1) && r->todo > 0;
    };
    auto walk_on = [&] {
        Runs *walk = runs + RUNS;
        r = runs + nth % RUNS;
        if (lane == 0) {
            if (nth == 0)
                *walk = Runs(*found);
            if (!walk->next(w))
                walk->todo = 0;
        }
        __syncwarp();
        if (lane < 16)
            reinterpret_cast<int *>(runs + nth % RUNS)[lane] = reinterpret_cast<const int *>(walk)[lane];
        __syncwarp();
        if (lane == 0)
            bar_arrive(known(nth % RUNS));
        return r->todo > 0;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGS));
        if (warp == KEY_WARP || warp == VALUE_WARP) {
            const bool keys = warp == KEY_WARP;
            const CUtensorMap *m = keys ? &map_k : &map_v;
            const int first = keys ? 0 : KS, count = keys ? KS : VS;
            int stage = 0;
            uint32_t phase = 0;
            auto key_of = [&](int i) { return tile_key(r->u, r->off + i); };
            auto look = [&](int i) { return i < r->todo ? page_of(w, r->u, key_of(i)) : 0; };
            uint32_t copied = 0, asked = 0;  // tiles, and rows
            auto load_rows = [&] {
                if (!warp_wait(gave_up, q_empty, (nth & 1) ^ 1))
                    dead = true;
                const bool two = PAIR && r->u.nt > w.TT;
                asked += !dead;
                if (!dead && lane == 0) {
                    bar_expect(q_full, (two ? 2u : 1u) * w.TT * w.a.G * D * 2);
                    for (int x = 0; x <= two; ++x)
                        for (int half = 0; half < HALVES; ++half)
                            copy_3d(q_at + x * TILE + half * HALF, &map_q, half * 64, r->h * w.a.G,
                                    r->u.b * w.a.T + r->u.t0 + x * w.TT, q_full);
                }
                __syncwarp();
            };
            Cut cut{};  // what the second launch has to join
            while (!dead && (keys ? walk_on() : next_run())) {
                if (r->todo == r->left && r->off == 0 && !r->whole)
                    cut = Cut{1 + (r->u.count - r->todo - 1) / found->per + 1, r->slot, r->u.b, r->u.t0, r->u.nt, r->h, {}};
                int id = look(0);
                // the rows before the first keys, which keep the memory busy; behind them where the
                // rows of the run before may still be read
                const bool early = nth == 0;
                if (keys && early)
                    load_rows();
                for (int i = 0; i < r->todo; ++i) {
                    const int next = look(i + 1);  // on its way while this tile is copied
                    if (!warp_wait(gave_up, empty(first + stage), phase ^ 1))
                        dead = true;
                    if (!dead) {
                        copy_tile<D>(w, r->u, r->h, key_of(i), id, m, ring + (first + stage) * TILE, full(first + stage));
                        ++copied;
                    }
                    if (++stage == count) {
                        stage = 0;
                        phase ^= 1;
                    }
                    id = next;
                    if (keys && !early && i == min(LEAD, r->todo) - 1)
                        load_rows();
                }
                ++nth;
            }
            if (!keys && lane == 0)
                w.cuts[blockIdx.x] = cut;
            // copies in flight land before the CTA ends, whatever was given up
            for (uint32_t i = copied > static_cast<uint32_t>(count) ? copied - count : 0; i < copied; ++i)
                bar_wait_long(gave_up, full(first + i % count), i / count & 1, true);
            if (asked > 0)
                bar_wait_long(gave_up, q_full, (asked - 1) & 1, true);
        } else if (warp == MMA_WARP) {
            // The whole warp walks; one lane issues.  One warp for both groups: with a warp each, their
            // products ran into each other (a prompt's chunk took 1078 us for 828 then).
            constexpr uint32_t SCORES = product_desc(BF16, KT, KT, false), VALUES = product_desc(BF16, KT, D, true);
            const uint32_t acc = uniform(tmem);
            uint32_t done = 0;  // bit g: the phase of group g's weights
            Ring<KS> key;
            Ring<VS> val;
            // (the next elect() brings the lanes together again)
            auto wait = [&](uint32_t bar, uint32_t parity) {
                if (!bar_try(bar, parity) && !bar_wait_long(gave_up, bar, parity, false))
                    dead = true;
            };
            // `math` false: a group without rows, which keeps step with the other
            auto scores = [&](int g, uint32_t q, bool math) {
                const uint64_t a = tile_desc(q, 16, 1024), b = tile_desc(ring + key.stage * TILE, 16, 1024);
                if (math) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t step = (k / 4 * HALF + k % 4 * 32) >> 4;
                        mma_ss(acc + g * KT, a + step, b + step, SCORES, k > 0);
                    }
                }
                mma_commit(s_full(g));
            };
            auto values = [&](int g, int half, bool add, bool math) {
                const uint64_t b = tile_desc(ring_v + val.stage * TILE, HALF, 1024);
                if (math) {
#pragma unroll
                    for (int k = 0; k < KT / 32; ++k)
                        mma_ts(acc + 2 * KT + g * KT, acc + g * KT + (half * KT / 32 + k) * 8,
                               b + ((half * KT / 32 + k) * 16 * 128 >> 4), VALUES, add || half > 0 || k > 0);
                }
                if (half == 1)
                    mma_commit(o_full(g));
            };
            while (next_run()) {
                const int todo = uniform(r->todo), lead = PAIR ? 0 : seq & 1;
                const bool two = uniform(r->u.nt > w.TT);
                wait(q_full, nth & 1);
                for (int i = 0; i < min(LEAD, todo); ++i) {
                    wait(full(key.stage), key.phase);
                    if (elect() && !dead) {
                        scores(PAIR ? 0 : i ^ lead, q_at, true);
                        if (PAIR)
                            scores(1, q_at + TILE, two);
                        mma_commit(empty(key.stage));
                        if (i == todo - 1)
                            mma_commit(q_empty);
                    }
                    key.step();
                }
                for (int i = 0; i < todo; ++i) {
                    const bool more = i + LEAD < todo;
                    wait(v_clean(val.stage), val.phase);
#pragma unroll
                    for (int x = 0; x < (PAIR ? 2 : 1); ++x) {
                        const int g = PAIR ? x : (i & 1) ^ lead;
                        const bool math = x == 0 || two, last = x == (PAIR ? 1 : 0);
                        wait(p_half(g), done >> g & 1);
                        fence_after();
                        if (elect() && !dead)
                            values(g, 0, i >= LEAD, math);
                        // few steps between the products: as one where the keys are at hand
                        wait(p_full(g), done >> g & 1);
                        done ^= 1u << g;
                        if (PAIR && more && x == 0)
                            wait(full(key.stage), key.phase);
                        fence_after();
                        if (elect() && !dead) {
                            values(g, 1, i >= LEAD, math);
                            if (last)
                                mma_commit(empty(KS + val.stage));
                            if (PAIR && more) {
                                scores(g, q_at + g * TILE, math);
                                if (last) {
                                    mma_commit(empty(key.stage));
                                    if (i + LEAD == todo - 1)
                                        mma_commit(q_empty);
                                }
                            }
                        }
                        if (!PAIR && more) {
                            wait(full(key.stage), key.phase);
                            if (elect() && !dead) {
                                scores(g, q_at, true);
                                mma_commit(empty(key.stage));
                                if (i + LEAD == todo - 1)
                                    mma_commit(q_empty);
                            }
                        }
                    }
                    val.step();
                    if (more)
                        key.step();
                }
                seq += todo;
                ++nth;
            }
            // products in flight end before the tensor memory is freed, whatever was given up
            if (elect())
                mma_commit(drained);
            __syncwarp();
            bar_wait_long(gave_up, drained, 0, true);
        } else if (warp == CLEAN_WARP) {
            // Value tiles pass from the copies to the products through this warp.  Values of keys that
            // no row sees become zeros (a weight of 0 times anything is then 0); of a key that only
            // some rows see, values that are not finite do too, and the key is marked: the rows that
            // see it become NaN at the end.
            Ring<VS> at;
            const int line = lane >> 3, chunk = lane & 7;  // 8 lanes a row, 4 rows at a time
            while (next_run()) {
                const Unit u = r->u;
                Poison &p = poison[nth % HELD];
                if (lane < 17)
                    (lane == 0 ? p.any : p.bits[(lane - 1) & 15]) = 0;
                __syncwarp();
                for (int i = 0; i < r->todo; ++i) {
                    const int j0 = tile_key(u, r->off + i);
                    warp_wait(gave_up, full(KS + at.stage), at.phase);
                    if (is_edge(w, u, j0)) {
                        unsigned char *tile = raw + (ring_v + at.stage * TILE - base);
                        auto place = [&](int row) {
                            return reinterpret_cast<uint4 *>(tile + row * 128 + ((chunk ^ row) & 7) * 16);
                        };
                        auto hide = [&](int from, int to) {  // keys that no row sees
                            const int end = min(to - j0, KT);
#pragma unroll 2
                            for (int row = max(from - j0, 0) + line; row < end; row += 4)
#pragma unroll
                                for (int half = 0; half < HALVES; ++half)
                                    place(row)[half * HALF / 16] = make_uint4(0, 0, 0, 0);
                        };
                        auto look = [&](int from, int to) {  // keys that some rows may not see
                            const int first = max(from - j0, 0), end = min(to - j0, KT);
                            uint32_t sum[4] = {0, 0, 0, 0};  // x * 0 is NaN where x is not finite, and stays
#pragma unroll 1
                            for (int row = first + line; row < end; row += 4)
#pragma unroll
                                for (int half = 0; half < HALVES; ++half) {
                                    const uint4 x = place(row)[half * HALF / 16];
                                    sum[0] = times_zero<BF16>(x.x, sum[0]);
                                    sum[1] = times_zero<BF16>(x.y, sum[1]);
                                    sum[2] = times_zero<BF16>(x.z, sum[2]);
                                    sum[3] = times_zero<BF16>(x.w, sum[3]);
                                }
                            const bool none = !(is_nan2<BF16>(sum[0]) || is_nan2<BF16>(sum[1]) ||
                                                is_nan2<BF16>(sum[2]) || is_nan2<BF16>(sum[3]));
                            if (__all_sync(0xffffffffu, none))
                                return;
#pragma unroll 1
                            for (int row0 = first; row0 < end; row0 += 4) {  // which ones
                                const int row = row0 + line, j = j0 + row;
                                bool bad = false;
                                if (row < end)
                                    for (int half = 0; half < HALVES; ++half) {
                                        const uint4 x = place(row)[half * HALF / 16];
                                        for (uint32_t e : {x.x, x.y, x.z, x.w})
                                            bad |= is_nan2<BF16>(times_zero<BF16>(e, 0u));
                                    }
                                const uint32_t lanes = __ballot_sync(0xffffffffu, bad) >> (8 * line) & 0xffu;
                                if (lanes && some_see(w, u, j) && !all_see(w, u, j)) {
                                    for (int half = 0; half < HALVES; ++half)
                                        place(row)[half * HALF / 16] = make_uint4(0, 0, 0, 0);
                                    if (chunk == 0) {
                                        const int bit = j > u.n + u.t0 ? j - (u.n + u.t0) : 256 + j - u.lo;
                                        atomicOr(&p.bits[bit >> 5], 1u << (bit & 31));
                                        p.any = 1;
                                    }
                                }
                                __syncwarp();
                            }
                        };
#pragma unroll 1
                        for (int side = 0; side < (w.a.seen.window ? 2 : 1); ++side) {
                            hide(side ? w.a.seen.sinks : u.hi, side ? u.lo : u.hi + KT);
                            look(side ? max(u.lo, w.a.seen.sinks) : u.n + u.t0 + 1,
                                 side ? min(u.lo + u.nt, u.n + u.t0 + 1) : u.hi);
                        }
                        fence_async();
                    }
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(v_clean(at.stage));
                    at.step();
                }
                ++nth;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(GROUP_REGS));
        const int g = warp >> 2, row = tid & 127;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);  // lane 32 (warp % 4)
        const uint32_t s_at = lanes + g * KT, o_at = lanes + 2 * KT + g * KT;
        const int rt = row / w.a.G, rg = row - rt * w.a.G;
        uint32_t done = 0, joins = 0;
        while (next_run()) {
            const Unit &u = r->u;
            const int t = (PAIR ? g * w.TT : 0) + rt;  // of the unit's rows
            const bool live = rt < w.TT && t < u.nt;
            const bool busy = __any_sync(0xffffffffu, live);
            const int p = u.n + u.t0 + t;
            const int p_low = w.a.seen.window ? max(0, p - w.a.seen.window + 1) : 0;
            // tiles alternate over all runs; the group with a run's first tile leads it
            const int lead = PAIR ? 0 : seq & 1, first = PAIR ? 0 : g ^ lead;
            const int tiles = PAIR ? r->todo : (r->todo + 1 - first) / 2;
            float m = -INFINITY, used = -INFINITY, l = 0.0f;
            auto key_of = [&](int i) { return tile_key(u, r->off + i); };
            for (int x = 0; x < tiles; ++x) {
                const int i = PAIR ? x : 2 * x + first;
                const int j0 = key_of(i);
                const bool edge = is_edge(w, u, j0);
                warp_wait(gave_up, s_full(g), (done + x) & 1);
                if (busy) {
                    fence_after();
                    uint32_t s[KT];
                    float top[4] = {m, -INFINITY, -INFINITY, -INFINITY};
                    tmem_ld32(s_at, s);
                    tmem_ld32(s_at + 32, s + 32);
                    tmem_ld32(s_at + 64, s + 64);
                    tmem_ld32(s_at + 96, s + 96);
                    tmem_wait_ld();
                    if (edge) {
                        const int end = p + 1 - j0, low = p_low - j0, sinks = w.a.seen.sinks - j0;
#pragma unroll
                        for (int k = 0; k < KT; k += 32) {
                            const uint32_t seen = bits_below(end - k) & (~bits_below(low - k) | bits_below(sinks - k));
                            if (!__all_sync(0xffffffffu, seen == 0xffffffffu))
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    s[k + e] = seen >> e & 1 ? s[k + e] : 0xff800000u;
                        }
                    }
                    highest(top, s);
                    highest(top, s + 64);
                    m = fmaxf(max3(top[0], top[1], top[2]), top[3]);
                    if (x == 0) {
                        used = m;
                    } else if (__any_sync(0xffffffffu, (m - used) * w.c > LAG || (used == -INFINITY && m > used))) {
                        warp_wait(gave_up, o_full(g), (done + x - 1) & 1);
                        fence_after();
                        const float f = m == used ? 1.0f : ex2((used - m) * w.c);
                        l *= f;
                        used = m;
#pragma unroll 1
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
                    const Two cc = two(w.c, w.c), minus = two(LIFT<BF16> - off, LIFT<BF16> - off);
                    Two sum[2] = {two(0.0f, 0.0f), two(0.0f, 0.0f)};
#pragma unroll
                    for (int k = 0; k < KT; k += 32) {
                        uint32_t weights[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 z = apart(fma2(two(s[k + 2 * e], s[k + 2 * e + 1]), cc, minus));
                            const float p0 = ex2(z.x), p1 = ex2(z.y);
                            sum[e & 1] = add2(sum[e & 1], two(p0, p1));
                            weights[e] = pack<BF16>(p0, p1);
                        }
                        if (k == 64) {  // the product with the first values may begin
                            tmem_wait_st();
                            fence_before();
                            __syncwarp();
                            if (lane == 0)
                                bar_arrive(p_half(g));
                        }
                        tmem_st16(s_at + k / 2, weights);
                    }
                    const float2 all = apart(add2(sum[0], sum[1]));
                    l += all.x + all.y;
                    tmem_wait_st();
                } else if (lane == 0) {
                    bar_arrive(p_half(g));
                }
                fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(p_full(g));
            }
            // the result of the run
            if (tiles > 0)
                warp_wait(gave_up, o_full(g), (done + tiles - 1) & 1);
            done += tiles;
            fence_after();
            const bool join = !PAIR && r->todo > 1;
            float f0 = 1.0f, f1 = 0.0f;
            if (join && g != lead) {
                other[row] = make_float2(used, l);
                fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(told);
            }
            if (join && g == lead) {
                warp_wait(gave_up, told, joins & 1);
                fence_after();
                const float2 o = other[row];
                const float both = fmaxf(used, o.x);
                if (both != -INFINITY) {
                    f0 = used == both ? 1.0f : ex2((used - both) * w.c);
                    f1 = o.x == both ? 1.0f : ex2((o.x - both) * w.c);
                }
                used = both;
                l = l * f0 + o.y * f1;
            }
            bool spoiled = false;
            const Poison &bad = poison[nth % HELD];
            if (bad.any)
                for (int k = 0; k < 16; ++k)
                    for (uint32_t left = bad.bits[k]; left; left &= left - 1) {
                        const int bit = 32 * (k & 7) + __ffs(left) - 1, j = k < 8 ? u.n + u.t0 + bit : u.lo + bit;
                        spoiled |= j <= p && (j >= p_low || j < w.a.seen.sinks);
                    }
            __syncwarp();
            if (busy && (PAIR || g == lead) && !__any_sync(0xffffffffu, *gave_up)) {
                const bool whole = r->whole;
                const int hq = r->h * w.a.G + rg;
                const long long to = (static_cast<long long>(u.b) * w.a.T + u.t0 + t) * w.a.Hq + hq;
                const long long slot = static_cast<long long>(r->slot) * (PAIR ? 2 * KT : KT) + (PAIR ? g * KT : 0) + row;
                const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
                f0 *= inv;
                f1 *= inv;
#pragma unroll 1  // code that runs once a run is waited for: short (with the rescaling's loop 93 us for 86,
                for (int k = 0; k < D; k += 32) {  // a window prompt's chunk)
                    uint32_t o[32];
                    tmem_ld32(o_at + k, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
                    if (join) {
                        uint32_t o1[32];
                        tmem_ld32(o_at + (g == 0 ? KT : -KT) + k, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
                    }
                    if (spoiled)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = 0x7fc00000u;
                    if (live && whole) {
                        uint32_t x[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            x[e] = pack<BF16>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                        store8(w.a.out + to * D + k, x, w.wide);
                        store8(w.a.out + to * D + k + 16, x + 8, w.wide);
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            store8(w.parts + slot * D + k + e, o + e, true);
                    }
                    __syncwarp();
                }
                if (live && whole && w.a.lse)
                    w.a.lse[to] = l == 0.0f ? -INFINITY : (used * w.c + log2f(l) - LIFT<BF16>) * LN2;
                if (live && !whole)
                    w.stats[slot] = make_float2(used, l);
            }
            if (join) {  // the other group's sums and statistics have been read
                fence_before();
                __syncwarp();
                if (g == lead) {
                    if (lane == 0)
                        bar_arrive(joined);
                } else {
                    warp_wait(gave_up, joined, joins & 1);
                    fence_after();
                }
                ++joins;
            }
            seq += r->todo;
            ++nth;
        }
    }
    fence_before();
    __syncthreads();
    if (warp < 8 && *gave_up) {
        if (tid == 0)
            raise(w.a.status, KDA_ST_TIMEOUT);
        spoil<D, PAIR>(w, *found);
    }
    if (warp == MMA_WARP) {
        __syncwarp();
        tmem_free<512>(tmem);
    }
}

// The second launch joins the parts of the units that were cut: CTAs for each, a warp a row of its
// tiles.  It is a chain of latencies, so no warp has a second row (with two to eight a warp a round of 8
// rows of 64 heads over 32768 keys took 44 us for 38, of 16 rows over 16384 46 for 31), and its code is
// short and loads early: two parts, the usual number where units are many, are joined without the
// exchange between lanes (a window's prompt chunk 96 us for 93).
constexpr int JOIN_T = 256;

template <int D, bool BF16>
__global__ void __launch_bounds__(JOIN_T) attend_join_kernel(const __grid_constant__ Walk w, int rows_a_part)
{
    after_previous();
    constexpr int E = D / 32;
    const Cut cut = w.cuts[blockIdx.x];
    const int lane = threadIdx.x & 31, row = blockIdx.y * (JOIN_T / 32) + (threadIdx.x >> 5);
    // a row's place in the tiles: the token and the head
    const int tile = row / KT, x = row % KT, rt = x / w.a.G, t = tile * w.TT + rt, g = x - rt * w.a.G;
    if (cut.n == 0 || rt >= w.TT || t >= cut.nt)
        return;
    const float *parts = w.parts + static_cast<size_t>(row) * D + lane * E;
    const size_t far = static_cast<size_t>(rows_a_part) * D;
    auto slot_of = [&](int k) { return k == 0 ? cut.slot : 2 * (static_cast<int>(blockIdx.x) + k); };
    float top = -INFINITY, l = 0.0f, o[E] = {};
    if (cut.n == 2) {
        const float2 s0 = w.stats[slot_of(0) * rows_a_part + row], s1 = w.stats[slot_of(1) * rows_a_part + row];
        float v[2][E];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < E; e += 2)
                *reinterpret_cast<float2 *>(v[k] + e) = *reinterpret_cast<const float2 *>(parts + slot_of(k) * far + e);
        top = fmaxf(s0.x, s1.x);
        const float f0 = s0.x == top ? 1.0f : ex2((s0.x - top) * w.c), f1 = s1.x == top ? 1.0f : ex2((s1.x - top) * w.c);
        l = s0.y * f0 + s1.y * f1;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = v[0][e] * f0 + v[1][e] * f1;
    }
    for (int k0 = 0; k0 < cut.n && cut.n != 2; k0 += 32) {
        // a lane a part: its maximum and sum; then a part after another
        const float2 s = k0 + lane < cut.n ? w.stats[slot_of(k0 + lane) * rows_a_part + row] : make_float2(-INFINITY, 0.0f);
        float most = fmaxf(top, s.x);
#pragma unroll
        for (int d = 16; d; d >>= 1)
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        const float again = top == most ? 1.0f : ex2((top - most) * w.c);
        const float f = s.x == most ? 1.0f : ex2((s.x - most) * w.c);
        float sum = s.y * f;
#pragma unroll
        for (int d = 16; d; d >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l = l * again + sum;
        top = most;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] *= again;
#pragma unroll 16
        for (int k = 0; k < min(32, cut.n - k0); ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
            const float *from = parts + slot_of(k0 + k) * far;
            if constexpr (E == 4) {
                const float4 v = *reinterpret_cast<const float4 *>(from);
                o[0] += v.x * fk;
                o[1] += v.y * fk;
                o[2] += v.z * fk;
                o[3] += v.w * fk;
            } else {
                const float2 v = *reinterpret_cast<const float2 *>(from);
                o[0] += v.x * fk;
                o[1] += v.y * fk;
            }
        }
    }
    const long long to = (static_cast<long long>(cut.b) * w.a.T + cut.t0 + t) * w.a.Hq + cut.h * w.a.G + g;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t *dst = reinterpret_cast<uint32_t *>(w.a.out + to * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2)
        dst[e / 2] = pack<BF16>(o[e] * inv, o[e + 1] * inv);
    if (lane == 0 && w.a.lse)
        w.a.lse[to] = l == 0.0f ? -INFINITY : (top * w.c + log2f(l) - LIFT<BF16>) * LN2;
}

// More than 128 rows of a session and kv head fill two tiles.  As two units of one tile, which read the
// keys twice: 2048 rows over 16384 keys 810 us for 731, 16 sessions of 24 rows over 4096 107 for 77.  One
// tile as a pair with an empty second: 32 sessions of 15 rows over 16384 keys 349 us for 335.
bool is_pair(int T, int G) { return static_cast<long long>(T) > KT / G; }

template <int D, bool PAIR, bool BF16>
int run(const Walk &w, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v, unsigned grid,
        cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, PAIR, BF16>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, shared_bytes(D, PAIR));
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string("attend_kernel shared memory: ") + cudaGetErrorString(e));
    if (int rc = launch(attend_kernel<D, PAIR, BF16>, dim3(grid), THREADS, shared_bytes(D, PAIR), stream, "attend_kernel", w,
                        q, k, v))
        return rc;
    const int rows = PAIR ? 2 * KT : w.a.T * w.a.G;
    return launch(attend_join_kernel<D, BF16>, dim3(grid, (rows - 1) / (JOIN_T / 32) + 1), JOIN_T, 0, stream,
                  "attend_join_kernel", w, PAIR ? 2 * KT : KT);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" size_t spec_attend_workspace_bytes(int B, int T, int Hq, int Hkv, int D)
{
    if (B < 1 || T < 1 || Hkv < 1 || Hq < Hkv || Hq / Hkv > KDA_GROUP_MAX)
        return 16;
    const size_t rows = 2 * pages::SMS * (is_pair(T, Hq / Hkv) ? 2 * KT : KT);
    return 32 + pages::SMS * sizeof(Cut) + rows * (8 + 4 * static_cast<size_t>(D));
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
    // q itself is read by the CTAs that write a unit's rows, before they do; rows that lie otherwise are not
    const double rows = static_cast<double>(a.c.B) * T, q_at = static_cast<double>(reinterpret_cast<uintptr_t>(q)),
                 out_at = static_cast<double>(reinterpret_cast<uintptr_t>(out)), width = static_cast<double>(Hq) * a.c.D;
    if (!(q == out && static_cast<double>(ld_q) == width) && q_at < out_at + 2 * rows * width &&
        out_at < q_at + 2 * ((rows - 1) * static_cast<double>(ld_q) + width))
        return fail(KDA_EINVAL, "out must be q itself, with dense rows, or lie apart from it");
    if (!workspace || !aligned16(workspace) ||
        workspace_bytes < spec_attend_workspace_bytes(a.c.B, T, Hq, a.c.Hkv, a.c.D))
        return fail(KDA_EINVAL, "workspace must hold spec_attend_workspace_bytes(...) bytes, 16-byte aligned");
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    const bool bf16 = cache->dtype == KDA_BF16, pair = is_pair(T, a.G);
    const int D = a.c.D;
    pages::lay_out(&w, pages::KT / a.G * (pair ? 2 : 1));
    // as many CTAs as there can be tiles, one an SM at most
    const double most = static_cast<double>(a.c.B) * w.nq * a.c.Hkv * ((a.c.capacity() + KT - 1) / KT);
    if (most > KDA_TILES_MAX)
        return fail(KDA_EINVAL, "too many tiles of keys for one call");
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    ws += 31 - (reinterpret_cast<uintptr_t>(ws) + 31) % 32;  // 32-byte stores
    w.wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    w.cuts = reinterpret_cast<Cut *>(ws);
    ws += pages::SMS * sizeof(Cut);
    w.stats = reinterpret_cast<float2 *>(ws);
    w.parts = reinterpret_cast<float *>(ws + sizeof(float2) * 2 * pages::SMS * (pair ? 2 * KT : KT));

    CUtensorMap map_q, map_k, map_v;
    if (int rc = pages::cache_map(&map_k, w, a.c.k, bf16))
        return rc;
    if (int rc = pages::cache_map(&map_v, w, a.c.v, bf16))
        return rc;
    if (int rc = pages::query_map(&map_q, w, bf16))
        return rc;
    const unsigned grid = static_cast<unsigned>(std::min(most, static_cast<double>(pages::SMS)));
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
