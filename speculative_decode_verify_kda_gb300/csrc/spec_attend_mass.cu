// spec_attend_mass.cu -- what every key of a paged cache was worth to a call's rows.
//
// The products are turned round: a tile of 128 keys times a tile of up to 128 rows gives each
// key's scores against the rows in one lane of tensor memory, so a thread sums its key's weights
// exp(s - lse) by itself, in the order of the rows: no sum depends on the order of blocks, and
// nothing is joined.  All sessions' key tiles, each counted as often as there are tiles of rows,
// are cut into equal shares, one a CTA.  Two key tiles share the row tiles that pass by; each has two
// groups of 128 threads, which take its products in turn and add their sums at the end (two warps a
// scheduler left it idle for 60 % of the cycles).  A warp copies keys, a warp rows, a warp issues the
// products.  A row's -lse / scale is part of the product, as four 16-bit terms of its own against a
// column of constants: read from shared memory by every thread it bound the kernel (128 bytes a cycle,
// as do the reads of tensor memory).  Bound by the keys' bytes for a verify round's rows (61 us for 16
// sessions of 8 rows of 64 heads over up to 16384 keys, 5.6 TB/s), by exp2 and the reads of scores before
// it, which add up, for a prompt's (68 us for 1024 rows of 32 heads over 8192 keys, 1.1 PFLOP/s; the
// tensor pipe and the exponentials' are busy half the time each).
#include "attend_common.cuh"

namespace kda {
namespace {

using namespace pages;
using namespace tiles;

constexpr int KEY_WARP = 16, ROW_WARP = 17, MMA_WARP = 18;
constexpr int THREADS = 608;

// Tiles in shared memory, keys and rows.
__host__ __device__ constexpr int key_stages(int D) { return D == 128 ? 4 : 8; }
__host__ __device__ constexpr int row_stages(int D) { return D == 128 ? 2 : 4; }
constexpr int TERMS = KT * 32;  // a tile of terms: 16 elements a row
__host__ __device__ constexpr int barrier_bytes(int D) { return (8 * (2 * key_stages(D) + 2 * row_stages(D) + 13) + 31) / 32 * 32; }
__host__ __device__ constexpr int shared_bytes(int D)
{
    return (key_stages(D) + row_stages(D)) * tile_bytes(D) + (row_stages(D) + 1) * TERMS + barrier_bytes(D) + 144 + 1024;
}

// The constants that a row's four terms are multiplied by: bf16 reaches as far as f32; f16 terms
// of 11 bits each begin at 2^15, so that 2 10^9 is reached and 10^-9 kept.
template <bool BF16>
__device__ __forceinline__ float term_unit(int i)
{
    return BF16 ? 1.0f : i == 0 ? 32768.0f : i == 1 ? 32.0f : i == 2 ? 0.03125f : 3.0517578125e-5f;
}

template <bool BF16>
__device__ __forceinline__ float rounded(float x)
{
    return BF16 ? __bfloat162float(__float2bfloat16_rn(x)) : __half2float(__float2half_rn(x));
}

// x as its four terms, two to a word
template <bool BF16>
__device__ __forceinline__ uint4 terms_of(float x)
{
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] = rounded<BF16>(x / term_unit<BF16>(i));
        // what is not finite, or past the first term's reach, is that term's alone
        x = isinf(t[i]) || t[i] != t[i] ? 0.0f : x - t[i] * term_unit<BF16>(i);
    }
    return make_uint4(pack<BF16>(t[0], t[1]), pack<BF16>(t[2], t[3]), 0, 0);
}

// Descriptor of a tile of terms: blocks of 8 rows of 16 bytes, the two halves of the 16 elements side by side.
__device__ __forceinline__ uint64_t terms_desc(uint32_t addr)
{
    return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | static_cast<uint64_t>(128 >> 4) << 16 |
           static_cast<uint64_t>(256 >> 4) << 32 | 1ull << 46;
}

struct Mass : Span {
    const float *lse;
    float *mass;
    long long ld;
    float over;  // 1 / scale
};

// Where a CTA's share of the tiles begins: the tiles whose place in the order (session, kv head,
// key tile), counted in tiles of rows, lies in [first, last).
struct Share {
    Unit u;
    int h, tile, at, last;
};

// The runs of one session's and kv head's key tiles within a share.
struct Runs {
    Unit u;
    int nr;         // tiles of rows
    int h, from, to;  // key tiles
    int at, last;
    __device__ explicit Runs(const Span &w, const Share &s)
        : u(s.u), nr((s.u.nt + w.TT - 1) / w.TT), h(s.h), from(s.tile), to(s.tile), at(s.at), last(s.last)
    {
    }
    __device__ __forceinline__ bool next(const Span &w)
    {
        at += (to - from) * nr;
        if (at >= last)
            return false;
        from = to;
        if (from == u.count) {
            from = 0;
            if (++h == w.a.c.Hkv) {
                h = 0;
                do
                    u = unit_of(w, u.b + 1);
                while (u.count == 0);
                nr = (u.nt + w.TT - 1) / w.TT;
            }
        }
        to = min(u.count, from + (last - at - 1) / nr + 1);
        return true;
    }
};

// The tiles of rows that see the key tile from j0 on: first .. second.
__device__ __forceinline__ int2 rows_of(const Span &w, const Unit &u, int nr, int j0)
{
    const int low = max(0, j0 - u.n) / w.TT;
    int high = nr - 1;
    if (w.a.seen.window && j0 >= w.a.seen.sinks)
        high = min(high, max(0, j0 + KT - 1 - u.n + w.a.seen.window - 1) / w.TT);
    return make_int2(low, high);
}

// The same of one or two tiles: what passes by a pair.
__device__ __forceinline__ int2 rows_of_pair(const Span &w, const Runs &r, int i)
{
    int2 x = rows_of(w, r.u, r.nr, tile_key(r.u, i));
    if (i + 1 < r.to) {
        const int2 y = rows_of(w, r.u, r.nr, tile_key(r.u, i + 1));
        x = make_int2(min(x.x, y.x), max(x.y, y.y));
    }
    return x;
}

__device__ __forceinline__ void share_of(const Span &w, int *part, Share *found)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = w.a.c.B, each = (B - 1) / THREADS + 1;
    const int i0 = tid * each, i1 = min(B, i0 + each);
    Unit u{};
    auto weight = [&] { return u.count * ((u.nt + w.TT - 1) / w.TT) * w.a.c.Hkv; };
    int mine = 0;
    for (int i = i0; i < i1; ++i) {
        u = unit_of(w, i);
        if (u.count > 0)
            mine += weight();
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
        found->at = found->last = found->tile = found->u.nt = 0;
    __syncthreads();
    int before = s - mine, total = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i == warp)
            before += total;
        total += part[i];
    }
    const int per = (total - 1) / static_cast<int>(gridDim.x) + 1;
    const long long begin = static_cast<long long>(per) * blockIdx.x;
    if (begin < total && before <= begin && begin < before + mine) {
        const int first = static_cast<int>(begin);
        for (int i = i0;; ++i) {
            u = unit_of(w, i);
            if (u.count == 0)
                continue;
            if (first < before + weight())
                break;
            before += weight();
        }
        const int nr = (u.nt + w.TT - 1) / w.TT, head = u.count * nr;
        const int h = (first - before) / head, tile = (first - before - h * head + nr - 1) / nr;
        *found = Share{u, h, tile, before + h * head + tile * nr, min(total, first + per)};
    }
    __syncthreads();
}

// A CTA that gave up: the masses that it had to add to become NaN.
__device__ __noinline__ void spoil(const Mass &w, const Share &found)
{
    for (Runs r(w, found); r.next(w);)
        for (int i = threadIdx.x; i < (r.to - r.from) * KT; i += THREADS) {
            const int j = tile_key(r.u, r.from + i / KT) + i % KT;
            if (some_see(w, r.u, j))
                w.mass[(static_cast<long long>(r.u.b) * w.a.c.Hkv + r.h) * w.ld + j] = __int_as_float(0x7fffffff);
        }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1) attend_mass_kernel(const __grid_constant__ Mass w,
                                                                 const __grid_constant__ CUtensorMap map_q,
                                                                 const __grid_constant__ CUtensorMap map_k)
{
    constexpr int TILE = tile_bytes(D), HALF = KT * 128, KS = key_stages(D), RS = row_stages(D);
    extern __shared__ __align__(1024) unsigned char raw[];
    const uint32_t base = smem_addr(raw), keys = base, rows = base + KS * TILE, units = rows + RS * TILE, terms = units + TERMS,
                   bars = terms + RS * TERMS;
    auto k_full = [&](int s) { return bars + 8u * s; };
    auto k_empty = [&](int s) { return bars + 8u * (KS + s); };
    auto q_full = [&](int s) { return bars + 8u * (2 * KS + s); };
    auto q_empty = [&](int s) { return bars + 8u * (2 * KS + RS + s); };
    auto s_full = [&](int g, int i) { return bars + 8u * (2 * KS + 2 * RS + 2 * g + i); };
    auto s_empty = [&](int g, int i) { return bars + 8u * (2 * KS + 2 * RS + 4 + 2 * g + i); };
    const uint32_t drained = bars + 8u * (2 * KS + 2 * RS + 8);
    auto told = [&](int g) { return drained + 8u * (1 + g); };
    auto joined = [&](int g) { return drained + 8u * (3 + g); };
    constexpr int BARS = barrier_bytes(D);
    unsigned char *spare = raw + (bars - base) + BARS;
    volatile int *gave_up = reinterpret_cast<volatile int *>(spare);
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(spare + 4);
    int *part = reinterpret_cast<int *>(spare + 8);  // [19]
    Share *found = reinterpret_cast<Share *>(spare + 88);
    float *other = reinterpret_cast<float *>(spare + 144);         // [2][128]: the second groups' sums
    static_assert(sizeof(Share) <= 56 && THREADS / 32 <= 20, "room behind the rings");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (warp == MMA_WARP)
        tmem_alloc<512>(smem_addr(tmem_at));
    if (tid == 0) {
        for (int s = 0; s < KS; ++s) {
            bar_init(k_full(s), 1);
            bar_init(k_empty(s), 1);
        }
        for (int s = 0; s < RS; ++s) {
            bar_init(q_full(s), 2);
            bar_init(q_empty(s), 1);
        }
        for (int g = 0; g < 2; ++g)
            for (int i = 0; i < 2; ++i) {
                bar_init(s_full(g, i), 1);
                bar_init(s_empty(g, i), 4);
            }
        bar_init(drained, 1);
        for (int g = 0; g < 2; ++g) {
            bar_init(told(g), 4);
            bar_init(joined(g), 4);
        }
        *gave_up = stopped();
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
        prefetch_map(&map_q);
        prefetch_map(&map_k);
    }
    // the constants, and zeros behind the terms
    for (int i = tid; i < (RS + 1) * TERMS / 16; i += THREADS) {
        const bool unit = i < TERMS / 16 && (i & 8) == 0;
        reinterpret_cast<uint4 *>(raw + (units - base))[i] =
            unit ? make_uint4(pack<BF16>(term_unit<BF16>(0), term_unit<BF16>(1)),
                              pack<BF16>(term_unit<BF16>(2), term_unit<BF16>(3)), 0, 0)
                 : make_uint4(0, 0, 0, 0);
    }
    fence_async();
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
    Runs r(w, *found);
    bool dead = false;  // a wait gave up: nothing more is issued
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!warp_wait(gave_up, bar, parity))
            dead = true;
    };

    if (warp == KEY_WARP) {
        Ring<KS> to;
        uint32_t copied = 0;
        while (r.next(w)) {
            int id = page_of(w, r.u, tile_key(r.u, r.from));
            for (int i = r.from; i < r.to; ++i) {
                const int next = i + 1 < r.to ? page_of(w, r.u, tile_key(r.u, i + 1)) : 0;
                wait(k_empty(to.stage), to.phase ^ 1);
                if (!dead) {
                    copy_tile<D>(w, r.u, r.h, tile_key(r.u, i), id, &map_k, keys + to.stage * TILE, k_full(to.stage));
                    ++copied;
                }
                to.step();
                id = next;
            }
        }
        // copies in flight land before the CTA ends, whatever was given up
        for (uint32_t i = copied > KS ? copied - KS : 0; i < copied; ++i)
            bar_wait_long(gave_up, k_full(i % KS), i / KS & 1, true);
    } else if (warp == ROW_WARP) {
        Ring<RS> to;
        uint32_t copied = 0;
        const int c0 = lane * 4;  // this lane's columns of a tile of rows
        int t_of[4], g_of[4];
        for (int e = 0; e < 4; ++e) {
            t_of[e] = (c0 + e) / w.a.G;
            g_of[e] = c0 + e - t_of[e] * w.a.G;
        }
        float l[4];  // lse of this lane's rows of the next tile
        auto fetch = [&](int x) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = x * w.TT + t_of[e];
                l[e] = 0.0f;  // of a row that is not there: its products are left out
                if (t_of[e] < w.TT && t < r.u.nt)
                    l[e] = w.lse[(static_cast<long long>(r.u.b) * w.a.T + t) * w.a.Hq + r.h * w.a.G + g_of[e]];
            }
        };
        auto load = [&](int x, int next) {
            uint4 f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)  // a row without any score has lse -inf and no weight
                f[e] = terms_of<BF16>(l[e] == -INFINITY ? -INFINITY : -l[e] * w.over);
            if (next >= 0)
                fetch(next);  // on its way while this tile is copied
            wait(q_empty(to.stage), to.phase ^ 1);
            if (!dead) {
                if (lane == 0) {
                    bar_expect(q_full(to.stage), static_cast<uint32_t>(w.TT) * w.a.G * D * 2);
                    for (int half = 0; half < D / 64; ++half)
                        copy_3d(rows + to.stage * TILE + half * HALF, &map_q, half * 64, r.h * w.a.G,
                                r.u.b * w.a.T + x * w.TT, q_full(to.stage));
                }
                uint4 *t = reinterpret_cast<uint4 *>(raw + (terms + to.stage * TERMS - base)) + (c0 >> 3) * 16 + (c0 & 7);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    t[e] = f[e];
                fence_async();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(q_full(to.stage));
                ++copied;
            }
            __syncwarp();
            to.step();
        };
        while (r.next(w)) {
            if (r.nr == 1) {  // one tile of rows stays for the whole run
                fetch(0);
                load(0, -1);
                continue;
            }
            for (int i = r.from; i < r.to; i += 2) {
                const int2 x = rows_of_pair(w, r, i);
                fetch(x.x);
                for (int y = x.x; y <= x.y; ++y)
                    load(y, y < x.y ? y + 1 : -1);
            }
        }
        for (uint32_t i = copied > RS ? copied - RS : 0; i < copied; ++i)
            bar_wait_long(gave_up, q_full(i % RS), i / RS & 1, true);
    } else if (warp == MMA_WARP) {
        // The whole warp walks; one lane issues.
        const uint32_t acc = uniform(tmem);
        Ring<KS> key;
        Ring<RS> row;
        uint32_t count[2] = {0, 0};  // products of a pair's first and second tiles
        // (the next elect() brings the lanes together again)
        auto see = [&](uint32_t bar, uint32_t parity) {
            if (!bar_try(bar, parity) && !bar_wait_long(gave_up, bar, parity, false))
                dead = true;
        };
        while (r.next(w)) {
            const bool hold = uniform(r.nr) == 1;
            const int from = uniform(r.from), to = uniform(r.to);
            const int cols = uniform((min(r.u.nt, w.TT) * w.a.G + 15) & ~15);
            const uint32_t desc = product_desc(BF16, KT, 0, false) | static_cast<uint32_t>(cols >> 3) << 17;
            for (int i = from; i < to; i += 2) {
                const int2 x = rows_of_pair(w, r, i);
                const bool two = i + 1 < to;
                Ring<KS> second = key;
                second.step();
                see(k_full(key.stage), key.phase);
                if (two)
                    see(k_full(second.stage), second.phase);
                const int last = uniform(x.y);
                for (int y = uniform(x.x); y <= last; ++y) {
                    if (!hold || i == from)
                        see(q_full(row.stage), row.phase);
                    const uint64_t b = tile_desc(rows + row.stage * TILE, 16, 1024);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (g == 1 && !two)
                            continue;
                        const uint32_t buf = count[g] & 1;
                        const uint64_t a = tile_desc(keys + (g == 1 ? second.stage : key.stage) * TILE, 16, 1024);
                        see(s_empty(g, buf), (count[g] >> 1 & 1) ^ 1);
                        ++count[g];
                        fence_after();
                        if (elect() && !dead) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint64_t step = (k / 4 * HALF + k % 4 * 32) >> 4;
                                mma_ss(acc + (2 * g + buf) * KT, a + step, b + step, desc, k > 0);
                            }
                            mma_ss(acc + (2 * g + buf) * KT, terms_desc(units), terms_desc(terms + row.stage * TERMS), desc,
                                   true);
                            mma_commit(s_full(g, buf));
                            if (g == 1 || !two) {  // the last that reads these rows, these keys
                                if (!hold)
                                    mma_commit(q_empty(row.stage));
                                if (y == last) {
                                    mma_commit(k_empty(key.stage));
                                    if (two)
                                        mma_commit(k_empty(second.stage));
                                }
                            }
                        }
                    }
                    if (!hold)
                        row.step();
                }
                key.step();
                if (two)
                    key.step();
            }
            if (hold) {
                if (elect() && !dead)
                    mma_commit(q_empty(row.stage));
                row.step();
            }
        }
        // products in flight end before the tensor memory is freed, whatever was given up
        if (elect())
            mma_commit(drained);
        __syncwarp();
        bar_wait_long(gave_up, drained, 0, true);
    } else {
        const int g = warp >> 3, half = warp >> 2 & 1, line = tid & 127;
        const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21) + (2 * g + half) * KT;
        const Two cc = two(w.c, w.c), zero = two(0.0f, 0.0f);
        uint32_t count = 0, joins = 0;  // products of this tile of the pairs, and pairs with sums to add
        while (r.next(w)) {
            const int cols = min(r.u.nt, w.TT) * w.a.G;
            for (int i = r.from; i < r.to; i += 2) {
                const int2 x = rows_of_pair(w, r, i);
                const bool on = i + g < r.to;
                const int j = tile_key(r.u, on ? i + g : i) + line;
                // the rows t0 .. t1 - 1 see this key
                const int t0 = max(0, j - r.u.n);
                const int t1 = w.a.seen.window && j >= w.a.seen.sinks ? min(r.u.nt, j - r.u.n + w.a.seen.window) : r.u.nt;
                Two sum[2] = {zero, zero};
                bool mine = false;
                for (int y = x.x; y <= x.y; ++y) {
                    if (on && (count++ & 1) == static_cast<uint32_t>(half)) {
                        mine = true;
                        wait(s_full(g, half), (count - 1) >> 1 & 1);
                        fence_after();
                        // its columns of this tile of rows
                        const int a = max(0, min(w.TT, t0 - y * w.TT)) * w.a.G, b = max(0, min(w.TT, t1 - y * w.TT)) * w.a.G;
#pragma unroll 1
                        for (int k = 0; k < cols; k += 32) {
                            uint32_t s[32];
                            tmem_ld32(at + k, s);
                            tmem_wait_ld();
                            if (k + 32 >= cols) {  // the last of it: the next product may come
                                fence_before();
                                __syncwarp();
                                if (lane == 0)
                                    bar_arrive(s_empty(g, half));
                            }
                            const uint32_t seen = bits_below(b - k) & ~bits_below(a - k);
                            if (__all_sync(0xffffffffu, seen == 0xffffffffu)) {
#pragma unroll
                                for (int e = 0; e < 32; e += 4) {
                                    const float2 u = apart(mul2(two(s[e], s[e + 1]), cc));
                                    const float2 v = apart(mul2(two(s[e + 2], s[e + 3]), cc));
                                    sum[0] = add2(sum[0], two(ex2(u.x), ex2(u.y)));
                                    sum[1] = add2(sum[1], two(ex2(v.x), ex2(v.y)));
                                }
                            } else if (__any_sync(0xffffffffu, seen != 0)) {
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 u = apart(mul2(two(s[e], s[e + 1]), cc));
                                    sum[e >> 1 & 1] = add2(sum[e >> 1 & 1], two(seen >> e & 1 ? ex2(u.x) : 0.0f,
                                                                                seen >> (e + 1) & 1 ? ex2(u.y) : 0.0f));
                                }
                            }
                        }
                    }
                }
                const float2 both = apart(add2(sum[0], sum[1]));
                float all = both.x + both.y;
                if (on && x.y > x.x) {  // two products or more: both groups have some
                    if (half == 1) {
                        other[g * KT + line] = all;
                        __syncwarp();
                        if (lane == 0)
                            bar_arrive(told(g));
                        wait(joined(g), joins & 1);
                        mine = false;
                    } else {
                        wait(told(g), joins & 1);
                        all += other[g * KT + line];
                        __syncwarp();
                        if (lane == 0)
                            bar_arrive(joined(g));
                    }
                    ++joins;
                }
                if (mine && some_see(w, r.u, j) && !*gave_up) {
                    float *to = w.mass + (static_cast<long long>(r.u.b) * w.a.c.Hkv + r.h) * w.ld + j;
                    *to = (j < r.u.n ? *to : 0.0f) + all;
                }
                __syncwarp();
            }
        }
    }
    fence_before();
    __syncthreads();
    if (*gave_up) {
        if (tid == 0)
            raise(w.a.status, KDA_ST_TIMEOUT);
        spoil(w, *found);
    }
    if (warp == MMA_WARP) {
        __syncwarp();
        tmem_free<512>(tmem);
    }
}

template <int D, bool BF16>
int run(const Mass &w, const CUtensorMap &q, const CUtensorMap &k, unsigned grid, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(attend_mass_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               shared_bytes(D));
    if (e != cudaSuccess)
        return fail(KDA_ECUDA, std::string("attend_mass_kernel shared memory: ") + cudaGetErrorString(e));
    return launch(attend_mass_kernel<D, BF16>, dim3(grid), THREADS, shared_bytes(D), stream, "attend_mass_kernel", w, q,
                  k);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int spec_attend_mass(const kda_cache *cache, const void *q, int T, int Hq, long long ld_q, const float *lse,
                                const int *t_rows, int window, int sinks, float scale, float *mass, long long ld_mass,
                                int *dev_status, cudaStream_t stream)
{
    Mass w{};
    if (int rc = pages::check_attend(cache, q, T, Hq, ld_q, t_rows, window, sinks, scale, dev_status, &w.a))
        return rc;
    if (ld_mass < w.a.c.capacity() || ld_mass >= (1ll << 40))
        return fail(KDA_EINVAL, "ld_mass must be at least table_cols * page");
    if (w.a.c.B == 0 || T == 0)
        return ok();
    if (!lse || !mass || !pages::aligned4(lse) || !pages::aligned4(mass))
        return fail(KDA_EINVAL, "lse and mass must not be NULL and must be 4-byte aligned");
    w.lse = lse;
    w.mass = mass;
    w.ld = ld_mass;
    w.over = 1.0f / scale;
    pages::lay_out(&w, T);
    const double tiles = static_cast<double>(w.a.c.B) * w.a.c.Hkv * ((w.a.c.capacity() + pages::KT - 1) / pages::KT);
    if (tiles * ((T - 1) / w.TT + 1) > KDA_TILES_MAX)
        return fail(KDA_EINVAL, "too many tiles of keys and rows for one call");
    const bool bf16 = cache->dtype == KDA_BF16;
    CUtensorMap map_q, map_k;
    if (int rc = pages::cache_map(&map_k, w, w.a.c.k, bf16))
        return rc;
    if (int rc = pages::query_map(&map_q, w, bf16))
        return rc;
    const unsigned grid = static_cast<unsigned>(std::min(tiles, static_cast<double>(pages::SMS)));
    if (w.a.c.D == 128)
        return bf16 ? run<128, true>(w, map_q, map_k, grid, stream) : run<128, false>(w, map_q, map_k, grid, stream);
    return bf16 ? run<64, true>(w, map_q, map_k, grid, stream) : run<64, false>(w, map_q, map_k, grid, stream);
}
