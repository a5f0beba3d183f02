"""spec_cache_append and spec_cache_evict, and verify rounds that use the cache's operators
together, against plain forms."""
import math

import pytest
import torch

from cache_ref import Case, kept_of, near
from libs import ensure_built

from speculative_decode_verify_kda_gb300 import binding as kb

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def bits(x):
    return x.contiguous().view(torch.int16)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "paired"])
@pytest.mark.parametrize("T,Hkv,D,page,dtype", [(1, 1, 64, 8, BF16), (3, 2, 128, 16, F16), (15, 8, 128, 64, BF16),
                                                (70, 3, 64, 32, F16), (300, 1, 128, 128, BF16)])
def test_append(T, Hkv, D, page, dtype, layout):
    t = [T, 0, (T + 1) // 2]
    c = Case([0, 40, 61], T=T, Hq=Hkv, Hkv=Hkv, D=D, page=page, dtype=dtype, t_rows=t, layout=layout, fused=T < 100,
             seed=T)
    want = [c.k.clone(), c.v.clone()]
    for b in range(3):  # what was there goes, the rows' places are marked
        for j in range(c.n[b], c.n[b] + t[b]):
            at = (c.table[b, j // page], slice(None), j % page)
            for x, w, rows in zip((c.k, c.v), want, (c.k_rows, c.v_rows)):
                w[at] = rows[b, j - c.n[b]]
                x[at] = 9.0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = c.cache()
    assert kb.spec_cache_append(cache, c.k_rows, c.v_rows, t_rows=c.t_rows, dev_status=status) is cache
    assert torch.equal(bits(c.k), bits(want[0])) and torch.equal(bits(c.v), bits(want[1]))
    assert int(status) == 0


def test_append_leaves_bad_sessions_and_pages_alone():
    c = Case([20, 20, 20, 20, 20, 20], T=4, Hq=2, Hkv=2, t_rows=[4] * 6, seed=1)
    c.lens[1], c.lens[2] = -3, c.cache().capacity - 3
    c.t_rows[3], c.t_rows[4] = 5, -1
    c.table[5, 1] = 2**31 - 1
    k, v = c.k.clone(), c.v.clone()
    for t in range(4):
        k[c.table[0, 1], :, 4 + t], v[c.table[0, 1], :, 4 + t] = c.k_rows[0, t], c.v_rows[0, t]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kb.spec_cache_append(c.cache(), c.k_rows, c.v_rows, t_rows=c.t_rows, dev_status=status)
    assert torch.equal(bits(c.k), bits(k)) and torch.equal(bits(c.v), bits(v))
    assert int(status) == kb.ST_BADKEEP | kb.ST_BADLEN | kb.ST_BADPAGE


def test_append_pages_past_32_bits():
    c = Case([14], T=4, Hq=2, Hkv=2, page=16, spare=1, seed=4)
    k, v = c.k.clone(), c.v.clone()
    c.spread(2**31 + 1024)
    for j in range(14, 18):
        for x in (c.k, c.v):
            x[c.table[0, j // 16], :, j % 16] = 9.0
    kb.spec_cache_append(c.cache(), c.k_rows, c.v_rows)
    assert torch.equal(bits(c.k), bits(k)) and torch.equal(bits(c.v), bits(v))


class Evict:
    """A cache of B sessions full of numbers, masses, and what an eviction has to leave."""

    def __init__(self, lens, Hkv=2, D=64, page=16, dtype=BF16, layout="hnd", seed=0, cols=None, kind="rand"):
        g = torch.Generator().manual_seed(seed)
        self.n, self.page, B = list(lens), page, len(lens)
        cols = -(-max(max(lens), 1) // page) if cols is None else cols
        pages = 2 * B * cols + 2
        both = torch.randn((2, pages, Hkv, page, D), generator=g).to(dtype).cuda()
        if layout == "nhd":
            both = both.transpose(2, 3).contiguous().transpose(2, 3)
        self.k, self.v = both[0], both[1]
        order = torch.randperm(pages, generator=g).int()
        self.table = order[:B * cols].view(B, cols).cuda()
        self.other = order[B * cols:2 * B * cols].view(B, cols).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        shape = (B, Hkv, cols * page)
        self.mass = {"rand": torch.rand(shape, generator=g).pow(8), "equal": torch.ones(shape),
                     "few": torch.randint(0, 3, shape, generator=g).float(),
                     "signed": torch.randn(shape, generator=g).mul(1e3).round().div(64),
                     "tiny": torch.randint(-3, 4, shape, generator=g).float() * 1e-45}[kind].cuda()
        self.cache = kb.PagedCache(self.k, self.v, self.table, self.lens)

    def rows(self, x, table, b, h, at):
        at = torch.tensor(at, dtype=torch.long, device="cuda")
        return x[table[b].long()[at // self.page], h, at % self.page]

    def check(self, budget, recent, sinks, in_place):
        mass, lens = self.mass.cpu(), list(self.n)
        k, v = self.k.clone(), self.v.clone()
        to = self.table if in_place else self.other[:, :-(-budget // self.page)].contiguous()
        want = [[kept_of(mass[b, h].tolist(), n, budget, recent, sinks) for h in range(mass.shape[1])]
                for b, n in enumerate(lens)]
        for b in range(len(lens)):
            for h, at in enumerate(want[b]):
                place = torch.arange(len(at), device="cuda")
                for x, old in ((k, self.k), (v, self.v)):
                    x[to[b].long()[place // self.page], h, place % self.page] = self.rows(old, self.table, b, h, at)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        more = {"mass_out": self.mass, "lens_out": self.lens} if in_place else {"dst_table": to}
        kept, mass_out, lens_out = kb.spec_cache_evict(self.cache, self.mass, budget, recent, sinks,
                                                       dev_status=status, **more)
        assert lens_out.tolist() == [min(n, budget) for n in lens]
        for b in range(len(lens)):
            for h, at in enumerate(want[b]):
                assert kept[b, h].tolist() == at + [-1] * (budget - len(at)), (b, h)
                assert torch.equal(mass_out[b, h, :len(at)].cpu().view(torch.int32),
                                   mass[b, h][torch.tensor(at, dtype=torch.long)].view(torch.int32))
        assert torch.equal(bits(self.k), bits(k)) and torch.equal(bits(self.v), bits(v))
        assert int(status) == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["rand", "equal", "few", "signed", "tiny"])
@pytest.mark.parametrize("budget,recent,sinks", [(1, 0, 0), (40, 8, 4), (100, 0, 0), (64, 60, 4), (64, 64, 0),
                                                 (200, 30, 1)])
def test_evict(budget, recent, sinks, kind, in_place):
    Evict([0, 1, budget, budget + 1, 333, 150], kind=kind, seed=budget, cols=22).check(budget, recent, sinks, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("Hkv,D,page,dtype,layout", [(1, 128, 8, F16, "nhd"), (8, 128, 64, BF16, "hnd"),
                                                     (3, 64, 128, F16, "nhd")])
def test_evict_layouts(Hkv, D, page, dtype, layout, in_place):
    Evict([700, 129, 50], Hkv, D, page, dtype, layout, seed=D).check(128, 32, 4, in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,budget", [(1023, 512), (1025, 1024), (5000, 1111), (20011, 3001), (70001, 9000)])
def test_evict_long(n, budget, in_place):
    Evict([n, n // 2], Hkv=1, seed=n, page=32).check(budget, 100, 4, in_place)


def test_evict_more_tokens_than_a_cluster_holds():
    Evict([400001], Hkv=1, seed=8, page=1024).check(3000, 100, 4, False)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_many_long_sessions(in_place):
    """More heads than clusters of eight have room for, more tokens than a block holds in registers."""
    Evict([9000 - 37 * b for b in range(40)], Hkv=1, page=64, seed=3).check(700, 20, 4, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_pages_past_32_bits(in_place):
    e = Evict([40], seed=6)
    stride, block = 2**31 + 512, e.k[0].numel()
    far = torch.empty(stride * (e.k.shape[0] - 1) + 2 * block, dtype=BF16, device="cuda")
    k, v = (far.as_strided(e.k.shape, (stride, *e.k.stride()[1:]), i * block).copy_(x)
            for i, x in enumerate((e.k, e.v)))
    e.k, e.v, e.cache = k, v, kb.PagedCache(k, v, e.table, e.lens)
    e.check(20, 4, 2, in_place)


def test_evict_orders_nan_zero_and_infinity():
    e = Evict([12, 12], Hkv=1, page=8)
    e.mass[0, 0, :12] = torch.tensor([math.nan, -0.0, 0.0, -math.inf, 3.0, math.inf, -0.0, math.nan, 0.0, -1.0, 2.0,
                                      -math.nan])
    e.mass[1, 0, :12] = math.nan
    kept, _, _ = kb.spec_cache_evict(e.cache, e.mass, 6, dst_table=e.other)
    assert kept[0, 0].tolist() == [1, 2, 4, 5, 6, 10]
    assert kept[1, 0].tolist() == [0, 1, 2, 3, 4, 5]
    kept, _, _ = kb.spec_cache_evict(e.cache, e.mass, 10, dst_table=e.other)
    assert kept[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 8, 9, 10]


def test_evict_leaves_bad_sessions_and_pages_alone():
    e = Evict([60, 60, 60, 60], Hkv=2, page=16)
    e.lens[1], e.lens[2] = -1, e.cache.capacity + 1
    to = e.other[:, :2].contiguous()
    to[3, 1] = 2**31 - 1
    k, v, lens = e.k.clone(), e.v.clone(), e.lens.clone()
    lens_out = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, _, _ = kb.spec_cache_evict(e.cache, e.mass, 30, 5, 2, dst_table=to, lens_out=lens_out, dev_status=status)
    assert lens_out.tolist() == [30, 77, 77, 30]
    assert torch.all(kept[1:3] == -1) and torch.equal(e.lens, lens)
    for b in (0, 3):
        for h in range(2):
            at = kept_of(e.mass[b, h].tolist(), 60, 30, 5, 2)
            assert kept[b, h].tolist() == at
            for i, j in enumerate(at):
                if b == 3 and i >= 16:
                    continue
                for x, old in ((k, e.k), (v, e.v)):
                    x[to[b, i // 16], h, i % 16] = old[e.table[b, j // 16], h, j % 16]
    assert torch.equal(bits(e.k), bits(k)) and torch.equal(bits(e.v), bits(v))
    assert int(status) == kb.ST_BADLEN | kb.ST_BADPAGE


def test_evict_captured_and_replayed():
    """In place, twice: the second replay finds the first one's lengths and masses."""
    e = Evict([300, 90], Hkv=2, seed=5)
    side = torch.cuda.Stream()
    plan = kb.CacheEvictPlan(e.cache, e.mass, 100, 10, 2, mass_out=e.mass, lens_out=e.lens, stream=side)
    start = [x.clone() for x in (e.k, e.v, e.mass, e.lens)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan()
    graph.replay()
    torch.cuda.synchronize()
    first = [x.clone() for x in (e.k, e.v, e.mass, e.lens)]
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(first, (e.k, e.v, e.mass, e.lens)):
        assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))
    for x, y in zip((e.k, e.v, e.mass, e.lens), start):
        x.copy_(y)
    e.check(100, 10, 2, True)


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
def test_rounds_together(window, sinks):
    """Verify rounds of a session batch as a serving loop runs them: append, attend, accept, the
    accepted rows' mass, commit, and an eviction when the caches are full.  A plain copy of every
    head's tokens in 64 bits goes through the same rounds."""
    B, T, Hq, Hkv, D, page, V, budget = 3, 5, 8, 2, 64, 16, 97, 48
    g = torch.Generator().manual_seed(1)
    cols = 5
    pages = B * cols
    k = torch.full((pages, Hkv, page, D), math.nan, dtype=BF16, device="cuda")
    v = k.clone()
    table = torch.randperm(pages, generator=g).int().view(B, cols).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = kb.PagedCache(k, v, table, lens)
    mass = torch.zeros((B, Hkv, cache.capacity), device="cuda")
    text = [[[] for _ in range(Hkv)] for _ in range(B)]  # a head's tokens: [k, v, mass]
    see = {"window": window, "sinks": sinks}
    for turn in range(25):
        normal = lambda *s: torch.randn(s, generator=g).to(BF16)  # noqa: E731
        q, kn, vn = normal(B, T, Hq, D) * 2, normal(B, T, Hkv, D), normal(B, T, Hkv, D)
        logits = torch.randn((B, T, V), generator=g)
        drafts = logits.argmax(-1)[:, :-1].int()
        miss = torch.randint(0, T, (B,), generator=g)
        for b in range(B):
            if miss[b] < T - 1:
                drafts[b, miss[b]] = (drafts[b, miss[b]] + 1) % V
        kb.spec_cache_append(cache, kn.cuda(), vn.cuda(), dev_status=status)
        out, lse = kb.spec_attend(cache, q.cuda(), dev_status=status, **see)
        _, _, keep = kb.spec_accept(logits.cuda(), drafts.cuda(), dev_status=status)
        kb.spec_attend_mass(cache, q.cuda(), lse, mass, t_rows=keep, dev_status=status, **see)
        assert keep.tolist() == [int(m) + 1 for m in miss]
        # the plain copy
        out, lse = out.cpu(), lse.cpu()
        for b in range(B):
            for h in range(Hkv):
                mine = text[b][h]
                n = len(mine)
                ks = torch.stack([x[0] for x in mine] + list(kn[b, :, h].double()))
                vs = torch.stack([x[1] for x in mine] + list(vn[b, :, h].double()))
                share = torch.zeros(n + T, dtype=torch.float64)
                for t in range(T):
                    p = n + t
                    seen = torch.tensor([j <= p and (not window or p - j < window or j < sinks)
                                         for j in range(n + T)])
                    for i in range(Hq // Hkv):
                        hq = h * (Hq // Hkv) + i
                        s = (ks @ q[b, t, hq].double() / D**0.5).masked_fill(~seen, -math.inf)
                        w = torch.softmax(s, 0)
                        want, size = w @ vs, w @ vs.abs()
                        # weights and result rounded to bf16, whose 8 significant bits put a value at most
                        # 2^-8 of itself off (half a step of 2^-7); scores of size 20 in f32
                        near(out[b, t, hq], want, 2.0**-8 * (want.abs() + size) * 1.01 + 1e-4 * size, f"{turn}")
                        assert abs(float(lse[b, t, hq]) - float(torch.logsumexp(s, 0))) < 1e-4
                        if t <= miss[b]:
                            share += w
                for j, x in enumerate(mine):
                    x[2] += float(share[j])
                for t in range(int(miss[b]) + 1):
                    mine.append([kn[b, t, h].double(), vn[b, t, h].double(), float(share[n + t])])
        lens += keep
        for b in range(B):
            got = mass[b, :, :int(lens[b])].cpu().double()
            near(got, torch.tensor([[x[2] for x in text[b][h]] for h in range(Hkv)]), 1e-4 + 1e-4 * got)
        if int(lens.max()) + T > cache.capacity:
            kept, _, _ = kb.spec_cache_evict(cache, mass, budget, recent=8, sinks=2, mass_out=mass, lens_out=lens,
                                             dev_status=status)
            for b in range(B):
                for h in range(Hkv):
                    at = [j for j in kept[b, h].tolist() if j >= 0]
                    values = [x[2] for x in text[b][h]]
                    if len(values) > budget:
                        # the same positions, or ones whose masses the sums' rounding cannot tell apart
                        want = kept_of(values, len(values), budget, 8, 2)
                        assert len(at) == budget
                        for x, y in zip(sorted(values[j] for j in at), sorted(values[j] for j in want)):
                            assert abs(x - y) < 1e-3
                    text[b][h] = [text[b][h][j] for j in at]
        assert int(status) == 0


@pytest.mark.parametrize("T,window", [(3, 0), (40, 100)])
def test_captured_rounds_are_the_eager_ones(T, window):
    """Append, attention, masses, the accept's lengths and an eviction in place as one graph: its replays
    leave the bits that the same calls leave one by one."""
    def state():
        c = Case([400, 37, 0], T=T, Hq=8, Hkv=2, t_rows=[T, T - 1, 0], window=window, sinks=4 if window else 0, seed=T,
                 cols=64)
        for x in (c.k, c.v):  # an eviction moves what a window has hidden too
            x.nan_to_num_(0.5)
        mass = torch.rand((3, 2, c.cache().capacity), generator=torch.Generator().manual_seed(3)).cuda()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        return c, mass, status

    def calls(c, mass, status, stream):
        kw = {"dev_status": status, "stream": stream}
        append = kb.CacheAppendPlan(c.cache(), c.k_rows, c.v_rows, t_rows=c.t_rows, **kw)
        attend = kb.AttendPlan(c.cache(), c.q, **c.see(), **kw)
        weigh = kb.AttendMassPlan(c.cache(), c.q, attend.out[1], mass, **c.see(), **kw)
        evict = kb.CacheEvictPlan(c.cache(), mass, 390, 50, 4, mass_out=mass, lens_out=c.lens, **kw)

        def step():
            append()
            attend()
            weigh()
            c.lens.add_(c.t_rows)
            evict()
        return attend, evict, step

    side = torch.cuda.Stream()
    one, two = state(), state()
    attend1, evict1, eager = calls(*one, None)
    attend2, evict2, captured = calls(*two, side)
    for plan in (attend1, attend2):
        for x in plan.out:
            x.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured()
    for _ in range(4):
        eager()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((one[0].k, one[0].v, one[1], one[0].lens, one[2], *attend1.out, evict1.out[0]),
                        (two[0].k, two[0].v, two[1], two[0].lens, two[2], *attend2.out, evict2.out[0])):
            assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))
    assert int(one[2]) == 0 and one[0].lens.tolist() == [390, 37 + 4 * (T - 1), 0]
