"""spec_attend and spec_attend_mass against the formulas in 64 bits: lengths, row counts, head
groups, pages, layouts, windows and sinks; whatever no row sees holds NaN."""
import ctypes
import math
import os
import random
import subprocess

import pytest
import torch

from cache_ref import Case, near
from libs import ensure_built

from speculative_decode_verify_kda_gb300 import binding as kb
from speculative_decode_verify_kda_gb300 import build

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def run(c, **kw):
    """out and lse of a call, checked; rows behind a session's last one keep what they held."""
    out = torch.full((c.B, c.T, c.Hq, c.D), 7.0, dtype=c.dtype, device="cuda")
    lse = torch.full((c.B, c.T, c.Hq), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kb.spec_attend(c.cache(), c.q, out=out, lse_out=lse, dev_status=status, **c.see(), **kw)
    assert got[0] is out and got[1] is lse
    want, want_lse, tol, tol_lse = c.attend()
    there = near(out, want, tol, "out")
    near(lse, want_lse, tol_lse, "lse")
    assert torch.all(out.cpu()[~there] == 7.0), "rows that are not the call's were written"
    assert torch.all(lse.cpu()[torch.isnan(want_lse)] == 7.0)
    assert int(status) == 0
    return out, lse


def weigh(c, lse):
    """mass after a call, checked against its shares."""
    cap = c.cache().capacity
    g = torch.Generator().manual_seed(5)
    before = torch.rand((c.B, c.Hkv, cap + 3), generator=g)
    for b in range(c.B):
        before[b, :, c.n[b]:] = math.nan  # what a rejected draft may have left
    mass = before.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert kb.spec_attend_mass(c.cache(), c.q, lse, mass, dev_status=status, **c.see()) is mass
    got = mass.cpu()
    for b in range(c.B):
        n, t = c.n[b], c.t[b]
        assert torch.isnan(got[b, :, n + t:]).all()
        if t == 0:
            assert torch.equal(got[b, :, :n], before[b, :, :n])
            continue
        share, tol = c.share(lse.cpu(), b)
        old = torch.cat((before[b, :, :n], torch.zeros(c.Hkv, t)), 1).double()
        near(got[b, :, :n + t], old + share, tol + 2.0**-23 * (old + share), f"mass of session {b}")
        unseen = [j for j in range(n) if not c.seen_by_any(b, j)]
        assert torch.equal(got[b][:, unseen], before[b][:, unseen])
    assert int(status) == 0


def both(c):
    _, lse = run(c)
    weigh(c, lse)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [8, 16, 64, 128, 256])
def test_pages_and_types(page, D, dtype):
    both(Case([0, 1, 15, 16, 129, 300], T=3, D=D, page=page, dtype=dtype, seed=page))


@pytest.mark.parametrize("n", [0, 1, 7, 63, 64, 126, 127, 128, 129, 255, 256, 257, 511, 1000])
def test_lengths(n):
    both(Case([n], T=2, Hq=8, Hkv=1, seed=n))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (3, 1), (5, 1), (6, 2), (7, 1), (16, 1), (64, 8), (100, 1),
                                    (128, 1)])
@pytest.mark.parametrize("T", [1, 4])
def test_groups(Hq, Hkv, T):
    both(Case([200, 77], T=T, Hq=Hq, Hkv=Hkv, seed=Hq))


@pytest.mark.parametrize("T,Hq,Hkv", [(15, 64, 8), (16, 8, 1), (17, 8, 1), (31, 9, 1), (33, 8, 1), (64, 4, 1),
                                      (130, 1, 1), (129, 2, 2), (257, 3, 1), (300, 4, 2), (5, 100, 1), (40, 65, 1)])
def test_rows(T, Hq, Hkv):
    both(Case([150, 0], T=T, Hq=Hq, Hkv=Hkv, seed=T))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (16, 0), (17, 4), (100, 16), (128, 128), (130, 200),
                                          (1000, 4), (3, 1000)])
@pytest.mark.parametrize("T", [1, 6, 70])
def test_windows(window, sinks, T):
    both(Case([0, 5, 140, 517], T=T, Hq=4, Hkv=2, window=window, sinks=sinks, seed=window))


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("T", [4, 90])
def test_sessions_with_fewer_rows(T, window):
    both(Case([0, 33, 250, 90, 128], T=T, Hq=6, Hkv=2, t_rows=[T, 0, 1, T - 1, T // 2], window=window, sinks=2,
              seed=T))


@pytest.mark.parametrize("layout", ["nhd", "paired"])
@pytest.mark.parametrize("D", [64, 128])
def test_layouts(layout, D):
    both(Case([260, 31], T=5, Hq=12, Hkv=3, D=D, layout=layout, fused=True, seed=D))


def test_many_sessions():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 200, (90,), generator=g).tolist()
    rows = torch.randint(0, 4, (90,), generator=g).tolist()
    both(Case(lens, T=3, Hq=4, Hkv=2, t_rows=rows, seed=11))


def test_more_sessions_than_a_block_has_threads():
    g = torch.Generator().manual_seed(4)
    both(Case(torch.randint(0, 150, (900,), generator=g).tolist(), T=1, Hq=2, Hkv=1, D=64, seed=12))


@pytest.mark.parametrize("seed", range(24))
def test_anywhere_in_the_range(seed):
    """Sizes drawn over the whole range, small enough for the plain form."""
    r = random.Random(seed)
    Hkv = r.choice((1, 2, 3))
    G, T = r.choice((1, 2, 3, 4, 6, 8, 16, 50)), r.choice((1, 2, 7, 15, 33, 100))
    lens = [r.choice((0, 1, r.randint(0, 300), r.randint(0, 1500))) for _ in range(r.randint(1, 5))]
    both(Case(lens, T=T, Hq=Hkv * G, Hkv=Hkv, D=r.choice((64, 128)), page=r.choice((8, 16, 32, 64, 128, 512, 1024)),
              dtype=r.choice((BF16, F16)), t_rows=r.choice((None, [r.randint(0, T) for _ in lens])),
              window=r.choice((0, 0, r.randint(1, 40), r.randint(1, 600))), sinks=r.choice((0, 3, 130)),
              layout=r.choice(("hnd", "nhd", "paired")), fused=r.random() < 0.5, seed=seed))


def test_sessions_of_one_row_in_a_call_of_many():
    """A decode step beside room for a prompt's chunk: 65535 units of two tokens without rows lie between two
    sessions with one.  They cost a few dozen microseconds, not milliseconds."""
    B, T, H, D, n = 3, 2**17, 128, 64, 30100
    g = torch.Generator("cuda").manual_seed(2)
    cols = n // 1024 + 1
    k, v = torch.randn((2, B * cols, 1, 1024, D), generator=g, device="cuda", dtype=BF16)
    table = torch.arange(B * cols, dtype=torch.int32, device="cuda").view(B, cols)
    cache = kb.PagedCache(k, v, table, torch.full((B,), n - 1, dtype=torch.int32, device="cuda"))
    q = torch.empty((B, T, H, D), dtype=BF16, device="cuda")
    q[:, 0] = torch.randn((B, H, D), generator=g, device="cuda", dtype=BF16)
    plan = kb.AttendPlan(cache, q, t_rows=torch.ones(B, dtype=torch.int32, device="cuda"))
    best = math.inf
    for _ in range(4):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        out, lse = plan()
        end.record()
        end.synchronize()
        best = min(best, start.elapsed_time(end))
    kd, vd = (x.double().view(B, -1, D)[:, :n] for x in (k, v))
    s = torch.einsum("bhd,bnd->bhn", q[:, 0].double(), kd) * D**-0.5
    total = torch.logsumexp(s, 2)
    p = (s - total[..., None]).exp()
    size, u = p @ vd.abs(), torch.finfo(BF16).eps / 2
    ds = (D + 4) * 2.0**-24 * D**-0.5 * float(q[:, 0].double().norm(dim=-1).max() * kd.norm(dim=-1).max())
    near(out[:, 0], p @ vd, u * (p @ vd).abs() + (u + 2 * ds + 2.0**-17) * size * (1 + u) + 1e-30)
    near(lse[:, 0], total, ds + 2.0**-17 + 2.0**-22 * total)
    assert best < 1.0, f"{best} ms"


def test_one_head_shared_by_many_sessions_pages():
    """Sessions that share their first pages, as those of one prompt do."""
    c = Case([160, 160, 160], T=2, Hq=8, Hkv=2, page=32, seed=21)
    c.table[1:, :4] = c.table[0, :4]
    for b in (1, 2):
        c.dense[b][:, :, :128] = c.dense[0][:, :, :128]
    both(c)


@pytest.mark.parametrize("n,T", [(5000, 1), (5000, 15), (3000, 40), (3000, 70), (2000, 193)])
def test_long_texts_are_split_and_joined(n, T):
    both(Case([n, 3], T=T, Hq=8, Hkv=2, page=64, seed=n + T))


@pytest.mark.parametrize("Hkv,D", [(1, 128), (2, 64)])
def test_pages_past_32_bits(Hkv, D):
    both(Case([40], T=3, Hq=4, Hkv=Hkv, D=D, page=16, spare=0, seed=D).spread(2**31 + 8 * D))


def test_rows_past_32_bits():
    """2.2 thousand million elements of q: the first rows, and the last, which begin past 2^31."""
    T, Hq, D, W = 2**17 + 3000, 128, 128, 16
    g = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn((T // 1024 + 1, 1, 1024, D), generator=g, device="cuda", dtype=BF16) for _ in range(2))
    table = torch.arange(len(k), dtype=torch.int32, device="cuda")[None]
    cache = kb.PagedCache(k, v, table, torch.zeros(1, dtype=torch.int32, device="cuda"))
    q = torch.randn((1, T, Hq, D), generator=g, device="cuda", dtype=BF16)
    out, lse = kb.spec_attend(cache, q, window=W)
    mass = kb.spec_attend_mass(cache, q, lse, torch.full((1, 1, cache.capacity), math.nan, device="cuda"), window=W)
    u = torch.finfo(BF16).eps / 2
    for t0 in (0, T // 2, T - 40):
        kk, vv = (x.view(-1, D)[t0:t0 + 40].double().cpu() for x in (k, v))
        qq = q[0, t0:t0 + 40].double().cpu()
        s = torch.einsum("thd,nd->thn", qq, kk) * D**-0.5
        p, j = torch.arange(40)[:, None], torch.arange(40)[None]
        s = s.masked_fill(((j > p) | (p - j >= W))[:, None], -math.inf)
        whole = slice(0 if t0 == 0 else W, 40)  # rows whose window lies in the slice
        total = torch.logsumexp(s, 2)
        w = (s - total[..., None]).exp()
        o, size = torch.einsum("thn,nd->thd", w, vv), torch.einsum("thn,nd->thd", w, vv.abs())
        ds = (D + 4) * 2.0**-24 * D**-0.5 * float(qq.norm(dim=-1).max() * kk.norm(dim=-1).max())
        rows = slice(t0 + whole.start, t0 + 40)
        # the bounds of Case.attend and Case.share; 2048 weights in a key's sum
        near(out[0, rows], o[whole], (u * o.abs() + (u + 2 * ds + 2.0**-17) * size * (1 + u) + 1e-30)[whole])
        near(lse[0, rows], total[whole], ds + 2.0**-17 + 2.0**-22 * total[whole].abs())
        seen = slice(whole.start, 40 if t0 == T - 40 else 40 - W)  # keys whose rows lie in the slice
        x = w.sum((0, 1))
        far = float(torch.where(s == -math.inf, 0.0, s.abs()).max() + total.abs().max())
        near(mass[0, 0, t0 + seen.start:t0 + seen.stop], x[seen], (x * (2 * ds + far * 2.0**-21 + 2.0**-14))[seen])


def test_a_text_of_sixteen_million_tokens():
    """Every page the same one: the attention is that page's, its lse larger by the log of their number."""
    N = 2**24
    c = Case([1024 - 2], T=2, Hq=4, Hkv=1, D=64, page=1024, spare=0, seed=2)
    want, _, tol, _ = c.attend()
    cache = kb.PagedCache(c.k, c.v, torch.zeros((1, N // 1024), dtype=torch.int32, device="cuda"),
                          torch.tensor([N - 2], dtype=torch.int32, device="cuda"))
    out, lse = kb.spec_attend(cache, c.q)
    # the last row sees N keys; a CTA adds up to N / 152 / 16 times to a sum, half an ulp lost each time or,
    # in the tensor cores, a whole one
    s, v, ds = c.head(0, 0)
    lost = N / 152 / 16 * 2.0**-23
    near(out[:, 1], want[:, 1], tol[:, 1] + lost * v.abs().max())
    total = torch.logsumexp(s[1], 1) + math.log(N // 1024)
    near(lse[0, 1], total, ds + 2.0**-17 + 2.0**-22 * total + lost)


@pytest.mark.parametrize("T,G,n,window", [(33, 16, 90, 0), (31, 16, 300, 0), (250, 16, 0, 0), (600, 4, 200, 0),
                                          (400, 8, 100, 70), (7, 64, 500, 0), (290, 1, 40, 0), (520, 1, 130, 0)])
def test_many_tiles_of_rows_for_few_keys(T, G, n, window):
    both(Case([n], T=T, Hq=G, Hkv=1, window=window, sinks=3 if window else 0, seed=T))


def test_scores_of_a_wide_range():
    """Scores of hundreds: the running maximum moves far at every tile."""
    run(Case([700], T=3, Hq=8, Hkv=2, q_scale=60.0, seed=2))
    run(Case([700], T=40, Hq=8, Hkv=2, q_scale=60.0, dtype=F16, seed=3))


def test_rising_scores():
    """Every key scores above the ones before it: the maximum moves in every tile, by little and by much."""
    for step in (0.01, 0.3):
        c = Case([900], T=4, Hq=4, Hkv=1, seed=4)
        unit = torch.zeros(c.D)
        unit[0] = 1.0
        for j in range(904):
            k = (c.dense[0][0, :, j].float() * 0.01 + unit * step * j).to(c.dtype)
            c.dense[0][0, :, j] = k
            c.k[c.table[0, j // c.page], :, j % c.page] = k.cuda()
        c.q_host = (c.q_host.float() * 0.01 + 4.0 * unit).to(c.dtype)
        c.fuse(False)
        run(c)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_many_small_weights_behind_a_strong_key(dtype):
    """The first of 2^18 keys scores 14.5 above the rest, which hold an eighth of the weight together;
    each alone is 8.5 steps of f16's least.  A session a CTA, so that all of it is one running sum."""
    N, D, B, gap = 2**18, 64, 152, 14.4921875
    g = torch.Generator().manual_seed(1)
    k, v = torch.zeros((2, 2, 1, 1024, D))
    k[0, 0, 0, 0] = gap
    v.copy_(1.0 + 0.1 * torch.randn(v.shape, generator=g))
    v[0, 0, 0] = 0.0
    k, v = k.to(dtype), v.to(dtype)
    q = torch.zeros((B, 1, 1, D), dtype=dtype)
    q[..., 0] = D**0.5
    table = torch.ones((B, N // 1024), dtype=torch.int32)
    table[:, 0] = 0
    cache = kb.PagedCache(k.cuda(), v.cuda(), table.cuda(), torch.full((B,), N - 1, dtype=torch.int32, device="cuda"))
    out, lse = kb.spec_attend(cache, q.cuda())
    strong = math.exp(float(k[0, 0, 0, 0]))
    total = strong + N - 1
    o = (v[0].double().sum(1) + (N // 1024 - 1) * v[1].double().sum(1))[None, None] / total
    # weights and result rounded to the type; f16's small weights off by 2^-32; sums of N / 16 steps, each
    # off by an ulp at most
    u, sums = torch.finfo(dtype).eps / 2, N / 16 * 2.0**-23
    near(out, o.expand(out.shape), (2 * u + 2.0**-17 + sums) * o.expand(out.shape) * (1 + u) + 2.0**-32 * N)
    near(lse, torch.full(lse.shape, math.log(total)), torch.full(lse.shape, 2.0**-17 + 2.0**-18 + sums))


def test_scale():
    c = Case([100], T=2)
    c.scale = 0.02
    out = kb.spec_attend(c.cache(), c.q, scale=0.02)[0]
    want, _, tol, _ = c.attend()
    near(out, want, tol)


def test_values_that_only_later_rows_see_do_not_reach_earlier_ones():
    """The second of three rows brings NaN and infinite values: the first row is as without it,
    the rows that see it are NaN."""
    for bad in (math.nan, math.inf, -math.inf):
        for T, G in ((3, 4), (80, 2)):
            c = Case([130], T=T, Hq=G, Hkv=1, seed=9)
            j = 131
            c.v[c.table[0, j // c.page], :, j % c.page, 5] = bad
            out, lse = kb.spec_attend(c.cache(), c.q)
            want, want_lse, tol, tol_lse = c.attend()
            near(out[:, :1], want[:, :1], tol[:, :1])
            near(lse, want_lse, tol_lse)
            assert torch.isnan(out[0, 1:, :, 5]).all() or math.isinf(bad)
            assert not torch.isfinite(out[0, 1:, :, 5]).any()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,window,at", [(6, 40, 92), (6, 40, 94), (90, 4, 150), (90, 40, 100), (90, 100, 60)])
def test_values_that_only_some_rows_see_reach_those_alone(T, window, at, dtype):
    """A value behind the window of the later rows, or of a key that is new: NaN where it is seen."""
    c = Case([130], T=T, Hq=4, Hkv=1, window=window, sinks=2, dtype=dtype, seed=T)
    c.v[c.table[0, at // c.page], :, at % c.page, 9] = math.inf
    out, lse = kb.spec_attend(c.cache(), c.q, **c.see())
    want, want_lse, tol, tol_lse = c.attend()
    near(lse, want_lse, tol_lse)
    sees = torch.tensor([c.sees(130 + t, at) for t in range(T)])
    assert sees.any() and not sees.all()
    near(out[:, ~sees], want[:, ~sees], tol[:, ~sees])
    assert not torch.isfinite(out[:, sees][..., 9]).any()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("T,G,window,at", [(200, 4, 0, 135), (200, 4, 100, 100), (31, 4, 0, 133), (300, 1, 0, 390),
                                           (40, 100, 0, 132), (200, 4, 0, 60), (150, 16, 70, 199)])
def test_how_far_a_value_that_is_not_finite_reaches(T, G, window, at, bad):
    """The whole row where only some of the unit's rows see the key, else its own element alone."""
    c = Case([130], T=T, Hq=G, Hkv=1, window=window, seed=T + at)
    c.v[c.table[0, at // c.page], :, at % c.page, 9] = bad
    out, lse = kb.spec_attend(c.cache(), c.q, **c.see())
    want, want_lse, tol, tol_lse = c.attend()
    near(lse, want_lse, tol_lse)
    unit = 128 // G * (2 if T > 128 // G else 1)
    sees = [c.sees(130 + t, at) for t in range(T)]
    out, parts = out.cpu(), 0
    for t in range(T):
        mates = sees[t // unit * unit:][:unit]
        if sees[t] and not all(mates):
            assert torch.isnan(out[0, t]).all(), t
            parts += 1
        else:
            if sees[t]:
                assert not torch.isfinite(out[0, t, :, 9]).any(), t
                out[0, t, :, 9] = want[0, t, :, 9].to(out.dtype)
            near(out[0, t], want[0, t], tol[0, t], f"row {t}")
    # 60 lies before the call; 132 is the first row of a unit of two: all rows of the units behind see them
    assert any(sees) and (parts == 0) == (at in (60, 132))


@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_not_finite_in_many_short_sessions(D):
    """Units of one key tile follow one another in a block: what one marks does not reach the others."""
    g = torch.Generator().manual_seed(D)
    B = 700
    c = Case(torch.randint(0, 120, (B,), generator=g).tolist(), T=3, Hq=4, Hkv=1, D=D, seed=D)
    bad = torch.rand(B, generator=g) < 0.5
    for b in bad.nonzero()[:, 0].tolist():  # the second row's own value
        j = c.n[b] + 1
        c.v[c.table[b, j // c.page], :, j % c.page, 9] = math.inf
    want, want_lse, tol, tol_lse = c.attend()
    for _ in range(3):
        out, lse = kb.spec_attend(c.cache(), c.q)
        near(lse, want_lse, tol_lse)
        out = out.cpu()
        near(out[~bad], want[~bad], tol[~bad])
        near(out[bad][:, :1], want[bad][:, :1], tol[bad][:, :1])
        assert not torch.isfinite(out[bad][:, 1:, :, 9]).any()


def test_keys_that_only_later_rows_see_do_not_reach_earlier_ones():
    c = Case([130], T=3, Hq=4, Hkv=1, seed=9)
    j = 131
    c.k[c.table[0, j // c.page], :, j % c.page, 5] = math.nan
    out, lse = kb.spec_attend(c.cache(), c.q)
    want, want_lse, tol, tol_lse = c.attend()
    near(out[:, :1], want[:, :1], tol[:, :1])
    near(lse[:, :1], want_lse[:, :1], tol_lse[:, :1])
    assert torch.isnan(out[:, 1:]).all() and torch.isnan(lse[:, 1:]).all()


def test_all_scores_minus_infinity():
    c = Case([40], T=2, Hq=4, Hkv=1, seed=1)
    unit = torch.zeros(c.D, dtype=c.dtype)
    unit[0] = -math.inf
    for j in range(42):
        c.k[c.table[0, j // c.page], :, j % c.page] = unit.cuda()
    c.q = c.q.abs() + 1.0
    c.q[..., 1:] = 1.0
    out, lse = kb.spec_attend(c.cache(), c.q)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    mass = torch.ones((1, 1, c.cache().capacity), device="cuda")
    kb.spec_attend_mass(c.cache(), c.q, lse, mass)
    assert torch.all(mass[..., :40] == 1.0) and torch.all(mass[..., 40:42] == 0.0)


@pytest.mark.parametrize("Hq,Hkv", [(3, 3), (8, 2)])
def test_mass_with_an_lse_of_any_strides(Hq, Hkv):
    """Heads before rows in memory, or part of a larger tensor: the bits of a dense lse, also when its
    values change between a plan's calls."""
    c = Case([150, 40], T=5, Hq=Hq, Hkv=Hkv, seed=Hq)
    _, lse = kb.spec_attend(c.cache(), c.q)
    turned = lse.transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.full((2, 5, Hq + 3), math.nan, device="cuda")
    wide[:, :, 2:2 + Hq] = lse
    want = kb.spec_attend_mass(c.cache(), c.q, lse, torch.zeros((2, Hkv, c.cache().capacity), device="cuda"))
    for x in (turned, wide[:, :, 2:2 + Hq]):
        assert not x.is_contiguous()
        mass = torch.zeros_like(want)
        plan = kb.AttendMassPlan(c.cache(), c.q, x, mass)
        plan()
        assert torch.equal(mass, want)
        x.add_(1.0)
        mass.zero_()
        plan()
        # exponents of size 64 at most on either side, off by 2^-21 of that
        near(mass, want.double() / math.e, 2.0**-14 * want)
        x.sub_(1.0)
    turned.copy_(lse)
    plan = kb.AttendMassPlan(c.cache(), c.q, turned.requires_grad_(), torch.zeros_like(want))
    assert torch.equal(plan(), want)
    assert not plan.out.requires_grad and not plan._dense.requires_grad


def test_mass_adds_up():
    """Twice the same rows: twice their shares on the tokens before, once on the rows' own."""
    c = Case([300, 90], T=4, Hq=8, Hkv=2, seed=6)
    _, lse = kb.spec_attend(c.cache(), c.q)
    mass = torch.zeros((2, 2, c.cache().capacity), device="cuda")
    plan = kb.AttendMassPlan(c.cache(), c.q, lse, mass)
    plan()
    once = mass.clone()
    plan()
    for b, n in enumerate(c.n):
        assert torch.equal(mass[b, :, :n], 2 * once[b, :, :n])
        assert torch.equal(mass[b, :, n:n + 4], once[b, :, n:n + 4])
        # every row and head hands out one
        assert torch.allclose(once[b].sum(1), torch.full((2,), 16.0, device="cuda"), rtol=1e-4)


def test_sessions_out_of_range_are_left_untouched():
    c = Case([100, 100, 100, 100, 100], T=3, Hq=4, Hkv=2, t_rows=[3, 3, 3, 3, 3], seed=8)
    cap = c.cache().capacity
    c.lens[1], c.lens[2] = -1, cap - 2
    c.t_rows[3], c.t_rows[4] = 4, -1
    out = torch.full((5, 3, 4, 128), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((5, 3, 4), 7.0, device="cuda")
    mass = torch.full((5, 2, cap), 7.0, device="cuda")
    want, want_lse, tol, tol_lse = c.attend()
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    kb.spec_attend(c.cache(), c.q, t_rows=c.t_rows, out=out, lse_out=lse, dev_status=status[:1])
    kb.spec_attend_mass(c.cache(), c.q, lse, mass, t_rows=c.t_rows, dev_status=status[1:])
    near(out[:1], want[:1], tol[:1])
    assert torch.all(out[1:] == 7.0) and torch.all(lse[1:] == 7.0) and torch.all(mass[1:] == 7.0)
    assert status.tolist() == [kb.ST_BADKEEP | kb.ST_BADLEN] * 2


def test_bad_pages_read_as_zeros():
    for bad in (-1, -(2**31), 2**31 - 1, None):
        c = Case([200, 200], T=3, Hq=4, Hkv=2, seed=12)
        c.table[0, 5] = c.k.shape[0] if bad is None else bad
        c.dense[0][:, :, 80:96] = 0.0
        out = torch.full((2, 3, 4, 128), 7.0, dtype=BF16, device="cuda")
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        mass = torch.zeros((2, 2, c.cache().capacity), device="cuda")
        _, lse = kb.spec_attend(c.cache(), c.q, out=out, dev_status=status[:1])
        want, want_lse, tol, tol_lse = c.attend()
        near(out, want, tol)
        near(lse, want_lse, tol_lse)
        kb.spec_attend_mass(c.cache(), c.q, lse, mass, dev_status=status[1:])
        share, tol = c.share(lse.cpu(), 0)
        near(mass[0, :, :203], share, tol + 1e-7)
        assert status.tolist() == [kb.ST_BADPAGE] * 2


def test_pages_behind_the_window_are_not_looked_at():
    c = Case([500], T=3, window=64, sinks=4, page=16, seed=13)
    gone = [i for i in range(c.table.shape[1]) if not any(c.seen_by_any(0, j) for j in range(16 * i, 16 * i + 16)
                                                          if j < 503)]
    assert len(gone) > 20
    c.table[0, gone] = 2**30
    both(c)


def test_a_call_on_another_stream_and_twice_the_same_bits():
    c = Case([900, 40], T=15, Hq=16, Hkv=2, seed=14)
    first, lse = kb.spec_attend(c.cache(), c.q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    again, lse2 = kb.spec_attend(c.cache(), c.q, stream=side)
    side.synchronize()
    assert torch.equal(first, again) and torch.equal(lse, lse2)


def test_captured_and_replayed_with_other_lengths():
    """One graph serves lengths, rows and pages that change between its replays."""
    a = Case([300, 20, 77], T=4, Hq=8, Hkv=2, t_rows=[4, 0, 2], seed=15)
    b = Case([17, 290, 0], T=4, Hq=8, Hkv=2, t_rows=[1, 4, 3], seed=16, cols=a.table.shape[1])
    out = torch.full((3, 4, 8, 128), 7.0, dtype=BF16, device="cuda")
    side = torch.cuda.Stream()
    live = Case([300, 20, 77], T=4, Hq=8, Hkv=2, t_rows=[4, 0, 2], seed=15)
    plan = kb.AttendPlan(live.cache(), live.q, t_rows=live.t_rows, out=out, stream=side)
    mass = torch.zeros((3, 2, live.cache().capacity), device="cuda")
    weigh_plan = kb.AttendMassPlan(live.cache(), live.q, plan.out[1], mass, t_rows=live.t_rows, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        plan()
        weigh_plan()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan()
        weigh_plan()
    for c in (b, a):
        for name in ("k", "v", "table", "lens", "t_rows", "q"):
            getattr(live, name).copy_(getattr(c, name))
        out.fill_(7.0)
        mass.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, _, tol, _ = c.attend()
        there = near(out, want, tol)
        assert torch.all(out.cpu()[~there] == 7.0)
        for s in range(3):
            if c.t[s]:
                share, tol = c.share(plan.out[1].cpu(), s)
                near(mass[s, :, :c.n[s] + c.t[s]], share, tol + 1e-7)


def test_calls_in_a_row_share_a_workspace():
    cases = [Case([n, 40], T=6, Hq=16, Hkv=2, seed=n) for n in (1200, 64, 700)]
    work = torch.empty(max(kb.AttendPlan.workspace_bytes(c.cache(), c.T, c.Hq) for c in cases), dtype=torch.uint8,
                       device="cuda")
    plans = [kb.AttendPlan(c.cache(), c.q, workspace=work) for c in cases]
    for _ in range(3):
        for p in plans:
            p()
    for c, p in zip(cases, plans):
        want, want_lse, tol, tol_lse = c.attend()
        near(p.out[0], want, tol)
        near(p.out[1], want_lse, tol_lse)


def test_two_calls_at_once():
    cases = [Case([800 + s, 100], T=8, Hq=16, Hkv=2, seed=s) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    plans = [kb.AttendPlan(c.cache(), c.q, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for _ in range(20):
        for p in plans:
            p()
    torch.cuda.synchronize()
    for c, p in zip(cases, plans):
        want, _, tol, _ = c.attend()
        near(p.out[0], want, tol)


@pytest.mark.parametrize("T,Hq,D", [(3, 8, 128), (60, 16, 128), (200, 4, 64)])
def test_results_in_the_place_of_the_rows(T, Hq, D):
    c = Case([3000, 17, 400, 0], T=T, Hq=Hq, Hkv=2, D=D, t_rows=[T, T, 0, T - 1], seed=T)
    out, lse = kb.spec_attend(c.cache(), c.q, t_rows=c.t_rows)
    for _ in range(3):
        q = c.q.clone()
        again, lse2 = kb.spec_attend(c.cache(), q, t_rows=c.t_rows, out=q)
        assert again is q
        for b, t in enumerate(c.t):
            assert torch.equal(q[b, :t], out[b, :t]) and torch.equal(lse2[b, :t], lse[b, :t])
            assert torch.isnan(q[b, t:]).all()


def test_no_rows_and_no_sessions():
    c = Case([10, 20], T=2)
    out, lse = kb.spec_attend(c.cache(), c.q[:, :0])
    assert out.shape == (2, 0, 4, 128) and lse.shape == (2, 0, 4)
    empty = kb.PagedCache(c.k, c.v, c.table[:0], c.lens[:0])
    assert kb.spec_attend(empty, c.q[:0])[0].shape == (0, 2, 4, 128)
    kb.spec_attend_mass(empty, c.q[:0], torch.empty((0, 2, 4), device="cuda"),
                        torch.empty((0, 2, empty.capacity), device="cuda"))


def test_a_workspace_that_is_too_small_is_refused():
    c = Case([10], T=2)
    need = kb.AttendPlan.workspace_bytes(c.cache(), 2, 4)
    with pytest.raises(kb.KdaError, match="workspace"):
        kb.spec_attend(c.cache(), c.q, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


@pytest.fixture(scope="module")
def stopping(tmp_path_factory):
    """The two attention kernels built so that every third CTA behaves as if its first wait had run out."""
    where = tmp_path_factory.mktemp("stopping")
    parts = [str(where / f"{src}.o") for src in ("spec_attend.cu", "spec_attend_mass.cu", "kda_abi.cpp")]
    jobs = [subprocess.Popen([build.nvcc(), *build.ARCH, *build.NVFLAGS, "-DKDA_STOP_EVERY=3", "-c",
                              os.path.join(build.CSRC, os.path.basename(o)[:-2]), "-o", o]) for o in parts]
    assert [j.wait() for j in jobs] == [0, 0, 0]
    path = str(where / "stopping.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-o", path, *parts], check=True)
    return ctypes.CDLL(path)


def through(L, plan):
    """The plan's call, made of another library."""
    fn = getattr(L, plan.name)
    fn.argtypes, fn.restype = plan._fn.argtypes, plan._fn.restype
    plan._fn = fn
    return plan


@pytest.mark.parametrize("D,T,Hq", [(128, 4, 8), (64, 4, 8), (128, 40, 16), (64, 40, 16)])
def test_what_a_stopped_block_had_to_compute_is_nan(stopping, D, T, Hq):
    """With a status word, and without one; every other row and mass is as it should be."""
    c = Case([5000, 3, 700, 128, 0, 100, 50, 20, 2000, 64, 30, 7], T=T, Hq=Hq, Hkv=2, D=D, page=32, seed=D + T,
             t_rows=[T, T, 1, T, T, T, 0, T, T - 1, T, T, T])
    want, want_lse, tol, tol_lse = c.attend()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    work = torch.zeros(kb.AttendPlan.workspace_bytes(c.cache(), T, Hq), dtype=torch.uint8, device="cuda")
    for told in (status, None):
        out = torch.full((c.B, T, Hq, D), 7.0, dtype=BF16, device="cuda")
        lse = torch.full((c.B, T, Hq), 7.0, device="cuda")
        through(stopping, kb.AttendPlan(c.cache(), c.q, t_rows=c.t_rows, out=out, lse_out=lse, dev_status=told,
                                        workspace=work))()
        lost = torch.isnan(lse).cpu()
        there = ~torch.isnan(want_lse)
        assert (lost & there).any() and (~lost & there).any() and not (lost & ~there).any()
        assert torch.isnan(out.cpu()[lost]).all()
        near(lse, want_lse.masked_fill(lost, math.nan), tol_lse, "lse")
        near(out, want.masked_fill(lost[..., None], math.nan), tol, "out")
        assert torch.all(out.cpu()[~there] == 7.0) and torch.all(lse.cpu()[~there] == 7.0)
    assert int(status) == kb.ST_TIMEOUT
    _, lse = run(c)  # the same call of the library proper
    status.zero_()
    for told in (status, None):
        mass = torch.full((c.B, 2, c.cache().capacity), 7.0, device="cuda")
        through(stopping, kb.AttendMassPlan(c.cache(), c.q, lse, mass, t_rows=c.t_rows, dev_status=told))()
        mass = mass.cpu()
        right = 0
        for b in range(c.B):
            n, t = c.n[b], c.t[b]
            assert torch.all(mass[b, :, n + t:] == 7.0)
            if t == 0:
                assert torch.all(mass[b] == 7.0)
                continue
            share, tol_share = c.share(lse.cpu(), b)
            old = torch.cat((torch.full((2, n), 7.0), torch.zeros(2, t)), 1).double()
            lost = torch.isnan(mass[b, :, :n + t])
            right += int((~lost).sum())
            near(mass[b, :, :n + t], (old + share).masked_fill(lost, math.nan), tol_share + 2.0**-23 * (old + share))
        assert right > 0 and torch.isnan(mass).any()
    assert int(status) == kb.ST_TIMEOUT
