"""What the entry points over a paged cache refuse before anything is launched."""
import ctypes
import math

import pytest
import torch

from libs import ensure_built
from test_logit_plans_cpu import fake

from speculative_decode_verify_kda_gb300 import binding as kb

FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    ensure_built()
    return kb.lib()


def cache(**kw):
    c = dict(k=FAKE, v=FAKE, table=FAKE, lens=FAKE, page_stride=2 * 16 * 128, head_stride=16 * 128, slot_stride=128,
             B=2, Hkv=2, D=128, page=16, pages=8, table_cols=4, dtype=kb.BF16)
    c.update(kw)
    return kb.KdaCache(*(c[name] for name, _ in kb.KdaCache._fields_))


def append(L, c, k=FAKE, v=FAKE, T=3, ld_k=256, ld_v=256, t_rows=None, status=None):
    return L.spec_cache_append(None if c is None else ctypes.byref(c), k, v, T, ld_k, ld_v, t_rows, status, None)


def attend(L, c, q=FAKE, T=3, Hq=4, ld=512, t_rows=None, window=0, sinks=0, scale=0.1, out=FAKE, lse=None, status=None,
           work=FAKE, size=1 << 40):
    return L.spec_attend(None if c is None else ctypes.byref(c), q, T, Hq, ld, t_rows, window, sinks, scale, out, lse,
                         status, work, size, None)


def mass(L, c, q=FAKE, T=3, Hq=4, ld=512, lse=FAKE, t_rows=None, window=0, sinks=0, scale=0.1, m=FAKE, ld_mass=64,
         status=None):
    return L.spec_attend_mass(None if c is None else ctypes.byref(c), q, T, Hq, ld, lse, t_rows, window, sinks, scale,
                              m, ld_mass, status, None)


def evict(L, c, m=FAKE, ld=64, budget=32, recent=4, sinks=2, dst=None, cols=0, kept=FAKE, m_out=None, ld_out=0,
          lens_out=FAKE, status=None):
    return L.spec_cache_evict(None if c is None else ctypes.byref(c), m, ld, budget, recent, sinks, dst, cols, kept,
                              m_out, ld_out, lens_out, status, None)


CALLS = [append, attend, mass, evict]

BAD_CACHES = [dict(B=-1), dict(Hkv=0), dict(Hkv=65536), dict(D=96), dict(D=256), dict(dtype=kb.F32), dict(dtype=9),
              dict(page=4), dict(page=24), dict(page=2048), dict(page=0), dict(page=-16), dict(pages=0),
              dict(table_cols=0), dict(table_cols=2**26 + 1), dict(page_stride=0), dict(page_stride=4100),
              dict(head_stride=64), dict(slot_stride=-128), dict(slot_stride=2**38), dict(k=None), dict(v=None),
              dict(table=None), dict(lens=None), dict(k=FAKE + 8), dict(v=FAKE + 2), dict(table=FAKE + 2),
              dict(lens=FAKE + 1)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches_are_refused(L, call, bad):
    assert call(L, cache(**bad)) == kb.EINVAL
    assert L.kda_last_error()


@pytest.mark.parametrize("call", CALLS)
def test_no_cache_is_refused_and_no_session_is_nothing_to_do(L, call):
    assert call(L, None) == kb.EINVAL
    assert call(L, cache(B=0, k=None, v=None, table=None, lens=None)) == kb.OK


@pytest.mark.parametrize("bad", [dict(T=-1), dict(T=2**30), dict(k=None), dict(v=None), dict(k=FAKE + 8),
                                 dict(ld_k=248), dict(ld_v=260), dict(ld_k=2**38), dict(t_rows=FAKE + 2),
                                 dict(status=FAKE + 1)], ids=str)
def test_append_refuses(L, bad):
    assert append(L, cache(), **bad) == kb.EINVAL


QUERY = [dict(T=-1), dict(T=2**30), dict(q=None), dict(q=FAKE + 4), dict(ld=504), dict(ld=516), dict(Hq=0),
         dict(Hq=1), dict(Hq=3), dict(Hq=258, ld=2**20), dict(window=-1), dict(sinks=-1), dict(scale=0.0),
         dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=9e-7), dict(scale=1.1e6),
         dict(t_rows=FAKE + 2), dict(status=FAKE + 2), dict(lse=FAKE + 2)]


@pytest.mark.parametrize("bad", [*QUERY, dict(out=None), dict(out=FAKE + 8), dict(work=None), dict(work=FAKE + 8),
                                 dict(size=0)], ids=str)
def test_attend_refuses(L, bad):
    assert attend(L, cache(), **bad) == kb.EINVAL


@pytest.mark.parametrize("bad", [*QUERY, dict(lse=None), dict(m=None), dict(m=FAKE + 2), dict(ld_mass=63),
                                 dict(ld_mass=2**40)], ids=str)
def test_mass_refuses(L, bad):
    assert mass(L, cache(), **bad) == kb.EINVAL


@pytest.mark.parametrize("bad", [dict(m=None), dict(ld=63), dict(budget=0), dict(budget=65), dict(budget=-5),
                                 dict(recent=-1), dict(sinks=-1), dict(recent=31, sinks=2),
                                 dict(recent=2**31 - 1, sinks=2**31 - 1), dict(dst=FAKE, cols=1), dict(dst=FAKE),
                                 dict(dst=FAKE + 2, cols=2), dict(kept=None), dict(lens_out=None),
                                 dict(m_out=1 << 20, ld_out=31), dict(m_out=FAKE + 4, ld_out=64),
                                 dict(m_out=FAKE, ld_out=65), dict(kept=FAKE + 1), dict(status=FAKE + 3)], ids=str)
def test_evict_refuses(L, bad):
    assert evict(L, cache(), **bad) == kb.EINVAL


@pytest.mark.parametrize("ld,out", [(520, 0), (512, 16), (512, -16), (512, 2 * 5 * 512), (4096, 2 * 5 * 4096 + 1008)])
def test_attend_refuses_an_out_that_overlaps_its_rows(L, ld, out):
    base = 1 << 24
    assert attend(L, cache(), q=base, ld=ld, out=base + out) == kb.EINVAL and b"apart" in L.kda_last_error()
    # q itself, and what lies behind or before it, pass this check (and fail the next)
    for q_ld, apart in ((512, 0), (ld, 2 * 5 * ld + 1024), (ld, -2 * 6 * 512)):
        assert attend(L, cache(), q=base, ld=q_ld, out=base + apart, work=None) == kb.EINVAL
        assert b"workspace" in L.kda_last_error()


def test_more_tiles_than_a_call_counts_are_refused(L):
    many = cache(B=2**20, Hkv=64, table_cols=2**16)
    assert attend(L, many, T=1, Hq=64, ld=64 * 128) == kb.EINVAL and b"tiles" in L.kda_last_error()
    assert mass(L, many, T=1, Hq=64, ld=64 * 128, ld_mass=2**20) == kb.EINVAL and b"tiles" in L.kda_last_error()


def test_more_rows_than_a_launch_moves_are_refused(L):
    """(Before the first of the two launches: without a device that one would be KDA_ECUDA.)"""
    many = cache(B=2**15, Hkv=2**15, table_cols=8)
    assert evict(L, many, ld=128, budget=128, dst=FAKE, cols=8) == kb.EINVAL and b"rows" in L.kda_last_error()


def test_no_rows_are_nothing_to_do(L):
    assert append(L, cache(), T=0, k=None, v=None) == kb.OK
    assert attend(L, cache(), T=0, q=None, out=None, work=None, size=0) == kb.OK
    assert mass(L, cache(), T=0, q=None, lse=None, m=None) == kb.OK


def paged(**kw):
    c = dict(k=fake(8, 2, 16, 128, dtype=torch.bfloat16), table=fake(2, 4, dtype=torch.int32),
             lens=fake(2, dtype=torch.int32))
    c.update(kw)
    c.setdefault("v", c["k"])
    return kb.PagedCache(c["k"], c["v"], c["table"], c["lens"])


@pytest.mark.parametrize("bad", [dict(k=torch.empty(8, 2, 16, 128)), dict(k=fake(8, 2, 16, 128)),
                                 dict(v=fake(8, 2, 16, 128, dtype=torch.float16)),
                                 dict(v=fake(8, 2, 16, 64, dtype=torch.bfloat16)),
                                 dict(k=fake(16, 16, 128, dtype=torch.bfloat16)),
                                 dict(v=fake(8, 16, 2, 128, dtype=torch.bfloat16).transpose(1, 2)),
                                 dict(k=fake(8, 2, 128, 16, dtype=torch.bfloat16).transpose(2, 3)),
                                 dict(table=fake(2, 4)), dict(table=fake(8, dtype=torch.int32)),
                                 dict(lens=fake(3, dtype=torch.int32)), dict(lens=fake(2, dtype=torch.int64)),
                                 dict(k=fake(2**31, 1, 16, 128, dtype=torch.bfloat16))], ids=lambda d: next(iter(d)))
def test_the_binding_refuses_caches(bad):
    with pytest.raises((TypeError, ValueError)):
        paged(**bad)


def test_the_binding_takes_strides():
    nhd = fake(8, 16, 2, 128, dtype=torch.bfloat16).transpose(1, 2)
    c = paged(k=nhd).c
    assert (c.page_stride, c.head_stride, c.slot_stride) == (16 * 2 * 128, 128, 2 * 128)
    one = paged(k=fake(8, 1, 16, 128, dtype=torch.bfloat16)).c
    assert (one.page_stride, one.head_stride, one.slot_stride) == (16 * 128, 128, 128)


@pytest.mark.parametrize("name", ["k", "v", "table", "lens"])
def test_a_caches_tensors_stay_the_ones_it_was_made_with(name):
    c = paged(v=fake(8, 2, 16, 128, dtype=torch.bfloat16))
    first = getattr(c, name)
    with pytest.raises(AttributeError, match=name):
        setattr(c, name, first[:])
    with pytest.raises(AttributeError):
        delattr(c, name)
    assert getattr(c, name) is first
    setattr(c, name, first)
    c.lens += fake(2, dtype=torch.int32)
    c.table[0, 1] = 3
    assert getattr(c, name) is first


def test_the_binding_refuses_rows(L):
    c, bf = paged(), torch.bfloat16
    kw = dict(out=fake(2, 3, 4, 128, dtype=bf), lse_out=fake(2, 3, 4), workspace=fake(16, dtype=torch.uint8), stream=0)
    for q in (fake(2, 3, 4, 128), fake(3, 3, 4, 128, dtype=bf), fake(2, 3, 4, 64, dtype=bf), fake(2, 12, 128, dtype=bf),
              fake(2, 4, 3, 128, dtype=bf).transpose(1, 2), fake(3, 2, 4, 128, dtype=bf).transpose(0, 1)):
        with pytest.raises((TypeError, ValueError)):
            kb.AttendPlan(c, q, **kw)
    q = fake(2, 3, 4, 128, dtype=bf)
    for more in (dict(t_rows=fake(3, dtype=torch.int32)), dict(t_rows=fake(2)), dict(out=fake(2, 3, 4, 128)),
                 dict(lse_out=fake(2, 3)), dict(window=2**32), dict(sinks=2**31)):
        with pytest.raises((TypeError, ValueError)):
            kb.AttendPlan(c, q, **{**kw, **more})
    with pytest.raises(ValueError, match="same number of rows"):
        kb.CacheAppendPlan(c, fake(2, 3, 2, 128, dtype=bf), fake(2, 4, 2, 128, dtype=bf), stream=0)
    with pytest.raises(ValueError, match="mass"):
        kb.AttendMassPlan(c, q, fake(2, 3, 4), fake(2, 2, 63), stream=0)
    with pytest.raises(ValueError, match="mass_out"):
        kb.CacheEvictPlan(c, fake(2, 2, 64), 32, kept_out=fake(2, 2, 32, dtype=torch.int32), mass_out=fake(2, 2, 31),
                          lens_out=fake(2, dtype=torch.int32), stream=0)


def test_the_binding_refuses_an_lse_of_another_shape_or_type(L):
    c, q = paged(), fake(2, 3, 4, 128, dtype=torch.bfloat16)
    for lse in (fake(2, 4, 3), fake(2, 4, 4).transpose(1, 2), fake(2, 4, 3, dtype=torch.float64).transpose(1, 2),
                torch.empty(2, 4, 3).transpose(1, 2)):
        with pytest.raises((TypeError, ValueError)):
            kb.AttendMassPlan(c, q, lse, fake(2, 2, 64), stream=0)


def test_a_plan_is_launched_on_the_device_of_its_tensors(monkeypatch, L):
    """(No sessions: nothing is launched.)"""
    current = [0]
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    c = paged(table=fake(0, 4, dtype=torch.int32), lens=fake(0, dtype=torch.int32))
    rows = fake(0, 3, 2, 128, dtype=torch.bfloat16)
    plan = kb.CacheAppendPlan(c, rows, rows, stream=0)
    plan()
    current[0] = 1
    with pytest.raises(RuntimeError, match="current device"):
        plan()
    with pytest.raises(RuntimeError, match="current device"):
        kb.CacheAppendPlan(c, rows, rows, stream=0)
