"""spec_logprobs and spec_logprobs_backward on the GPU against 64-bit definitions.

Tolerances, derived before the first run (u = 2^-24).  A weight exp(z - m) carries the
rounding of its argument (three roundings of at most |d| = 30 in base 2: 62 u) and of
the exponential (2^-22 = 4 u); a sum of V terms in a block's order has a random-walk
error of about sqrt(V / 256 + 13) u, 23 u at V = 131072, and at most 525 u.  ln S, and
with it every log-probability, is then within about 1e-5; the quotient and
subtraction of the logit itself add 4 u of its size.  The entropy multiplies the weights'
errors by |d| <= 20 nats: 2e-5.  Whole numbers are exact."""
import numpy as np
import pytest
import torch

import score_ref as ref
from gpu_util import to_dev
from libs import ensure_built

from speculative_decode_verify_kda_gb300 import binding as kb

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def dev(x, dtype):
    return to_dev(np.asarray(x, np.float32)).to(DT[dtype])


def near(got, want, atol, rtol, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = (np.isnan(got) & np.isnan(want)) | (got == want)
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - want) <= atol + rtol * np.abs(want))
    assert ok.all(), f"{what}: {np.argwhere(~ok)[:4].tolist()} got {got[~ok][:4]} want {want[~ok][:4]}"


def check(x, tokens, K, tau, dtype, t=None, **kw):
    t = dev(x, dtype) if t is None else t
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tok = None if tokens is None else to_dev(np.asarray(tokens, np.int32))
    lp, H, stats, ids, top = kb.spec_logprobs(t, tok, K, tau, dev_status=st, **kw)
    torch.cuda.synchronize()
    want = ref.score(x, tokens, K, tau)
    scale = 4 * 2.0**-24
    assert np.array_equal(ids.cpu().numpy(), want[3])
    if tokens is not None:
        near(lp, want[0], 1e-5, scale, "logprob")
    near(H, want[1], 2e-5, 1e-6, "entropy")
    assert np.array_equal(stats[..., 0].cpu().numpy(), want[2][:, 0].astype(np.float32), equal_nan=True)
    near(stats[..., 1], want[2][:, 1], 1e-5, scale, "ln S")
    near(top, want[4], 1e-5, scale, "top_logprobs")
    return int(st.item()), (lp, H, stats, ids, top)


def tokens_for(N, V, seed):
    return np.random.default_rng(seed).integers(0, V, N)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 2), (2, 5, 8), (5, 32, 5), (5, 37, 7), (4, 257, 128),
                                   (4, 1001, 20), (70, 1000, 3), (2, 2049, 32), (2, 4099, 128), (3, 16384, 33),
                                   (1, 32768, 5), (8, 32768, 20), (2, 50021, 64), (2, 100003, 1), (700, 777, 5),
                                   (37, 131072, 64), (330, 33000, 20), (2, 262147, 128), (1, 600011, 9)])
def test_sizes(N, V, K, dtype):
    x = ref.rows("normal", N, V, dtype, 11 * N + V)
    assert check(x, tokens_for(N, V, 3), K, 1.0, dtype)[0] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K", [(2, 37, 5), (3, 1001, 20), (2, 32768, 20), (200, 8200, 20), (2, 70001, 128)])
@pytest.mark.parametrize("kind", [k for k in ref.KINDS if k != "huge"])
def test_kinds_of_rows(kind, N, V, K, dtype):
    x = ref.rows(kind, N, V, dtype, 5)
    assert check(x, tokens_for(N, V, 4), K, 1.0, dtype)[0] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [1e-4, 0.5, 0.7, 2.0, 1e4])
def test_temperatures(tau, dtype):
    # at 1e-4 a logit's own rounding of z is 4 u of |z| = 1e5: the differences to the maximum
    # are exact in f32 for bf16 logits and within 2 u of |d| otherwise
    x = ref.rows("normal", 4, 5003, dtype, 9)
    check(x, tokens_for(4, 5003, 2), 20, float(np.float32(tau)), dtype)


def test_huge_logits_stay_finite():
    x = ref.rows("huge", 3, 4099, "f32", 6)
    _, (lp, H, stats, ids, top) = check(x, tokens_for(3, 4099, 7), 6, 1.0, "f32")
    assert torch.isfinite(stats).all() and torch.isfinite(H).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [37, 1001, 40000])
def test_nan_and_infinite_rows_are_reported(V, dtype):
    x = ref.rows("normal", 6, V, dtype, 8)
    x[0, 0] = np.nan
    x[2, V - 1] = np.nan
    x[3, V // 2] = np.inf
    x[4, V // 2] = -np.nan
    x[4, V // 3] = np.inf
    st, _ = check(x, tokens_for(6, V, 1), 4, 1.0, dtype)
    assert st == kb.ST_NAN


def test_tokens_that_are_none_or_out_of_range():
    x = ref.rows("normal", 5, 300, "bf16", 2)
    assert check(x, [-1, 3, -100, 299, 0], 2, 1.0, "bf16")[0] == 0
    assert check(x, [-1, 3, 300, 299, 2**31 - 1], 2, 1.0, "bf16")[0] == kb.ST_BADTOKEN
    out = kb.spec_logprobs(dev(x, "bf16"), None, 0)
    assert out[0] is None and out[3].shape == (5, 0)
    near(out[2], ref.score(x, None, 0, 1.0)[2], 1e-5, 1e-6, "stats")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,ld,off", [(1001, 1001, 1), (1001, 1003, 3), (4096, 4104, 8), (4095, 5000, 5),
                                      (33, 40, 7), (33000, 33001, 1)])
def test_row_strides_and_offsets(V, ld, off, dtype):
    N = 5
    buf = torch.full((off + N * ld + 16,), float("nan"), dtype=DT[dtype], device="cuda")  # NaN around the rows
    t = buf[off:off + N * ld].view(N, ld)[:, :V] if ld > V else buf[off:off + N * ld].view(N, V)
    x = ref.rows("peaked", N, V, dtype, V + off)
    t.copy_(dev(x, dtype))
    assert check(x, tokens_for(N, V, 3), 9, 0.7, dtype, t=t)[0] == 0


def test_three_dimensions_and_views():
    x = ref.rows("normal", 4 * 6, 517, "bf16", 3)
    t = dev(x, "bf16").view(4, 6, 517)
    lp, H, stats, ids, top = kb.spec_logprobs(t, torch.zeros(4, 6, dtype=torch.int32, device="cuda"), 3)
    assert lp.shape == H.shape == (4, 6) and stats.shape == (4, 6, 2) and ids.shape == top.shape == (4, 6, 3)
    want = ref.score(x, np.zeros(24), 3, 1.0)
    near(lp.reshape(-1), want[0], 1e-5, 1e-6, "logprob")
    assert np.array_equal(ids.cpu().numpy().reshape(24, 3), want[3])
    near(kb.spec_logprobs(t[:, 2], None, 0)[2], want[2].reshape(4, 6, 2)[:, 2], 1e-5, 1e-6, "one row of each")
    near(kb.spec_logprobs(t[1], None, 0)[2], want[2].reshape(4, 6, 2)[1], 1e-5, 1e-6, "one session")
    near(kb.spec_logprobs(t.view(24, 517)[::3], None, 0)[2], want[2][::3], 1e-5, 1e-6, "every third row")
    for bad in (t[..., ::2], t.transpose(1, 2), t[:, 1:4], t[0, :1].expand(3, 517)):
        with pytest.raises(ValueError):
            kb.spec_logprobs(bad, None, 0)


def test_offsets_past_32_bits():
    V, ld = 1001, 2**30 + 24
    buf = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    t = buf.as_strided((3, V), (ld, 1))
    x = ref.rows("normal", 3, V, "bf16", 1)
    t.copy_(dev(x, "bf16"))
    tok = tokens_for(3, V, 3)
    _, out = check(x, tok, 5, 1.0, "bf16", t=t)
    g = torch.ones(3, device="cuda")
    got = kb.spec_logprobs_backward(t, to_dev(tok.astype(np.int32)), out[2], grad_logprob=g, dlogits=t)
    want = ref.score_grad(x, tok, np.ones(3), None, 1.0)
    near(got.float(), want, 1e-6, 2.0**-8, "gradient in place")


def test_no_rows_and_repeatability():
    e = kb.spec_logprobs(torch.empty(0, 100, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), 4)
    assert e[0].shape == (0,) and e[3].shape == (0, 4)
    x = ref.rows("two_values", 40, 33001, "bf16", 2)
    t = dev(x, "bf16")
    a = kb.spec_logprobs(t, torch.zeros(40, dtype=torch.int32, device="cuda"), 50)
    b = kb.spec_logprobs(t, torch.zeros(40, dtype=torch.int32, device="cuda"), 50)
    for p, q in zip(a, b):
        assert torch.equal(p.view(torch.int32), q.view(torch.int32))


def test_own_stream_and_graph():
    x1, x2 = (ref.rows("normal", 8, 32768, "bf16", s) for s in (1, 2))
    s = torch.cuda.Stream()
    tok = to_dev(tokens_for(8, 32768, 3).astype(np.int32))
    t = dev(x1, "bf16")
    s.wait_stream(torch.cuda.current_stream())
    plan = kb.LogprobsPlan(t, tok, 20, stream=s)
    g = torch.cuda.CUDAGraph()
    plan()
    s.synchronize()
    with torch.cuda.graph(g, stream=s):
        plan()
    for x in (x1, x2):
        with torch.cuda.stream(s):
            t.copy_(dev(x, "bf16"))
            g.replay()
        s.synchronize()
        want = ref.score(x, tok.cpu().numpy(), 20, 1.0)
        assert np.array_equal(plan.out[3].cpu().numpy(), want[3])
        near(plan.out[0], want[0], 1e-5, 1e-6, "logprob")


# ---------------------------------------------------------------------------
# backward.  An element is scale * p_i * (...): relative error of p as above (4e-5 covers
# 62 u + 4 u + 525 u), and ln S's own error (1e-5 at most) is common to the row; bf16
# results add half a unit in the last place, 2^-9 (2^-8 allowed).
# ---------------------------------------------------------------------------
def grad_near(got, want, size, dtype, what):
    got = got.double().cpu().numpy()
    tol = 5e-5 * size + 1e-30 + (2.0**-8 * np.abs(want) if dtype == "bf16" else 0.0)
    with np.errstate(invalid="ignore"):
        ok = (np.isnan(got) & np.isnan(want)) | (np.abs(got - want) <= tol)
    assert ok.all(), f"{what}: {np.argwhere(~ok)[:4].tolist()} got {got[~ok][:4]} want {want[~ok][:4]}"


def sizes_of(x, tokens, g, h, tau):
    """|g| (1{i=t} + p) + |h| p (|ln p| + H), over tau: what the gradient's rounding is relative to."""
    N, V = x.shape
    out = np.zeros((N, V))
    for n in range(N):
        p, lp = ref.probs(x[n], tau)
        lp = np.where(p > 0, lp, 0.0)
        H = -(p * lp).sum()
        out[n] = abs(0 if g is None else g[n]) * p + abs(0 if h is None else h[n]) * p * (np.abs(lp) + H)
        if tokens is not None and 0 <= tokens[n] < V and g is not None:
            out[n, tokens[n]] += abs(g[n])
    return out / tau


def check_grad(x, tokens, tau, dtype, with_g=True, with_h=True, kind="", seed=1):
    N, V = x.shape
    rng = np.random.default_rng(seed)
    g = rng.standard_normal(N).astype(np.float32) if with_g else None
    h = rng.standard_normal(N).astype(np.float32) if with_h else None
    t, tok = dev(x, dtype), to_dev(np.asarray(tokens, np.int32))
    _, H, stats, _, _ = kb.spec_logprobs(t, tok, 0, tau)
    got = kb.spec_logprobs_backward(t, tok, stats, H, None if g is None else to_dev(g), None if h is None else to_dev(h),
                                    tau)
    want = ref.score_grad(x, tokens, g, h, tau)
    grad_near(got, want, sizes_of(x, tokens, g, h, tau), dtype, f"gradient {kind}")
    keep = t.clone()
    inplace = kb.spec_logprobs_backward(t, tok, stats, H, None if g is None else to_dev(g),
                                        None if h is None else to_dev(h), tau, dlogits=t)
    assert inplace.data_ptr() == t.data_ptr() and torch.equal(inplace.view(torch.uint8), got.view(torch.uint8))
    assert keep.shape == t.shape


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(1, 1), (3, 2), (5, 37), (4, 1001), (2, 4099), (3, 32768), (2, 100003), (400, 513),
                                 (1, 600011)])
def test_backward_sizes(N, V, dtype):
    check_grad(ref.rows("peaked", N, V, dtype, N + V), tokens_for(N, V, 5), 0.7, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [k for k in ref.KINDS if k != "huge"])
def test_backward_kinds_of_rows(kind, dtype):
    x = ref.rows(kind, 3, 2050, dtype, 4)
    check_grad(x, tokens_for(3, 2050, 6), 1.0, dtype, kind=kind)


@pytest.mark.parametrize("with_g,with_h", [(True, False), (False, True)])
def test_backward_one_gradient_alone(with_g, with_h):
    x = ref.rows("normal", 4, 999, "f32", 4)
    check_grad(x, [5, -1, 998, 0], 2.0, "f32", with_g, with_h)


def test_backward_of_rows_left_out_and_bad_rows():
    x = ref.rows("normal", 4, 301, "f32", 3)
    x[1, 7] = np.nan
    x[2, 9] = np.nan
    t = dev(x, "f32")
    tok = to_dev(np.array([3, 4, 5, -1], np.int32))
    _, H, stats, _, _ = kb.spec_logprobs(t, tok, 0)
    g = to_dev(np.array([1.0, 0.0, 1.0, 1.0], np.float32))
    got = kb.spec_logprobs_backward(t, tok, stats, H, grad_logprob=g).cpu().numpy()
    assert np.isfinite(got[0]).all() and (got[1] == 0).all() and np.isnan(got[2]).all() and (got[3] == 0).all()


def test_backward_writes_its_rows_alone():
    N, V, ld = 4, 1001, 1010
    x = ref.rows("normal", N, V, "bf16", 12)
    buf = torch.full((N * ld + 3,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[3:].view(N, ld)[:, :V]
    tok = tokens_for(N, V, 1)
    t, td = dev(x, "bf16"), to_dev(tok.astype(np.int32))
    stats = kb.spec_logprobs(t, td, 0)[2]
    g = torch.ones(N, device="cuda")
    kb.spec_logprobs_backward(t, td, stats, grad_logprob=g, dlogits=out)
    grad_near(out.float(), ref.score_grad(x, tok, np.ones(N), None, 1.0),
              sizes_of(x, tok, np.ones(N), None, 1.0), "bf16", "strided gradient")
    assert (buf[:3] == 7).all() and (buf[3:].view(N, ld)[:, V:] == 7).all()
    with pytest.raises(kb.KdaError):  # overlapping rows that are not the logits themselves
        kb.spec_logprobs_backward(t.view(-1)[:2 * V].view(2, V), td[:2], stats[:2], grad_logprob=g[:2],
                                  dlogits=t.view(-1)[1:1 + 2 * V].view(2, V))


def test_backward_against_differences():
    """Central differences of the forward call, h = 2^-5 in every coordinate: truncation at most
    h^2/6 |f'''| with third derivatives of log p and H up to about 2 and 8, 1.4e-3; the
    forward's rounding 2e-5 / h = 7e-4 at most."""
    V, h = 37, 2.0**-5
    x = ref.rows("peaked", 1, V, "f32", 21)
    tok, eye = 4, np.eye(V, dtype=np.float32)
    both = np.concatenate([x + h * eye, x - h * eye]).astype(np.float32)
    t = torch.full((2 * V,), tok, dtype=torch.int32, device="cuda")
    lp, H, _, _, _ = kb.spec_logprobs(dev(both, "f32"), t, 0)
    one = dev(x, "f32")
    _, H0, stats, _, _ = kb.spec_logprobs(one, t[:1], 0)
    a, b = 0.8, -0.6
    f = (a * lp + b * H).double().cpu().numpy()
    diff = (f[:V] - f[V:]) / (2 * h)
    got = kb.spec_logprobs_backward(one, t[:1], stats, H0, torch.tensor([a], device="cuda"),
                                    torch.tensor([b], device="cuda"))
    assert np.abs(got.double().cpu().numpy()[0] - diff).max() < 2.5e-3


# ---------------------------------------------------------------------------
# many long rows.  The 64-bit values are formed for some of the rows.
# ---------------------------------------------------------------------------
def some(N):
    return sorted({0, 1, N // 3, N // 2, N - 2, N - 1})


def check_some(x, tokens, K, tau, dtype, t=None):
    t = dev(x, dtype) if t is None else t
    rows = some(x.shape[0])
    out = kb.spec_logprobs(t, to_dev(np.asarray(tokens, np.int32)), K, tau)
    lp, H, stats, ids, top = (o[rows] for o in out)
    want = ref.score(x[rows], np.asarray(tokens)[rows], K, tau)
    assert np.array_equal(ids.cpu().numpy(), want[3])
    near(lp, want[0], 1e-5, 4 * 2.0**-24, "logprob")
    near(H, want[1], 2e-5, 1e-6, "entropy")
    near(stats[:, 1], want[2][:, 1], 1e-5, 4 * 2.0**-24, "ln S")
    near(top, want[4], 1e-5, 4 * 2.0**-24, "top_logprobs")
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K", [(153, 16384, 20), (160, 16391, 128), (1300, 8192, 1), (3000, 8193, 7),
                                   (700, 40001, 0), (200, 131072, 64), (170, 300007, 33)])
def test_many_long_rows(N, V, K, dtype):
    x = ref.rows("peaked", N, V, dtype, N + K)
    check_some(x, tokens_for(N, V, 3), K, 0.7, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [k for k in ref.KINDS if k != "normal"])
def test_many_long_rows_of_kinds(kind, dtype):
    x = ref.rows(kind, 180, 16391, dtype, 7)
    for n in (1, 90, 179):  # beside rows of another kind
        x[n] = ref.rows("normal", 1, 16391, dtype, n)[0]
    check_some(x, tokens_for(180, 16391, 4), 50, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_long_rows_with_bad_rows_and_strides(dtype):
    N, V, ld, off = 200, 16385, 16411, 3
    buf = torch.full((off + N * ld,), float("nan"), dtype=DT[dtype], device="cuda")
    t = buf[off:].view(N, ld)[:, :V]
    x = ref.rows("some_masked", N, V, dtype, 7)
    x[N // 3, V - 1] = np.nan
    x[1, 0] = np.inf
    t.copy_(dev(x, dtype))
    out = check_some(x, tokens_for(N, V, 4), 5, 1.0, dtype, t=t)
    bad = torch.isnan(out[0]).nonzero()[:, 0].tolist()
    assert bad == [1, N // 3]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_long_rows_give_what_few_give(dtype):
    """The kernel that is chosen for the number of rows changes no alternative and no more than
    the last places of the sums."""
    x = ref.rows("normal", 400, 20011, dtype, 7)
    t, tok = dev(x, dtype), to_dev(tokens_for(400, 20011, 4).astype(np.int32))
    many = kb.spec_logprobs(t, tok, 30)
    few = kb.spec_logprobs(t[100:110], tok[100:110], 30)
    assert torch.equal(many[3][100:110], few[3])
    for a, b in zip(many, few):
        assert torch.allclose(a[100:110].float(), b.float(), atol=2e-6, rtol=1e-6)
    again = kb.spec_logprobs(t, tok, 30)
    for a, b in zip(many, again):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 19, 20, 38, 39, 304, 305])
@pytest.mark.parametrize("V,K", [(24576, 20), (24584, 128), (12289, 33), (65535, 5), (770, 16), (1281, 17)])
def test_around_every_choice_of_kernel(N, V, K, dtype):
    """Rows, lengths and numbers of alternatives on both sides of where the launch changes."""
    if N * V > 8e6:
        N = N % 100 + 1
    x = ref.rows("peaked", N, V, dtype, N + V)
    check_some(x, tokens_for(N, V, 3), K, 1.0, dtype) if N > 2 else check(x, tokens_for(N, V, 3), K, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("K", [16, 17, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("V", [40, 130, 257, 511, 1000, 1100, 2100])
def test_short_rows_with_many_alternatives(V, K, dtype):
    for kind in ("normal", "two_values"):
        for N in (3, 310):
            x = ref.rows(kind, N, V, dtype, V + K)
            check_some(x, tokens_for(N, V, 3), K, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [2, 30, 400])
@pytest.mark.parametrize("V", [20000, 150001])
def test_large_logits_in_the_vectors_of_few_threads(V, N, dtype):
    """More logits than a list holds, above all others, repeat at the distance at which threads
    take vectors: no threshold from the threads' maxima tells them apart."""
    if N * V > 2e7:
        N = 40
    i = np.arange(V)
    row = np.where(i % 512 < 96, 8.0 + (i % 6007) * 2.0**-10, (i % 13) * 0.25).astype(np.float32)
    x = ref.typed(np.tile(row, (N, 1)), dtype)
    check_some(x, tokens_for(N, V, 3), 20, 1.0, dtype) if N > 2 else check(x, tokens_for(N, V, 3), 20, 1.0, dtype)


def test_calls_from_several_host_threads():
    """Calls of different shapes from several threads, each on a stream of its own."""
    import threading
    shapes = [(400, 33000, 20), (400, 9000, 20), (3, 33000, 5), (400, 100, 5)]
    xs = [ref.rows("normal", N, V, "bf16", N + V) for N, V, _ in shapes]
    ts = [dev(x, "bf16") for x in xs]
    ones = torch.ones(400, device="cuda")
    torch.cuda.synchronize()
    got, wrong = {}, []

    def work(j):
        try:
            N, V, K = shapes[j]
            s = torch.cuda.Stream()
            for _ in range(20):
                out = kb.spec_logprobs(ts[j], None, K, stream=s)
                d = kb.spec_logprobs_backward(ts[j], None, out[2], out[1],
                                              grad_entropy=ones[:N], stream=s)
            s.synchronize()
            got[j] = (out, d)
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    for j, (N, V, K) in enumerate(shapes):
        want = ref.score(xs[j][:2], None, K, 1.0)
        assert np.array_equal(got[j][0][3][:2].cpu().numpy(), want[3])
        near(got[j][0][2][:2], want[2], 1e-5, 1e-6, "stats")
        assert torch.isfinite(got[j][1].float()).all()


def test_the_longest_row():
    """2^30 logits: 0 but for three, so that every result can be written down."""
    V = 2**30
    x = torch.zeros((1, V), dtype=torch.bfloat16, device="cuda")
    at = [V - 1, 5, V // 2 + 3]
    x[0, at] = torch.tensor([20.0, 22.0, 21.0], dtype=torch.bfloat16, device="cuda")
    tok = torch.tensor([V - 1], dtype=torch.int32, device="cuda")
    lp, H, stats, ids, top = kb.spec_logprobs(x, tok, 4)
    z = np.array([20.0, 22.0, 21.0])
    S = (V - 3) * np.exp(-22.0) + np.exp(z - 22.0).sum()
    lnS = np.log(S)
    assert ids[0].tolist() == [5, V // 2 + 3, V - 1, 0]
    # 2^30 equal terms: a lane adds 2^19 of them or so, in sums of 32
    near(stats, np.array([[22.0, lnS]]), 1e-3, 0.0, "stats")
    near(lp, np.array([-2.0 - lnS]), 1e-3, 0.0, "logprob")
    want = -((V - 3) * np.exp(-22.0 - lnS) * (-22.0 - lnS) + (np.exp(z - 22.0 - lnS) * (z - 22.0 - lnS)).sum())
    near(H, np.array([want]), 2e-2, 0.0, "entropy")
    kb.spec_logprobs_backward(x, tok, stats, grad_logprob=torch.ones(1, device="cuda"), dlogits=x)
    p = np.exp(z - 22.0 - lnS)
    got = x[0, at].float().cpu().numpy()
    assert np.abs(got - np.array([1 - p[0], -p[1], -p[2]])).max() < 4e-3
    assert abs(float(x[0, 77]) + np.exp(-22.0 - lnS)) < 4e-12


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(3, 40, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    f = torch.zeros(3, device="cuda")
    stats = torch.zeros(3, 2, device="cuda")
    with pytest.raises(ValueError):
        kb.spec_logprobs(x, torch.zeros(4, **i32), 2)
    with pytest.raises(TypeError):
        kb.spec_logprobs(x, torch.zeros(3, dtype=torch.int64, device="cuda"), 2)
    with pytest.raises(ValueError):
        kb.spec_logprobs(x, torch.zeros(3, 2, **i32)[:, 0], 2)
    with pytest.raises(ValueError):
        kb.spec_logprobs(x, None, 129)
    with pytest.raises(ValueError):
        kb.spec_logprobs(x, None, 2, logprob_out=f)
    with pytest.raises(ValueError):
        kb.spec_logprobs(x, None, 2, top_ids_out=torch.zeros(3, 3, **i32))
    with pytest.raises(TypeError):
        kb.spec_logprobs(x.half(), None, 2)
    with pytest.raises(ValueError):
        kb.spec_logprobs(x[0], None, 2)
    with pytest.raises(ValueError):
        kb.spec_logprobs_backward(x, None, f, f, grad_entropy=f)
    with pytest.raises(ValueError):
        kb.spec_logprobs_backward(x, None, stats, f, grad_entropy=f, dlogits=x.bfloat16())
    with pytest.raises(kb.KdaError):
        kb.spec_logprobs_backward(x, None, stats, f)
    for tau in (0.0, -1.0, float("nan"), 1e6):
        with pytest.raises(kb.KdaError):
            kb.spec_logprobs(x, None, 2, temperature=tau)
    ids, v = torch.zeros(3, 2, **i32), torch.zeros(3, 2, device="cuda")
    for bad in (dict(ids=ids[0]), dict(ids=ids[:2]), dict(values=v[:, :1]), dict(weight=v), dict(values=None)):
        with pytest.raises((ValueError, TypeError)):
            kb.spec_distill_step(x, **{**dict(ids=ids, values=v), **bad})
    with pytest.raises(TypeError):
        kb.spec_distill(x, ids, v.half())
    with pytest.raises(kb.KdaError):
        kb.spec_distill(x, torch.zeros(3, 129, **i32), torch.zeros(3, 129, device="cuda"))
    with pytest.raises(kb.KdaError):
        kb.spec_distill(x, ids, v, kind=2)
