"""spec_distill, spec_distill_backward and spec_distill_step on the GPU against 64-bit
definitions.  Tolerances as in test_gpu_scores.py, derived there: log-probabilities within
1e-5 and 4 u of the logit, weights within 5e-5 of themselves; a loss is tau^2 w times a
q-weighted mean of such log-probabilities and of ln q (both within 1e-5, u of their size)."""
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


def dev(x, dtype="f32"):
    return to_dev(np.asarray(x, np.float32)).to(DT[dtype])


def entries(N, V, K, seed, kind="distinct"):
    rng = np.random.default_rng(seed)
    if kind == "repeated":
        ids = rng.integers(0, max(1, min(V, K // 2 + 1)), (N, K))
    else:
        ids = np.stack([rng.permutation(V)[:K] if V >= K else rng.integers(0, V, K) for _ in range(N)])
    if kind == "short":
        ids[rng.random((N, K)) < 0.4] = -1
        ids[0] = -1
    values = -np.cumsum(rng.random((N, K)), 1) + 3 * rng.standard_normal((N, 1))
    return ids.astype(np.int32), values.astype(np.float32)


def same_or_near(got, want, tol, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    with np.errstate(invalid="ignore"):
        ok = (np.isnan(got) & np.isnan(want)) | (got == want) | (np.abs(got - want) <= tol)
    assert ok.all(), f"{what}: {np.argwhere(~ok)[:4].tolist()} got {got[~ok][:4]} want {want[~ok][:4]}"


def check(x, ids, values, tau, dtype, weight=None, g=None, logprobs=False, vdtype="f32", t=None, status=0):
    values = ref.typed(values, vdtype)
    loss, stats, grad, P, D = ref.distill(x, ids, values, tau, weight, g, logprobs)
    N = x.shape[0]
    w = np.ones(N) if weight is None else np.abs(weight)
    gg = np.ones(N) if g is None else np.abs(g)
    kw = {"weight": None if weight is None else to_dev(weight), "temperature": tau,
          "kind": kb.TEACHER_LOGPROBS if logprobs else kb.TEACHER_LOGITS}
    gd = None if g is None else to_dev(g)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = dev(x, dtype) if t is None else t
    i, v = to_dev(ids), dev(values, vdtype)
    with np.errstate(invalid="ignore"):
        # |loss| <= sum of q |ln q| + q |lp|: relative to the sizes that are subtracted
        size = w * tau * tau * (2e-5 + 1e-6 * np.nan_to_num(np.abs(stats[:, 0]), posinf=0, neginf=0)) + 1e-5 * np.abs(loss)
        ltol = 1e-5 + 4 * 2.0**-24 * np.abs(stats)
        gtol = (gg * w * tau)[:, None] * (5e-5 * (P + D) + 1e-30)
    if dtype == "bf16":
        gtol = gtol + 2.0**-8 * np.abs(grad)
    l1, z1 = kb.spec_distill(t, i, v, dev_status=st, **kw)
    same_or_near(l1, loss, size, "loss")
    same_or_near(z1, stats, ltol, "stats")
    assert int(st.item()) == status
    d1 = kb.spec_distill_backward(t, i, v, z1, grad_loss=gd, dev_status=st, **kw)
    same_or_near(d1, grad, gtol, "gradient")
    l2, z2, d2 = kb.spec_distill_step(t, i, v, grad_loss=gd, dev_status=st, **kw)
    same_or_near(l2, loss, size, "loss of the step")
    same_or_near(z2, stats, ltol, "stats of the step")
    same_or_near(d2, grad, gtol, "gradient of the step")
    assert int(st.item()) == status
    u = t.clone()
    kb.spec_distill_backward(u, i, v, z1, grad_loss=gd, dlogits=u, **kw)
    assert torch.equal(u.view(torch.uint8), d1.view(torch.uint8)), "in place"
    u = t.clone()
    kb.spec_distill_step(u, i, v, grad_loss=gd, dlogits=u, **kw)
    assert torch.equal(u.view(torch.uint8), d2.view(torch.uint8)), "step in place"
    return l2, z2, d2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K", [(1, 1, 1), (3, 2, 2), (5, 32, 5), (5, 37, 37), (4, 257, 128), (15, 1001, 8),
                                   (70, 1000, 3), (2, 2049, 32), (2, 4099, 128), (3, 16384, 33), (1, 32768, 5),
                                   (8, 32768, 20), (2, 50021, 64), (2, 100003, 1), (700, 777, 5), (37, 131072, 64),
                                   (330, 33000, 20), (2, 262147, 128), (1, 600011, 9)])
def test_sizes(N, V, K, dtype):
    rng = np.random.default_rng(N + V)
    x = ref.rows("peaked", N, V, dtype, 3 * N + V)
    ids, values = entries(N, V, K, V)
    check(x, ids, values, 1.0, dtype, (0.5 + rng.random(N)).astype(np.float32),
          rng.standard_normal(N).astype(np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [37, 2050, 33001])
@pytest.mark.parametrize("kind", [k for k in ref.KINDS if k != "huge"])
def test_kinds_of_rows(kind, V, dtype):
    x = ref.rows(kind, 4, V, dtype, 4)
    ids, values = entries(4, V, 12, 9)
    check(x, ids, values, 1.0, dtype)


@pytest.mark.parametrize("kind", ["short", "repeated"])
@pytest.mark.parametrize("logprobs", [False, True])
@pytest.mark.parametrize("vdtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_entries(kind, logprobs, vdtype, tau):
    x = ref.rows("normal", 9, 3001, "bf16", 4)
    ids, values = entries(9, 3001, 40, 2, kind)
    if logprobs:
        values = values - 6.0
    check(x, ids, values, tau, "bf16", logprobs=logprobs, vdtype=vdtype)


def test_masked_values_and_ids_out_of_range():
    x = ref.rows("normal", 5, 777, "f32", 4)
    ids, values = entries(5, 777, 6, 5)
    values[1, :3] = -np.inf
    values[2, :] = -np.inf  # no entry with a probability: no loss
    check(x, ids, values, 1.0, "f32")
    ids[3, 2] = 777
    ids[4, 0] = 2**31 - 1
    check(x, ids, values, 1.0, "f32", status=kb.ST_BADTOKEN)


def test_rows_of_weight_zero_are_not_read():
    x = ref.rows("normal", 6, 5001, "bf16", 4)
    x[1] = np.nan
    x[4, 17] = np.nan
    ids, values = entries(6, 5001, 10, 5)
    values[1] = np.nan
    w = np.array([1, 0, 0.5, 2, 0, 1], np.float32)
    loss, stats, grad = check(x, ids, values, 2.0, "bf16", w)
    assert (loss[[1, 4]] == 0).all() and (stats[[1, 4]] == 0).all() and (grad[[1, 4]] == 0).all()
    g = np.array([1, 1, 0, 1, 1, -2], np.float32)
    check(x, ids, values, 2.0, "bf16", w, g)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [37, 1001, 40000])
def test_bad_rows_are_reported(V, dtype):
    x = ref.rows("normal", 5, V, dtype, 4)
    x[0, V - 1] = np.nan
    x[3, 0] = np.inf
    ids, values = entries(5, V, 7, 5)
    check(x, ids, values, 1.0, dtype, status=kb.ST_NAN)


@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_teacher_values_that_are_no_numbers(what):
    x = ref.rows("normal", 3, 500, "f32", 4)
    ids, values = entries(3, 500, 7, 5)
    values[1, 3] = what
    loss, stats, grad = kb.spec_distill_step(dev(x), to_dev(ids), to_dev(values))
    loss, grad = loss.cpu().numpy(), grad.cpu().numpy()
    assert np.isnan(loss[1]) and np.isnan(grad[1]).all()
    assert np.isfinite(loss[[0, 2]]).all() and np.isfinite(grad[[0, 2]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,ld,off,ldg,goff", [(1001, 1001, 1, 1001, 0), (1001, 1003, 3, 1005, 2),
                                               (4096, 4104, 8, 4096, 0), (33000, 33001, 1, 33007, 5)])
def test_strides_of_rows_and_gradients(V, ld, off, ldg, goff, dtype):
    N = 4
    x = ref.rows("normal", N, V, dtype, V)
    src = torch.full((off + N * ld,), float("nan"), dtype=DT[dtype], device="cuda")
    t = src[off:].view(N, ld)[:, :V]
    t.copy_(dev(x, dtype))
    ids, values = entries(N, V, 9, 3)
    _, _, want, P, D = ref.distill(x, ids, values, 1.0)
    tol = 5e-5 * (P + D) + 1e-30 + (2.0**-8 * np.abs(want) if dtype == "bf16" else 0.0)
    for step in (True, False):
        dst = torch.full((goff + N * ldg + 8,), 7.0, dtype=DT[dtype], device="cuda")
        out = dst[goff:goff + N * ldg].view(N, ldg)[:, :V]
        if step:
            kb.spec_distill_step(t, to_dev(ids), to_dev(values), dlogits=out)
        else:
            _, stats = kb.spec_distill(t, to_dev(ids), to_dev(values))
            kb.spec_distill_backward(t, to_dev(ids), to_dev(values), stats, dlogits=out)
        same_or_near(out, want, tol, "strided gradient")
        rest = torch.ones_like(dst, dtype=torch.bool)
        rest[goff:goff + N * ldg].view(N, ldg)[:, :V] = False
        assert (dst[rest] == 7).all(), "written outside its rows"


def test_offsets_past_32_bits():
    V, ld = 1001, 2**30 + 24
    buf = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda")
    t = buf.as_strided((3, V), (ld, 1))
    x = ref.rows("normal", 3, V, "bf16", 1)
    t.copy_(dev(x, "bf16"))
    ids, values = entries(3, V, 9, 3)
    loss, stats, grad, P, D = ref.distill(x, ids, values, 1.0)
    l1, z1, d1 = kb.spec_distill_step(t, to_dev(ids), to_dev(values), dlogits=t)
    same_or_near(d1, grad, 5e-5 * (P + D) + 2.0**-8 * np.abs(grad), "gradient")
    same_or_near(l1, loss, 3e-5 + 1e-5 * np.abs(loss), "loss")


def test_repeatability_streams_and_graph():
    x = ref.rows("normal", 33, 33001, "bf16", 2)
    ids, values = entries(33, 33001, 20, 3, "repeated")
    t, i, v = dev(x, "bf16"), to_dev(ids), to_dev(values)
    a = kb.spec_distill_step(t, i, v)
    b = kb.spec_distill_step(t, i, v)
    for p, q in zip(a, b):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan = kb.DistillStepPlan(t, i, v, stream=s)
    plan()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        plan()
    for o in plan.out:
        o.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(a, plan.out):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_no_rows():
    e = kb.spec_distill_step(torch.empty(0, 9, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                             torch.empty(0, 3, device="cuda"))
    assert e[0].shape == (0,) and e[2].shape == (0, 9)


def test_gradient_against_differences():
    """Central differences of the loss call, h = 2^-5 in every coordinate: the truncation is at
    most h^2/6 |f'''| <= 1e-3 tau^-1 (third derivatives of ln S are at most 1), the loss's
    rounding 2e-5 / h at most."""
    V, h, tau = 37, 2.0**-5, 1.5
    x = ref.rows("peaked", 1, V, "f32", 21)
    eye = np.eye(V, dtype=np.float32)
    both = np.concatenate([x + h * eye, x - h * eye]).astype(np.float32)
    ids, values = entries(1, V, 9, 3, "repeated")
    many = lambda a: to_dev(np.repeat(a, 2 * V, 0))  # noqa: E731
    loss, _ = kb.spec_distill(dev(both), many(ids), many(values), temperature=tau)
    f = loss.double().cpu().numpy()
    diff = (f[:V] - f[V:]) / (2 * h)
    got = kb.spec_distill_step(dev(x), to_dev(ids), to_dev(values), temperature=tau)[2]
    assert np.abs(got.double().cpu().numpy()[0] - diff).max() < 2e-3


def test_scores_are_a_teacher():
    """The alternatives of spec_logprobs are a teacher's entries: against its own row, as
    log-probabilities, the loss is 0 and the gradient is what the entries leave out."""
    x = ref.rows("peaked", 6, 2001, "f32", 3)
    t = dev(x)
    _, _, _, ids, top = kb.spec_logprobs(t, None, 128, 2.0)
    loss, _, grad = kb.spec_distill_step(t, ids, top, kind=kb.TEACHER_LOGPROBS, temperature=2.0)
    assert loss.abs().max().item() < 4 * 4e-5
    at = grad.gather(1, ids.long())
    p = top.exp()
    assert torch.allclose(at, 2.0 * p * (p.sum(1, keepdim=True) - 1), atol=1e-5)


# ---------------------------------------------------------------------------
# many long rows.  The 64-bit values are formed for some of the rows.
# ---------------------------------------------------------------------------
def copy_of(t):
    """The same values at the same place within a vector (whose sums are formed alike)."""
    whole = torch.empty(0, dtype=t.dtype, device=t.device).set_(t.untyped_storage()).clone()
    return whole.as_strided(t.shape, t.stride(), t.storage_offset())


def check_some(x, ids, values, tau, dtype, weight, g, t=None, which=None):
    N = x.shape[0]
    rows = sorted({0, 1, N // 3, N // 2, N - 2, N - 1}) if which is None else which
    w, gg = weight[rows], g[rows]
    loss, stats, grad, P, D = ref.distill(x[rows], ids[rows], values[rows], tau, w, gg)
    t = dev(x, dtype) if t is None else t
    kw = {"weight": to_dev(weight), "temperature": tau}
    i, v, gd = to_dev(ids), dev(values), to_dev(g)
    size = np.abs(w) * tau * tau * 4e-5 + 1e-5 * np.abs(loss)
    gtol = (np.abs(gg) * np.abs(w) * tau)[:, None] * (5e-5 * (P + D) + 1e-30)
    if dtype == "bf16":
        gtol = gtol + 2.0**-8 * np.abs(grad)
    l1, z1 = kb.spec_distill(t, i, v, **kw)
    same_or_near(l1[rows], loss, size, "loss")
    same_or_near(z1[rows][:, 1], stats[:, 1], 1e-5 + 1e-6 * np.abs(stats[:, 1]), "ln S")
    d1 = kb.spec_distill_backward(t, i, v, z1, grad_loss=gd, **kw)
    same_or_near(d1[rows], grad, gtol, "gradient")
    l2, z2, d2 = kb.spec_distill_step(t, i, v, grad_loss=gd, **kw)
    same_or_near(l2[rows], loss, size, "loss of the step")
    same_or_near(d2[rows], grad, gtol, "gradient of the step")
    # every row: the step and the two calls agree, a row's gradient sums to g w tau (Q - Q) = 0
    same = (l1 == l2) | (torch.isnan(l1) & torch.isnan(l2)) | ((l1 - l2).abs() <= 1e-6 + 1e-5 * l1.abs())
    assert same.all()
    a, b = d1.float(), d2.float()
    assert ((a == b) | (torch.isnan(a) & torch.isnan(b)) | ((a - b).abs() <= 1e-7 + 0.01 * a.abs())).all()
    u = copy_of(t)
    kb.spec_distill_step(u, i, v, grad_loss=gd, dlogits=u, **kw)
    assert torch.equal(u.view(torch.uint8), d2.view(torch.uint8)), "step in place"
    u = copy_of(t)
    kb.spec_distill_backward(u, i, v, z1, grad_loss=gd, dlogits=u, **kw)
    assert torch.equal(u.view(torch.uint8), d1.view(torch.uint8)), "in place"
    return l2, z2, d2


def weights(N, seed):
    rng = np.random.default_rng(seed)
    w = (0.5 + rng.random(N)).astype(np.float32)
    w[15::16] = 0
    return w, rng.standard_normal(N).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K", [(153, 16384, 20), (160, 16391, 128), (500, 33000, 3), (1000, 16400, 64),
                                   (200, 131072, 64), (170, 300007, 33), (155, 600011, 5)])
def test_many_long_rows(N, V, K, dtype):
    """Shares that stay in one CTA, in clusters of two, four and eight, with and without whole
    vectors; every sixteenth row has no weight."""
    x = ref.rows("peaked", N, V, dtype, N + K)
    rng = np.random.default_rng(K)
    ids = ((rng.integers(0, V, (N, 1)) + np.arange(K) * rng.integers(1, V // K, (N, 1))) % V).astype(np.int32)
    values = (3 * rng.standard_normal((N, K))).astype(np.float32)
    w, g = weights(N, K)
    _, _, d = check_some(x, ids, values, 2.0, dtype, w, g)
    assert (d[15::16] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_are_read_twice(dtype):
    """Shares beyond what eight CTAs hold between the sum and the gradient."""
    N, V, K = 153, 1600011 // (2 if dtype == "f32" else 1), 16
    x = np.tile(ref.rows("peaked", 3, V, dtype, 1), (N // 3, 1))
    rng = np.random.default_rng(K)
    ids = rng.integers(0, V, (N, K)).astype(np.int32)
    values = (3 * rng.standard_normal((N, K))).astype(np.float32)
    w, g = weights(N, K)
    check_some(x, ids, values, 1.0, dtype, w, g, which=[0, 77, 152])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", [k for k in ref.KINDS if k not in ("huge", "normal")])
def test_many_long_rows_of_kinds(kind, dtype):
    N, V, K = 180, 16391, 12
    x = ref.rows(kind, N, V, dtype, 7)
    for n in (1, 90, 179):  # beside rows of another kind
        x[n] = ref.rows("normal", 1, V, dtype, n)[0]
    ids, values = entries(N, V, K, 9)
    ids[60], values[90] = -1, -np.inf  # rows without entries
    check_some(x, ids, values, 1.0, dtype, *weights(N, 3))


def test_many_long_rows_with_bad_rows_and_strides():
    N, V, ld, off = 200, 16385, 16411, 3
    x = ref.rows("normal", N, V, "bf16", 7)
    x[1, V - 1] = np.nan
    x[15] = np.nan  # of weight 0
    x[N // 3, 0] = np.inf
    buf = torch.full((off + N * ld,), float("nan"), dtype=torch.bfloat16, device="cuda")
    t = buf[off:].view(N, ld)[:, :V]
    t.copy_(dev(x, "bf16"))
    ids, values = entries(N, V, 9, 5, "repeated")
    w, g = weights(N, 3)
    loss, _, d = check_some(x, ids, values, 1.0, "bf16", w, g, t=t)
    bad = torch.isnan(loss).nonzero()[:, 0].tolist()
    assert bad == [1, N // 3] and (d[15] == 0).all()
    dst = torch.full((7 + N * ld + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = dst[7:7 + N * ld].view(N, ld)[:, :V]
    kb.spec_distill_step(t, to_dev(ids), to_dev(values), weight=to_dev(w), grad_loss=to_dev(g), dlogits=out)
    assert torch.equal(torch.nan_to_num(out.float(), 5.0), torch.nan_to_num(d.float(), 5.0))
    rest = torch.ones_like(dst, dtype=torch.bool)
    rest[7:7 + N * ld].view(N, ld)[:, :V] = False
    assert (dst[rest] == 7).all(), "written outside its rows"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 19, 38, 76, 77, 153, 305])
@pytest.mark.parametrize("V,K", [(257, 5), (3201, 33), (12288, 20), (23041, 64), (35840, 7), (35848, 128)])
def test_around_every_choice_of_kernel(N, V, K, dtype):
    """Rows and lengths on both sides of where the launch changes."""
    if N * V > 8e6:
        N = N % 100 + 1
    x = ref.rows("peaked", N, V, dtype, N + V)
    ids, values = entries(N, V, K, V, "repeated" if K == 33 else "short" if K == 20 else "distinct")
    w, g = weights(N, 3)
    check_some(x, ids, values, 1.0, dtype, w, g, which=sorted({0, N // 2, N - 1}))


def test_a_step_of_several_host_threads():
    """Held runs of different sizes are launched from several threads at once."""
    import threading
    shapes = [(200, 33000), (200, 60000), (200, 9000), (4, 33000)]
    data = []
    for N, V in shapes:
        x = ref.rows("normal", N, V, "bf16", N + V)
        ids, values = entries(N, V, 9, 4)
        data.append((x, ids, values, dev(x, "bf16"), to_dev(ids), to_dev(values)))
    torch.cuda.synchronize()
    got, wrong = {}, []

    def work(j):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got[j] = kb.spec_distill_step(*data[j][3:], stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    for j in range(len(shapes)):
        x, ids, values = (a[:2] for a in data[j][:3])
        loss, _, grad, P, D = ref.distill(x, ids, values, 1.0)
        same_or_near(got[j][0][:2], loss, 4e-5 + 1e-5 * np.abs(loss), "loss")
        same_or_near(got[j][2][:2].float(), grad, 5e-5 * (P + D) + 1e-30 + 2.0**-8 * np.abs(grad), "gradient")


def test_the_longest_row():
    """2^30 logits: 0 but for three, so that every result can be written down."""
    V = 2**30
    x = torch.zeros((1, V), dtype=torch.bfloat16, device="cuda")
    at = [V - 1, 5, V // 2 + 3]
    x[0, at] = torch.tensor([20.0, 22.0, 21.0], dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([[V - 1, 7]], dtype=torch.int32, device="cuda")
    values = torch.tensor([[0.0, 0.0]], device="cuda")
    z = np.array([20.0, 22.0, 21.0])
    lnS = np.log((V - 3) * np.exp(-22.0) + np.exp(z - 22.0).sum())
    loss, stats, grad = kb.spec_distill_step(x, ids, values)
    same_or_near(stats, np.array([[22.0, lnS]]), 1e-3, "stats")
    same_or_near(loss, np.array([np.log(0.5) - 0.5 * (-2.0 - lnS) - 0.5 * (-22.0 - lnS)]), 2e-3, "loss")
    p = np.exp(z - 22.0 - lnS)
    got = grad[0, at].float().cpu().numpy()
    assert np.abs(got - np.array([p[0] - 0.5, p[1], p[2]])).max() < 4e-3
    assert abs(float(grad[0, 7]) + 0.5) < 4e-3 and abs(float(grad[0, 8]) - np.exp(-22.0 - lnS)) < 4e-12
