"""Scores and distillation where f32 ends: logits of the type's lowest and largest finite
values, temperatures from 1e-4 to 1e4, weights far from 1, teacher values that are no numbers.
The 64-bit values, brought into the range of f32 as each test says, are the reference.

Tolerances, derived before the first run (u = 2^-24).  A teacher's q: the argument
(v - top) / tau carries three roundings (of the difference, of 1 / tau and of the
product) of at most |d| = 20 each, 60 u; expf 4 u; a sum of at most 128 terms by lanes 7 u,
quotient 2 u: within 80 u, 5e-6 of itself (1e-5 allowed), and ln q within 1e-5 and 4 u of its
size.  ln p = (x - m) / tau - ln S: 1e-5 for ln S (derived in test_gpu_scores.py) and 4 u of the
size of the quotient.  A loss w tau^2 sum q (ln q - ln p) is then within
w tau^2 (2e-5 + 1e-5 sum q (|ln q| + |ln p|))."""
import numpy as np
import pytest
import torch

import score_ref as ref
from gpu_util import to_dev
from libs import ensure_built

from speculative_decode_verify_kda_gb300 import binding as kb

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FLT_MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def dev(x, dtype="f32"):
    return to_dev(np.asarray(x, np.float32)).to(DT[dtype])


def near(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    with np.errstate(invalid="ignore"):
        ok = (np.isnan(got) & np.isnan(want)) | (got == want) | (np.abs(got - want) <= tol)
    assert ok.all(), f"{what}: {np.argwhere(~ok)[:4].tolist()} got {got[~ok][:4]} want {want[~ok][:4]}"


def end_rows(kind, N, V, dtype, seed):
    """score_ref's rows, and rows whose logits lie at both ends of the type's range."""
    if kind != "both_ends":
        return ref.rows(kind, N, V, dtype, seed)
    top = np.random.default_rng(seed).random((N, V)) < 4.0 / V
    top[:, V // 2] = True
    return ref.typed(np.where(top, 3e38, ref.LOWEST[dtype]), dtype)


def spread(N, V, K, seed):
    """K ids a row, none twice."""
    rng = np.random.default_rng(seed)
    return np.stack([rng.permutation(V)[:K] for _ in range(N)]).astype(np.int32)


def loss_tolerance(x, ids, values, tau, weight, logprobs=False):
    q, lnq = ref.teacher(ids, values, x.shape[1], tau, logprobs)
    lp = np.stack([ref.probs(r, tau)[1][i] for r, i in zip(x, np.maximum(ids, 0))])
    with np.errstate(invalid="ignore"):
        size = np.where(q > 0, q * (np.abs(lnq) + np.abs(lp)), 0.0).sum(1)
        return np.abs(weight) * tau * tau * (2e-5 + 1e-5 * np.nan_to_num(size, posinf=0.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [1e-4, 0.5, 1.0, 2.0, 1e4])
@pytest.mark.parametrize("V", [37, 33001])
@pytest.mark.parametrize("kind", ["few_allowed_lowest", "all_lowest", "both_ends"])
def test_a_loss_at_the_ends_of_the_range(kind, V, tau, dtype):
    """Finite logits give the finite loss, or the end of the range that it passes, whatever the
    order in which its factors are taken; +inf is left to entries that the student masks."""
    tau = float(np.float32(tau))
    N, K = 7, 12
    x = end_rows(kind, N, V, dtype, 5)
    ids = spread(N, V, K, 3)
    values = (2 * tau * np.random.default_rng(4).standard_normal((N, K))).astype(np.float32)
    x[3, ids[3, 2]] = -np.inf
    w = np.array([1.0, 3.5, 1 / 64, 2.0, 1e-8, 0.75, 1e-30], np.float32)
    want, _, _, _, _ = ref.distill(x, ids, values, tau, w)
    assert np.isposinf(want[3]) and np.isfinite(np.delete(want, 3)).all()
    tol = loss_tolerance(x, ids, values, tau, w)
    held = np.where(np.isfinite(want), np.clip(want, -FLT_MAX, FLT_MAX), want)
    args = dev(x, dtype), to_dev(ids), dev(values)
    kw = {"weight": to_dev(w), "temperature": tau}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    near(kb.spec_distill(*args, dev_status=st, **kw)[0], held, tol, "loss")
    near(kb.spec_distill_step(*args, dev_status=st, **kw)[0], held, tol, "loss of the step")
    assert int(st) == 0


def test_a_loss_past_the_range_keeps_its_sign():
    """Weights may be negative; one that is infinite or no number, and an empty row, stay so."""
    x = ref.typed(np.full((6, 50), ref.LOWEST["f32"]), "f32")
    x[:, 7] = 1.0
    x[4] = -np.inf
    ids, values = np.tile(np.int32([[3, 9]]), (6, 1)), np.zeros((6, 2), np.float32)
    w = np.array([2.0, -2.0, np.inf, np.nan, 2.0, 1e-38], np.float32)
    loss = kb.spec_distill(dev(x), to_dev(ids), dev(values), weight=to_dev(w), temperature=2.0)[0].cpu().numpy()
    assert loss[0] == FLT_MAX and loss[1] == -FLT_MAX and np.isposinf(loss[2]) and np.isnan(loss[3])
    assert np.isposinf(loss[4])
    assert abs(loss[5] - 2 * 1e-38 * -ref.LOWEST["f32"]) <= 1e-5 * loss[5]


@pytest.mark.parametrize("vdtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [1e-4, 1e-3, 1e-2, 0.5, 1e4])
@pytest.mark.parametrize("offset", [0.0, 25.0, -1000.0])
def test_teacher_logits_of_a_common_offset(offset, tau, vdtype):
    """q depends on the differences of a row's values alone, at every temperature."""
    tau = float(np.float32(tau))
    N, V, K = 6, 3001, 20
    rng = np.random.default_rng(7)
    x = ref.rows("normal", N, V, "f32", 4)
    ids = spread(N, V, K, 3)
    values = ref.typed(offset + 3 * tau * rng.standard_normal((N, K)), vdtype)
    want, _, grad, P, D = ref.distill(x, ids, values, tau)
    tol = loss_tolerance(x, ids, values, tau, np.ones(N))
    gtol = tau * (1e-5 * D + 5e-5 * P + 1e-30)
    args = dev(x), to_dev(ids), dev(values, vdtype)
    loss, stats = kb.spec_distill(*args, temperature=tau)
    near(loss, want, tol, "loss")
    near(kb.spec_distill_backward(*args, stats, temperature=tau), grad, gtol, "gradient")
    loss, _, got = kb.spec_distill_step(*args, temperature=tau)
    near(loss, want, tol, "loss of the step")
    near(got, grad, gtol, "gradient of the step")


@pytest.mark.parametrize("vdtype", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [1e-4, 0.5, 1.0, 1e4])
def test_finite_teacher_logits_are_numbers(tau, vdtype):
    """Values at the ends of their type's range: a mask of the lowest value leaves q = 0, a row of
    nothing else a flat q; no row is left out and none becomes NaN."""
    tau = float(np.float32(tau))
    N, V, K = 4, 500, 6
    low = ref.LOWEST[vdtype]
    x = ref.rows("normal", N, V, "f32", 4)
    ids = spread(N, V, K, 3)
    values = ref.typed(np.random.default_rng(2).standard_normal((N, K)), vdtype)
    values[0, 3:] = low
    values[1] = low
    values[2, :3], values[2, 3:] = -low, low
    values[3] = -low
    want, _, grad, P, D = ref.distill(x, ids, values, tau)
    assert np.isfinite(want).all() and np.allclose(D.sum(1), 1.0)
    tol = loss_tolerance(x, ids, values, tau, np.ones(N))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dev(x), to_dev(ids), dev(values, vdtype)
    near(kb.spec_distill(*args, temperature=tau, dev_status=st)[0], want, tol, "loss")
    loss, _, got = kb.spec_distill_step(*args, temperature=tau, dev_status=st)
    near(loss, want, tol, "loss of the step")
    near(got, grad, tau * (1e-5 * D + 5e-5 * P + 1e-30), "gradient of the step")
    assert int(st) == 0


@pytest.mark.parametrize("kind", [kb.TEACHER_LOGITS, kb.TEACHER_LOGPROBS])
@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_teacher_rows_that_are_no_numbers(what, kind):
    """A NaN or +inf among a row's values: NaN for the row's loss and gradient, and the status
    says so, in every call; the other rows are as without it."""
    x = ref.rows("normal", 4, 500, "f32", 4)
    ids = spread(4, 500, 7, 5)
    values = -np.random.default_rng(6).random((4, 7)).astype(np.float32) - 1.0
    args = dev(x), to_dev(ids)
    good = kb.spec_distill(*args, dev(values), kind=kind)[0], kb.spec_distill_step(*args, dev(values), kind=kind)[0]
    values[1, 3] = what
    values[2, 2], ids[2, 2] = what, -1  # no entry: its value is not looked at
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dev(x), to_dev(ids), dev(values)
    loss, stats = kb.spec_distill(*args, kind=kind, dev_status=st)
    assert int(st) == kb.ST_NAN
    grad = kb.spec_distill_backward(*args, stats, kind=kind)
    st.zero_()
    loss2, _, grad2 = kb.spec_distill_step(*args, kind=kind, dev_status=st)
    assert int(st) == kb.ST_NAN
    for a, d, before in ((loss, grad, good[0]), (loss2, grad2, good[1])):
        assert torch.isnan(a[1]) and torch.isnan(d[1]).all()
        assert torch.isfinite(a[[0, 2, 3]]).all() and torch.isfinite(d[[0, 2, 3]]).all()
        assert torch.equal(a[[0, 3]], before[[0, 3]])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0, 1e4])
@pytest.mark.parametrize("N,V,K", [(5, 37, 37), (5, 3001, 128), (2, 33001, 20), (330, 33001, 9)])
@pytest.mark.parametrize("kind", ["both_ends", "few_allowed_lowest", "all_lowest"])
def test_log_probabilities_at_both_ends_of_the_range(kind, N, V, K, tau, dtype):
    """A log-probability that f32 holds is given, however far its logit lies from the row's
    maximum; one past the range is -inf, as in rounding."""
    tau = float(np.float32(tau))
    x = end_rows(kind, N, V, dtype, 5)
    tokens = np.random.default_rng(1).integers(0, V, N).astype(np.int32)
    rows = [0, 1, N // 2, N - 1]
    want = ref.score(x[rows], tokens[rows], K, tau)
    with np.errstate(over="ignore"):
        held = [np.asarray(a, np.float64).astype(np.float32).astype(np.float64) for a in want]
    lp, H, stats, ids, top = kb.spec_logprobs(dev(x, dtype), to_dev(tokens), K, tau)
    u = 2.0**-24
    assert np.array_equal(ids[rows].cpu().numpy(), want[3])
    with np.errstate(invalid="ignore"):
        near(lp[rows], held[0], 1e-5 + 4 * u * np.abs(want[0]), "logprob")
        near(top[rows], held[4], 1e-5 + 4 * u * np.abs(want[4]), "top_logprobs")
    near(H[rows], want[1], 2e-5 + 1e-6 * np.abs(want[1]), "entropy")
    near(stats[rows][:, 1], want[2][:, 1], 1e-5 + 4 * u * np.abs(want[2][:, 1]), "ln S")
