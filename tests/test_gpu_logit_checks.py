"""Scores and distillation: what calls leave alone, gradients of every row, and how large the
errors are on the whole.

The other files bound each element by the worst case.  Here the root mean square over many
elements is bounded, which a result held in too few bits does not pass.  Derived before the
first run, u = 2^-24:
  ln S below 16: a term's exponent is rounded once below 16 in base 2, at most 5.5 u of the
    weight and averaged over the row's terms; exp2 4 u at most, which may be common; sums by
    tiles, groups, lanes and warps of 50 additions or so, 3 u as a random walk; log1p 2 u; the
    result's own rounding 4.6 u (half a unit of 16 u, uniform).  Together 9 u; 16 u allowed.
  ln p down to -32: the quotient and its subtraction add roundings of 4.6 u and 9 u: 14 u;
    24 u allowed.
  entropy: weights' errors of 4 u common and 3 u random, times exponents up to 10; its own
    rounding 4.6 u: 41 u; 64 u allowed.
  a gradient's p above 2^-32, relative to itself, f32: the exponent's rounding below 32 in base 2
    6.4 u, the difference's 6 u, ln S in base 2 5 u, exp2 4 u, ln S itself 9 u: 20 u at most;
    40 u allowed (temperature 1, at which 1 / temperature carries no rounding)."""
import threading

import numpy as np
import pytest
import torch

import score_ref as ref
from gpu_util import to_dev
from libs import ensure_built

from speculative_decode_verify_kda_gb300 import binding as kb

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0**-24


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def dev(x, dtype="f32"):
    return to_dev(np.asarray(x, np.float32)).to(DT[dtype])


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def rms(a):
    return float(a.double().square().mean().sqrt())


def teacher(N, V, K, seed):
    rng = np.random.default_rng(seed)
    ids = ((rng.integers(0, V, (N, 1)) + np.arange(K) * rng.integers(1, max(2, V // K), (N, 1))) % V).astype(np.int32)
    return ids, (3 * rng.standard_normal((N, K))).astype(np.float32)


SIZES = [(1, 37, 5), (8, 32768, 20), (3, 100003, 64), (400, 513, 8), (500, 33001, 20), (200, 131072, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K", SIZES)
def test_calls_leave_their_inputs_alone(N, V, K, dtype):
    t = dev(ref.rows("peaked", N, V, dtype, 3), dtype)
    ids, values = teacher(N, V, K, 4)
    tok, g = to_dev(ids[:, 0].copy()), torch.linspace(-1, 1, N, device="cuda")
    i, v, w = to_dev(ids), dev(values), g.abs() + 0.5
    inputs = [t, tok, g, i, v, w]
    kept = [a.clone() for a in inputs]
    _, H, stats, _, _ = kb.spec_logprobs(t, tok, K)
    inputs += [H, stats]
    kept += [H.clone(), stats.clone()]
    kb.spec_logprobs_backward(t, tok, stats, H, g, g)
    _, z = kb.spec_distill(t, i, v, w)
    kb.spec_distill_backward(t, i, v, z, g, w)
    kb.spec_distill_step(t, i, v, g, w)
    for a, b in zip(inputs, kept):
        assert same_bits(a, b)


def test_score_gradients_from_several_host_threads():
    """What a thread gets is, bit for bit, what the call gives when it is made alone."""
    shapes = [(400, 33000), (400, 9000), (3, 33000), (400, 100)]
    ts = [dev(ref.rows("normal", N, V, "bf16", N + V), "bf16") for N, V in shapes]
    toks = [to_dev(np.random.default_rng(V).integers(0, V, N).astype(np.int32)) for N, V in shapes]
    g = torch.linspace(-1, 1, 400, device="cuda")

    def both(j, stream=None):
        N = shapes[j][0]
        out = kb.spec_logprobs(ts[j], toks[j], 7, stream=stream)
        return out, kb.spec_logprobs_backward(ts[j], toks[j], out[2], out[1], g[:N], g[:N], stream=stream)

    alone = [both(j) for j in range(len(shapes))]
    torch.cuda.synchronize()
    got, wrong = {}, []

    def work(j):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got[j] = both(j, s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(shapes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    for j, (out, d) in enumerate(alone):
        for a, b in zip((*out, d), (*got[j][0], got[j][1])):
            assert same_bits(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,K", SIZES)
def test_every_row_of_a_distillation_gradient(N, V, K, dtype):
    """Each element of each row against the definition in 64 bits (elementary torch), from the
    step and from the two calls, and each row's sum, which is g w tau (Q - Q) = 0: within the
    elements' tolerance summed over a row whose p and q add up to 1 each."""
    tau = 2.0
    t = dev(ref.rows("peaked", N, V, dtype, 3), dtype)
    ids, values = teacher(N, V, K, 4)
    i, v = to_dev(ids), dev(values)
    rng = np.random.default_rng(1)
    g, w = dev(rng.standard_normal(N)), dev(0.5 + rng.random(N))
    _, _, step = kb.spec_distill_step(t, i, v, g, w, temperature=tau)
    _, stats = kb.spec_distill(t, i, v, w, temperature=tau)
    two = kb.spec_distill_backward(t, i, v, stats, g, w, temperature=tau)
    bf16 = 2.0**-8 if dtype == "bf16" else 0.0
    q = torch.softmax(v.double() / tau, 1)
    scale = (g.double() * w.double() * tau)[:, None]
    for a in range(0, N, 50):
        r = slice(a, a + 50)
        p = torch.softmax(t[r].double() / tau, 1)
        d = torch.zeros_like(p).scatter_add_(1, i[r].long(), q[r])
        want = scale[r] * (p - d)
        tol = scale[r].abs() * 5e-5 * (p + d) + bf16 * want.abs() + 1e-30
        for got in (step, two):
            got = got[r].double()
            assert ((got - want).abs() <= tol).all()
            assert (got.sum(1).abs() <= scale[r, 0].abs() * 2 * (5e-5 + bf16)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(8, 32768), (38, 131072), (400, 5000), (480, 32768), (200, 131072)])
def test_errors_of_scores_on_the_whole(N, V, dtype):
    t = dev(ref.rows("normal", N, V, dtype, 3), dtype)
    tok = to_dev(np.random.default_rng(V).integers(0, V, N).astype(np.int32))
    lp, H, stats, ids, top = kb.spec_logprobs(t, tok, 20)
    for a in range(0, N, 50):
        r = slice(a, a + 50)
        logp = torch.log_softmax(t[r].double(), 1)
        lnS = torch.logsumexp(t[r].double() - stats[r, :1].double(), 1)
        assert lnS.max() < 16
        assert rms(stats[r, 1] - lnS) <= 16 * U
        assert rms(lp[r] - logp.gather(1, tok[r].long()[:, None])[:, 0]) <= 24 * U
        assert rms(top[r] - logp.gather(1, ids[r].long())) <= 24 * U
        assert rms(H[r] + (logp.exp() * logp).sum(1)) <= 64 * U


@pytest.mark.parametrize("N,V", [(8, 32768), (400, 5000), (480, 32768), (200, 131072)])
def test_errors_of_f32_gradients_on_the_whole(N, V):
    t = dev(ref.rows("normal", N, V, "f32", 3))
    ids, values = teacher(N, V, 8, 4)
    i, v, one = to_dev(ids), dev(values), torch.ones(N, device="cuda")
    tok = to_dev(ids[:, 0].copy())
    _, _, stats, _, _ = kb.spec_logprobs(t, tok, 0)
    score = kb.spec_logprobs_backward(t, tok, stats, grad_logprob=one)
    _, _, step = kb.spec_distill_step(t, i, v)
    two = kb.spec_distill_backward(t, i, v, stats)
    for a in range(0, N, 50):
        r = slice(a, a + 50)
        p = torch.softmax(t[r].double(), 1)
        at = p > 2.0**-32
        at.scatter_(1, i[r].long(), False)  # elsewhere the gradients are -p and p
        for got, sign in ((score, -1.0), (step, 1.0), (two, 1.0)):
            assert rms((sign * got[r].double() - p)[at] / p[at]) <= 40 * U
