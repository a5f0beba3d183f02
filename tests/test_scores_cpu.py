"""Refusals of the score and distillation entry points on the host: nothing is launched."""
import ctypes

import numpy as np
import pytest
import torch

import score_ref as ref
from libs import ensure_built

from speculative_decode_verify_kda_gb300 import binding as kb

FAKE = 0x10000  # never dereferenced: every call below fails validation or has no rows


@pytest.fixture(scope="module")
def L():
    ensure_built()
    return kb.lib()


def score(L, **k):
    return L.spec_logprobs(k.get("x", FAKE), k.get("dt", kb.BF16), k.get("N", 2), k.get("V", 100), k.get("ld", 100),
                           k.get("tok", FAKE), k.get("K", 5), k.get("tau", 1.0), k.get("lp", FAKE), k.get("H", FAKE),
                           k.get("stats", FAKE), k.get("ids", FAKE), k.get("top", FAKE), k.get("st"), None)


BAD = [{"N": -1}, {"V": 0}, {"V": -5}, {"V": 2**30 + 1, "ld": 2**31}, {"ld": 99}, {"dt": 2}, {"dt": -1}, {"x": None}, {"x": FAKE + 1},
       {"x": FAKE + 2, "dt": kb.F32}, {"tau": 0.0}, {"tau": -1.0}, {"tau": float("nan")}, {"tau": float("inf")},
       {"tau": 1e-5}, {"tau": 1e5}]


@pytest.mark.parametrize("bad", BAD + [{"K": -1}, {"K": 129}, {"ids": None}, {"top": None}, {"tok": None},
                                       {"tok": FAKE + 2}, {"stats": FAKE + 1}, {"st": FAKE + 3}, {"top": FAKE + 2}])
def test_scores_reject(L, bad):
    assert score(L, **bad) == kb.EINVAL
    assert L.kda_last_error()


def test_scores_of_no_rows(L):
    assert score(L, N=0, x=None) == kb.OK
    assert score(L, N=0, K=200) == kb.EINVAL


def backward(L, **k):
    return L.spec_logprobs_backward(k.get("x", FAKE), k.get("dt", kb.BF16), k.get("N", 2), k.get("V", 100),
                                    k.get("ld", 100), k.get("tok", FAKE), k.get("stats", FAKE), k.get("H", FAKE),
                                    k.get("g", FAKE), k.get("h", FAKE), k.get("tau", 1.0), k.get("dx", FAKE),
                                    k.get("ldg", 100), None)


GRAD = [{"dx": None}, {"ldg": 99}, {"dx": FAKE + 1}, {"dx": FAKE + 2}, {"dx": FAKE, "ldg": 101},
        {"dx": FAKE + 2 * 199}, {"dx": FAKE - 2 * 199}, {"stats": None}]


@pytest.mark.parametrize("bad", BAD + GRAD + [{"g": None, "h": None}, {"tok": None}, {"H": None}, {"H": FAKE + 2},
                                              {"g": FAKE + 1}])
def test_scores_backward_rejects(L, bad):
    assert backward(L, **bad) == kb.EINVAL


def distill(L, which, **k):
    te = None
    if k.get("teacher", True):
        te = ctypes.byref(kb.KdaTeacher(k.get("ids", FAKE), k.get("vals", FAKE), k.get("w"), k.get("vdt", kb.F32),
                                        k.get("kind", 0), k.get("K", 4)))
    head = (k.get("x", FAKE), k.get("dt", kb.BF16), k.get("N", 2), k.get("V", 100), k.get("ld", 100), te,
            k.get("tau", 1.0))
    loss, stats, g, dx = k.get("loss", FAKE), k.get("stats", FAKE), k.get("g"), k.get("dx", FAKE + 0x8000)
    if which == "loss":
        return L.spec_distill(*head, loss, stats, k.get("st"), None)
    if which == "backward":
        return L.spec_distill_backward(*head, stats, g, dx, k.get("ldg", 100), k.get("st"), None)
    return L.spec_distill_step(*head, g, loss, stats, dx, k.get("ldg", 100), k.get("st"), None)


@pytest.mark.parametrize("which", ["loss", "backward", "step"])
@pytest.mark.parametrize("bad", BAD + [{"teacher": False}, {"K": 0}, {"K": 129}, {"vdt": 3}, {"kind": 2}, {"ids": None},
                                       {"vals": None}, {"ids": FAKE + 2}, {"w": FAKE + 2}, {"vals": FAKE + 2},
                                       {"vals": FAKE + 1, "vdt": kb.BF16}, {"stats": FAKE + 2}, {"st": FAKE + 1}])
def test_distill_rejects(L, which, bad):
    assert distill(L, which, **bad) == kb.EINVAL
    assert L.kda_last_error()


def test_distill_gradients_and_losses_reject(L):
    for bad in GRAD[:-1]:
        assert distill(L, "backward", **bad) == kb.EINVAL and distill(L, "step", **bad) == kb.EINVAL
    assert distill(L, "backward", stats=None) == kb.EINVAL
    for which in ("loss", "step"):
        assert distill(L, which, loss=None) == kb.EINVAL and distill(L, which, loss=FAKE + 1) == kb.EINVAL
    for which in ("loss", "backward", "step"):
        assert distill(L, which, N=0, x=None, ids=None, vals=None) == kb.OK


def test_binding_refuses_host_tensors_and_bad_types():
    x = torch.zeros(2, 8)
    with pytest.raises(TypeError):
        kb.spec_logprobs(x, None, 2)
    with pytest.raises(TypeError):
        kb.spec_distill(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))


def test_reference_definitions():
    """The tests' own 64-bit definitions on a case that can be written down."""
    x = np.log(np.array([[1.0, 2.0, 1.0]])).astype(np.float64)
    lp, H, stats, ids, top = ref.score(x, [1], 3, 1.0)
    assert np.allclose(lp, np.log(0.5)) and np.allclose(stats, [[np.log(2.0), np.log(2.0)]]) and np.allclose(H, 1.5 * np.log(2.0))
    assert ids.tolist() == [[1, 0, 2]] and np.allclose(np.exp(top), [[0.5, 0.25, 0.25]])
    g = ref.score_grad(x, [1], [1.0], None, 1.0)
    assert np.allclose(g, [[-0.25, 0.5, -0.25]])
    loss, _, grad, _, _ = ref.distill(x, np.array([[1, 0]]), np.array([[0.0, 0.0]]), 1.0)
    assert np.allclose(loss, 0.5 * np.log(0.5 / 0.5) + 0.5 * np.log(0.5 / 0.25))
    assert np.allclose(grad, [[0.25 - 0.5, 0.5 - 0.5, 0.25]])
