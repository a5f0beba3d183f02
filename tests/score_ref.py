"""Plain 64-bit (numpy) definitions of the score and distillation operators, and the rows
that their tests use.  No value here comes from the CUDA path."""
from __future__ import annotations

import numpy as np

LOWEST = {"f32": -3.4028234663852886e38, "bf16": -3.3895313892515355e38}


def bf16_round(x: np.ndarray) -> np.ndarray:
    """float32 values rounded to bfloat16 (to nearest, ties to even), as float32."""
    x = np.ascontiguousarray(x, np.float32)
    b = x.view(np.uint32)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, x)


def typed(x, dtype: str) -> np.ndarray:
    """float32 array holding values that the type has."""
    x = np.asarray(x, np.float32)
    return bf16_round(x) if dtype == "bf16" else x


def score(x, tokens, K, tau):
    """(logprob, entropy, stats, top_ids, top_logprobs) of rows x [N][V]; stats [N][2] are the
    maximum m and ln sum exp((x - m) / tau)."""
    N, V = x.shape
    lp, H, stats = np.zeros(N), np.zeros(N), np.zeros((N, 2))
    ids, top = np.full((N, K), -1, np.int64), np.full((N, K), -np.inf)
    for n in range(N):
        z = x[n].astype(np.float64) / tau
        t = -1 if tokens is None else int(tokens[n])
        has = 0 <= t < V
        if np.isnan(z).any() or np.isposinf(z).any():
            stats[n] = H[n] = np.nan
            top[n] = np.nan
            lp[n] = np.nan if has else 0.0
            continue
        m = z.max()
        if np.isneginf(m):
            stats[n] = -np.inf
            lp[n] = -np.inf if has else 0.0
            continue
        e = np.exp(z - m)
        S = e.sum()
        stats[n] = x[n].max(), np.log(S)
        d = np.where(e > 0, z - m, 0.0)
        H[n] = np.log(S) - (e * d).sum() / S
        if has:
            lp[n] = (z[t] - m) - np.log(S)
        order = np.lexsort((np.arange(V), -z))[:K]
        order = order[np.isfinite(z[order])]
        ids[n, :len(order)] = order
        top[n, :len(order)] = (z[order] - m) - np.log(S)
    return lp, H, stats, ids, top


def probs(x, tau):
    """p and ln p of one row (an empty row: p = 0)."""
    z = np.asarray(x, np.float64) / tau
    m = z.max()
    if np.isnan(z).any() or np.isposinf(m):
        return np.full(z.shape, np.nan), np.full(z.shape, np.nan)
    if np.isneginf(m):
        return np.zeros(z.shape), np.full(z.shape, -np.inf)
    lp = z - m - np.log(np.exp(z - m).sum())
    return np.exp(lp), lp


def score_grad(x, tokens, g, h, tau):
    """d logits from g = dL/dlogprob and h = dL/dentropy (either None)."""
    N, V = x.shape
    out = np.zeros((N, V))
    for n in range(N):
        t = -1 if tokens is None else int(tokens[n])
        gn = float(g[n]) if g is not None and 0 <= t < V else 0.0
        hn = float(h[n]) if h is not None else 0.0
        if gn == 0 and hn == 0:
            continue
        p, lp = probs(x[n], tau)
        if not np.isnan(p).any() and p.sum() == 0:
            continue
        plp = p * np.where(p > 0, lp, 0.0)
        out[n] = -p * gn - hn * (plp - p * plp.sum())
        if 0 <= t < V:
            out[n, t] += gn
    return out / tau


def teacher(ids, values, V, tau, logprobs=False):
    """(q, ln q) of every entry; q = 0 where there is none."""
    ids = np.asarray(ids)
    v = np.asarray(values, np.float64) / (1.0 if logprobs else tau)
    v = np.where((ids >= 0) & (ids < V), v, -np.inf)
    if not logprobs:
        top = v.max(1, keepdims=True)
        with np.errstate(invalid="ignore", divide="ignore"):
            v = v - top - np.log(np.exp(v - top).sum(1, keepdims=True))
        v = np.where(np.isneginf(top), -np.inf, v)
    return np.exp(v), v


def distill(x, ids, values, tau, weight=None, g=None, logprobs=False):
    """(loss [N], stats [N][2], gradient [N][V], p [N][V], dense q [N][V])."""
    N, V = x.shape
    q, lnq = teacher(ids, values, V, tau, logprobs)
    loss, stats = np.zeros(N), np.zeros((N, 2))
    grad, P, D = np.zeros((N, V)), np.zeros((N, V)), np.zeros((N, V))
    for n in range(N):
        w = 1.0 if weight is None else float(weight[n])
        gn = 1.0 if g is None else float(g[n])
        if w == 0:
            continue
        p, lp = probs(x[n], tau)
        z = x[n].astype(np.float64) / tau
        empty = not np.isnan(p).any() and p.sum() == 0
        if np.isnan(p).any():
            stats[n] = np.nan
        elif empty:
            stats[n] = -np.inf
        else:
            stats[n] = x[n].max(), np.log(np.exp(z - z.max()).sum())
        on = q[n] != 0
        if not on.any():
            continue
        at = np.asarray(ids[n])[on]
        loss[n] = w * tau * tau * (q[n][on] * (lnq[n][on] - lp[at])).sum()
        np.add.at(D[n], at, q[n][on])
        P[n] = p
        if not empty and gn != 0:
            Q = q[n][on].sum()
            grad[n] = gn * w * tau * (Q * p - D[n])
    return loss, stats, grad, P, D


def rows(kind: str, N: int, V: int, dtype: str, seed: int) -> np.ndarray:
    """Rows of logits of one kind, float32 holding values of the type."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((N, V)) * 1.8).astype(np.float32)
    low = np.float32(LOWEST[dtype])
    if kind == "peaked":
        x[np.arange(N), rng.integers(0, V, N)] += 12.0
    elif kind == "constant":
        x[:] = 0.25
    elif kind == "two_values":  # more equal maxima than any list holds
        x = np.where(rng.random((N, V)) < 0.4, 1.0, -1.0).astype(np.float32)
    elif kind == "few_allowed_inf":
        keep = rng.random((N, V)) < 5.0 / V
        keep[:, V // 2] = True
        x = np.where(keep, x, -np.inf).astype(np.float32)
    elif kind == "few_allowed_lowest":
        keep = rng.random((N, V)) < 5.0 / V
        keep[:, V // 3] = True
        x = np.where(keep, x, low).astype(np.float32)
    elif kind == "all_lowest":
        x[:] = low
    elif kind == "all_masked":
        x[:] = -np.inf
    elif kind == "some_masked":
        x[rng.random((N, V)) < 0.3] = -np.inf
        x[N // 2] = -np.inf
    elif kind == "zeros_of_both_signs":
        x = np.where(rng.random((N, V)) < 0.5, np.float32(0.0), np.float32(-0.0))
    elif kind == "ascending":
        x = np.tile(np.arange(V, dtype=np.float32) * (16.0 / V), (N, 1))
    elif kind == "descending":
        x = np.tile(-np.arange(V, dtype=np.float32) * (16.0 / V), (N, 1))
    elif kind == "periodic":  # the largest logits repeat with a power-of-two period
        i = np.arange(V)
        x = np.tile(np.where(i % 1024 < 16, 4.0 + (i % 7919) * 1e-3, 0.0).astype(np.float32), (N, 1))
    elif kind == "huge":
        x = (x * 1e37).astype(np.float32)
    else:
        assert kind == "normal", kind
    return typed(x, dtype)


KINDS = ("normal", "peaked", "constant", "two_values", "few_allowed_inf", "few_allowed_lowest", "all_lowest",
         "all_masked", "some_masked", "zeros_of_both_signs", "ascending", "descending", "periodic", "huge")
