"""Performance cases of the logit operators: token scores and distillation.

``listed()`` names the measured cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` makes a case's inputs on the GPU, ``run`` makes one pass and ``exact`` gives
the same results from the definitions in 64 bits.  With ``own`` false a pass is made of
elementary torch operations in 32 bits; with ``own`` true it calls this package.

Operators (x a row of logits, m = max x, d = (x - m) / temperature, s = ln sum exp d,
ln p = d - s; the row's stats are m and s):

  score          ln p of given tokens, entropy, stats, top alternatives
  score_grad     d logits from the gradients of ln p and entropy
  distill        KL from a teacher's top entries to p, per row
  distill_grad   d logits of that loss
  distill_step   loss and d logits in one call
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": (torch.bfloat16, 2), "f32": (torch.float32, 4)}
OPS = ("score", "score_grad", "distill", "distill_grad", "distill_step")


def _case(name, op, rows, vocab, k, dtype="bf16", temperature=1.0, mask=False):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "k": k, "dtype": dtype,
            "temperature": temperature, "mask": mask}


def listed():
    return [
        # the token that one session emits, with five alternatives: a call's latency
        _case("score_token", "score", 1, 32768, 5),
        # the eight verify rows of one session (T = 8), twenty alternatives a row
        _case("score_round", "score", 8, 32768, 20),
        # a batched verify round: 32 sessions of T = 15 rows
        _case("score_batch", "score", 480, 32768, 20),
        # constrained sampling of 64 sessions of T = 15 rows: f32 logits of an odd vocabulary with
        # masked tokens and rows whose mask leaves nothing
        _case("score_masked_f32", "score", 960, 100003, 10, "f32", 0.7, True),
        # collecting a teacher's top 64 over a long text, wide vocabulary
        _case("score_harvest", "score", 4096, 131072, 64),
        # the gradient of a policy loss with an entropy term
        _case("score_grad_batch", "score_grad", 2048, 32768, 0),
        # validation loss of a drafter on one batched round
        _case("distill_eval", "distill", 480, 32768, 32),
        # backward after a separate forward: f32 logits of an odd vocabulary
        _case("distill_grad_f32", "distill_grad", 1024, 65537, 32, "f32", 2.0),
        # one session's round in a small test vocabulary
        _case("step_small_f32", "distill_step", 15, 1001, 8, "f32"),
        # training a drafter online on one batched round
        _case("step_batch", "distill_step", 480, 32768, 20),
        # a training batch of drafter rows
        _case("step_train", "distill_step", 8192, 32768, 64, "bf16", 2.0),
        # the same in a wide vocabulary: the largest case
        _case("step_wide", "distill_step", 4096, 131072, 64),
    ]


#: the bytes of logits of the largest listed case
MOST_BYTES = 4096 * 131072 * 2


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    es = DTYPES[dtype][1]
    vocab = int(math.exp(rng.uniform(math.log(32), math.log(200000))))
    if rng.random() < 0.5:
        vocab = max(32, vocab // 64 * 64)
    most = min(8192, MOST_BYTES // (vocab * es))
    rows = max(1, int(math.exp(rng.uniform(0.0, math.log(most)))))
    k = 0 if op == "score_grad" else int(math.exp(rng.uniform(0.0, math.log(min(128, vocab)))))
    case = _case("", op, rows, vocab, k, dtype, rng.choice((1.0, 1.0, 0.7, 2.0)), op == "score" and rng.random() < 0.3)
    del case["name"]
    return case


def _unread(case):
    """Rows of a distillation batch that are padding (weight 0): every sixteenth."""
    return case["rows"] // 16 if case["op"].startswith("distill") else 0


def work(case):
    n, v, k, es = case["rows"], case["vocab"], case["k"], DTYPES[case["dtype"]][1]
    logits = (n - _unread(case)) * v * es
    if case["op"] == "score":
        return {"bytes": logits + n * (4 + 16 + 8 * k), "flops": 6 * n * v}
    if case["op"] == "score_grad":
        return {"bytes": logits + n * v * es + n * 24, "flops": 6 * n * v}
    small = n * (8 * k + 16)
    if case["op"] == "distill":
        return {"bytes": logits + small, "flops": 4 * n * v}
    flops = 4 * n * v if case["op"] == "distill_grad" else 8 * n * v
    return {"bytes": logits + n * v * es + small, "flops": flops}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    n, v, k, op, tau = (case[c] for c in ("rows", "vocab", "k", "op", "temperature"))
    dtype = DTYPES[case["dtype"]][0]
    # a broad bulk and a few likely tokens a row, which the teacher's entries are made of too
    x = torch.randn((n, v), generator=g, device=DEVICE, dtype=dtype).mul_(1.8)
    few = max(1, k or 8)
    start = torch.randint(0, v, (n, 1), generator=g, device=DEVICE)
    step = torch.randint(1, max(2, v // few), (n, 1), generator=g, device=DEVICE)
    ids = (start + step * torch.arange(few, device=DEVICE)) % v  # distinct within a row
    bump = 5.0 + 3.0 * torch.randn((n, few), generator=g, device=DEVICE)
    x.scatter_(1, ids, bump.to(dtype))
    s = {"op": op, "tau": tau, "k": k, "logits": x, "plan": None}
    row = torch.arange(n, device=DEVICE)
    if op in ("score", "score_grad"):
        pick = torch.randint(0, few, (n, 1), generator=g, device=DEVICE)
        s["tokens"] = ids.gather(1, pick)[:, 0].to(torch.int32)
        if case["mask"]:
            x[torch.rand((n, v), generator=g, device=DEVICE) < 0.3] = -math.inf
            x[row % 16 == 7] = -math.inf
        if op == "score_grad":
            _, s["entropy"], s["stats"] = _scores(x, s["tokens"], tau)
            s["grad_logprob"] = torch.randn(n, generator=g, device=DEVICE)
            s["grad_entropy"] = 0.1 * torch.randn(n, generator=g, device=DEVICE)
        return s
    # the teacher's entries: values falling along the list, the last ones of some rows absent
    drop = torch.rand((n, k), generator=g, device=DEVICE)
    s["values"] = 4.0 + 2.0 * torch.randn((n, 1), generator=g, device=DEVICE) - torch.cumsum(drop, 1)
    absent = (row[:, None] % 8 == 3) & (torch.arange(k, device=DEVICE) >= max(1, k // 2))
    s["ids"] = torch.where(absent, -1, ids).to(torch.int32)
    s["weight"] = torch.where(row % 16 == 15, 0.0, 0.5 + torch.rand(n, generator=g, device=DEVICE))
    if op != "distill":
        s["grad_loss"] = torch.randn(n, generator=g, device=DEVICE)
    if op == "distill_grad":
        s["stats"] = torch.where(s["weight"][:, None] == 0, 0.0, _scores(x, None, tau)[2])
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _scores(x, tokens, tau):
    """ln p of the tokens (or None), entropy and stats; a row of -inf has stats -inf and entropy 0."""
    x = x.float()
    top = x.amax(1, keepdim=True)
    d = (x - torch.where(top == -math.inf, 0.0, top)) / tau
    e = torch.exp(d)
    total = e.sum(1)
    log_total = torch.log(total)
    mean = torch.where(e > 0, e * d, 0.0).sum(1) / total
    entropy = torch.where(total > 0, log_total - mean, 0.0)
    logprob = None
    if tokens is not None:
        at = d.gather(1, tokens.long()[:, None])[:, 0]
        logprob = torch.where(at == -math.inf, at, at - log_total)
    return logprob, entropy, torch.stack((top[:, 0], log_total), 1)


def _ordered(x):
    """Whole numbers in the order of the floats (the two zeros equal)."""
    bits = (x + 0.0).view(torch.int32)
    return torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()


def _plain_score(s):
    x = s["logits"].float()
    logprob, entropy, stats = _scores(x, s["tokens"], s["tau"])
    # the largest logits, the lowest id first among equal ones
    ids = torch.arange(x.shape[1], device=x.device)
    key = (_ordered(x) << 32) - ids
    best = torch.topk(key, s["k"], dim=1).values
    top = -((best + (1 << 31)) % (1 << 32) - (1 << 31))
    at = x.gather(1, top)
    masked = at == -math.inf
    top_logprobs = torch.where(masked, at, (at - stats[:, :1]) / s["tau"] - stats[:, 1:])
    return {"logprob": logprob, "entropy": entropy, "stats": stats,
            "top_ids": torch.where(masked, -1, top).to(torch.int32), "top_logprobs": top_logprobs}


def _plain_score_grad(s):
    logp = (s["logits"].float() - s["stats"][:, :1]) / s["tau"] - s["stats"][:, 1:]
    p = torch.exp(logp)
    g, h = s["grad_logprob"][:, None], s["grad_entropy"][:, None]
    grad = -p * (g + h * (logp + s["entropy"][:, None]))
    grad.scatter_add_(1, s["tokens"].long()[:, None], g)
    return {"grad": (grad / s["tau"]).to(s["logits"].dtype)}


def _teacher(s):
    """The teacher's probabilities over its entries, 0 where there is none."""
    v = torch.where(s["ids"] >= 0, s["values"] / s["tau"], -math.inf)
    e = torch.exp(v - v.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_loss(s, logp, q):
    at = logp.gather(1, s["ids"].long().clamp(min=0))
    log_q = torch.log(torch.where(q > 0, q, 1.0))
    kl = torch.where(q > 0, q * (log_q - at), 0.0).sum(1)
    return kl * s["tau"] ** 2 * s["weight"]


def _plain_distill_grad(s, logp, q):
    grad = torch.exp(logp)
    grad.scatter_add_(1, s["ids"].long().clamp(min=0), -q)
    scale = s["grad_loss"] * s["weight"] * s["tau"]
    return (grad * scale[:, None]).to(s["logits"].dtype)


def _plain(s):
    if s["op"] == "score":
        return _plain_score(s)
    if s["op"] == "score_grad":
        return _plain_score_grad(s)
    x, q = s["logits"].float(), _teacher(s)
    if s["op"] == "distill_grad":
        return {"grad": _plain_distill_grad(s, (x - s["stats"][:, :1]) / s["tau"] - s["stats"][:, 1:], q)}
    d = (x - x.amax(1, keepdim=True)) / s["tau"]
    logp = d - torch.log(torch.exp(d).sum(1, keepdim=True))
    out = {"loss": _plain_loss(s, logp, q)}
    if s["op"] == "distill_step":
        out["grad"] = _plain_distill_grad(s, logp, q)
    return out


# ---------------------------------------------------------------------------
# this package's operators
# ---------------------------------------------------------------------------
def _plan(s):
    """The plan that a serving or training loop keeps for its buffers: it holds pointers and outputs."""
    from speculative_decode_verify_kda_gb300 import binding as kb
    if s["op"] == "score":
        return kb.LogprobsPlan(s["logits"], s["tokens"], top_k=s["k"], temperature=s["tau"])
    if s["op"] == "score_grad":
        return kb.LogprobsBackwardPlan(s["logits"], s["tokens"], s["stats"], s["entropy"],
                                       grad_logprob=s["grad_logprob"], grad_entropy=s["grad_entropy"],
                                       temperature=s["tau"])
    common = {"weight": s["weight"], "temperature": s["tau"]}
    if s["op"] == "distill":
        return kb.DistillPlan(s["logits"], s["ids"], s["values"], **common)
    if s["op"] == "distill_grad":
        return kb.DistillBackwardPlan(s["logits"], s["ids"], s["values"], s["stats"], grad_loss=s["grad_loss"],
                                      **common)
    return kb.DistillStepPlan(s["logits"], s["ids"], s["values"], grad_loss=s["grad_loss"], **common)


def run(state):
    if not own:
        return _plain(state)
    if state["plan"] is None:
        state["plan"] = _plan(state)
    out = state["plan"]()
    if state["op"] == "score":
        return dict(zip(("logprob", "entropy", "stats", "top_ids", "top_logprobs"), out))
    if state["op"] == "distill":
        return {"loss": out[0]}
    if state["op"] == "distill_step":
        return {"loss": out[0], "grad": out[2]}
    return {"grad": out}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rows(s, r):
    x = s["logits"][r].double() / s["tau"]
    logp = torch.log_softmax(x, 1)
    if s["op"] == "score":
        empty = torch.isinf(x).all(1)
        logp = torch.where(empty[:, None], -math.inf, logp)
        entropy = -torch.special.xlogy(logp.exp(), logp.exp()).sum(1)
        logprob = logp.gather(1, s["tokens"][r].long()[:, None])[:, 0]
        top = x.amax(1)
        stats = torch.stack((top * s["tau"], torch.where(empty, top, torch.logsumexp(x - top[:, None], 1))), 1)
        return {"logprob": logprob, "entropy": entropy + 0.0, "stats": stats,
                "top_logprobs": torch.topk(logp, s["k"], dim=1).values}
    if s["op"] == "score_grad":
        p = logp.exp()
        h = -torch.special.xlogy(p, p).sum(1, keepdim=True)
        hot = torch.zeros_like(p).scatter_(1, s["tokens"][r].long()[:, None], 1.0)
        grad = (hot - p) * s["grad_logprob"][r].double()[:, None]
        grad -= s["grad_entropy"][r].double()[:, None] * p * (logp + h)
        return {"grad": grad / s["tau"]}
    ids, w = s["ids"][r].long(), s["weight"][r].double()
    q = torch.softmax((s["values"][r].double() / s["tau"]).masked_fill(ids < 0, -math.inf), 1)
    dense = torch.zeros_like(logp).scatter_add_(1, ids.clamp(min=0), q)
    kl = (torch.special.xlogy(q, q) - q * logp.gather(1, ids.clamp(min=0))).sum(1)
    out = {"loss": w * kl * s["tau"] ** 2}
    if s["op"] != "distill":
        out["grad"] = (logp.exp() - dense) * (s["tau"] * w * s["grad_loss"][r].double())[:, None]
    if s["op"] == "distill_grad":
        del out["loss"]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    n, block = case["rows"], max(1, (1 << 26) // case["vocab"])
    parts = [_exact_rows(s, slice(a, min(n, a + block))) for a in range(0, n, block)]
    out = {name: torch.cat([p[name] for p in parts]) for name in parts[0]}
    if case["op"] == "score":
        out["top_ids"] = None
    return out
