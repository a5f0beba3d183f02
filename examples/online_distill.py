"""A drafter's head that learns from the target while it serves: one loop over verify rounds.

Each round drafts T - 1 tokens a session with the drafter's logits, accepts them against the
target's logits (spec_accept), scores the target's rows (spec_logprobs: log-probabilities of
the tokens handed out, entropy, top alternatives) and takes those alternatives as the teacher
of the drafter's rows (spec_distill_step: loss and d logits in one launch).  The rows behind
the first rejected draft belong to a text that was thrown away: they have weight 0.  The
head's gradient is one matrix product.

Target and drafter are stand-ins: linear heads over the same random features, the drafter's
starting at zero, so that every round costs what a round costs and the drafts get better.

    python examples/online_distill.py [--rounds 400] [--sessions 32] [--vocab 512]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from speculative_decode_verify_kda_gb300 import binding as kb  # noqa: E402


class Round:
    """The buffers of a verify round and the plans over them, made once."""

    def __init__(self, sessions: int, rows: int, vocab: int, top_k: int, temperature: float, device="cuda"):
        f32, i32 = torch.float32, torch.int32
        shape = (sessions, rows)
        self.target = torch.empty((*shape, vocab), dtype=torch.bfloat16, device=device)
        self.draft = torch.empty_like(self.target)
        self.tokens = torch.empty(shape, dtype=i32, device=device)
        self.weight = torch.empty(shape, dtype=f32, device=device)
        self.status = torch.zeros(1, dtype=i32, device=device)
        self.scores = kb.LogprobsPlan(self.target, self.tokens, top_k=top_k, dev_status=self.status)
        _, _, _, ids, top = self.scores.out
        # log-probabilities are logits up to a constant of the row: any temperature may be put on them
        self.step = kb.DistillStepPlan(self.draft, ids, top, weight=self.weight, temperature=temperature,
                                       dlogits=self.draft, dev_status=self.status)


def train(rounds=400, sessions=32, rows=8, vocab=512, features=32, top_k=32, temperature=1.0, rate=4.0, seed=0,
          device="cuda"):
    """Returns per round (mean accepted drafts, mean loss, mean log-probability of the tokens)."""
    g = torch.Generator(device=device).manual_seed(seed)
    target = torch.randn((features, vocab), generator=g, device=device) * 0.7
    head = torch.zeros((features, vocab), device=device)
    r = Round(sessions, rows, vocab, top_k, temperature, device)
    place = torch.arange(rows, device=device)
    history = []
    for _ in range(rounds):
        h = torch.randn((sessions, rows, features), generator=g, device=device)
        r.target.copy_(h @ target)
        r.draft.copy_(h @ head)
        drafts = r.draft.argmax(-1)[:, :-1].to(torch.int32).contiguous()
        j, bonus, _ = kb.spec_accept(r.target, drafts, dev_status=r.status)
        # handed out: the accepted drafts and the bonus token; behind them no token and no weight
        r.tokens[:, :-1] = torch.where(place[:-1] < j[:, None], drafts, -1)
        r.tokens.scatter_(1, j.long()[:, None], bonus[:, None])
        r.tokens.masked_fill_(place > j[:, None], -1)
        used = place <= j[:, None]
        r.weight.copy_(used / used.sum())
        logprob, entropy, _, _, _ = r.scores()
        loss, _, dlogits = r.step()
        head -= rate * (h.view(-1, features).T @ dlogits.view(-1, vocab).float())
        history.append((j.float().mean(), loss.sum(), logprob[used].mean()))
    if int(r.status):
        raise RuntimeError(f"device status {int(r.status):#x}")
    return [tuple(float(v) for v in t) for t in history]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rounds", type=int, default=400)
    ap.add_argument("--sessions", type=int, default=32)
    ap.add_argument("--vocab", type=int, default=512)
    a = ap.parse_args()
    history = train(rounds=a.rounds, sessions=a.sessions, vocab=a.vocab)
    for i in range(0, len(history), max(1, len(history) // 10)):
        print("round %4d  accepted %.2f  loss %.3f  log p %.3f" % (i, *history[i]))
    print("last        accepted %.2f  loss %.3f  log p %.3f" % history[-1])


if __name__ == "__main__":
    main()
