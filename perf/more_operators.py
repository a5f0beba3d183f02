"""Performance cases of the paged-cache operators: append, attention, attention mass, eviction.

``listed()`` names the measured cases, ``draw(rng)`` gives more of the same ranges,
``prepare`` makes a case's inputs on the GPU, ``run`` makes one pass and ``exact`` gives
the same results from the definitions in 64 bits.  With ``own`` false a pass is made of
elementary torch operations in 32 bits; with ``own`` true it calls this package.

A cache holds keys and values k, v [pages][kv heads][page][D]; session b's token j lies in
page table[b][j / page], slot j % page, and lens[b] tokens are held.  A call brings t_b <= T
new rows a session; row t stands at position p = lens[b] + t.  Key j is visible to it when
j <= p and (no window, or p - j < window, or j < sinks).

  append   the rows' keys and values go to their places in the pages
  attend   o = sum_j softmax_j(scale q.k_j) v_j over the visible keys, and ln sum_j exp(scale q.k_j)
  mass     every key's share of the rows' attention, summed over the rows and the heads that read it
  evict    a session's cache cut to a budget: first tokens, last tokens and the heaviest between
"""
import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
OPS = ("append", "attend", "attend", "attend", "mass", "evict")


def _case(name, op, sessions, rows, context, heads, kv_heads, dim=128, page=64, dtype="bf16", ragged=False, window=0,
          sinks=0, budget=0):
    return {"name": name, "op": op, "sessions": sessions, "rows": rows, "context": context, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "ragged": ragged, "window": window,
            "sinks": sinks, "budget": budget}


def listed():
    return [
        # the rows of a batched verify round (32 sessions, T = 15) enter the cache
        _case("append_round", "append", 32, 15, 8192, 64, 8, ragged=True),
        # four prompts' chunks enter the cache
        _case("append_prompt", "append", 4, 2048, 4096, 32, 8, dtype="f16"),
        # one session decodes one token: a call's latency
        _case("attend_token", "attend", 1, 1, 4096, 64, 8),
        # one session's verify round (T = 8) far into a text
        _case("attend_round", "attend", 1, 8, 32768, 64, 8),
        # a batched verify round: 32 sessions of up to T = 15 rows, lengths of their own
        _case("attend_batch", "attend", 32, 15, 16384, 64, 8, ragged=True),
        # a chunk of a long prompt: the largest case
        _case("attend_prompt", "attend", 1, 2048, 16384, 64, 8),
        # verify rounds of window layers: f16, six heads a kv head, D = 64, small pages
        _case("attend_window_batch", "attend", 64, 8, 16384, 24, 4, 64, 16, "f16", True, 4096, 4),
        # two prompts' chunks of an odd length in window layers
        _case("attend_window_prompt", "attend", 2, 1501, 8192, 32, 8, 128, 32, "bf16", True, 1024, 16),
        # what a batch's verify rows paid attention to
        _case("mass_round", "mass", 16, 8, 16384, 64, 8, ragged=True),
        # the same of a prompt's chunk
        _case("mass_prompt", "mass", 1, 1024, 8192, 32, 8, dtype="f16"),
        # one long session cut to an eighth
        _case("evict_session", "evict", 1, 0, 32768, 64, 8, window=256, sinks=4, budget=4096),
        # a batch of sessions cut to 2000 tokens, the shorter ones kept whole
        _case("evict_batch", "evict", 32, 0, 8000, 32, 8, page=16, dtype="f16", ragged=True, window=128, sinks=4,
              budget=2000),
    ]


#: what the largest listed case costs: multiply-adds of the attention, bytes of a cache
MOST_PAIRS = 64 * 2048 * (16384 + 1024)
MOST_CACHE = 32 * (16384 + 64) * 8 * 128 * 2


def _log(rng, low, high):
    return int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))


def draw(rng):
    op = rng.choice(OPS)
    kv_heads = rng.choice((1, 2, 4, 8))
    heads = kv_heads * rng.choice((1, 2, 4, 5, 6, 8, 16))
    dim, page = rng.choice((64, 128, 128)), rng.choice((16, 32, 64, 128))
    dtype, ragged = rng.choice(("bf16", "bf16", "f16")), rng.random() < 0.7
    context = _log(rng, 16, 32768)
    window, sinks, budget = 0, 0, 0
    if op == "evict":
        rows = 0
        budget = max(8, int(context * rng.uniform(0.1, 0.9)))
        sinks, window = rng.randint(0, 4), rng.randint(1, budget // 2)
    else:
        rows = rng.choice((1, _log(rng, 1, 15), _log(rng, 16, 2048)))
        if op != "append" and rng.random() < 0.4:
            window, sinks = _log(rng, 16, max(16, min(8192, context + rows))), rng.choice((0, 4, 16))
    pairs = heads * max(1, rows) * (context + rows)
    cache = kv_heads * dim * 2 * (context + rows + page)
    most = max(1, min(64, MOST_CACHE // cache, (MOST_PAIRS if op in ("attend", "mass") else 1 << 62) // pairs))
    case = _case("", op, _log(rng, 1, most), rows, context, heads, kv_heads, dim, page, dtype, ragged, window, sinks,
                 budget)
    del case["name"]
    return case


def _sizes(case):
    """Lengths and row counts of the sessions, as host lists that depend on the case alone."""
    n, t = case["context"], case["rows"]
    count = range(case["sessions"])
    if not case["ragged"]:
        return [n for _ in count], [t for _ in count]
    # between half and the whole of the context; every eighth session has fewer rows, every 16th none
    lens = [max(1, n - (b * 7919) % (n // 2 + 1)) for b in count]
    rows = [0 if b % 16 == 11 else max(1, t - t // 3) if b % 8 == 5 else t for b in count]
    return lens, rows


def _visible(n, t, window, sinks):
    """(row, key) pairs that t rows behind n tokens see, and the keys that some row sees."""
    if t == 0:
        return 0, 0
    if not window:
        return t * n + t * (t + 1) // 2, n + t
    pairs = sum(min(p + 1, window) + min(sinks, max(0, p + 1 - window)) for p in range(n, n + t))
    low = max(0, n - window + 1)
    return pairs, n + t - low + min(sinks, low)


def work(case):
    hq, hkv, d, op = (case[c] for c in ("heads", "kv_heads", "dim", "op"))
    lens, rows = _sizes(case)
    if op == "append":
        return {"bytes": 8 * sum(rows) * hkv * d, "flops": 0}
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": hkv * (4 * sum(lens) + kept * (8 * d + 8)), "flops": 0}
    seen = [_visible(n, t, case["window"], case["sinks"]) for n, t in zip(lens, rows)]
    pairs, keys = (sum(s[i] for s in seen) for i in (0, 1))
    if op == "mass":
        return {"bytes": keys * hkv * (2 * d + 8) + sum(rows) * hq * (2 * d + 4), "flops": 2 * d * hq * pairs}
    return {"bytes": keys * hkv * 4 * d + sum(rows) * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    b, t, hq, hkv, d, page = (case[c] for c in ("sessions", "rows", "heads", "kv_heads", "dim", "page"))
    dtype, op = DTYPES[case["dtype"]], case["op"]
    lens, rows = _sizes(case)
    cols = -(-(case["context"] + t) // page)
    short = -(-case["budget"] // page)
    pages = b * (cols + short)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=DEVICE, dtype=dtype).mul_(scale)

    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    s = {"op": op, "case": case, "plan": None, "k": normal(pages, hkv, page, d), "v": normal(pages, hkv, page, d),
         "table": order[:b * cols].view(b, cols).contiguous(), "lens": torch.tensor(lens, device=DEVICE).int(),
         "t_rows": torch.tensor(rows, device=DEVICE).int(), "scale": d**-0.5}
    if op == "append":
        s["k_rows"], s["v_rows"] = normal(b, t, hkv, d), normal(b, t, hkv, d)
        return s
    if op == "evict":
        # shares of attention: a few tokens hold most of it
        s["mass"] = torch.rand((b, hkv, cols * page), generator=g, device=DEVICE).pow_(8).mul_(4.0)
        s["dst"] = order[b * cols:].view(b, short).contiguous()
        s["kept"] = torch.empty((b, hkv, case["budget"]), dtype=torch.int32, device=DEVICE)
        s["mass_out"] = torch.zeros((b, hkv, case["budget"]), device=DEVICE)
        s["lens_out"] = torch.empty_like(s["lens"])
        return s
    s["q"] = normal(b, t, hq, d, scale=2.0)
    # rows behind a session's last one are neither read nor written
    s["out"] = torch.zeros((b, t, hq, d), dtype=dtype, device=DEVICE)
    s["lse"] = torch.zeros((b, t, hq), device=DEVICE)
    if case["window"]:
        # pages that no row sees have been handed back
        at = torch.arange(cols, device=DEVICE) * page
        low = (s["lens"] - case["window"] + 1)[:, None]
        s["table"] = torch.where((at + page > low) | (at < case["sinks"]), s["table"], -1).contiguous()
    if op == "mass":
        s["lse"] = _plain_attend(s)["lse"]
        s["mass"] = torch.rand((b, hkv, cols * page), generator=g, device=DEVICE)
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _places(s):
    """Positions [B][N] that the rows may see, and which of them each row sees [B][T][N]."""
    case = s["case"]
    n, t, w, first = s["lens"].long()[:, None], case["rows"], case["window"], case["sinks"]
    if w:
        near = n - w + 1 + torch.arange(w - 1 + t, device=DEVICE)
        far = torch.arange(first, device=DEVICE).expand(n.shape[0], first)
        pos = torch.cat((torch.where(far < near[:, :1], far, -1), near), 1)
    else:
        pos = torch.arange(case["context"] + t, device=DEVICE).expand(n.shape[0], -1)
    row = torch.arange(t, device=DEVICE)
    at = (n + row)[:, :, None]
    key = pos[:, None, :]
    seen = (key >= 0) & (key <= at) & (row[:, None] < s["t_rows"][:, None, None])
    if w:
        seen &= (at - key < w) | (key < first)
    return pos, seen


def _gather(s, x, pos):
    """Rows of the pages at the positions: [B][Hkv][N][D] in f32."""
    page = s["case"]["page"]
    pos = pos.clamp(0, s["table"].shape[1] * page - 1)
    at = s["table"].long().gather(1, pos // page).clamp(min=0)
    return x[at, :, pos % page].permute(0, 2, 1, 3).float()


def _scores(s):
    """Scores [B][Hkv][T G][N] of the rows, -inf where a key is not visible; the positions and the mask."""
    case = s["case"]
    b, t, hkv = case["sessions"], case["rows"], case["kv_heads"]
    group = case["heads"] // hkv
    pos, seen = _places(s)
    k = _gather(s, s["k"], pos)
    q = s["q"].float().view(b, t, hkv, group, -1).transpose(1, 2).reshape(b, hkv, t * group, -1)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, t, group, -1)
    x = x.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    return x.view(b, hkv, t * group, -1), pos, seen


def _plain_attend(s):
    case = s["case"]
    b, t, hkv = case["sessions"], case["rows"], case["kv_heads"]
    x, pos, _ = _scores(s)
    top = x.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = x.sub_(top).exp_()
    total = e.sum(3, keepdim=True)
    o = (e @ _gather(s, s["v"], pos)) / total

    def rows_first(y):  # [B][Hkv][T G][...] to [B][T][Hq][...]
        return y.view(b, hkv, t, case["heads"] // hkv, -1).transpose(1, 2).reshape(b, t, case["heads"], -1)

    live = torch.arange(t, device=DEVICE) < s["t_rows"][:, None]
    out = torch.where(live[:, :, None, None], rows_first(o), 0.0).to(s["out"].dtype)
    lse = torch.where(live[:, :, None], rows_first(top + torch.log(total))[..., 0], 0.0)
    return {"out": out, "lse": lse}


def _plain_mass(s):
    case = s["case"]
    b, t, hkv = case["sessions"], case["rows"], case["kv_heads"]
    x, pos, _ = _scores(s)
    lse = s["lse"].view(b, t, hkv, -1).transpose(1, 2).reshape(b, hkv, -1, 1)
    share = x.sub_(lse).exp_().sum(2)
    place = torch.arange(s["mass"].shape[2], device=DEVICE)
    n = s["lens"][:, None]
    new = (place >= n) & (place < n + s["t_rows"][:, None])
    s["mass"].masked_fill_(new[:, None], 0.0)
    s["mass"].scatter_add_(2, pos.clamp(0, place.numel() - 1)[:, None].expand_as(share), share)
    return {"mass": s["mass"]}


def _plain_append(s):
    case = s["case"]
    row = torch.arange(case["rows"], device=DEVICE)
    pos = s["lens"].long()[:, None] + row
    b, t = torch.nonzero(row < s["t_rows"][:, None], as_tuple=True)
    at = s["table"].long().gather(1, pos // case["page"])[b, t]
    slot = (pos % case["page"])[b, t]
    s["k"][at, :, slot] = s["k_rows"][b, t]
    s["v"][at, :, slot] = s["v_rows"][b, t]
    return {"k": s["k"], "v": s["v"]}


def _ordered(x):
    """Whole numbers in the order of the floats (the two zeros equal)."""
    bits = (x + 0.0).view(torch.int32)
    return torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()


def _plain_evict(s):
    case = s["case"]
    budget, page = case["budget"], case["page"]
    b, hkv, wide = s["mass"].shape
    n = s["lens"].long()[:, None]
    place = torch.arange(wide, device=DEVICE)
    key = (_ordered(s["mass"]) << 20) - place  # the lowest position first among equal masses
    always = ((place < case["sinks"]) | (place >= n - case["window"])) | (n <= budget)
    key = torch.where(always[:, None], (1 << 60) - place, key)
    key = torch.where((place < n)[:, None], key, -(1 << 60) - place)
    width = min(budget, wide)
    best, at = key.sort(2, descending=True)
    kept = torch.where(best[:, :, :width] > -(1 << 59), at[:, :, :width], wide).sort(2).values
    there = kept < wide
    kept = torch.where(there, kept, -1)
    s["kept"][:, :, width:] = -1
    s["kept"][:, :, :width] = kept
    s["lens_out"].copy_(n[:, 0].clamp(max=budget))
    i, h, r = torch.nonzero(there, as_tuple=True)
    src, from_page, to_page = kept[i, h, r], s["table"].long(), s["dst"].long()
    for x in (s["k"], s["v"]):
        x[to_page[i, r // page], h, r % page] = x[from_page[i, src // page], h, src % page]
    s["mass_out"][i, h, r] = s["mass"][i, h, src]
    return {"kept": s["kept"], "lens": s["lens_out"], "mass": s["mass_out"], "k": s["k"], "v": s["v"]}


_PLAIN = {"append": _plain_append, "attend": _plain_attend, "mass": _plain_mass, "evict": _plain_evict}


# ---------------------------------------------------------------------------
# this package's operators
# ---------------------------------------------------------------------------
def _plan(s):
    """The plan that a serving loop keeps for its buffers: it holds pointers and outputs."""
    from speculative_decode_verify_kda_gb300 import binding as kb
    case = s["case"]
    cache = kb.PagedCache(s["k"], s["v"], s["table"], s["lens"])
    if s["op"] == "append":
        return kb.CacheAppendPlan(cache, s["k_rows"], s["v_rows"], t_rows=s["t_rows"])
    if s["op"] == "evict":
        return kb.CacheEvictPlan(cache, s["mass"], case["budget"], recent=case["window"], sinks=case["sinks"],
                                 dst_table=s["dst"], kept_out=s["kept"], mass_out=s["mass_out"],
                                 lens_out=s["lens_out"])
    seen = {"t_rows": s["t_rows"], "window": case["window"], "sinks": case["sinks"], "scale": s["scale"]}
    if s["op"] == "mass":
        return kb.AttendMassPlan(cache, s["q"], s["lse"], s["mass"], **seen)
    return kb.AttendPlan(cache, s["q"], out=s["out"], lse_out=s["lse"], **seen)


def run(state):
    if not own:
        return _PLAIN[state["op"]](state)
    if state["plan"] is None:
        state["plan"] = _plan(state)
    state["plan"]()
    names = {"append": ("k", "v"), "attend": ("out", "lse"), "mass": ("mass",),
             "evict": ("kept", "lens_out", "mass_out", "k", "v")}[state["op"]]
    return {{"lens_out": "lens", "mass_out": "mass"}.get(name, name): state[name] for name in names}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _cached(s, name, b, h, n):
    """The first n rows of session b, kv head h, in 64 bits (unread where a page was handed back)."""
    at = s["table"][b].long()
    x = s[name][at.clamp(min=0), h].double()
    return x.reshape(-1, x.shape[-1])[:n]


def _exact_head(s, b, h, n, t):
    """Scores [t][group][n + t] of one session and kv head."""
    case = s["case"]
    group = case["heads"] // case["kv_heads"]
    q = s["q"][b, :t, h * group:(h + 1) * group].double()
    x = torch.einsum("tgd,nd->tgn", q, _cached(s, "k", b, h, n + t)) * s["scale"]
    key, at = torch.arange(n + t, device=DEVICE)[None], n + torch.arange(t, device=DEVICE)[:, None]
    hidden = key > at
    if case["window"]:
        hidden |= (at - key >= case["window"]) & (key >= case["sinks"])
    return x.masked_fill_(hidden[:, None], -math.inf)


def exact(case, seed):
    s = prepare(case, seed)
    lens, rows = _sizes(case)
    if case["op"] == "append":
        for b, (n, t) in enumerate(zip(lens, rows)):
            for i in range(0, t):
                at, slot = s["table"][b, (n + i) // case["page"]], (n + i) % case["page"]
                s["k"][at, :, slot] = s["k_rows"][b, i]
                s["v"][at, :, slot] = s["v_rows"][b, i]
        return {"k": s["k"].double(), "v": s["v"].double()}
    if case["op"] == "evict":
        return None  # nothing is computed: what is kept is compared as whole numbers, the rest is moved
    group = case["heads"] // case["kv_heads"]
    out, lse = s["q"].double().zero_(), s["lse"].double()
    mass = s["mass"].double() if case["op"] == "mass" else None
    for b, (n, t) in enumerate(zip(lens, rows)):
        for h in range(case["kv_heads"] if t else 0):
            x, mine = _exact_head(s, b, h, n, t), slice(h * group, (h + 1) * group)
            if mass is not None:
                mass[b, h, n:n + t] = 0.0
                mass[b, h, :n + t] += (x - lse[b, :t, mine, None]).exp().sum((0, 1))
                continue
            lse[b, :t, mine] = torch.logsumexp(x, 2)
            p = torch.softmax(x, 2)
            out[b, :t, mine] = torch.einsum("tgn,nd->tgd", p, _cached(s, "v", b, h, n + t))
    return {"mass": mass} if mass is not None else {"out": out, "lse": lse}
