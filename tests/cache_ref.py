"""The paged-cache operators in 64 bits, a session and a key-value head at a time, and the
tolerances of the kernels' results against them."""
import math

import torch

from speculative_decode_verify_kda_gb300 import binding as kb

DEV = "cuda"
F64 = torch.float64


class Case:
    """A cache and rows for it.  Whatever no row of the call sees holds NaN: unused pages, the
    slots behind a session's last row, keys behind a window, rows behind a session's last."""

    def __init__(self, lens, T=1, Hq=4, Hkv=2, D=128, page=16, dtype=torch.bfloat16, t_rows=None, window=0, sinks=0,
                 layout="hnd", seed=0, spare=3, fused=False, q_scale=2.0, cols=None):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.B, self.T, self.Hq, self.Hkv, self.D, self.page, self.dtype = B, T, Hq, Hkv, D, page, dtype
        self.G, self.window, self.sinks, self.scale = Hq // Hkv, window, sinks, D**-0.5
        self.n = list(lens)
        self.t = [T] * B if t_rows is None else list(t_rows)
        cols = max(1, -(-(max(self.n, default=0) + T) // page)) if cols is None else cols
        pages = B * cols + spare
        normal = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        both = torch.full((2, pages, Hkv, page, D), math.nan)
        table = torch.randperm(pages, generator=g)[:B * cols].view(B, cols).int()
        self.dense = []  # per session the tokens' k and v [2][Hkv][n + t][D] as the cache's type holds them
        for b in range(B):
            total = self.n[b] + self.t[b]
            x = normal(2, Hkv, total, D).to(dtype)
            self.dense.append(x)
            for j in range(total):
                if self.t[b] == 0 or not self.seen_by_any(b, j):
                    continue
                both[:, table[b, j // page], :, j % page] = x[:, :, j].float()
        both = both.to(dtype).to(DEV)
        if layout == "hnd":
            self.k, self.v = both[0], both[1]
        elif layout == "nhd":  # [pages][page][Hkv][D] in memory
            both = both.transpose(2, 3).contiguous().transpose(2, 3)
            self.k, self.v = both[0], both[1]
        elif layout == "paired":  # a page's keys and values side by side
            both = both.permute(1, 2, 0, 3, 4).contiguous().permute(2, 0, 1, 3, 4)
            self.k, self.v = both[0], both[1]
        self.table, self.lens = table.to(DEV), torch.tensor(self.n, dtype=torch.int32, device=DEV)
        self.t_rows = None if t_rows is None else torch.tensor(self.t, dtype=torch.int32, device=DEV)
        self.q_host = (normal(B, T, Hq, D) * q_scale).to(dtype)
        for b in range(B):
            self.q_host[b, self.t[b]:] = math.nan
        self.fuse(fused)

    def fuse(self, fused):
        B, T, Hq, Hkv, D = self.B, self.T, self.Hq, self.Hkv, self.D
        new = torch.full((B, T, 2, Hkv, D), math.nan, dtype=self.dtype)
        for b in range(B):
            x = self.dense[b][:, :, self.n[b]:]
            new[b, :self.t[b]] = x.permute(2, 0, 1, 3)
        if fused:  # q, k and v as parts of one projection's output
            x = torch.cat((self.q_host.flatten(2), new.flatten(2)), 2).to(DEV)
            self.q = x[:, :, :Hq * D].unflatten(2, (Hq, D))
            self.k_rows = x[:, :, Hq * D:(Hq + Hkv) * D].unflatten(2, (Hkv, D))
            self.v_rows = x[:, :, (Hq + Hkv) * D:].unflatten(2, (Hkv, D))
        else:
            self.q = self.q_host.to(DEV)
            self.k_rows, self.v_rows = (new[:, :, i].contiguous().to(DEV) for i in (0, 1))

    def spread(self, stride):
        """Pages `stride` elements apart, a page's keys and values side by side."""
        pages, block = self.k.shape[0], self.k[0].numel()
        far = torch.empty(stride * (pages - 1) + 2 * block, dtype=self.dtype, device=DEV)
        for i, name in enumerate("kv"):
            x = far.as_strided(self.k.shape, (stride, *self.k[0].contiguous().stride()), i * block)
            setattr(self, name, x.copy_(getattr(self, name)))
        return self

    def sees(self, p, j):
        return j <= p and (self.window == 0 or p - j < self.window or j < self.sinks)

    def seen_by_any(self, b, j):
        return any(self.sees(self.n[b] + t, j) for t in range(self.t[b]))

    def cache(self):
        return kb.PagedCache(self.k, self.v, self.table, self.lens)

    def see(self):
        return {"t_rows": self.t_rows, "window": self.window, "sinks": self.sinks}

    def hidden(self, b):
        p = self.n[b] + torch.arange(self.t[b])[:, None]
        j = torch.arange(self.n[b] + self.t[b])[None]
        hide = j > p
        if self.window:
            hide |= (p - j >= self.window) & (j >= self.sinks)
        return hide

    def head(self, b, h):
        """Scores [t][G][n + t] (hidden ones -inf), values, and a bound of the scores' error."""
        k, v = (self.dense[b][i, h].to(F64) for i in (0, 1))
        q = self.q_host[b, :self.t[b], h * self.G:(h + 1) * self.G].to(F64)
        s = torch.einsum("tgd,nd->tgn", q, k) * self.scale
        s = s.masked_fill(self.hidden(b)[:, None], -math.inf)
        # D products and their sum in f32, then two roundings more: each half an ulp of a partial sum
        ds = (self.D + 4) * 2.0**-24 * self.scale * float((q.norm(dim=-1).max() * k.norm(dim=-1).max()))
        return s, v, ds

    def attend(self):
        """out, lse and their tolerances [B][T][Hq]..., NaN in rows that stay as they are."""
        u = torch.finfo(self.dtype).eps / 2
        shape = (self.B, self.T, self.Hq, self.D)
        out, tol = (torch.full(shape, math.nan, dtype=F64) for _ in range(2))
        lse, tol_lse = (torch.full(shape[:3], math.nan, dtype=F64) for _ in range(2))
        for b in range(self.B):
            for h in range(self.Hkv if self.t[b] else 0):
                s, v, ds = self.head(b, h)
                mine = slice(h * self.G, (h + 1) * self.G)
                total = torch.logsumexp(s, 2)
                p = (s - total[..., None]).exp()
                o = torch.einsum("tgn,nd->tgd", p, v)
                size = torch.einsum("tgn,nd->tgd", p, v.abs())
                # the weights' rounding u, the scores' error in weights and in their sum, f32 sums and
                # exponentials 2^-17; a weight under the type's smallest normal number is off by half of its
                # least step at most, the largest weight being 1; the result's own rounding
                step = torch.finfo(self.dtype).smallest_normal * torch.finfo(self.dtype).eps / 2
                lost = step * (v.abs().sum(0) + 1)
                out[b, :self.t[b], mine] = o
                tol[b, :self.t[b], mine] = u * o.abs() + (u + 2 * ds + 2.0**-17) * size * (1 + u) + lost
                lse[b, :self.t[b], mine] = total
                tol_lse[b, :self.t[b], mine] = ds + 2.0**-17 + 2.0**-22 * total.abs()
        return out, lse, tol, tol_lse

    def share(self, lse, b):
        """Shares [Hkv][n + t] with the given lse [B][T][Hq], and their tolerance."""
        share, tol = [], []
        for h in range(self.Hkv):
            s, _, ds = self.head(b, h)
            l = lse[b, :self.t[b], h * self.G:(h + 1) * self.G].to(F64)
            x = torch.where(l[..., None] == -math.inf, 0.0, (s - l[..., None]).exp()).sum((0, 1))
            share.append(x)
            # exponents of size |s| + |lse| in f32, the sums
            far = float(torch.where(s == -math.inf, 0.0, s.abs()).max() + l.abs().max())
            tol.append(x * (2 * ds + far * 2.0**-21 + 2.0**-17))
        return torch.stack(share), torch.stack(tol)


def near(got, want, tol, what=""):
    got, want, tol = (x.to(F64).cpu() for x in (got, want, tol))
    there = ~torch.isnan(want)
    bad = there & ~((got - want).abs() <= tol) & ~((want == got))
    if bad.any():
        at = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {int(there.sum())} off, first at {at}: "
                             f"{float(got[at])} for {float(want[at])}, tolerance {float(tol[at]):.3g}")
    return there


def kept_of(mass, n, budget, recent, sinks):
    """Positions that an eviction keeps of n tokens with these masses (a list of floats)."""
    if n <= budget:
        return list(range(n))
    value = lambda j: -math.inf if math.isnan(mass[j]) else mass[j]  # noqa: E731
    middle = sorted(range(sinks, n - recent), key=lambda j: (math.isnan(mass[j]), -value(j), j))
    return sorted([*range(sinks), *middle[:budget - sinks - recent], *range(n - recent, n)])
