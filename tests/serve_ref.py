"""Plain forms of the operators around windows with sinks, drafted trees and
shared pages, and their kernels' error bounds, for the tests (see paged_ref for
how the attention's and the rotation's bounds are counted)."""
import torch

import paged_ref as ref
from paged_ref import F32, half_step


def attend_seen(q, k, v, seen, scale, cache_dtype, out_dtype, shift):
    """q [n, h, d], k, v [m, kv_heads, d], seen [n, m] bool -> out, lse and
    their bounds in float64.  Unseen tokens take no part; a row that sees
    nothing gives zeros and -infinity."""
    parts = []
    for i in range(q.shape[0]):
        at = seen[i].nonzero()[:, 0]
        parts.append(ref.attend(q[i:i + 1], k[at], v[at], [at.numel() - 1], scale, 0, cache_dtype,
                                out_dtype, shift))
    return tuple(torch.cat(x) for x in zip(*parts))


def sinks_seen(pos, m, window, sinks, device):
    """Row at position p sees j <= p with j > p - window or j < sinks."""
    j = torch.arange(m, device=device)[None]
    p = torch.tensor(pos, device=device)[:, None]
    near = (j > p - window) if window else torch.ones_like(j, dtype=torch.bool)
    return (j <= p) & (near | (j < sinks))


def ancestors(parent):
    """see[i][t]: token i of a tree follows token t or is it."""
    see = []
    for i, p in enumerate(parent):
        row = list(see[p]) if p >= 0 else [False] * len(parent)
        row[i] = True
        see.append(row)
    return see


def depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def normed(x, weight, eps):
    """x [n, heads, d] float64."""
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * weight.double()


def norm_error(y, d):
    """|error| of a normed value before the rotation: a sum of d squares (at
    most d binary32 additions), halved by the root; the mean, eps, the root (2
    steps) and the two products."""
    return y.abs() * ((d / 2 + 8) * F32)


def rotate_error(err, cos_sin, pos, interleaved):
    """Errors of the rotation's inputs carried through it."""
    r = cos_sin.shape[1]
    cs = cos_sin.double()[pos].abs()
    c, s = cs[:, None, : r // 2], cs[:, None, r // 2:]
    out = err.clone()
    i = torch.arange(r // 2, device=err.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    a, b = err[..., ia], err[..., ib]
    out[..., ia], out[..., ib] = a * c + b * s, b * c + a * s
    return out


def append_norm(x, weight, eps, cos_sin, pos, interleaved, dtype):
    """Normed and turned rows with their bound: x [n, heads, d] any type."""
    y = x.double() if weight is None else normed(x.double(), weight, eps)
    err = torch.zeros_like(y) if weight is None else norm_error(y, x.shape[-1])
    mag = y.abs()
    if cos_sin is not None:
        err = rotate_error(err, cos_sin, pos, interleaved)
        y, turned = ref.rotate(y, cos_sin, pos, interleaved)
        mag = torch.maximum(turned, mag)
    return y, err * (1 + half_step(dtype)) + ref.rotate_bound(y, mag, dtype)


class Ledger:
    """The page ledger in plain lists: rows fork and resize one after another."""

    def __init__(self, table, lens, refs, page):
        self.table, self.lens, self.refs, self.page = table, lens, refs, page
        self.copies = []  # (page from, page to, tokens)

    def pages(self, n):
        return (n + self.page - 1) // self.page

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            if s < 0:
                continue
            for e in range(self.pages(self.lens[d])):
                self.refs[self.table[d][e]] -= 1
            for e in range(self.pages(self.lens[s])):
                self.table[d][e] = self.table[s][e]
                self.refs[self.table[s][e]] += 1
            self.lens[d] = self.lens[s]

    def take(self):
        new = self.refs.index(0)
        self.refs[new] = 1
        return new

    def resize(self, new_lens):
        for r, n in enumerate(new_lens):
            if n < self.lens[r]:
                for e in range(self.pages(n), self.pages(self.lens[r])):
                    self.refs[self.table[r][e]] -= 1
                self.lens[r] = n
        # a page counts as taken before any row lets go of a shared one: that
        # never frees a page, since the last holder keeps it
        for r, n in enumerate(new_lens):
            old = self.lens[r]
            if n <= old:
                continue
            e = old // self.page
            if old % self.page and self.refs[self.table[r][e]] > 1:
                new = self.take()
                self.copies.append((self.table[r][e], new, old % self.page))
                self.refs[self.table[r][e]] -= 1
                self.table[r][e] = new
            for e in range(self.pages(old), self.pages(n)):
                self.table[r][e] = self.take()
            self.lens[r] = n
