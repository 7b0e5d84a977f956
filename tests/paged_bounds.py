"""64-bit attention over BF16 pages with a bound of the kernels' error for each output, and caches to test it on.

Queries and keys are small integers, so that every q.k is exact in the kernel's fp32 sums. What is left, relative to a
weight 2^(x - m), x the logit in log2 units, `span` the range of a head's logits, eps = 2^-24 (half a step of fp32):
- x: the scale and the product are rounded, 2 eps |x|; the reference m cancels between numerator and denominator;
- x - m: eps (span + 8), as the reference is at most 8 below the largest logit; exp2f: two units, 4 eps;
- the reference is raised at the first page (nothing is scaled yet) and when a head's logit passes it by 8: at most
  span / 8 + 1 times for each of the g heads of a group, never where span < 8. A raise scales by exp2f of the
  difference: 4 eps + eps, and eps of the difference, whose sum is at most span;
- a warp's and a split's part are joined by such factors: twice 5 eps + eps span.
Numerator, relative to sum p |v|: the three bf16 pieces leave 2^-27; a tensor-core product of 16 terms and an
accumulator truncates each of the 17 by at most 2^-23 of their sum, the lower pieces' by 2^-8 of that; a page's sums
are added with one rounding, as are the parts of at most `adds` warps and splits. The sum of weights has four
roundings a page and as many joins. The division rounds once. All this is for an fp32 output; a bf16 one is that, rounded
to nearest even.
"""

import numpy as np
import torch

from oracle import paged

P = 16
EPS = 2.0 ** -24
WARP_PAGES = 128         # pages that one warp takes at most
JOINS = 72               # additions that join warps and splits at most


def attention(q, k, v, sm_scale, g, logits=None, weights=None):
    """(out, bound) for q [g, d], k and v [n, d] of one KV head in float64. `logits` and `weights` plant a mistake: they
    map the exact ones."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    x = (q @ k.T) * (sm_scale * 1.4426950408889634)
    if logits is not None:
        x = logits(x)
    top = x.max(1, keepdim=True).values
    p = torch.exp2(x - top)
    if weights is not None:
        p = weights(p)
    total = p.sum(1, keepdim=True)
    p = p / total
    out = p @ v
    span = float((x.max(1).values - x.min(1).values).max())
    raises = g * (int(span / 8) + 1) if span >= 8 else 0
    ln2 = 0.6931471805599453
    fixed = 4 * EPS + ln2 * EPS * (span + 8) + raises * 5 * EPS + ln2 * EPS * span + 2 * (5 * EPS + ln2 * EPS * span)
    w = 2 * EPS * ln2 * x.abs() + fixed                                   # per weight
    pages = min(-(-k.shape[0] // P), WARP_PAGES)
    sums = (p * w) @ v.abs()
    size = p @ v.abs()
    bound = sums + size * (2.0 ** -27 + 17 * 2.0 ** -23 * (1 + 2.0 ** -7) + (pages + JOINS) * EPS)
    bound = bound + out.abs() * ((p * w).sum(1, keepdim=True) + (4 * pages + JOINS) * EPS + 2 * EPS)
    return out, bound * (1 + 2.0 ** -10)                                  # second-order terms


class IntCache:
    """Sequences of any length over a small pool: integer keys within +-2, normal values. Logical pages alias the pool's
    but for each sequence's last one, whose values are 32 times as large and whose rows behind the length hold NaN, so
    that the last token and what lies behind it both show. Table entries behind the length are junk."""

    def __init__(self, seed, lens, h_q, h_kv, d, pool_pages=300, pad=0, q_values=1):
        r = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        self.h_q, self.h_kv, self.d, self.g = h_q, h_kv, d, h_q // h_kv
        batch = len(lens)
        pages = pool_pages + batch
        pool = torch.empty(pages, h_kv, 2, P, d, dtype=torch.bfloat16)
        gen = torch.Generator().manual_seed(seed)
        pool[:, :, 0] = torch.randint(-2, 3, (pages, h_kv, P, d), generator=gen).to(torch.bfloat16)
        pool[:, :, 1] = torch.randn(pages, h_kv, P, d, generator=gen).to(torch.bfloat16)
        self.q = torch.randint(-q_values, q_values + 1, (batch, h_q, d), generator=gen).to(torch.bfloat16)
        stride = max([paged.pages_for(int(n)) for n in lens] + [1]) + pad
        tables = r.integers(-5, 2 * pages, (batch, stride))
        for b, n in enumerate(map(int, lens)):
            need = paged.pages_for(n)
            if need == 0:
                continue
            tables[b, :need - 1] = r.integers(0, pool_pages, need - 1)
            last, rows = pool_pages + b, n - (need - 1) * P
            tables[b, need - 1] = last
            pool[last, :, 1] *= 32
            pool[last, :, :, rows:] = float("nan")
        self.pool, self.tables = pool, torch.from_numpy(tables.astype(np.int32))
        self.steps = torch.zeros(h_kv, d, dtype=torch.int8)
        b = np.sort(r.integers(-127, 128, (pages, h_kv, 2, d)), 2)
        self.bounds = torch.from_numpy(b.astype(np.int8))

    def rows(self, b, h, pages=None, device="cpu"):
        """K and V rows of the given logical pages (all of them) in float64."""
        n = int(self.lens[b])
        pages = torch.arange(paged.pages_for(n)) if pages is None else torch.as_tensor(pages, dtype=torch.long)
        ids = self.tables[b].long()[pages]
        real = (ids >= 0) & (ids < self.pool.shape[0])
        pages, ids = pages[real], ids[real]
        kv = self.pool[:, h].to(device)[ids.to(device)].double()                       # [pages, 2, 16, d]
        inside = (pages[:, None] * P + torch.arange(P) < n).reshape(-1).to(device)
        return kv[:, 0].reshape(-1, self.d)[inside], kv[:, 1].reshape(-1, self.d)[inside]

    def reference(self, sm_scale, chosen=None, device="cpu"):
        """(out, bound), [B, H_q, d] in float64, over the chosen[b][h] logical pages (all of them)."""
        out, bound = (torch.zeros(len(self.lens), self.h_q, self.d, dtype=torch.float64, device=device) for _ in range(2))
        for b in range(len(self.lens)):
            for h in range(self.h_kv):
                k, v = self.rows(b, h, None if chosen is None else chosen[b][h], device)
                q = self.q[b, h * self.g:(h + 1) * self.g].to(device).double()
                at = slice(h * self.g, (h + 1) * self.g)
                out[b, at], bound[b, at] = attention(q, k, v, sm_scale, self.g)
        return out, bound


def choose(q, steps, bounds, table, length, top, sink, recent):
    """oracle.paged.select for a whole sequence at once: q [H_q, d], bounds [pages, H_kv, 2, d]; a list for each head."""
    h_kv = bounds.shape[1]
    g = q.shape[0] // h_kv
    n = paged.pages_for(length)
    kept = min(n, paged.pages_for(sink))
    first = min(n, max(length - recent, 0) // P)
    cand = np.arange(kept, max(first, kept))
    ids = np.asarray(table)[cand]
    real = (ids >= 0) & (ids < bounds.shape[0])
    got = []
    for h in range(h_kv):
        b = bounds[np.where(real, ids, 0), h].astype(np.float64)                       # integers: exact
        score = np.full(len(cand), -np.inf)
        for x in q[h * g:(h + 1) * g]:
            u, e = paged.query_codes(x, steps[h])
            u = u.astype(np.float64)
            score = np.maximum(score, (b[:, 1] @ np.maximum(u, 0) + b[:, 0] @ np.minimum(u, 0)) * 2.0 ** e)
        score = np.where(real, score, -np.inf)
        best = cand[np.lexsort((cand, -score))[:top]]
        got.append(np.sort(np.concatenate([np.arange(kept), best, np.arange(max(first, kept), n)])).tolist())
    return got
