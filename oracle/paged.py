"""fp64 oracle of the BF16 paged-cache operators: planning, key bounds, page selection, attention.

Written from the definitions, one request, page and head at a time, with Python integers and NumPy
float64; it shares no code with the GPU path.
"""

import math

import numpy as np

P = 16


def pages_for(n):
    return -(-n // P)


def plan_append(seq_len, new_len, free_pages, free_head, tables, slot_cap):
    """(tables, slots, row_start, total_len, state): requests in order, pages in the free list's order."""
    tables = np.array(tables, np.int32, copy=True)
    slots = np.full(slot_cap, -1, np.int64)
    avail = len(free_pages) - free_head if 0 <= free_head < len(free_pages) else 0
    row_start, total_len, rejected = [0], [], []
    taken = wanted = 0
    for b, (s, n) in enumerate(zip(map(int, seq_len), map(int, new_len))):
        row = row_start[-1]
        row_start.append(row + max(n, 0))
        ok = s >= 0 and n >= 0 and s + n <= P * tables.shape[1] and row + n <= slot_cap
        if ok:
            need = pages_for(s + n) - pages_for(s)
            wanted += need
            ok = need == 0 or wanted <= avail
        if not ok:
            rejected.append(b)
            total_len.append(s)
            continue
        for j in range(need):
            tables[b, pages_for(s) + j] = free_pages[free_head + taken + j]
        taken += need
        for i in range(n):
            t = s + i
            slots[row + i] = int(tables[b, t // P]) * P + t % P
        total_len.append(s + n)
    state = [free_head + taken, row_start[-1], len(rejected), rejected[0] if rejected else -1]
    return tables, slots, np.array(row_start, np.int32), np.array(total_len, np.int32), np.array(state, np.int32)


def key_codes(k, steps):
    """Integer codes of keys [..., d] in steps 2^steps: clamp(rint(k 2^-step), -127, 127), 0 for NaN."""
    with np.errstate(invalid="ignore", over="ignore"):
        c = np.rint(np.asarray(k, np.float64) * np.exp2(-np.asarray(steps, np.float64)))
    return np.clip(np.where(np.isnan(c), 0.0, c), -127, 127).astype(np.int64)


def append(pool, bounds, k, v, slots, steps=None):
    """New rows into pool [pages, H, 2, 16, d] and bounds [pages, H, 2, d] (or None), in place."""
    last = None
    fresh = set()
    for i, slot in enumerate(map(int, slots)):
        if not 0 <= slot < pool.shape[0] * P:
            last = None
            continue
        page, row = divmod(slot, P)
        pool[page, :, 0, row], pool[page, :, 1, row] = k[i], v[i]
        if bounds is None:
            continue
        if page != last:                        # a new run: with row 0 in it, the page's bounds start anew
            run = [slot]
            for s in map(int, slots[i + 1:]):
                if s < 0 or s // P != page:
                    break
                run.append(s)
            if any(s % P == 0 for s in run):
                fresh.add(page)
                bounds[page, :, 0], bounds[page, :, 1] = 127, -127
        last = page
        c = key_codes(k[i], steps)
        bounds[page, :, 0] = np.minimum(bounds[page, :, 0], c)
        bounds[page, :, 1] = np.maximum(bounds[page, :, 1], c)


def attend(q, k, v, sm_scale):
    """softmax(sm_scale q k^T) v for q [g, d], k and v [n, d]; zeros for n = 0."""
    if len(k) == 0:
        return np.zeros_like(q)
    x = (q @ k.T) * sm_scale
    w = np.exp(x - x.max(axis=1, keepdims=True))
    return (w @ v) / w.sum(axis=1, keepdims=True)


def rows_of(pool, table, pages, length, h, kind):
    """Rows of one head over the given logical pages, [n, d]; a page id outside the pool has none."""
    got = [pool[table[p], h, kind, :max(0, min(P, length - p * P))] for p in pages if 0 <= table[p] < pool.shape[0]]
    return np.concatenate(got).astype(np.float64) if got else np.zeros((0, pool.shape[-1]))


def decode(q, pool, tables, lens, sm_scale):
    """Dense decode: q [B, H_q, d] -> [B, H_q, d]."""
    out = np.zeros(q.shape)
    h_kv = pool.shape[1]
    g = q.shape[1] // h_kv
    for b, n in enumerate(map(int, lens)):
        for h in range(h_kv):
            k, v = (rows_of(pool, tables[b], range(pages_for(n)), n, h, i) for i in (0, 1))
            out[b, h * g:(h + 1) * g] = attend(np.asarray(q[b, h * g:(h + 1) * g], np.float64), k, v, sm_scale)
    return out


def query_codes(q, steps):
    """(codes, e) of one query head: x = q 2^steps, codes in units of 2^e."""
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.asarray(q, np.float64) * np.exp2(np.asarray(steps, np.float64))
        x = np.where(np.isfinite(x.astype(np.float32)), x, 0.0)
    top = float(np.abs(x).max())
    if top < 2.0 ** -60:
        return np.zeros(len(x), np.int64), 0
    e = min(math.frexp(top)[1] - 7, 60)
    return np.clip(np.rint(x * 2.0 ** -e), -127, 127).astype(np.int64), e


def select(q, steps, bounds, table, length, top, sink, recent):
    """Ascending logical pages of one KV head: q [g, d], bounds [pages, 2, d] of this head, its block table."""
    n = pages_for(length)
    kept = [p for p in range(n) if p < pages_for(sink) or p >= max(length - recent, 0) // P]
    cand = [p for p in range(n) if p not in set(kept)]
    codes = [query_codes(x, steps) for x in q]

    def score(p):
        if not 0 <= table[p] < bounds.shape[0]:
            return -math.inf
        lo, hi = (bounds[table[p], i].astype(np.int64) for i in (0, 1))
        return max(int(np.maximum(u * lo, u * hi).sum()) * 2.0 ** e for u, e in codes)

    best = sorted(cand, key=lambda p: (-score(p), p))[:top]
    return sorted(kept + best)


def decode_sparse(q, pool, bounds, steps, tables, lens, top, sink, recent, sm_scale):
    """(out, chosen): chosen[b][h] the list of logical pages."""
    out = np.zeros(q.shape)
    h_kv = pool.shape[1]
    g = q.shape[1] // h_kv
    chosen = []
    for b, n in enumerate(map(int, lens)):
        chosen.append([])
        for h in range(h_kv):
            qh = np.asarray(q[b, h * g:(h + 1) * g], np.float64)
            pages = select(qh, steps[h], bounds[:, h], tables[b], n, top, sink, recent)
            k, v = (rows_of(pool, tables[b], pages, n, h, i) for i in (0, 1))
            out[b, h * g:(h + 1) * g] = attend(qh, k, v, sm_scale)
            chosen[-1].append(pages)
    return out, chosen
