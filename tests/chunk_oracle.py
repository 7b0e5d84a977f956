"""fp64 definition of oscar_extend_bf16 for the tests, and the error that its arithmetic allows."""

import numpy as np

P = 16


def rows_of(pool, table, length, h):
    """(k, v, there) of one head's first `length` tokens; tokens of a page id outside the pool are not there."""
    t = np.arange(length)
    page = np.asarray(table, np.int64)[t // P] if length else np.zeros(0, np.int64)
    there = (page >= 0) & (page < len(pool))
    at = np.where(there, page, 0)
    return pool[at, h, 0, t % P], pool[at, h, 1, t % P], there


def extend(q, pool, tables, row_start, total_len, sm_scale, exact_weights=False):
    """(out, bound), [n, H_q, d] each; rows of no request are NaN in out.

    q [n, H_q, d], pool [pages, H_kv, 2, 16, d]: float64. bound, derived from the arithmetic: products of bf16 are
    exact; a logit is a sum of d of them in d / 16 tensor-core steps, each off by at most 9 * 2^-23 of the sum of
    magnitudes A (natural units), scaled and exponentiated in fp32: a weight is off by w = A (9 d / 16 + 2) 2^-23 + 4 * 2^-23
    relative, and by 2^-8 by its rounding to bf16, e = w + 2^-8 together (2^-8 w apart). A normalised mean whose weights
    are off by e is off by e sum(w |v - out|) / (1 - e) <= e (mean |v| + |out|) (1 + 2 e). Sums take 8 tensor-core steps a
    tile of 128 tokens, off by at most 9 * 2^-23 of the magnitudes each, and a few rounded operations: (72 tiles + 64) 2^-23
    of mean |v|. The output is rounded once: 2^-8 of it. With exact_weights (sm_scale ln 2, whole logits) weights are
    powers of two and both sums exact, here too; what is left are two roundings of the normalisation and the one to
    bf16."""
    n, h_q, d = q.shape
    h_kv = pool.shape[1]
    g = h_q // h_kv
    out, bound = np.full(q.shape, np.nan), np.zeros(q.shape)
    for b in range(len(total_len)):
        lo, hi, total = int(row_start[b]), int(row_start[b + 1]), int(total_len[b])
        if hi == lo:
            continue
        pos = total - hi + np.arange(lo, hi)
        for h in range(h_kv):
            k, v, there = rows_of(pool, tables[b], total, h)
            for j in range(h * g, (h + 1) * g):
                with np.errstate(invalid="ignore"):
                    x = (q[lo:hi, j] @ k.T) * (1.0 if exact_weights else sm_scale)
                    size = (np.abs(q[lo:hi, j]) @ np.abs(k).T).max(1, initial=0.0) * sm_scale
                seen = (np.arange(total)[None] <= pos[:, None]) & there[None]
                x = np.where(seen, x, -np.inf)
                top = x.max(1, initial=-np.inf, keepdims=True)
                p = (np.exp2 if exact_weights else np.exp)(x - np.where(np.isneginf(top), 0.0, top))
                total_p = np.maximum(p.sum(1, keepdims=True), 1e-300)
                values = np.where(there[:, None], v, 0.0)
                if not np.isfinite(values).all():            # tokens without weight do not count, whatever they hold
                    y = np.stack([(np.where(w[:, None] > 0, w[:, None] * values, 0.0)).sum(0) for w in p]) / total_p
                    mean = np.abs(y)
                else:
                    y, mean = (p @ values) / total_p, (p @ np.abs(values)) / total_p
                out[lo:hi, j] = y
                e = 0.0 if exact_weights else size[:, None] * (9 * d / 16 + 2) * 2.0 ** -23 + 4 * 2.0 ** -23 + 1.01 * 2.0 ** -8
                steps = 2.0 ** -22 * np.abs(y) if exact_weights else (72 * (total // 128 + 1) + 64) * 2.0 ** -23 * mean
                err = e * (mean + np.abs(y)) * (1 + 2 * e) + steps
                bound[lo:hi, j] = err + 2.0 ** -8 * (np.abs(y) + err)
    return out, bound
