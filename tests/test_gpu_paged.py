"""The BF16 paged-cache operators against their fp64 oracle: plan, append, dense and sparse decode.

Tolerance of a decode, derived from the arithmetic. Products of bf16 are exact; a logit is a sum of d of
them in d / 16 tensor-core steps, each off by at most 9 * 2^-23 of the sum of magnitudes A (in units of the
logit, natural), then scaled in fp32 and exponentiated: a weight is off by at most
w = A (9 d / 16 + 2) 2^-23 + 4 * 2^-23 relative. Numerator and denominator both carry it, the page sums of
the numerator are truncated at 9 * 2^-23 for each of three steps and added with one rounding a page and
three a split join: |error| <= max|v| (2 w + (pages + 64) 2^-23). A bf16 output is rounded once: 2^-8 of it.
"""

import math

import numpy as np
import pytest
import torch

import cases
from bit_kv_cache_write_gb300 import oscar as O
from oracle import paged

pytestmark = pytest.mark.gpu
P = 16
BF, I32, I64, I8 = torch.bfloat16, torch.int32, torch.int64, torch.int8


def context(h_q, h_kv, d, **over):
    c = dict(n_layers=1, n_q_heads=h_q, n_kv_heads=h_kv, head_dim=d, group=32)
    c.update(over)
    return O.Oscar(**c)


def dev(a, cuda, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(cuda)
    return t if dtype is None else t.to(dtype)


def bf16(x):
    """The values rounded to bf16, as float64."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(BF).double().numpy()


# ---------------------------------------------------------------------------------------------- planning

def run_plan(ctx, cuda, seq, new, free, head, tables, cap):
    batch = len(seq)
    t = dev(np.asarray(tables, np.int32), cuda)
    slots = torch.full((cap,), 77, dtype=I64, device=cuda)
    rows, total, state = (torch.full((n,), 77, dtype=I32, device=cuda) for n in (batch + 1, batch, 4))
    ctx.plan_append(dev(np.asarray(seq, np.int32), cuda), dev(np.asarray(new, np.int32), cuda),
                    dev(np.asarray(free, np.int32), cuda), dev(np.asarray([head], np.int32), cuda), t, slots, rows,
                    total, state)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, slots, rows, total, state)]


def same_plan(got, want):
    for g, w, name in zip(got, want, ("tables", "slots", "row_start", "total_len", "state")):
        assert np.array_equal(g, w), name


@pytest.mark.parametrize("batch,hi,new_hi", [(1, 1, 1), (3, 40, 20), (64, 900, 1), (5, 300, 700), (1000, 60, 5),
                                             (1025, 33, 3), (2500, 20, 2)])
def test_plan_matches_the_oracle(cuda, batch, hi, new_hi):
    r = np.random.default_rng(batch)
    seq, new = r.integers(0, hi + 1, batch), r.integers(0, new_hi + 1, batch)
    stride = paged.pages_for(hi + new_hi)
    tables = r.integers(0, 1 << 20, (batch, stride)).astype(np.int32)
    need = int(sum(paged.pages_for(s + n) - paged.pages_for(s) for s, n in zip(seq, new)))
    free = r.permutation(1 << 16)[:need + 4].astype(np.int32)
    cap = int(new.sum()) + 5
    ctx = context(4, 2, 64)
    for head in (0, 4):
        same_plan(run_plan(ctx, cuda, seq, new, free, head, tables, cap),
                  paged.plan_append(seq, new, free, head, tables, cap))


@pytest.mark.parametrize("case", ["few_pages", "no_pages", "bad_lengths", "short_map", "narrow_table", "bad_head", "mixed"])
def test_plan_rejections_match_the_oracle(cuda, case):
    r = np.random.default_rng(5)
    batch, stride = 70, 6
    seq, new = r.integers(0, 50, batch), r.integers(0, 40, batch)
    tables = r.integers(0, 1000, (batch, stride)).astype(np.int32)
    free, head, cap = r.permutation(5000)[:200].astype(np.int32), 0, int(new.sum()) + 3
    if case in ("few_pages", "mixed"):
        free = free[:30]
    if case == "no_pages":
        free = free[:0]
    if case in ("bad_lengths", "mixed"):
        seq[[3, 60]], new[[0, 9]] = -1, -7
        new[30] = seq[31] = 2 ** 31 - 1                 # rows past 32 bits behind it, pages past the table
    if case == "short_map":
        cap = int(new.sum()) // 2
    if case == "narrow_table":
        seq[[5, 6, 69]] = [96, 81, 97]
    if case == "bad_head":
        head = -3
    got = run_plan(context(4, 2, 64), cuda, seq, new, free, head, tables, cap)
    want = list(paged.plan_append(seq, new, free, head, tables, cap)) if case not in ("bad_lengths", "mixed") else None
    if want is None:                                    # the oracle's row starts are not clamped to 32 bits
        t, s, total = tables.copy(), np.full(cap, -1, np.int64), []
        row = taken = wanted = rejected = 0
        first = -1
        rows = [0]
        for b in range(batch):
            ok = seq[b] >= 0 and new[b] >= 0 and seq[b] + new[b] <= P * stride and row + new[b] <= cap
            need = paged.pages_for(int(seq[b] + new[b])) - paged.pages_for(int(seq[b])) if ok else 0
            wanted += need
            ok = ok and (need == 0 or wanted <= len(free))
            if ok:
                t[b, paged.pages_for(int(seq[b])):][:need] = free[taken:taken + need]
                taken += need
                for i in range(new[b]):
                    s[row + i] = int(t[b, (seq[b] + i) // P]) * P + (seq[b] + i) % P
            else:
                rejected, first = rejected + 1, b if first < 0 else first
            total.append(seq[b] + new[b] if ok else seq[b])
            row += max(int(new[b]), 0)
            rows.append(min(row, 2 ** 31 - 1))
        want = [t, s, np.array(rows), np.array(total), np.array([taken, rows[-1], rejected, first])]
    same_plan(got, want)


def test_plan_of_no_request_and_of_no_room(cuda):
    ctx = context(4, 2, 64)
    got = run_plan(ctx, cuda, [], [], [4, 5], 1, np.zeros((0, 3)), 4)
    assert (got[1] == -1).all() and got[2].tolist() == [0] and got[4].tolist() == [1, 0, 0, -1]
    got = run_plan(ctx, cuda, [0, 16], [0, 0], [], 0, np.zeros((2, 1)), 0)
    assert got[2].tolist() == [0, 0, 0] and got[3].tolist() == [0, 16] and got[4].tolist() == [0, 0, 0, -1]


def test_captured_plan_carries_its_state(cuda):
    """One graph, replayed: lengths and free head move on the device."""
    ctx = context(4, 2, 64)
    batch, steps = 9, 40
    r = np.random.default_rng(3)
    start = r.integers(0, 40, batch)
    stride = paged.pages_for(int(start.max()) + steps)
    free = r.permutation(500)[:batch * 5].astype(np.int32)
    tables0 = r.integers(500, 600, (batch, stride)).astype(np.int32)
    seq, new, f, t = dev(start.astype(np.int32), cuda), torch.ones(batch, dtype=I32, device=cuda), dev(free, cuda), dev(tables0, cuda)
    slots, rows, state = torch.empty(batch, dtype=I64, device=cuda), torch.empty(batch + 1, dtype=I32, device=cuda), torch.zeros(4, dtype=I32, device=cuda)
    total = torch.empty(batch, dtype=I32, device=cuda)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.plan_append(seq, new, f, state[:1], t, slots, rows, total, state)
        seq.copy_(total)
    head, tables, lens = 0, tables0, start
    for _ in range(steps):
        graph.replay()
        tables, want, _, lens, st = paged.plan_append(lens, [1] * batch, free, head, tables, batch)
        head = int(st[0])
        torch.cuda.synchronize()
        assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(state.cpu().numpy(), st)
    assert np.array_equal(t.cpu().numpy(), tables)


# --------------------------------------------------------------------------------------------- appending

def append_case(seed, h_kv, d, slots, pages, odd=False):
    r = np.random.default_rng(seed)
    n = len(slots)
    k, v = (bf16(r.standard_normal((n, h_kv, d)) * 3) for _ in range(2))
    if odd and n > 3:
        k[0, 0, :4] = [np.nan, np.inf, -np.inf, 3e38]
        k[1, -1, 1], v[1, 0, 0] = np.nan, np.nan
    steps = r.integers(-7, -1, (h_kv, d)).astype(np.int8)
    pool = bf16(r.standard_normal((pages, h_kv, 2, P, d)))
    bounds = np.stack([r.integers(-90, -5, (pages, h_kv, d)), r.integers(5, 90, (pages, h_kv, d))], 2)
    return k, v, steps, pool, bounds


def slots_of(runs):
    return np.array([s for page, lo, hi in runs for s in (range(page * P + lo, page * P + hi) if page >= 0 else [-1] * hi)],
                    np.int64)


@pytest.mark.parametrize("h_kv,d", [(1, 64), (2, 128), (8, 128), (3, 64)])
@pytest.mark.parametrize("runs", [
    [(4, 0, 1)], [(4, 7, 8)], [(2, 0, 16), (9, 0, 16), (3, 0, 5)],
    [(5, 3, 16), (6, 0, 16), (0, 0, 2), (-1, 0, 3), (7, 15, 16), (8, 0, 1)],
    [(-1, 0, 2), (11, 9, 12), (-1, 0, 1)], [(p, 0, 16) for p in range(40)], [(p, p % 16, p % 16 + 1) for p in range(41)],
], ids=lambda r: "%druns" % len(r))
@pytest.mark.parametrize("with_bounds", [False, True])
def test_append_matches_the_oracle(cuda, h_kv, d, runs, with_bounds):
    slots = slots_of(runs)
    pages = 42
    k, v, steps, pool, bounds = append_case(len(slots), h_kv, d, slots, pages, odd=True)
    ctx = context(h_kv, h_kv, d)
    kv = torch.stack([dev(k, cuda, BF), dev(v, cuda, BF)], 1)          # token stride 2 h_kv d
    gp, gb = dev(pool, cuda, BF), dev(bounds.astype(np.int8), cuda)
    args = (dev(steps, cuda), gb) if with_bounds else (None, None)
    ctx.append_bf16(kv[:, 0], kv[:, 1], dev(slots, cuda), gp, *args)
    torch.cuda.synchronize()
    want_b = bounds.copy()
    paged.append(pool, want_b if with_bounds else None, k, v, slots, steps)
    got, want = gp.cpu().view(torch.int16), torch.from_numpy(pool.astype(np.float32)).to(BF).view(torch.int16)
    nan = torch.from_numpy(np.isnan(pool))
    assert torch.equal(got[~nan], want[~nan]) and bool(gp.cpu()[nan].isnan().all())
    assert np.array_equal(gb.cpu().numpy(), want_b)


def test_append_skips_slots_behind_the_pool(cuda):
    ctx = context(2, 2, 64, debug_bounds=1)
    pool = torch.zeros(2, 2, 2, P, 64, dtype=BF, device=cuda)
    k = torch.ones(3, 2, 64, dtype=BF, device=cuda)
    ctx.append_bf16(k, k, torch.tensor([32, 1, -5], device=cuda), pool)
    st, kind, index = ctx.debug_error()
    assert (st, kind, index) == (-5, 1, 32)
    assert float(pool.float().sum()) == 2 * 2 * 64 and float(pool[0, :, :, 1].float().sum()) == 2 * 2 * 64


def test_append_of_a_long_prefill(cuda):
    """More tokens than a wave of units: the units' shares of runs join without gaps."""
    h_kv, d, n = 4, 128, 9001
    r = np.random.default_rng(0)
    pages = 700
    perm = r.permutation(pages)
    t = np.arange(5, 5 + n)                                          # the first page holds five tokens already
    slots = perm[t // P] * P + t % P
    k, v, steps, _, _ = append_case(7, h_kv, d, slots, 1)
    pool, bounds = np.zeros((pages, h_kv, 2, P, d)), np.tile(np.array([-3, 3])[None, None, :, None], (pages, h_kv, 1, d))
    ctx = context(4, 4, 128)
    gp, gb = dev(pool, cuda, BF), dev(bounds.astype(np.int8), cuda)
    ctx.append_bf16(dev(k, cuda, BF), dev(v, cuda, BF), dev(slots, cuda), gp, dev(steps, cuda), gb)
    torch.cuda.synchronize()
    pool[slots // P, :, 0, slots % P], pool[slots // P, :, 1, slots % P] = k, v
    c = paged.key_codes(k, steps)
    for lp in range(t[0] // P, t[-1] // P + 1):
        rows = c[(t // P) == lp]
        b = bounds[perm[lp]]
        lo, hi = rows.min(0), rows.max(0)
        bounds[perm[lp], :, 0], bounds[perm[lp], :, 1] = (np.minimum(lo, b[:, 0]), np.maximum(hi, b[:, 1])) if lp == 0 else (lo, hi)
    assert np.array_equal(gp.cpu().double().numpy(), pool) and np.array_equal(gb.cpu().numpy(), bounds)


@pytest.mark.parametrize("h_kv,d", [(8, 128), (3, 64)])
@pytest.mark.parametrize("with_bounds", [False, True])
def test_append_of_many_ragged_runs(cuda, h_kv, d, with_bounds):
    """Enough tokens that a warp takes sixteen: runs of every length, in and across the warps' shares, with padding."""
    r = np.random.default_rng(d)
    pages, runs = 2600, []
    for p in r.permutation(pages)[:2500]:
        lo = int(r.integers(0, 16)) if r.random() < 0.5 else 0
        runs.append((int(p), lo, int(r.integers(lo + 1, 17))))
        if r.random() < 0.2:
            runs.append((-1, 0, int(r.integers(1, 4))))
    slots = slots_of(runs)
    assert len(slots) > 64 * 152
    k, v, steps, _, bounds = append_case(3, h_kv, d, slots, pages)
    pool = np.zeros((pages, h_kv, 2, P, d))
    gp, gb = dev(pool, cuda, BF), dev(bounds.astype(np.int8), cuda)
    context(h_kv, h_kv, d).append_bf16(dev(k, cuda, BF), dev(v, cuda, BF), dev(slots, cuda), gp,
                                       *((dev(steps, cuda), gb) if with_bounds else ()))
    torch.cuda.synchronize()
    paged.append(pool, bounds if with_bounds else None, k, v, slots, steps)
    assert np.array_equal(gp.cpu().double().numpy(), pool) and np.array_equal(gb.cpu().numpy(), bounds)


# ---------------------------------------------------------------------------------------------- decoding

class Cache:
    """Random pages for sequences of the given lengths; rows behind a length hold NaN."""

    def __init__(self, seed, lens, h_q, h_kv, d, pad=0, gain=1.0):
        r = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        need = [paged.pages_for(n) for n in lens]
        pages = sum(need) + 3
        self.pool = np.full((pages, h_kv, 2, P, d), np.nan)
        self.tables = r.integers(-5, 2 * pages, (len(lens), max(need + [1]) + pad)).astype(np.int32)   # junk behind the length
        perm, at = r.permutation(pages), 0
        for b, n in enumerate(lens):
            ids = perm[at:at + need[b]]
            at += need[b]
            self.tables[b, :need[b]] = ids
            rows = bf16(r.standard_normal((need[b] * P, h_kv, 2, d)) * gain)
            rows[n:] = np.nan
            self.pool[ids] = rows.reshape(need[b], P, h_kv, 2, d).transpose(0, 2, 3, 1, 4)
        self.q = bf16(r.standard_normal((len(lens), h_q, d)) * gain)
        self.steps = np.full((h_kv, d), -5, np.int8)
        c = paged.key_codes(self.pool[:, :, 0], self.steps[None, :, None])
        live = ~np.isnan(self.pool[:, :, 0])
        self.bounds = np.stack([np.where(live, c, 127).min(2), np.where(live, c, -127).max(2)], 2).astype(np.int8)

    def tolerance(self, want, out_type, sm_scale):
        k = np.nan_to_num(np.abs(self.pool[:, :, 0]))
        d = k.shape[-1]
        a = float((np.abs(self.q).max((0, 1)) * k.max((0, 1, 2))).sum()) * sm_scale
        w = a * (9 * d / 16 + 2) * 2.0 ** -23 + 4 * 2.0 ** -23
        pages = max(paged.pages_for(int(n)) for n in self.lens)
        tol = float(np.nan_to_num(np.abs(self.pool[:, :, 1])).max()) * (2 * w + (pages + 64) * 2.0 ** -23)
        return tol + (np.abs(want) * 2.0 ** -8 if out_type == BF else 0.0)


def run_dense(ctx, c, cuda, out_type, max_len=None, q=None):
    max_len = int(c.lens.max()) if max_len is None else max_len
    b, h_q, d = c.q.shape
    out = torch.full((b, h_q, d), float("nan"), dtype=out_type, device=cuda)
    ws = torch.full((max(1, ctx.decode_bf16_workspace_size(b, max_len)),), 255, dtype=torch.uint8, device=cuda)
    ctx.decode_bf16(dev(c.q, cuda, BF) if q is None else q, dev(c.pool, cuda, BF), dev(c.tables, cuda), dev(c.lens, cuda),
                    max_len, out, ws)
    torch.cuda.synchronize()
    return out.cpu().double().numpy()


def run_sparse(ctx, c, cuda, out_type, top, max_len=None):
    max_len = int(c.lens.max()) if max_len is None else max_len
    b, h_q, d = c.q.shape
    h_kv = c.pool.shape[1]
    cap = ctx.sparse_capacity(top)
    out = torch.full((b, h_q, d), float("nan"), dtype=out_type, device=cuda)
    chosen, n = torch.full((b, h_kv, cap), 77, dtype=I32, device=cuda), torch.full((b, h_kv), 77, dtype=I32, device=cuda)
    ws = torch.full((max(1, ctx.decode_bf16_sparse_workspace_size(b, max_len, top)),), 255, dtype=torch.uint8, device=cuda)
    ctx.decode_bf16_sparse(dev(c.q, cuda, BF), dev(c.pool, cuda, BF), dev(c.steps, cuda), dev(c.bounds, cuda),
                           dev(c.tables, cuda), dev(c.lens, cuda), max_len, top, chosen, n, out, ws)
    torch.cuda.synchronize()
    chosen, n = chosen.cpu().numpy(), n.cpu().numpy()
    lists = [[chosen[i, h, :n[i, h]].tolist() for h in range(h_kv)] for i in range(b)]
    assert all((chosen[i, h, n[i, h]:] == -1).all() for i in range(b) for h in range(h_kv))
    return out.cpu().double().numpy(), lists


def close(got, want, tol):
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) - tol).max()
    assert worst <= 0, "off by %.3g (output up to %.3g), %.3g over the bound" % (np.abs(got - want).max(), np.abs(want).max(), worst)


LENS = [[0], [1], [15, 16, 17], [0, 1, 300, 64], [1344], [777, 0, 2100, 33, 5], [4099]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("h_kv,g,d", [(2, 2, 64), (1, 8, 128), (8, 4, 128), (3, 1, 128), (2, 8, 64)])
def test_dense_matches_the_oracle(cuda, lens, h_kv, g, d):
    c = Cache(len(lens) + d, lens, h_kv * g, h_kv, d)
    ctx = context(h_kv * g, h_kv, d)
    want = paged.decode(c.q, c.pool, c.tables, c.lens, d ** -0.5)
    for out_type in (torch.float32, BF):
        close(run_dense(ctx, c, cuda, out_type), want, c.tolerance(want, out_type, d ** -0.5))


def test_dense_with_more_room_than_tokens(cuda):
    c = Cache(4, [200, 33, 0], 8, 2, 128, pad=300)
    want = paged.decode(c.q, c.pool, c.tables, c.lens, 128 ** -0.5)
    ctx = context(8, 2, 128)
    close(run_dense(ctx, c, cuda, torch.float32, max_len=16 * c.tables.shape[1]), want, c.tolerance(want, None, 128 ** -0.5))


def test_dense_with_sharp_logits(cuda):
    """Logits far apart, and rising along the sequence: the running reference is raised again and again."""
    c = Cache(5, [900], 8, 2, 64, gain=4.0)
    ids = c.tables[0, :paged.pages_for(900)]
    for i, p in enumerate(ids):
        c.pool[p, :, 0] = bf16(c.pool[p, :, 0] * (0.05 + i / len(ids)))
    want = paged.decode(c.q, c.pool, c.tables, c.lens, 0.125)
    close(run_dense(context(8, 2, 64), c, cuda, torch.float32), want, c.tolerance(want, None, 0.125))


def test_own_scale_and_strided_queries(cuda):
    c = Cache(6, [100, 500], 8, 4, 64)
    ctx = context(8, 4, 64, sm_scale=0.3)
    wide = torch.zeros(2, 8 + 4 + 4, 64, dtype=BF, device=cuda)          # q, k, v of one projection
    wide[:, :8] = dev(c.q, cuda, BF)
    want = paged.decode(c.q, c.pool, c.tables, c.lens, 0.3)
    close(run_dense(ctx, c, cuda, torch.float32, q=wide[:, :8]), want, c.tolerance(want, None, 0.3))


def test_masked_logits_and_a_row_without_weight(cuda):
    """Keys that send logits to -inf: no weight; all of a head's logits at -inf: zeros, as for no token."""
    c = Cache(7, [40], 4, 2, 64)
    c.q[0, :, 0] = 1.0
    for t in range(40):
        c.pool[c.tables[0, t // P], 0, 0, t % P, 0] = -np.inf if t != 21 else 0.0
        c.pool[c.tables[0, t // P], 1, 0, t % P, 0] = -np.inf
    got = run_dense(context(4, 2, 64), c, cuda, torch.float32)
    v = c.pool[c.tables[0, 21 // P], 0, 1, 21 % P]
    assert np.array_equal(got[0, :2], np.stack([v, v])) and (got[0, 2:] == 0).all()


def test_lengths_outside_their_range_count_as_the_nearer_end(cuda):
    c = Cache(8, [50, 50, 50], 4, 2, 64)
    want = paged.decode(c.q, c.pool, c.tables, [50, 0, 50], 0.125)
    ctx = context(4, 2, 64, debug_bounds=1)
    c.lens[:] = [50, -4, 5000]
    got = run_dense(ctx, c, cuda, torch.float32, max_len=50)
    c.lens[:] = 50
    close(got, want, c.tolerance(want, None, 0.125))
    st, kind, index = ctx.debug_error()
    assert st == -5 and kind == 3 and index in (-4, 5000)


@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_page_ids_outside_the_pool_are_masked(cuda, bad):
    c = Cache(9, [100, 60], 4, 2, 64)
    c.tables[0, 3], c.tables[1, :] = bad, bad
    want = paged.decode(c.q, c.pool, c.tables, c.lens, 0.125)
    ctx = context(4, 2, 64, debug_bounds=1)
    got = run_dense(ctx, c, cuda, torch.float32)
    close(got, want, c.tolerance(want, None, 0.125))
    assert (got[1] == 0).all() and ctx.debug_error()[:2] == (-5, 2)


def test_shared_pages_and_aliased_sequences(cuda):
    c = Cache(10, [320, 200], 8, 2, 128)
    c.tables[1, :12] = c.tables[0, :12]                        # a prefix that both read
    want = paged.decode(c.q, c.pool, c.tables, c.lens, 128 ** -0.5)
    close(run_dense(context(8, 2, 128), c, cuda, torch.float32), want, c.tolerance(want, None, 128 ** -0.5))


def test_pages_past_32_bits(cuda):
    """Page ids whose byte and element offsets pass 2^32, in a pool of 9.1 GB."""
    h_kv, d, pages = 8, 128, 139000                            # 65,536 bytes a page
    ctx = context(32, h_kv, d)
    pool = torch.empty(pages, h_kv, 2, P, d, dtype=BF, device=cuda)
    r = np.random.default_rng(11)
    ids = np.array([[pages - 1, 3, 70000, 66000, 138000]], np.int32)
    k, v = (bf16(r.standard_normal((70, h_kv, d))) for _ in range(2))
    q = bf16(r.standard_normal((1, 32, d)))
    t = np.arange(70)
    slots = ids[0, t // P].astype(np.int64) * P + t % P
    steps = torch.full((h_kv, d), -5, dtype=I8, device=cuda)
    bounds = torch.zeros(pages, h_kv, 2, d, dtype=I8, device=cuda)
    ctx.append_bf16(dev(k, cuda, BF), dev(v, cuda, BF), dev(slots, cuda), pool, steps, bounds)
    out = torch.empty(1, 32, d, device=cuda)
    ws = torch.empty(max(1, ctx.decode_bf16_workspace_size(1, 70)), dtype=torch.uint8, device=cuda)
    ctx.decode_bf16(dev(q, cuda, BF), pool, dev(ids, cuda), torch.tensor([70], dtype=I32, device=cuda), 70, out, ws)
    torch.cuda.synchronize()
    want = np.concatenate([paged.attend(q[0, h * 4:h * 4 + 4], k[:, h], v[:, h], d ** -0.5) for h in range(h_kv)])
    assert np.abs(out.cpu().numpy()[0] - want).max() <= 9e-3       # |v| <= 5, A <= 100: 5 * 2 * 100 * 74 * 2^-23
    assert np.array_equal(bounds[ids[0, 2]].cpu().numpy()[:, 0], paged.key_codes(k[32:48], -5).min(0))


SPARSE = [([1344], 8), ([0, 1, 300, 64, 330], 3), ([2000, 700, 4100, 37], 20), ([1000], 0), ([1000], 500), ([321], 1),
          ([17000, 900], 33)]


@pytest.mark.parametrize("lens,top", SPARSE, ids=str)
@pytest.mark.parametrize("h_kv,g,d", [(2, 2, 64), (1, 8, 128), (4, 4, 128), (3, 1, 64)])
def test_sparse_matches_the_oracle(cuda, lens, top, h_kv, g, d):
    c = Cache(len(lens) + top + d, lens, h_kv * g, h_kv, d)
    ctx = context(h_kv * g, h_kv, d)
    want, lists = paged.decode_sparse(c.q, c.pool, c.bounds, c.steps, c.tables, c.lens, top, 64, 256, d ** -0.5)
    for out_type in (torch.float32, BF):
        got, chosen = run_sparse(ctx, c, cuda, out_type, top)
        assert chosen == lists
        close(got, want, c.tolerance(want, out_type, d ** -0.5))


def test_sparse_with_the_longest_sequences_first(cuda):
    """Lengths far apart and enough heads that not all clusters run at once (they start with the longest): lists and
    outputs in the sequences' own order, for equal and empty ones too."""
    lens = [100, 50000, 0, 16, 50000, 7000, 1, 49000, 300, 300, 20000, 64, 900, 0, 31000, 12]
    c = Cache(16, lens, 8, 8, 64)
    want, lists = paged.decode_sparse(c.q, c.pool, c.bounds, c.steps, c.tables, c.lens, 60, 64, 256, 0.125)
    got, chosen = run_sparse(context(8, 8, 64), c, cuda, torch.float32, 60)
    assert chosen == lists
    close(got, want, c.tolerance(want, None, 0.125))
    wide = Cache(16, lens, 8, 8, 64, pad=6000)                       # a bound of 131k, as a server passes it
    got, chosen = run_sparse(context(8, 8, 64), wide, cuda, torch.float32, 60, max_len=131072)
    want, lists = paged.decode_sparse(wide.q, wide.pool, wide.bounds, wide.steps, wide.tables, wide.lens, 60, 64, 256, 0.125)
    assert chosen == lists
    close(got, want, wide.tolerance(want, None, 0.125))


def test_sparse_beyond_the_keys_that_shared_memory_holds(cuda):
    c = Cache(15, [265001, 40000], 2, 1, 64)
    ctx = context(2, 1, 64)
    want, lists = paged.decode_sparse(c.q, c.pool, c.bounds, c.steps, c.tables, c.lens, 70, 64, 256, 0.125)
    got, chosen = run_sparse(ctx, c, cuda, torch.float32, 70)
    assert chosen == lists
    close(got, want, c.tolerance(want, None, 0.125))


@pytest.mark.parametrize("sink,recent", [(0, 0), (0, 1), (5, 0), (16, 17), (64, 448)])
def test_sparse_windows(cuda, sink, recent):
    c = Cache(12, [1000, 1008, 3], 4, 2, 64)
    ctx = context(4, 2, 64, sink=sink, recent=recent)
    for top in (0, 7):
        want, lists = paged.decode_sparse(c.q, c.pool, c.bounds, c.steps, c.tables, c.lens, top, sink, recent, 0.125)
        got, chosen = run_sparse(ctx, c, cuda, torch.float32, top)
        assert chosen == lists
        close(got, want, c.tolerance(want, None, 0.125))


@pytest.mark.parametrize("kind", ["equal", "two_values", "zero_query", "tiny_query", "odd_query", "bad_page", "extreme"])
def test_sparse_ties_and_odd_values(cuda, kind):
    c = Cache(13, [2500, 900], 8, 2, 64)
    r = np.random.default_rng(1)
    if kind == "equal":
        c.bounds[:] = 5
    if kind == "two_values":
        c.bounds[:] = r.integers(0, 2, (len(c.bounds), 1, 1, 1))
    if kind == "zero_query":
        c.q[:] = 0
    if kind == "tiny_query":
        c.q[:] = bf16(np.sign(c.q) * 2.0 ** -58)
        c.q[0, 0] *= 2.0 ** -10
    if kind == "odd_query":
        c.q[0, 3, 5], c.q[1, 0, 0] = np.inf, np.nan
    if kind == "bad_page":
        c.tables[0, [20, 21, 22]] = -1
    if kind == "extreme":
        c.bounds[:, :, 0], c.bounds[:, :, 1] = -128, 127
        c.steps[:] = r.integers(-100, 101, c.steps.shape)
    ctx = context(8, 2, 64)
    _, lists = paged.decode_sparse(np.nan_to_num(c.q, posinf=0.0), c.pool, c.bounds, c.steps, c.tables, c.lens, 50, 64, 256, 0.125)
    got, chosen = run_sparse(ctx, c, cuda, torch.float32, 50)
    assert chosen == lists
    if kind != "odd_query":
        want, _ = paged.decode_sparse(c.q, c.pool, c.bounds, c.steps, c.tables, c.lens, 50, 64, 256, 0.125)
        close(got, want, c.tolerance(want, None, 0.125))


@pytest.mark.parametrize("h_kv,d", [(3, 64), (4, 128)])
def test_many_short_sequences(cuda, h_kv, d):
    """More (sequence, KV head) units than the card has room for at once."""
    r = np.random.default_rng(9)
    lens = r.integers(0, 900, 160)
    lens[[0, 5]] = 0, 1500
    c = Cache(17, lens, h_kv * 2, h_kv, d)
    ctx = context(h_kv * 2, h_kv, d)
    want = paged.decode(c.q, c.pool, c.tables, c.lens, d ** -0.5)
    close(run_dense(ctx, c, cuda, torch.float32), want, c.tolerance(want, None, d ** -0.5))
    want, lists = paged.decode_sparse(c.q, c.pool, c.bounds, c.steps, c.tables, c.lens, 11, 64, 256, d ** -0.5)
    got, chosen = run_sparse(ctx, c, cuda, torch.float32, 11)
    assert chosen == lists
    close(got, want, c.tolerance(want, None, d ** -0.5))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_one_apart_are_told_apart(cuda, d, sign):
    """Scores near the largest magnitude that differ by one unit: the product over the bounds is exact."""
    c = Cache(18, [16 * 220], 2, 1, d)
    r = np.random.default_rng(d)
    codes = sign * np.where(np.arange(d) < d - 2, 127, 1)                    # the query's codes, e = 0
    c.q[0, :] = bf16(codes[None] * 2.0 ** -5)                                # steps of 2^-5 below undo the scale
    c.steps[:] = 5
    c.bounds[:] = 127 if sign > 0 else -128
    rank = r.permutation(220)                                                # two channels of weight one: 0 .. 219
    low = np.minimum(rank, 120)
    for p in range(220):
        c.bounds[c.tables[0, p], 0, :, d - 2] = low[p] - (0 if sign > 0 else 120)
        c.bounds[c.tables[0, p], 0, :, d - 1] = rank[p] - low[p] - (0 if sign > 0 else 120)
    for top in (1, 17, 100):
        want = paged.select(c.q[0], c.steps[0], c.bounds[:, 0], c.tables[0], 16 * 220, top, 64, 256)
        _, chosen = run_sparse(context(2, 1, d), c, cuda, torch.float32, top)
        assert chosen[0][0] == want
        middle = [p for p in range(4, 204)]
        best = sorted(middle, key=lambda p: -sign * rank[p])[:top]
        assert want == sorted(set(range(4)) | set(range(204, 220)) | set(best))


def test_results_do_not_change_from_run_to_run(cuda):
    c = Cache(14, [3000, 1, 700, 2222], 8, 2, 128)
    ctx = context(8, 2, 128)
    first = run_dense(ctx, c, cuda, torch.float32), run_sparse(ctx, c, cuda, torch.float32, 40)[0]
    for _ in range(5):
        assert np.array_equal(first[0], run_dense(ctx, c, cuda, torch.float32))
        assert np.array_equal(first[1], run_sparse(ctx, c, cuda, torch.float32, 40)[0])


def test_streams_with_a_workspace_each(cuda):
    """Two decodes at once on two streams, and a captured one replayed with other lengths."""
    ctx = context(8, 2, 128)
    cs = [Cache(20 + i, [2000, 500], 8, 2, 128) for i in range(2)]
    want = [paged.decode(c.q, c.pool, c.tables, c.lens, 128 ** -0.5) for c in cs]
    held, streams = [], [torch.cuda.Stream() for _ in cs]
    for c in cs:
        held.append(dict(q=dev(c.q, cuda, BF), pool=dev(c.pool, cuda, BF), t=dev(c.tables, cuda), n=dev(c.lens, cuda),
                         out=torch.zeros(2, 8, 128, device=cuda),
                         ws=torch.empty(ctx.decode_bf16_workspace_size(2, 2000), dtype=torch.uint8, device=cuda)))
    torch.cuda.synchronize()
    for _ in range(20):
        for h, s in zip(held, streams):
            ctx.decode_bf16(h["q"], h["pool"], h["t"], h["n"], 2000, h["out"], h["ws"], stream=s)
    torch.cuda.synchronize()
    for c, h, w in zip(cs, held, want):
        close(h["out"].cpu().double().numpy(), w, c.tolerance(w, None, 128 ** -0.5))
    c, h = cs[0], held[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.decode_bf16(h["q"], h["pool"], h["t"], h["n"], 2000, h["out"], h["ws"])
    for lens in ([100, 0], [1999, 17]):
        h["n"].copy_(torch.tensor(lens, dtype=I32))
        graph.replay()
        torch.cuda.synchronize()
        w = paged.decode(c.q, c.pool, c.tables, lens, 128 ** -0.5)
        close(h["out"].cpu().double().numpy(), w, c.tolerance(w, None, 128 ** -0.5))


# --------------------------------------------------------------------------------------------- refusals

def test_refusals(cuda):
    ctx = context(4, 2, 64)
    q = torch.zeros(1, 4, 64, dtype=BF, device=cuda)
    pool = torch.zeros(4, 2, 2, P, 64, dtype=BF, device=cuda)
    t, n = torch.zeros(1, 4, dtype=I32, device=cuda), torch.full((1,), 64, dtype=I32, device=cuda)
    out = torch.zeros(1, 4, 64, device=cuda)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=cuda)
    steps, bounds = torch.zeros(2, 64, dtype=I8, device=cuda), torch.zeros(4, 2, 2, 64, dtype=I8, device=cuda)

    def status(call, *args):
        with pytest.raises(O.OscarError) as e:
            call(*args)
        return e.value.status

    assert status(ctx.decode_bf16, q, pool, t, n, 65, out, ws) == -1                  # past the table
    assert status(ctx.decode_bf16, q, pool, t, n, -1, out, ws) == -1
    assert status(ctx.decode_bf16, q, pool, t, n, (1 << 30) + 1, out, ws) == -2
    wide = torch.zeros(1, 1024, dtype=I32, device=cuda)
    assert status(ctx.decode_bf16, q, pool, wide, n, 16384, out, ws[:16]) == -7
    assert status(ctx.decode_bf16, q, pool, wide, n, 16384, out, None) == -7
    assert status(ctx.decode_bf16, q, pool, wide, n, 16384, out, torch.zeros(1 << 23, dtype=torch.uint8, device=cuda)[8:]) == -1
    assert status(ctx.decode_bf16, q, pool[:0], t, n, 64, out, ws) == -1
    odd = torch.zeros(1 + 4 * 64, dtype=BF, device=cuda)[1:].view(1, 4, 64)
    assert status(ctx.decode_bf16, odd, pool, t, n, 64, out, ws) == -1
    cap = ctx.sparse_capacity(2)
    chosen, count = torch.zeros(1, 2, cap, dtype=I32, device=cuda), torch.zeros(1, 2, dtype=I32, device=cuda)
    sparse = lambda top, *a: ctx.decode_bf16_sparse(q, pool, steps, bounds, t, n, 64, top, *a, out, ws)
    assert status(sparse, -1, chosen, count) == -1
    assert status(sparse, 65537, chosen, count) == -2
    with pytest.raises(ValueError, match="chosen"):
        sparse(3, chosen, count)
    with pytest.raises(ValueError, match="q must be"):
        ctx.decode_bf16(q[:, :3], pool, t, n, 64, out, ws)
    with pytest.raises(ValueError, match="out must"):
        ctx.decode_bf16(q, pool, t, n, 64, out.half(), ws)
    with pytest.raises(ValueError, match="tables"):
        ctx.decode_bf16(q, pool, t[0], n, 64, out, ws)
    with pytest.raises(ValueError, match="tables"):
        ctx.decode_bf16(q, pool, t.expand(2, 4), n, 64, out, ws)
    with pytest.raises(ValueError, match="out must hold"):
        ctx.decode_bf16(q, pool, t, n, 64, out[:, :3].contiguous(), ws)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        ctx.decode_bf16(q, pool, t, n, 64, out, ws[::2])
    with pytest.raises(ValueError, match="seq_len must be torch.int32"):
        ctx.decode_bf16(q, pool, t, n.long(), 64, out, ws)
    with pytest.raises(ValueError, match="bf16_pool must be a CUDA tensor"):
        ctx.decode_bf16(q, pool.cpu(), t, n, 64, out, ws)
    k = torch.zeros(2, 2, 64, dtype=BF, device=cuda)
    slots = torch.zeros(2, dtype=I64, device=cuda)
    with pytest.raises(ValueError, match="key_bounds"):
        ctx.append_bf16(k, k, slots, pool, steps, bounds[:3])
    with pytest.raises(ValueError, match="key_bounds"):
        ctx.append_bf16(k, k, slots, pool, steps)
    with pytest.raises(ValueError, match="heads must be contiguous"):
        ctx.append_bf16(torch.zeros(2, 2, 128, dtype=BF, device=cuda)[:, :, ::2], k, slots, pool)
    wide = torch.zeros(2, 2 * 64 + 4, dtype=BF, device=cuda)[:, :128].unflatten(1, (2, 64))
    assert status(ctx.append_bf16, wide, k, slots, pool) == -1                        # stride not a multiple of 8
    with pytest.raises(ValueError, match="slots"):
        ctx.append_bf16(k, k, slots[:1], pool)
    z = lambda m, dt=I32: torch.zeros(m, dtype=dt, device=cuda)
    with pytest.raises(ValueError, match="row_start"):
        ctx.plan_append(n, n, z(1), z(1), t, z(4, I64), z(1), z(1), z(4))
    lens, starts = z(3), z(4)
    plan = lambda seq, total, rows, state: ctx.plan_append(seq, z(3), z(1), z(1), z(12).view(3, 4), z(4, I64), rows, total, state)
    assert status(plan, lens, lens, starts, z(4)) == -1                               # in place
    both = z(8)
    assert status(plan, both[:3], both[2:5], starts, z(4)) == -1
    assert status(plan, lens, z(3), both[:4], both[3:7]) == -1
    for bad in (1 << 31, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="32 bits"):
            ctx.decode_bf16(q, pool, t, n, bad, out, ws)
        with pytest.raises(ValueError, match="32 bits"):
            sparse(bad, chosen, count)
    big = 65536
    assert status(ctx.plan_append, z(big), z(big), z(1), z(1), z(big).view(big, 1), z(4, I64), z(big + 1), z(big), z(4)) == -2


def test_injected_launch_failure(cuda, monkeypatch):
    ctx = context(4, 2, 64)
    k, slots = torch.zeros(1, 2, 64, dtype=BF, device=cuda), torch.zeros(1, dtype=I64, device=cuda)
    pool = torch.ones(1, 2, 2, P, 64, dtype=BF, device=cuda)
    monkeypatch.setenv("OSCAR_FAULT", "launch")
    with pytest.raises(O.OscarError) as e:
        ctx.append_bf16(k, k, slots, pool)
    assert e.value.status == -4 and float(pool.float().min()) == 1.0


def test_a_workspace_serves_smaller_calls(cuda):
    """Sized once for the largest batch and lengths; the sizes never fall as either grows."""
    ctx = context(8, 2, 128)
    sizes = [[ctx.decode_bf16_workspace_size(b, n) for n in (0, 16, 60, 500, 3000, 20000, 131072)] for b in (0, 1, 2, 7, 40, 500, 65535)]
    assert (np.diff(np.array(sizes, np.float64), axis=0) >= 0).all() and (np.diff(np.array(sizes, np.float64), axis=1) >= 0).all()
    sizes = [[ctx.decode_bf16_sparse_workspace_size(b, n, t) for n in (16, 500, 20000, 131072, 400000) for t in (0, 9, 300)] for b in (1, 7, 500)]
    assert (np.diff(np.array(sizes, np.float64), axis=0) >= 0).all()
    ws = torch.full((ctx.decode_bf16_workspace_size(200, 4000),), 255, dtype=torch.uint8, device=cuda)
    big = torch.full((ctx.decode_bf16_sparse_workspace_size(200, 4000, 100),), 255, dtype=torch.uint8, device=cuda)
    for lens in ([4000], [3999, 10], [100] * 30, [2000, 1500] * 8, [600] * 160, [60] * 200):
        c = Cache(len(lens), lens, 8, 2, 128)
        want = paged.decode(c.q, c.pool, c.tables, c.lens, 128 ** -0.5)
        q, pool, t, n = dev(c.q, cuda, BF), dev(c.pool, cuda, BF), dev(c.tables, cuda), dev(c.lens, cuda)
        out = torch.empty(len(lens), 8, 128, device=cuda)
        ctx.decode_bf16(q, pool, t, n, int(c.lens.max()), out, ws)
        close(out.cpu().double().numpy(), want, c.tolerance(want, None, 128 ** -0.5))
        for top in (3, 100):
            cap = ctx.sparse_capacity(top)
            chosen, count = torch.empty(len(lens), 2, cap, dtype=I32, device=cuda), torch.empty(len(lens), 2, dtype=I32, device=cuda)
            ctx.decode_bf16_sparse(q, pool, dev(c.steps, cuda), dev(c.bounds, cuda), t, n, int(c.lens.max()), top, chosen, count, out, big)
            want, _ = paged.decode_sparse(c.q, c.pool, c.bounds, c.steps, c.tables, c.lens, top, 64, 256, 128 ** -0.5)
            close(out.cpu().double().numpy(), want, c.tolerance(want, None, 128 ** -0.5))


def test_no_room_for_tokens(cuda):
    """max_len 0, no tables: zeros, and lists of nothing."""
    ctx = context(4, 2, 64)
    q, pool = torch.ones(3, 4, 64, dtype=BF, device=cuda), torch.ones(1, 2, 2, P, 64, dtype=BF, device=cuda)
    t, n = torch.zeros(3, 0, dtype=I32, device=cuda), torch.zeros(3, dtype=I32, device=cuda)
    out = torch.ones(3, 4, 64, device=cuda)
    ctx.decode_bf16(q, pool, t, n, 0, out, None)
    assert float(out.abs().max()) == 0
    out.fill_(1)
    chosen, count = torch.zeros(3, 2, ctx.sparse_capacity(2), dtype=I32, device=cuda), torch.ones(3, 2, dtype=I32, device=cuda)
    ctx.decode_bf16_sparse(q, pool, torch.zeros(2, 64, dtype=I8, device=cuda), torch.zeros(1, 2, 2, 64, dtype=I8, device=cuda),
                           t, n, 0, 2, chosen, count, out, None)
    assert float(out.abs().max()) == 0 and int(chosen.max()) == -1 and int(count.max()) == 0


def test_empty_calls_do_nothing(cuda):
    ctx = context(4, 2, 64)
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device=cuda)
    ctx.append_bf16(e(0, 2, 64), e(0, 2, 64), e(0, dt=I64), e(1, 2, 2, P, 64))
    ctx.decode_bf16(e(0, 4, 64), e(1, 2, 2, P, 64), e(0, 3, dt=I32), e(0, dt=I32), 48, e(0, 4, 64, dt=torch.float32), None)


# ------------------------------------------------------------------------------------------- all together

def test_serving_loop(cuda):
    """Prefill, then decode steps as a server runs them: plan, append, dense and sparse decode on one stream with no
    wait between, the step captured once and replayed; tables, pool, bounds and outputs against the oracle's loop."""
    h_q, h_kv, d, batch, top = 8, 2, 64, 5, 6
    ctx = context(h_q, h_kv, d)
    r = np.random.default_rng(21)
    prompt = np.array([700, 3, 0, 333, 1500])
    steps, stride = 36, 100
    need = sum(paged.pages_for(int(p) + steps) for p in prompt)
    free = r.permutation(need + 7).astype(np.int32)
    pages = need + 7
    step_codes = np.full((h_kv, d), -5, np.int8)
    i = lambda *s: torch.zeros(*s, dtype=I32, device=cuda)
    pool, bounds = torch.zeros(pages, h_kv, 2, P, d, dtype=BF, device=cuda), torch.zeros(pages, h_kv, 2, d, dtype=I8, device=cuda)
    g = dict(free=dev(free, cuda), tables=i(batch, stride), state=i(4), seq=i(batch), total=i(batch), rows=i(batch + 1))
    max_len = stride * P
    cap = ctx.sparse_capacity(top)
    ks = dev(step_codes, cuda)
    ws = torch.empty(max(ctx.decode_bf16_sparse_workspace_size(batch, max_len, top),
                         ctx.decode_bf16_workspace_size(batch, max_len), 1), dtype=torch.uint8, device=cuda)
    dense, sparse = (torch.zeros(batch, h_q, d, device=cuda) for _ in range(2))
    chosen, count = i(batch, h_kv, cap), i(batch, h_kv)
    qkv = torch.zeros(batch, h_q + 2 * h_kv, d, dtype=BF, device=cuda)
    slots = torch.zeros(batch, dtype=I64, device=cuda)
    ones = torch.ones(batch, dtype=I32, device=cuda)

    # the oracle's side
    o_pool, o_bounds = np.zeros((pages, h_kv, 2, P, d)), np.zeros((pages, h_kv, 2, d), np.int64)
    n = int(prompt.sum())
    k, v = (bf16(r.standard_normal((n, h_kv, d))) for _ in range(2))
    o_tables, o_slots, _, lens, st = paged.plan_append([0] * batch, prompt, free, 0, np.zeros((batch, stride)), n + 11)
    paged.append(o_pool, o_bounds, np.concatenate([k, k[:11]]), np.concatenate([v, v[:11]]), o_slots, step_codes)

    # prefill, with eleven rows of padding
    pslots = torch.zeros(n + 11, dtype=I64, device=cuda)
    ctx.plan_append(g["seq"], dev(prompt.astype(np.int32), cuda), g["free"], g["state"][:1], g["tables"], pslots, g["rows"],
                    g["total"], g["state"])
    pad = lambda x: torch.cat([dev(x, cuda, BF), torch.full((11, h_kv, d), float("nan"), dtype=BF, device=cuda)])
    ctx.append_bf16(pad(k), pad(v), pslots, pool, ks, bounds)
    g["seq"].copy_(g["total"])
    torch.cuda.synchronize()
    assert np.array_equal(bounds.cpu().numpy(), o_bounds) and np.array_equal(g["tables"].cpu().numpy(), o_tables)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.plan_append(g["seq"], ones, g["free"], g["state"][:1], g["tables"], slots, g["rows"], g["total"], g["state"])
        ctx.append_bf16(qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:], slots, pool, ks, bounds)
        ctx.decode_bf16(qkv[:, :h_q], pool, g["tables"], g["total"], max_len, dense, ws)
        ctx.decode_bf16_sparse(qkv[:, :h_q], pool, ks, bounds, g["tables"], g["total"], max_len, top, chosen, count, sparse, ws)
        g["seq"].copy_(g["total"])
    head = int(st[0])
    for step in range(steps):
        x = bf16(r.standard_normal((batch, h_q + 2 * h_kv, d)))
        qkv.copy_(dev(x, cuda, BF))
        graph.replay()
        o_tables, o_slots, _, lens, st = paged.plan_append(lens, [1] * batch, free, head, o_tables, batch)
        head = int(st[0])
        paged.append(o_pool, o_bounds, x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:], o_slots, step_codes)
        if step % 7 and step != steps - 1:
            continue
        torch.cuda.synchronize()
        q = x[:, :h_q]
        assert np.array_equal(g["tables"].cpu().numpy(), o_tables) and np.array_equal(g["total"].cpu().numpy(), lens)
        want = paged.decode(q, o_pool, o_tables, lens, 0.125)
        assert np.abs(dense.cpu().numpy() - want).max() <= 2.2e-3     # |v| <= 6, A <= 40: 6 * 2 * 40 * 38 * 2^-23
        want, lists = paged.decode_sparse(q, o_pool, o_bounds, step_codes, o_tables, lens, top, 64, 256, 0.125)
        assert [[chosen[b, h, :count[b, h]].tolist() for h in range(h_kv)] for b in range(batch)] == lists
        assert np.abs(sparse.cpu().numpy() - want).max() <= 2.2e-3
    assert np.array_equal(pool.cpu().double().numpy(), o_pool) and np.array_equal(bounds.cpu().numpy(), o_bounds)


def test_plan_and_append_feed_the_three_segment_decode(cuda):
    """The slots of two plans, for the INT2 history and the BF16 segment, into oscar_write_tokens, oscar_append_bf16
    and oscar_decode, one after the other on the stream: the cache and the output of the oracle's own case."""
    cfg = cases.workload("tiny")
    case = cases.DecodeCase(cfg, [300, 1000], [320, 37])
    h_kv, d, batch = cfg["h_kv"], cfg["d"], 2
    ctx = O.Oscar(n_layers=1, n_q_heads=cfg["h_q"], n_kv_heads=h_kv, head_dim=d, group=cfg["group"])
    ctx.calibrate_upload(0, case.rk, case.rv, case.tk, case.tv)
    i = lambda *s: torch.zeros(*s, dtype=I32, device=cuda)

    def plan(lens, tables, stride):
        ids = np.concatenate([tables[b, :paged.pages_for(int(n))] for b, n in enumerate(lens)])
        t, slots, total = i(batch, stride), torch.zeros(int(lens.sum()), dtype=I64, device=cuda), i(batch)
        ctx.plan_append(i(batch), dev(lens, cuda), dev(ids, cuda), i(1), t, slots, i(batch + 1), total, i(4))
        return t, slots, total

    rows = lambda kind, lens: [dev(np.concatenate(x), cuda, BF) for x in
                               zip(*(case.li.kv("%s/%d" % (kind, b), int(n)) for b, n in enumerate(lens)))]
    int2, bf = torch.zeros(case.int2_pool.size, dtype=torch.uint8, device=cuda), torch.zeros(case.bf16_pool.size, dtype=BF, device=cuda)
    t2, s2, n2 = plan(case.hist_lens, case.int2_tables, case.int2_stride)
    tb, sb, nb = plan(case.bf16_lens, case.bf16_tables, case.bf16_stride)
    ctx.write_tokens(0, *rows("hist", case.hist_lens), s2, int2)
    ctx.append_bf16(*rows("bf16", case.bf16_lens), sb, bf)
    ws = torch.empty(ctx.decode_workspace_size(batch, 1000), dtype=torch.uint8, device=cuda)
    out = torch.empty(batch, cfg["h_q"], d, device=cuda)
    ctx.decode(0, dev(case.q, cuda, BF), int2, t2, n2, 1000, bf, tb, nb, out, ws)
    torch.cuda.synchronize()
    assert np.array_equal(bf.float().cpu().numpy(), case.bf16_pool)
    case.int2_pool = int2.cpu().numpy()
    cases.check_decode(out.cpu().numpy(), case.oracle_out())
