"""The paged decodes close to their rounding: values at the edges, outputs held to the bound of paged_bounds, and the
variants that only long or many sequences take."""

import numpy as np
import pytest
import torch

from bit_kv_cache_write_gb300 import oscar as O
from oracle import paged
from paged_bounds import P, IntCache, choose

pytestmark = pytest.mark.gpu
BF, I32, I64, I8 = torch.bfloat16, torch.int32, torch.int64, torch.int8
SINK, RECENT = 64, 256


def context(c, sm_scale=0.0, **over):
    cfg = dict(n_layers=1, n_q_heads=c.h_q, n_kv_heads=c.h_kv, head_dim=c.d, group=32, sink=SINK, recent=RECENT,
               sm_scale=sm_scale)
    cfg.update(over)
    return O.Oscar(**cfg)


def dense(ctx, c, cuda, out_type=torch.float32, max_len=None):
    max_len = int(c.lens.max()) if max_len is None else max_len
    batch = len(c.lens)
    out = torch.full((batch, c.h_q, c.d), 7.0, dtype=out_type, device=cuda)
    ws = torch.full((max(1, ctx.decode_bf16_workspace_size(batch, max_len)),), 255, dtype=torch.uint8, device=cuda)
    ctx.decode_bf16(c.q.to(cuda), c.pool.to(cuda), c.tables.to(cuda), torch.from_numpy(c.lens).to(cuda), max_len, out, ws)
    return out


def sparse(ctx, c, cuda, top, out_type=torch.float32, max_len=None):
    """(out, lists)"""
    max_len = int(c.lens.max()) if max_len is None else max_len
    batch, cap = len(c.lens), ctx.sparse_capacity(top)
    out = torch.full((batch, c.h_q, c.d), 7.0, dtype=out_type, device=cuda)
    chosen, n = torch.full((batch, c.h_kv, cap), 77, dtype=I32, device=cuda), torch.full((batch, c.h_kv), 77, dtype=I32, device=cuda)
    ws = torch.full((max(1, ctx.decode_bf16_sparse_workspace_size(batch, max_len, top)),), 255, dtype=torch.uint8, device=cuda)
    ctx.decode_bf16_sparse(c.q.to(cuda), c.pool.to(cuda), c.steps.to(cuda), c.bounds.to(cuda), c.tables.to(cuda),
                           torch.from_numpy(c.lens).to(cuda), max_len, top, chosen, n, out, ws)
    chosen, n = chosen.cpu(), n.cpu()
    assert all(bool((chosen[b, h, n[b, h]:] == -1).all()) for b in range(batch) for h in range(c.h_kv))
    return out, [[chosen[b, h, :n[b, h]].tolist() for h in range(c.h_kv)] for b in range(batch)]


def within(out, want, bound):
    got = out.double().cpu()
    want, bound = want.cpu(), bound.cpu()
    assert bool(got.isfinite().all())
    off = ((got - want).abs() / bound.clamp(min=1e-30)).max()
    assert float(off) <= 1, "%.3g of the bound (errors up to %.3g)" % (off, (got - want).abs().max())


def check_dense(ctx, c, cuda, scale, max_len=None):
    """fp32 within the bound; the same again; bf16 the same rounded."""
    out = dense(ctx, c, cuda, max_len=max_len)
    within(out, *c.reference(scale, device=cuda))
    assert torch.equal(dense(ctx, c, cuda, max_len=max_len), out)
    assert torch.equal(dense(ctx, c, cuda, BF, max_len), out.to(BF))


def check_sparse(ctx, c, cuda, top, scale, max_len=None):
    """The pages that choose() gives, outputs over them within the bound; the same again; bf16 the same rounded."""
    out, lists = sparse(ctx, c, cuda, top, max_len=max_len)
    q, steps, bounds, tables = c.q.double().numpy(), c.steps.numpy(), c.bounds.numpy(), c.tables.numpy()
    for b, n in enumerate(map(int, c.lens)):
        assert lists[b] == choose(q[b], steps, bounds, tables[b], n, top, SINK, RECENT), b
    within(out, *c.reference(scale, lists, cuda))
    again, other = sparse(ctx, c, cuda, top, max_len=max_len)
    assert other == lists and torch.equal(again, out)
    assert torch.equal(sparse(ctx, c, cuda, top, BF, max_len)[0], out.to(BF))


# each takes another way to join: a cluster, one split, splits joined by one, eight and 32 warps, one-kernel sparse
SHAPES = [([5], 2, 2, 64), ([700], 8, 2, 128), ([300] * 9, 64, 64, 64), ([4000, 4000], 8, 2, 128), ([40000], 16, 8, 128),
          ([9000], 2, 1, 64)]


@pytest.mark.parametrize("lens,h_q,h_kv,d", SHAPES, ids=str)
def test_logits_of_any_finite_size_count(cuda, lens, h_q, h_kv, d):
    """All logits near -1e35: equal ones share the weight, and where one is the largest by far it alone has it."""
    c = IntCache(31, lens, h_q, h_kv, d)
    c.pool[:, :, 0] = 0
    c.pool[:, :, 0, :, 0] = -2.0 ** 60
    ctx = context(c, 0.125)
    c.q[:] = 0
    want, bound = c.reference(0.125)                # no logit at all weighs like equal ones
    c.q[:, :, 0] = 2.0 ** 60                        # -2^117 at every token
    within(dense(ctx, c, cuda), want, bound)
    out, lists = sparse(ctx, c, cuda, 40)
    q, c.q = c.q, torch.zeros_like(c.q)
    within(out, *c.reference(0.125, lists))
    c.q = q
    c.pool[:300, :, 0, :, 0] *= 2.0                 # every page but the sequences' last ones: far below
    want, _ = c.reference(0.125)
    out = dense(ctx, c, cuda).double().cpu()
    for b, n in enumerate(lens):
        last = (n - 1) % P + 1
        v = c.pool[300 + b, :, 1, :last].double()
        assert torch.allclose(want[b].view(h_kv, -1, d), v.mean(1)[:, None].expand(-1, h_q // h_kv, -1), rtol=1e-12, atol=1e-12)
        size = v.abs().mean(1)[:, None].expand(-1, h_q // h_kv, -1).reshape(h_q, d)
        assert bool(((out[b] - want[b]).abs() <= size * 64 * 2.0 ** -23).all())       # 17 truncations and the joins' roundings


def same_values(out, want, bound):
    """Infinities and NaN at the same places, the rest within the bound; zeros' bounds are zeros."""
    got, want, bound = out.double().cpu(), want.cpu(), bound.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    odd = ~want.isfinite()
    assert torch.equal(got[odd & ~want.isnan()], want[odd & ~want.isnan()])
    within(got[~odd], want[~odd], bound[~odd])
    return odd


def spread_infinities(c, seed):
    """Infinities of both signs and a few NaN among the values, at places that leave most outputs finite."""
    r = np.random.default_rng(seed)
    inf = float("inf")
    for x in (inf, -inf, inf, -inf, float("nan")):
        page, h, row, ch = r.integers(300), r.integers(c.h_kv), r.integers(P), r.integers(4, c.d)
        c.pool[page, h, 1, row, ch] = x
    for b, n in enumerate(map(int, c.lens)):
        if n == 0:
            continue
        last, h = 300 + b, int(r.integers(c.h_kv))
        c.pool[last, h, 1, (n - 1) % P, 0] = -inf                          # the last token
        first = int(c.tables[b, 0])
        c.pool[first, h, 1, 0, 1] = inf                                    # the first one
        c.pool[first, h, 1, 0, 2], c.pool[last, h, 1, (n - 1) % P, 2] = inf, -inf      # both: NaN
        c.pool[first, -1 - h, 1, 0, 3] = c.pool[last, -1 - h, 1, (n - 1) % P, 3] = inf


@pytest.mark.parametrize("scale", [2.0 ** -5, 4.0])
@pytest.mark.parametrize("lens,h_q,h_kv,d", SHAPES + [([0, 1, 33, 500], 4, 2, 64)], ids=str)
def test_infinite_values(cuda, lens, h_q, h_kv, d, scale):
    """softmax(..) V with infinities in V: the output's channel is infinite, of either sign, however small the token's
    weight (scale 4: far below what fp32 holds), NaN where both signs or a NaN meet; other channels and heads as ever."""
    c = IntCache(41, lens, h_q, h_kv, d)
    ctx = context(c, scale)
    clean = dense(ctx, c, cuda), sparse(ctx, c, cuda, 40)
    spread_infinities(c, 5)
    for out_type in (torch.float32, BF):
        out = dense(ctx, c, cuda, out_type)
        want, bound = c.reference(scale)
        if out_type == torch.float32:
            odd = same_values(out, want, bound)
            assert bool(odd.any()) and torch.equal(out.cpu()[~odd], clean[0].cpu()[~odd])
            full = out
        else:
            assert torch.equal(out.isnan(), full.isnan()) and torch.equal(out[~out.isnan()], full.to(BF)[~full.isnan()])
    out, lists = sparse(ctx, c, cuda, 40)
    assert lists == clean[1][1]
    odd = same_values(out, *c.reference(scale, lists))
    assert torch.equal(out.cpu()[~odd], clean[1][0].cpu()[~odd])


@pytest.mark.parametrize("lens", [[20], [3000, 77]], ids=str)
def test_infinite_values_of_tokens_without_weight(cuda, lens):
    """A logit of -infinity weighs zero: with a finite value it adds nothing, zero times infinity is NaN. Behind the
    length and on pages outside the pool nothing counts."""
    c = IntCache(42, lens, 4, 2, 64)
    c.q[:, :, 0] = 1
    c.pool[:, :, 0, :, 0] = 0
    c.tables[:, 0] = torch.arange(len(lens), dtype=torch.int32)            # first pages of their own
    if len(lens) > 1:
        c.tables[0, 5] = -1
        for b in range(len(lens)):                                         # and nowhere else
            rest = c.tables[b, 1:paged.pages_for(lens[b]) - 1]
            rest[(rest >= 0) & (rest < len(lens))] += 2
    ctx = context(c, 0.0625)
    pool = c.pool.clone()
    c.pool[:len(lens), 0, 0, 4, 0] = -float("inf")
    without = dense(ctx, c, cuda)
    assert bool(without.isfinite().all())
    c.pool[:len(lens), 0, 1, 4, 9] = float("inf")
    out = dense(ctx, c, cuda)
    nan = torch.zeros(len(lens), 4, 64, dtype=torch.bool, device=cuda)
    nan[:, :2, 9] = True
    assert bool(out[nan].isnan().all()) and torch.equal(out[~nan], without[~nan])
    c.pool = pool
    c.pool[:len(lens), :, 1, 4, 9] = float("inf")                          # now it has its weight
    out = dense(ctx, c, cuda)
    assert bool((out[:, :, 9] == float("inf")).all()) and bool(out[:, :, :9].isfinite().all())


# Dense plans on 152 SMs: 57 splits of 144 pages (36 a warp: ids are looked up a second time); over 400 splits of few
# pages, joined by 32 warps; splits of 256 pages; one split for each of many sequences; three of some 60 pages
LONG = [([131072], 16, 8, 128), ([131072], 2, 1, 128), ([131071], 2, 1, 64), ([131000, 2049, 2111, 4097, 0, 8209], 16, 8, 128),
        ([900] * 100, 8, 8, 128), ([3000] * 12, 8, 8, 128), ([2900] * 60, 16, 8, 64), ([33000, 100, 17], 8, 1, 64), ([70000, 65537], 64, 8, 64)]


@pytest.mark.parametrize("scale", [2.0 ** -5, 0.25])
@pytest.mark.parametrize("lens,h_q,h_kv,d", SHAPES + LONG, ids=lambda x: str(x) if len(str(x)) < 40 else "many")
def test_dense_is_within_its_rounding(cuda, lens, h_q, h_kv, d, scale):
    """The last token, every page and every bit of the weights: the bound is below what each of them changes."""
    c = IntCache(51, lens, h_q, h_kv, d)
    check_dense(context(c, scale), c, cuda, scale)


def test_pages_outside_the_pool_late_in_a_split(cuda):
    """Ids that are looked up with the second and the third 32 of a warp's pages."""
    c = IntCache(52, [131000, 30000], 8, 4, 128)
    for i in (3, 127, 128, 131, 133, 200, 256 + 129, 256 + 130, 1000):
        c.tables[:, i] = -1 if i % 2 else 10 ** 6
    check_dense(context(c, 2.0 ** -5), c, cuda, 2.0 ** -5)
    ctx = context(c, 2.0 ** -5, debug_bounds=1)
    dense(ctx, c, cuda)
    assert ctx.debug_error()[:2] == (-5, 2)


# Sparse plans: splits of 73 pages (37 a warp) behind clusters of four CTAs of 512 threads; clusters of two of 256 threads
# where all run at once and where they do not; keys in the workspace; 861 splits joined by 32 warps; the one-kernel form
# with one, two, four and eight CTAs
SELECT = [([30000, 20001, 29999, 5000, 30000, 0, 25000, 17], 16, 8, 128, 1000), ([4096] * 10 + [4000, 17, 900] * 4, 8, 8, 128, 30),
          ([50000] * 30 + [49000, 300, 0, 9000, 50000, 33333, 2, 16, 400, 50000], 8, 8, 128, 20), ([270001, 300], 2, 1, 128, 90),
          ([131072], 2, 1, 128, 6000), ([400], 4, 2, 128, 3), ([400] * 100, 1, 1, 64, 3), ([900] * 60, 2, 1, 64, 9),
          ([1500] * 30, 8, 1, 128, 9), ([3000] * 25, 2, 1, 128, 20), ([8000] * 18, 4, 1, 64, 300), ([100000], 32, 8, 128, 256)]


@pytest.mark.parametrize("lens,h_q,h_kv,d,top", SELECT, ids=lambda x: str(x) if len(str(x)) < 40 else "many")
def test_sparse_is_within_its_rounding(cuda, lens, h_q, h_kv, d, top):
    c = IntCache(53, lens, h_q, h_kv, d)
    c.bounds[5:9] = 100                                                   # ties
    check_sparse(context(c, 2.0 ** -5), c, cuda, top, 2.0 ** -5)


@pytest.mark.parametrize("lens,h_q,h_kv,d,top", SELECT[:3], ids=lambda x: str(x) if len(str(x)) < 40 else "many")
def test_sparse_with_room_for_more(cuda, lens, h_q, h_kv, d, top):
    """A bound of the lengths as a server passes it, twice the longest."""
    c = IntCache(54, lens, h_q, h_kv, d, pad=paged.pages_for(max(lens)))
    c.tables[1, 40:43] = torch.tensor([-1, 10 ** 6, -9], dtype=I32)
    check_sparse(context(c, 0.25), c, cuda, top, 0.25, 2 * max(lens))


# ---------------------------------------------------------------------------------------------- plans of many CTAs

def plan(ctx, cuda, seq, new, free, head, tables, cap):
    dev = lambda x, dt=I32: torch.as_tensor(np.ascontiguousarray(x)).to(dt).to(cuda)
    batch = len(seq)
    t, slots = dev(tables), torch.full((cap,), 77, dtype=I64, device=cuda)
    rows, total, state = (torch.full((n,), 77, dtype=I32, device=cuda) for n in (batch + 1, batch, 4))
    ctx.plan_append(dev(seq), dev(new), dev(free), dev([head]), t, slots, rows, total, state)
    return [x.cpu().numpy() for x in (t, slots, rows, total, state)]


@pytest.mark.parametrize("batch,new_hi,spare", [(40, 4000, 9), (96, 1500, 5000), (600, 200, 3), (700, 20, 60000), (2100, 60, 11),
                                                (5000, 3, 9), (5000, 9, 70000)])
@pytest.mark.parametrize("kind", ["fits", "few_pages", "short_map", "bad_lengths", "all_of_it"])
def test_plans_of_many_ctas_match_the_oracle(cuda, batch, new_hi, spare, kind):
    """Slot maps of up to 80,000, clusters of up to 16 CTAs, several chunks of requests, in each some rejected."""
    r = np.random.default_rng(batch + new_hi)
    seq, new = r.integers(0, 90, batch), r.integers(0, new_hi + 1, batch)
    stride = paged.pages_for(90 + new_hi)
    tables = r.integers(0, 1 << 20, (batch, stride))
    need = int(sum(paged.pages_for(int(s + n)) - paged.pages_for(int(s)) for s, n in zip(seq, new)))
    free, head, cap = r.permutation(1 << 17)[:need + 7], 5, int(new.sum()) + spare
    if kind in ("few_pages", "all_of_it"):
        free = free[:need // 2]
    if kind in ("short_map", "all_of_it"):
        cap = int(new[:-batch // 3].sum())
    if kind in ("bad_lengths", "all_of_it"):
        seq[::7], new[3::11] = -1 - seq[::7], -3
        seq[5::13] = 16 * stride + 1
    c = IntCache(1, [1], 4, 2, 64)
    got = plan(context(c), cuda, seq, new, free, head, tables, cap)
    want = paged.plan_append(seq, new, free, head, tables, cap)
    for g, w, name in zip(got, want, ("tables", "slots", "row_start", "total_len", "state")):
        assert np.array_equal(g, w), name
    assert (kind == "fits") == (want[4][2] == 0)


@pytest.mark.parametrize("lens,h_q,h_kv,d", SHAPES, ids=str)
@pytest.mark.parametrize("odd", [False, True])
def test_output_in_the_place_of_the_queries(cuda, lens, h_q, h_kv, d, odd):
    """A bf16 output may be the queries' own tensor, also where an infinite value takes a second look at the pages."""
    c = IntCache(61, lens, h_q, h_kv, d)
    ctx = context(c, 0.25)
    if odd:
        spread_infinities(c, 3)
    want, lists = dense(ctx, c, cuda, BF), sparse(ctx, c, cuda, 40, BF)
    pool, tables, n, batch, top = c.pool.to(cuda), c.tables.to(cuda), torch.from_numpy(c.lens).to(cuda), len(lens), 40
    ws = torch.empty(max(1, ctx.decode_bf16_workspace_size(batch, max(lens)),
                         ctx.decode_bf16_sparse_workspace_size(batch, max(lens), top)), dtype=torch.uint8, device=cuda)
    same = lambda a, b: torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])
    q = c.q.to(cuda)
    ctx.decode_bf16(q, pool, tables, n, max(lens), q, ws)
    assert same(q, want)
    q = c.q.to(cuda)
    chosen, count = torch.empty(batch, h_kv, ctx.sparse_capacity(top), dtype=I32, device=cuda), torch.empty(batch, h_kv, dtype=I32, device=cuda)
    ctx.decode_bf16_sparse(q, pool, c.steps.to(cuda), c.bounds.to(cuda), tables, n, max(lens), top, chosen, count, q, ws)
    assert same(q, lists[0])
