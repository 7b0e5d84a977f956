"""oscar_extend_bf16: blocks that rows fill in part, rows that infinities and NaN reach."""

import math

import numpy as np
import pytest
import torch

import chunk_oracle
from test_gpu_extend import BF, I32, P, Case, bf16, context

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cached", [200, 20000])
@pytest.mark.parametrize("h_q", [1, 2])
def test_partly_filled_warps(cuda, d, cached, h_q):
    """Row counts around those of a warp and a block, in whole items and in parts: lanes with a row beside lanes without
    one."""
    new = [1, 2, 31, 32, 33, 63, 97, 127, 128, 129, 161, 255, 257]
    c = Case([(cached if m < 40 else cached % 301, m) for m in new], h_q, 1, d, seed=cached + h_q, spare=2)
    c.check(c.run(cuda))


def odd_values(c, scale):
    """Per output: 0, or what the infinities and NaN among the values that it sees make of it, by the decode's rule: one
    counts whole however small its token's weight; the logit -infinity has none, and zero times infinity is NaN."""
    g, out = c.h_q // c.h_kv, np.zeros(c.q.shape)
    for b, total in enumerate(c.total):
        lo, hi = c.start[b], c.start[b + 1]
        for h in range(c.h_kv):
            k, v, there = chunk_oracle.rows_of(c.pool, c.tables[b], total, h)
            for t in np.flatnonzero(there & ~np.isfinite(v).all(1)):
                rows = slice(max(lo, lo + t - (total - (hi - lo))), hi)
                with np.errstate(invalid="ignore"):
                    x = (c.q[rows, h * g:(h + 1) * g] @ k[t]) * scale
                    one = np.where(x > -np.inf, 1.0, 0.0)[..., None]
                    out[rows, h * g:(h + 1) * g] += np.where(np.isfinite(v[t]), 0.0, one * np.where(np.isfinite(v[t]), 0.0, v[t]))
    return out


def check_odd(c, out, scale):
    """Infinities and NaN where odd_values has them, the rest within the bound."""
    odd, got = odd_values(c, scale), out.double().cpu().numpy()
    some = odd != 0
    assert some.any() and np.array_equal(got[some], odd[some], equal_nan=True)
    pool, c.pool = c.pool, np.where(np.isfinite(c.pool), c.pool, 0.0)
    c.pool[:, :, 0][np.isneginf(pool[:, :, 0])] = -3000.0    # a weight of nothing in 64 bits too
    want, bound = chunk_oracle.extend(c.q, c.pool, c.tables, c.start, c.total, scale)
    c.pool = pool
    n = len(got) - c.spare
    assert (np.abs(got - want) <= bound)[:n][~some[:n]].all() and (got[n:] == 7).all()
    return some


def spread_infinities(c, seed):
    """Infinities of both signs and NaN among the values: a few anywhere, the requests' first, last and middle tokens."""
    r = np.random.default_rng(seed)
    for x in (np.inf, -np.inf, np.nan):
        c.pool[r.integers(len(c.pool)), r.integers(c.h_kv), 1, r.integers(P), r.integers(5, c.d)] = x
    at = lambda b, t: (c.tables[b, t // P], int(r.integers(c.h_kv)), 1, t % P)
    for b, total in enumerate(c.total):
        if total == 0 or b > 40:
            continue
        c.pool[at(b, 0)][0] = np.inf
        c.pool[at(b, total - 1)][1] = -np.inf
        c.pool[at(b, total // 2)][2] = np.nan
        c.pool[c.tables[b, 0], 0, 1, 0, 3], c.pool[c.tables[b, (total - 1) // P], 0, 1, (total - 1) % P, 3] = np.inf, -np.inf


ODD = [([(20, 300)], 4, 2, 64), ([(0, 1)], 2, 1, 128), ([(300, 200), (4000, 3), (0, 40)], 8, 2, 128), ([(9000, 2)], 8, 1, 128),
       ([(5000, 150)], 2, 1, 64), ([(40 * i + 5, 2) for i in range(60)], 4, 2, 64), ([(i * 7 % 90, i % 3) for i in range(200)], 4, 2, 64),
       ([(150, 40)] * 45, 8, 2, 128)]


@pytest.mark.parametrize("scale", [2.0 ** -5, 4.0])
@pytest.mark.parametrize("lens,h_q,h_kv,d", ODD, ids=lambda x: str(x) if len(str(x)) < 50 else "many")
def test_infinite_values_of_any_weight(cuda, lens, h_q, h_kv, d, scale):
    """At scale 4 most weights are far below what fp32 holds. In whole items and in parts, by either plan."""
    c = Case(lens, h_q, h_kv, d, seed=len(lens) + d, spare=2)
    spread_infinities(c, 5)
    check_odd(c, c.run(cuda, context(h_q, h_kv, d, sm_scale=scale)), scale)


@pytest.mark.parametrize("lens", [[(20, 30)], [(3000, 5), (0, 77)]], ids=str)
def test_infinite_values_without_weight(cuda, lens):
    """A logit of -infinity weighs zero: with a finite value it adds nothing, zero times infinity is NaN. On pages outside
    the pool nothing counts, and a row that sees no weight at all is zeros."""
    c = Case(lens, 4, 2, 64, seed=2)
    c.q[..., 0] = 1.0
    c.pool[:, :, 0, :, 0] = 0.0
    for b, total in enumerate(c.total):
        page = c.tables[b, total // 2 // P]
        c.pool[page, :, 0, 4, 0] = -np.inf
        c.pool[page, 0, 1, 4, 9] = np.inf
    some = check_odd(c, c.run(cuda), 1 / 8)
    assert some[..., 9].any() and not some[..., :9].any()
    c.pool[c.tables[0, :2], :, 0, :, 0] = -np.inf            # the first tokens of all
    c.pool[c.tables[0, :2], :, 1, :, 3] = -np.inf
    c.total[0] = c.new[0] + 1                                # row i sees i + 2 tokens
    got = c.run(cuda).double().cpu().numpy()
    rows = min(31, c.new[0])
    assert (got[:rows] == 0).all()


@pytest.mark.parametrize("lens,h_q,h_kv,d", [([(9000, 2)], 8, 1, 128), ([(3000, 1)] * 12, 4, 2, 64)], ids=["cut", "line"])
def test_infinite_values_of_a_part_without_weight(cuda, lens, h_q, h_kv, d):
    """All logits of the first tokens, more than a part's, are -infinity, and one of their values is infinite."""
    c = Case(lens, h_q, h_kv, d, seed=6)
    c.q[..., 0] = 1.0
    c.pool[:, :, 0, :, 0] = 0.0
    for b, total in enumerate(c.total):
        c.pool[c.tables[b, :total // 2 // P], :, 0, :, 0] = -np.inf
        c.pool[c.tables[b, 3], 0, 1, 5, 9] = np.inf
    some = check_odd(c, c.run(cuda), 1 / math.sqrt(d))
    g = h_q // h_kv
    assert some[:, :g, 9].all() and some.sum() == g * len(c.q)


def test_infinite_values_as_in_the_decode(cuda):
    """Single tokens: infinite and NaN at the same places."""
    lens = [(0, 1), (15, 1), (4000, 1), (16, 1), (77, 1), (9000, 1)]
    c = Case(lens, 8, 2, 128, seed=1)
    spread_infinities(c, 6)
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(cuda).to(dt)
    c.pool[c.tables[4, 1], 1, 0, 3] = -np.inf                # logits of either infinity, and NaN
    c.pool[c.tables[4, 1], 1, 1, 3, 7] = np.inf
    for scale in (1 / math.sqrt(128), 4.0):
        ctx = context(8, 2, 128, sm_scale=scale)
        got = c.run(cuda, ctx)
        out = torch.empty(6, 8, 128, device=cuda)
        ws = torch.empty(max(1, ctx.decode_bf16_workspace_size(6, 9001)), dtype=torch.uint8, device=cuda)
        ctx.decode_bf16(t(c.q, BF), t(c.pool, BF), t(c.tables, I32), t(c.total, I32), 9001, out, ws)
        odd = ~torch.isfinite(out)
        assert odd.any() and torch.equal(torch.isnan(out), torch.isnan(got)) and torch.equal(odd, ~torch.isfinite(got))
        same = odd & ~torch.isnan(out)
        assert torch.equal(out[same], got[same].float())


def spoiled(c, what):
    """The case's pool with values that reach every row (but the first ones)."""
    pool = torch.from_numpy(c.pool).to(BF)
    if what == "past fp32":
        pool[:, :, 1, :, 3] = 3.0e38
    else:
        pool[int(c.tables[0, 0]), :, 1, 10, 3] = float(what)
    return pool


@pytest.mark.parametrize("what,times", [("inf", 100), ("nan", 100), ("past fp32", 1000)])
def test_a_bad_value_stalls_nothing(cuda, what, times):
    """A prompt of 4,096 tokens whose rows an infinity, a NaN or a sum past fp32 reaches takes longer, but not as long as
    if each row were formed by itself (over 10,000 times). Its other channels keep their bits."""
    c = Case([(0, 4096)], 32, 8, 128, seed=4, more_pages=0)
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(cuda).to(dt)
    ctx, q, out = context(32, 8, 128), t(c.q, BF), [torch.empty(c.q.shape, dtype=BF, device=cuda) for _ in range(2)]
    args = t(c.tables, I32), t(c.start, I32), t(c.total, I32)
    ws = torch.empty(ctx.extend_bf16_workspace_size(1, 4096), dtype=torch.uint8, device=cuda)
    spent = []
    for pool, o in zip((torch.from_numpy(c.pool).to(BF).to(cuda), spoiled(c, what).to(cuda)), out):
        events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ctx.extend_bf16(q, pool, *args, o, ws)
        torch.cuda.synchronize()
        events[0].record()
        for _ in range(3):
            ctx.extend_bf16(q, pool, *args, o, ws)
        events[1].record()
        torch.cuda.synchronize()
        spent.append(events[0].elapsed_time(events[1]))
    assert spent[1] < times * spent[0], spent
    rest = [i for i in range(128) if i != 3]
    assert torch.equal(out[0][..., rest], out[1][..., rest])
    if what == "past fp32":                                  # the mean of equal values, weights off by 2^-8 at most in all
        assert (out[1][..., 3].double() / float(torch.tensor(3.0e38).to(BF)) - 1).abs().max() <= 2.0 ** -7
    else:
        assert torch.equal(out[1][10:, :, 3], torch.full_like(out[1][10:, :, 3], float(what))) or torch.isnan(out[1][10:, :, 3]).all()
        assert (out[1][:10, :, 3] - out[0][:10, :, 3]).abs().max() <= 2.0 ** -6 * out[0][:10].abs().max()


def test_a_long_sum_past_fp32(cuda):
    """A row over 2^20 tokens whose values' sum passes fp32, formed in 2^15 steps of 32 tokens: a step's sum is off by at
    most 32 * 2^-24 of it, each addition of one by 2^-24 of the sum; weights are ones and their sum exact."""
    d, length, pages = 64, 1 << 20, 40
    gen = torch.Generator(device=cuda).manual_seed(5)
    pool = torch.zeros(pages, 1, 2, P, d, dtype=BF, device=cuda)
    pool[:, 0, 1] = ((1 + torch.rand(pages, P, d, generator=gen, device=cuda, dtype=torch.float64)) * 2.0 ** 125).to(BF)
    pool[:, 0, 1, :, 7] = 1.0
    tables = torch.randint(0, pages, (1, length // P), dtype=I32, device=cuda, generator=gen)
    q, start = torch.zeros(1, 1, d, dtype=BF, device=cuda), torch.tensor([0, 1], dtype=I32, device=cuda)
    out, ctx = torch.empty_like(q), context(1, 1, d)
    ws = torch.empty(ctx.extend_bf16_workspace_size(1, 1), dtype=torch.uint8, device=cuda)
    ctx.extend_bf16(q, pool, tables, start, torch.tensor([length], dtype=I32, device=cuda), out, ws)
    torch.cuda.synchronize()
    assert ctx.debug_error()[0] == 0
    count = torch.bincount(tables[0], minlength=pages).double()
    want = torch.einsum("p,pd->d", count, pool[:, 0, 1].double().mean(1)) / count.sum()
    relative = 2.0 ** -9 + 2.0 ** -19 + 2.0 ** -21
    assert ((out[0, 0].double() / want - 1).abs() <= relative + 2.0 ** -8 * (1 + relative)).all()


@pytest.mark.parametrize("d", [64, 128])
def test_small_values_beside_a_bad_one(cuda, d):
    """Rows in front of a token whose values are NaN, over values near the smallest numbers, and others beside them whose
    sum passes fp32."""
    c = Case([(0, 100), (60, 50)], 4, 2, d, seed=d)
    r = np.random.default_rng(d)
    c.pool[:, :, 1, :, :8] = bf16(r.uniform(1, 2, c.pool.shape[:2] + (P, 8)) * 2.0 ** -120)
    c.pool[:, :, 1, :, 8:12] = bf16(r.uniform(1, 2, c.pool.shape[:2] + (P, 4)) * 2.0 ** 126)
    want, bound = chunk_oracle.extend(c.q, c.pool, c.tables, c.start, c.total, 1 / math.sqrt(d))
    for b, t in ((0, 90), (1, 100)):
        c.pool[c.tables[b, t // P], :, 1, t % P] = np.nan
    got = c.run(cuda).double().cpu().numpy()
    for rows in (slice(0, 90), slice(100, 140)):
        assert (np.abs(got - want) <= bound)[rows].all()
    assert np.isnan(got[90:100]).all() and np.isnan(got[140:]).all()


def test_formed_rows_weigh_alike(cuda):
    """A row over two tokens, with a token of NaN behind it and without: the same bits. Weights 1 and 2^-0.75, rounded for
    the product with V and summed unrounded; the first value is 0, so that there is one product, exact in fp32."""
    d = 64
    q, pool = torch.zeros(3, 1, d, dtype=BF, device=cuda), torch.zeros(1, 1, 2, P, d, dtype=BF, device=cuda)
    q[..., 0], pool[0, 0, 0, 1, 0] = 1.0, -0.75
    v = 1 + torch.arange(d, dtype=torch.float64) / d
    pool[0, 0, 1, 1] = v.to(BF)
    w = 2.0 ** -0.75
    rounded = float(torch.tensor(w).to(BF))
    want, other = (rounded * v / (1 + w)).to(BF), (rounded * v / (1 + rounded)).to(BF)
    assert not torch.equal(want, other)
    t = lambda *x: torch.tensor(x, dtype=I32, device=cuda)
    ctx = context(1, 1, d, sm_scale=math.log(2))
    ws = torch.empty(ctx.extend_bf16_workspace_size(1, 3), dtype=torch.uint8, device=cuda)
    for value in (0.0, float("nan")):
        pool[0, 0, 1, 2] = value
        out = torch.empty_like(q)
        ctx.extend_bf16(q, pool, t(0)[None], t(0, 3), t(3), out, ws)
        assert torch.equal(out[1, 0].cpu(), want)


@pytest.mark.parametrize("lens,h_q,h_kv,d", [([(9000, 2)], 8, 1, 128), ([(0, 700), (300, 40)], 8, 2, 64), ([(300, 3)] * 30, 4, 2, 128),
                                             ([(i * 7 % 90, 1 + i % 3) for i in range(200)], 4, 2, 64)],
                         ids=["cut", "whole", "line", "many"])
def test_a_wait_that_runs_out(cuda, monkeypatch, lens, h_q, h_kv, d):
    """Every other CTA's loader stops in its first item: the call ends, says so afterwards, and writes nothing beyond its rows
    and workspace, whatever the workspace held; the next call of the same context and workspace is as ever."""
    c, ctx = Case(lens, h_q, h_kv, d, seed=3, spare=2), context(h_q, h_kv, d)
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(cuda).to(dt)
    n, size = len(c.q), ctx.extend_bf16_workspace_size(len(c.total), len(c.q))
    q, pool, tables, start, total = t(c.q, BF), t(c.pool, BF), t(c.tables, I32), t(c.start, I32), t(c.total, I32)
    outs = torch.full((n + 64, h_q, d), 7.0, dtype=BF, device=cuda)
    space = torch.full((size + 4096,), 255, dtype=torch.uint8, device=cuda)
    out, ws = outs[32:32 + n], space[:size]

    def call():
        ctx.extend_bf16(q, pool, tables, start, total, out, ws)
        torch.cuda.synchronize()
        assert (outs[:32] == 7).all() and (outs[32 + n - 2:] == 7).all() and (space[size:] == 255).all()
        return ctx.debug_error()[:2]

    for again in range(2):                                   # over a workspace of nothing, and one of an earlier call
        monkeypatch.setenv("OSCAR_FAULT", "wait")
        assert call() == (-5, 4)
        monkeypatch.delenv("OSCAR_FAULT")
        out.fill_(7.0)
        assert call()[0] == 0
        c.check(out)
        out.fill_(7.0)


def test_every_row_of_the_largest_batch(cuda):
    """65,535 requests of 256 rows: all 16.8 million against the definition in 64 bits, with chunk_oracle's bound."""
    batch, new, d, pages, per = 65535, 256, 64, 512, 19
    n, scale = batch * new, 1 / 8
    gen = torch.Generator(device=cuda).manual_seed(8)
    lens = torch.randint(0, 40, (batch,), generator=gen, device=cuda, dtype=I32)
    pool = torch.randn(pages, 1, 2, P, d, generator=gen, device=cuda).to(BF)
    tables = torch.randint(0, pages, (batch, per), generator=gen, device=cuda, dtype=I32)
    q = torch.randn(n, 1, d, generator=gen, device=cuda, dtype=BF)
    out, ctx = torch.full_like(q, 7.0), context(1, 1, d)
    ws = torch.full((ctx.extend_bf16_workspace_size(batch, n),), 255, dtype=torch.uint8, device=cuda)
    ctx.extend_bf16(q, pool, tables, torch.arange(0, n + 1, new, dtype=I32, device=cuda), lens + new, out, ws)
    torch.cuda.synchronize()
    assert ctx.debug_error()[0] == 0
    token, wide = torch.arange(per * P, device=cuda), pool.double()
    for b in range(0, batch, 1024):
        rows, some = slice(b * new, min(b + 1024, batch) * new), slice(b, min(b + 1024, batch))
        k, v = (wide[tables[some].long(), 0, i].flatten(1, 2) for i in (0, 1))
        x = q[rows, 0].double().view(-1, new, d)
        seen = token[None, None] <= (lens[some, None] + torch.arange(new, device=cuda))[..., None]
        size = torch.where(seen, x.abs() @ k.abs().mT, 0.0).amax(-1, keepdim=True) * scale
        p = torch.softmax(torch.where(seen, (x @ k.mT) * scale, -math.inf), -1)
        y, mean = p @ v, p @ v.abs()
        e = size * (9 * d / 16 + 2) * 2.0 ** -23 + 4 * 2.0 ** -23 + 1.01 * 2.0 ** -8
        err = e * (mean + y.abs()) * (1 + 2 * e) + (72 * 4 + 64) * 2.0 ** -23 * mean
        assert ((out[rows, 0].double().view_as(y) - y).abs() <= err + 2.0 ** -8 * (y.abs() + err)).all(), b


@pytest.mark.parametrize("lens,h_q,h_kv,d", [([(30, 90), (2000, 2), (0, 5)], 8, 2, 64), ([(i * 7 % 90, 1 + i % 3) for i in range(200)], 4, 2, 128)],
                         ids=["few", "many"])
def test_bad_values_come_and_go(cuda, lens, h_q, h_kv, d):
    """One captured call, queries at a stride, values that are finite, spoiled and finite again: nothing of an earlier
    replay is left."""
    c = Case(lens, h_q, h_kv, d, seed=17, spare=2)
    clean = c.pool.copy()
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(cuda).to(dt)
    wide = torch.full((len(c.q), h_q * d + 40), float("nan"), dtype=BF, device=cuda)
    q = wide[:, 16:16 + h_q * d].unflatten(1, (h_q, d))
    q.copy_(t(c.q, BF))
    pool, out = t(c.pool, BF), torch.empty(c.q.shape, dtype=BF, device=cuda)
    ctx, side = context(h_q, h_kv, d), torch.cuda.Stream()
    ws = torch.full((ctx.extend_bf16_workspace_size(len(c.total), len(c.q)),), 255, dtype=torch.uint8, device=cuda)
    args = t(c.tables, I32), t(c.start, I32), t(c.total, I32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ctx.extend_bf16(q, pool, *args, out, ws)
    first = None
    for step in range(5):
        c.pool = clean.copy()
        if step % 2:
            spread_infinities(c, step)
        pool.copy_(t(c.pool, BF))
        out.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        if step % 2:
            check_odd(c, out, 1 / math.sqrt(d))
        else:
            c.check(out)
            first = out.clone() if first is None else first
            assert torch.equal(out, first)
