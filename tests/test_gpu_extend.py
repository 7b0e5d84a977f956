"""oscar_extend_bf16 against its fp64 definition (chunk_oracle.py, which derives the tolerances)."""

import math

import numpy as np
import pytest
import torch

import chunk_oracle
import rope_oracle
from bit_kv_cache_write_gb300 import oscar as O
from bit_kv_cache_write_gb300 import rope

pytestmark = pytest.mark.gpu
P = 16
BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64


def context(h_q, h_kv, d, **over):
    c = dict(n_layers=1, n_q_heads=h_q, n_kv_heads=h_kv, head_dim=d, group=32)
    c.update(over)
    return O.Oscar(**c)


def bf16(x):
    """The values rounded to bf16, as float64."""
    return torch.from_numpy(np.asarray(x, np.float32)).to(BF).double().numpy()


class Case:
    """Requests of (cached, new) tokens over shuffled pages; rows and pages beyond them hold what `fill` says."""

    def __init__(self, lens, h_q, h_kv, d, seed=0, spare=0, spread=1.0, integers=False, more_pages=2):
        r = np.random.default_rng(seed)
        self.h_q, self.h_kv, self.d, self.spare = h_q, h_kv, d, spare
        self.new = np.array([n for _, n in lens])
        self.total = np.array([c + n for c, n in lens])
        self.start = np.concatenate([[0], np.cumsum(self.new)])
        n = int(self.start[-1]) + spare
        count = -(-self.total // P)
        ids = r.permutation(int(count.sum()) + more_pages)
        self.tables = np.zeros((len(lens), max(1, int(count.max(initial=0)))), np.int32)
        at = 0
        for b, c in enumerate(count):
            self.tables[b, :c] = ids[at:at + c]
            at += c
        shape = (int(count.sum()) + more_pages, h_kv, 2, P, d)
        if integers:
            # q = e_c scaled, k small integers: logits are small whole numbers, weights powers of two
            self.q = np.zeros((n, h_q, d))
            self.q[np.arange(n)[:, None], np.arange(h_q)[None], r.integers(0, d, (n, h_q))] = 1.0
            self.pool = r.integers(-4, 5, shape).astype(np.float64)
        else:
            self.q, self.pool = bf16(r.normal(0, spread, (n, h_q, d))), bf16(r.normal(0, 1, shape))

    def run(self, cuda, ctx=None, stream=None, out=None, total=None, start=None, q=None):
        ctx = ctx or context(self.h_q, self.h_kv, self.d)
        t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(cuda).to(dt)
        q = t(self.q, BF) if q is None else q
        out = torch.full(q.shape, 7.0, dtype=BF, device=cuda) if out is None else out
        ws = torch.full((ctx.extend_bf16_workspace_size(len(self.total), len(self.q)),), 255, dtype=torch.uint8, device=cuda)
        ctx.extend_bf16(q, t(self.pool, BF), t(self.tables, I32), t(self.start if start is None else start, I32),
                        t(self.total if total is None else total, I32), out, ws, stream)
        torch.cuda.synchronize()
        assert ctx.debug_error()[0] == 0
        return out

    def check(self, out, sm_scale=None, exact=False):
        want, bound = chunk_oracle.extend(self.q, self.pool, self.tables, self.start, self.total,
                                          sm_scale or 1 / math.sqrt(self.d), exact)
        got = out.double().cpu().numpy()
        n = len(got) - self.spare
        assert (got[n:] == 7).all()
        err = np.abs(got[:n] - want[:n])
        assert (err <= bound[:n]).all(), ("off by", err.max(), "rows", np.unique(np.where(~(err <= bound[:n]))[0])[:8])


SHAPES = [([(0, 1)], 4, 2, 64), ([(1339, 5)], 4, 2, 64), ([(0, 16)], 1, 1, 128), ([(0, 17)], 8, 1, 128),
          ([(0, 128)], 2, 2, 64), ([(0, 129)], 2, 1, 128), ([(127, 1)], 8, 8, 128), ([(128, 1)], 16, 2, 128),
          ([(0, 300)], 4, 4, 128), ([(37, 333)], 8, 2, 64), ([(0, 0), (5, 0), (0, 3), (40, 1), (513, 70), (0, 0), (2, 1)], 8, 2, 128),
          ([(5000, 3)], 8, 1, 128), ([(9000, 1), (20, 200), (3000, 2)], 4, 1, 64), ([(i * 13 % 300, i % 4) for i in range(90)], 4, 2, 64),
          ([(1000, 700), (0, 900)], 4, 2, 128)]


@pytest.mark.parametrize("lens,h_q,h_kv,d", SHAPES)
def test_matches_the_definition(cuda, lens, h_q, h_kv, d):
    c = Case(lens, h_q, h_kv, d, seed=len(lens) + d, spare=3)
    c.check(c.run(cuda))


@pytest.mark.parametrize("lens,h_q,h_kv,d", SHAPES)
def test_exact_weights(cuda, lens, h_q, h_kv, d):
    """Logits that are whole in log2 units: weights and sums are exact, so that every token counts to the last bit."""
    c = Case(lens, h_q, h_kv, d, seed=d, integers=True)
    scale = math.log(2)
    c.check(c.run(cuda, context(h_q, h_kv, d, sm_scale=scale)), scale, exact=True)


def test_runs_are_alike_and_streams_apart(cuda):
    c = Case([(3000, 5), (0, 200), (700, 1)], 8, 2, 128, seed=4)
    ctx, a = context(8, 2, 128), None
    side = torch.cuda.Stream()
    for stream in (None, None, side):
        b = c.run(cuda, ctx, stream=stream)
        assert a is None or torch.equal(a, b)
        a = b


@pytest.mark.parametrize("d", [64, 128])
def test_nothing_unseen_matters(cuda, d):
    """NaN and infinity behind the sequences, in unused pages and in tokens that come after a row's own."""
    lens = [(0, 150), (130, 5), (1000, 40), (5, 1), (2000, 2)]
    c = Case(lens, 4, 2, d, seed=d, more_pages=3)
    want = c.run(cuda).double().cpu().numpy()
    used = np.zeros(len(c.pool), bool)
    for b, total in enumerate(c.total):
        pages = c.tables[b, :-(-total // P)]
        used[pages] = True
        if total % P:
            c.pool[pages[-1], :, :, total % P:] = np.nan
    c.pool[~used] = np.inf
    got = c.run(cuda).double().cpu().numpy()
    assert np.array_equal(got, want)
    # the last token of the first and third request: rows in front of it do not see it, its own row does
    for b, bad in ((0, np.nan), (2, np.inf)):
        t = c.total[b] - 1
        c.pool[c.tables[b, t // P], :, 1, t % P, 3] = bad
    n = c.run(cuda).double().cpu().numpy()
    last = [c.start[1] - 1, c.start[3] - 1]
    rows = np.setdiff1d(np.arange(len(n)), last)
    oracle, bound = chunk_oracle.extend(c.q, np.where(np.isfinite(c.pool), c.pool, 0.0), c.tables, c.start, c.total, 1 / math.sqrt(d))
    assert (np.abs(n[rows] - oracle[rows]) <= bound[rows]).all()
    assert np.isnan(n[last[0], :, 3]).all() and np.isposinf(n[last[1], :, 3]).all()
    rest = np.setdiff1d(np.arange(d), [3])
    assert (np.abs(n[last][:, :, rest] - oracle[last][:, :, rest]) <= bound[last][:, :, rest]).all()


def test_unseen_keys_of_nan(cuda):
    """A NaN key gives its rows NaN and the rows in front of it nothing."""
    c = Case([(20, 300)], 4, 2, 64, seed=8)
    want = c.run(cuda)
    t = 20 + 250
    c.pool[c.tables[0, t // P], 1, 0, t % P, 5] = np.nan
    got = c.run(cuda)
    assert torch.equal(got[:250], want[:250]) and torch.equal(got[:, :2], want[:, :2])
    assert torch.isnan(got[250:, 2:]).all()


def test_pages_outside_the_pool_are_masked(cuda):
    c = Case([(700, 30), (50, 9), (10, 3)], 8, 2, 128, seed=5)
    c.tables[0, 3], c.tables[0, 40], c.tables[1, 0], c.tables[2, 0] = -1, len(c.pool), 2 ** 31 - 1, -2 ** 31
    c.check(c.run(cuda))                                 # the third request sees nothing at all: zeros
    ctx = context(8, 2, 128, debug_bounds=1)
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(cuda).to(dt)
    out = torch.empty(c.q.shape, dtype=BF, device=cuda)
    ws = torch.empty(ctx.extend_bf16_workspace_size(3, len(c.q)), dtype=torch.uint8, device=cuda)
    ctx.extend_bf16(t(c.q, BF), t(c.pool, BF), t(c.tables, I32), t(c.start, I32), t(c.total, I32), out, ws)
    st, kind, index = ctx.debug_error()
    assert (st, kind) == (-5, 2) and index in (-1, len(c.pool), 2 ** 31 - 1, -2 ** 31)


def test_rows_without_room_and_bad_lengths(cuda):
    """Positions below 0 see nothing; lengths outside the table count as the nearer end; starts that do not ascend or
    pass the rows touch nothing else."""
    c = Case([(0, 40), (0, 30), (4, 20)], 4, 2, 64, seed=6, spare=2)
    total = c.total.copy()
    total[0] = 7
    got = c.run(cuda, total=total).double().cpu().numpy()
    c.total[0] = 7
    want, bound = chunk_oracle.extend(c.q, c.pool, c.tables, c.start, c.total, 1 / 8)
    assert (got[:33] == 0).all() and (np.abs(got - want)[:90] <= bound[:90]).all() and (got[90:] == 7).all()
    total[:] = [-5, 30, 2 ** 31 - 1]
    got = c.run(cuda, total=total).double().cpu().numpy()
    assert (got[:40] == 0).all() and (np.abs(got - want)[40:70] <= bound[40:70]).all() and (got[90:] == 7).all()
    for start in ([0, 70, 40, 2 ** 31 - 1], [-9, 40, 30, 92], [92, 0, 92, 0], [0, 0, 0, 0]):
        c.run(cuda, start=np.array(start))
    assert (c.run(cuda, start=np.zeros(4, int)) == 7).all()


def test_infinite_values(cuda):
    """Infinite values of tokens with weight, in whole and in cut items: their channels are infinite, the others are not."""
    c = Case([(300, 200), (4000, 3)], 8, 2, 128, seed=7)
    c.pool[c.tables[0, 31], :, 1, 3, 9] = np.inf         # token 499 of 500
    c.pool[c.tables[1, 250], :, 1, 2, 100] = -np.inf     # token 4,002 of 4,003
    got = c.run(cuda).double().cpu().numpy()
    want, bound = chunk_oracle.extend(c.q, np.where(np.isfinite(c.pool), c.pool, 0.0), c.tables, c.start, c.total, 1 / math.sqrt(128))
    assert np.isposinf(got[199, :, 9]).all() and np.isneginf(got[202, :, 100]).all()
    got[199, :, 9], got[202, :, 100] = want[199, :, 9], want[202, :, 100]
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("lens,h_q,h_kv,d", [([(0, 300), (40, 3)], 4, 2, 64), ([(9000, 2)], 8, 1, 128), ([(5000, 150)], 2, 1, 64)])
def test_values_whose_sum_passes_fp32(cuda, lens, h_q, h_kv, d):
    """Their mean does not. Rows of one item and of parts; a channel of the largest numbers and one of ordinary ones."""
    c = Case(lens, h_q, h_kv, d, seed=21)
    c.pool[:, :, 1] = bf16(c.pool[:, :, 1] * 2.0 ** 122)
    c.pool[:, :, 1, :, 3] = float(torch.finfo(BF).max)
    c.pool[:, :, 1, :, 4] = bf16(np.random.default_rng(1).normal(0, 1, c.pool.shape[:2] + (P,)))
    c.check(c.run(cuda))


def test_large_logits(cuda):
    """Logits far apart: references that rise again and again, weights that vanish."""
    for spread in (30.0, 1000.0):
        c = Case([(900, 300), (0, 70)], 4, 1, 128, seed=int(spread), spread=spread)
        c.check(c.run(cuda))


def test_infinite_logits(cuda):
    """A token of logit -inf has no weight; a row without any other gives zeros, and +inf gives NaN."""
    c = Case([(0, 33)], 2, 1, 64, seed=3)
    c.q[:], c.pool[:, :, 0] = 1.0, 0.0
    c.pool[c.tables[0, 0], 0, 0, 0, 0] = -np.inf
    want, bound = chunk_oracle.extend(c.q, c.pool, c.tables, c.start, c.total, 1 / 8)
    got = c.run(cuda).double().cpu().numpy()
    assert (got[0] == 0).all() and (np.abs(got - want)[1:] <= bound[1:]).all()
    c.pool[c.tables[0, 0], 0, 0, 5, 0] = np.inf
    got = c.run(cuda).double().cpu().numpy()
    assert (np.abs(got - want)[1:5] <= bound[1:5]).all() and np.isnan(got[5:]).all()


def test_query_rows_at_a_stride(cuda):
    c = Case([(40, 90), (800, 2)], 4, 2, 64, seed=2)
    wide = torch.full((92, 4 * 64 + 24), float("nan"), dtype=BF, device=cuda)
    q = wide[:, 8:264].unflatten(1, (4, 64))
    q.copy_(torch.from_numpy(c.q).to(BF))
    c.check(c.run(cuda, q=q, out=torch.empty(92, 4, 64, dtype=BF, device=cuda)))


def test_agrees_with_the_decode(cuda):
    """Single tokens: the decode's fp32 outputs are the definition to 2^-20."""
    lens = [(0, 1), (15, 1), (4000, 1), (16, 1), (77, 1)]
    c = Case(lens, 8, 2, 128, seed=1)
    got = c.run(cuda)
    ctx = context(8, 2, 128)
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(cuda).to(dt)
    out = torch.empty(5, 8, 128, device=cuda)
    ws = torch.empty(max(1, ctx.decode_bf16_workspace_size(5, 4001)), dtype=torch.uint8, device=cuda)
    ctx.decode_bf16(t(c.q, BF), t(c.pool, BF), t(c.tables, I32), t(c.total, I32), 4001, out, ws)
    _, bound = chunk_oracle.extend(c.q, c.pool, c.tables, c.start, c.total, 1 / math.sqrt(128))
    assert (np.abs(got.double().cpu().numpy() - out.double().cpu().numpy()) <= bound + 2.0 ** -20 * out.abs().max().item()).all()


@pytest.mark.parametrize("h_q,h_kv,d,layout", [(4, 2, 64, 0), (8, 1, 128, 1)])
def test_prompt_and_tokens_in_one_captured_loop(cuda, h_q, h_kv, d, layout):
    """plan, norm and rotation, append, attention: two prompts in chunks, then single tokens, from one captured graph a
    chunk size, against the whole definition in 64 bits."""
    r = np.random.default_rng(d)
    steps = [(70, 33), (1, 40), (1, 1), (1, 1), (0, 1)]
    n_max = max(sum(s) for s in steps)
    stride, pages, batch = 8, 20, 2
    ctx = context(h_q, h_kv, d)
    turns, scale = rope.rope_turns(d, 1e4, dict(kind="yarn", factor=2, trained=64))
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(cuda).to(dt)
    z = lambda *s, dt=I32: torch.zeros(s, dtype=dt, device=cuda)
    free, pool, tables = t(r.permutation(pages), I32), torch.full((pages, h_kv, 2, P, d), float("nan"), dtype=BF, device=cuda), z(batch, stride)
    seq, new, state, start, total = z(batch), z(batch), z(4), z(batch + 1), z(batch)
    slots = z(n_max, dt=I64)
    qkv = torch.zeros(n_max, h_q + 2 * h_kv, d, dtype=BF, device=cuda)
    qw, kw = (t(r.normal(1, 0.2, d), torch.float32) for _ in range(2))
    qr, kr, out = z(n_max, h_q, d, dt=BF), z(n_max, h_kv, d, dt=BF), z(n_max, h_q, d, dt=BF)
    ws = torch.empty(ctx.extend_bf16_workspace_size(batch, n_max), dtype=torch.uint8, device=cuda)
    tt = torch.from_numpy(turns).to(cuda)

    def step():
        ctx.plan_append(seq, new, free, state[:1], tables, slots, start, total, state)
        ctx.norm_rope(qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qr, kr, tt, row_start=start, total_len=total, q_weight=qw,
                      k_weight=kw, layout=layout, scale=scale)
        ctx.append_bf16(kr, qkv[:, h_q + h_kv:], slots, pool)
        ctx.extend_bf16(qr, pool, tables, start, total, out, ws)
        seq.copy_(total)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (seq, state, tables):
        x.zero_()
    have = [np.zeros((0, 2, h_kv, d)) for _ in range(batch)]
    for counts in steps:
        new.copy_(t(np.array(counts), I32))
        x = bf16(r.normal(0, 1, (n_max, h_q + 2 * h_kv, d)))
        qkv.copy_(t(x, BF))
        graph.replay()
        torch.cuda.synchronize()
        assert state[2].item() == 0 and ctx.debug_error()[0] == 0
        got_q, got_k, got = (a.double().cpu().numpy() for a in (qr, kr, out))
        row = 0
        for b, m in enumerate(counts):
            rows = slice(row, row + m)
            pos = len(have[b]) + np.arange(m)
            for y, g, w in ((x[rows, :h_q], got_q[rows], qw), (x[rows, h_q:h_q + h_kv], got_k[rows], kw)):
                want, bound = rope_oracle.norm_rope(y, w.cpu().numpy(), 1e-6, turns.view(np.uint64).tolist(), layout == 1, scale, pos)
                assert (np.abs(g - want) <= bound).all()
            have[b] = np.concatenate([have[b], np.stack([got_k[rows], x[rows, h_q + h_kv:]], 1)])
            row += m
        for b, m in enumerate(counts):
            k = len(have[b])
            one = np.zeros((-(-k // P), h_kv, 2, P, d))
            for i in range(k):
                one[i // P, :, :, i % P] = have[b][i].transpose(1, 0, 2)
            lo = sum(counts[:b])
            want, bound = chunk_oracle.extend(got_q[lo:lo + m], one, np.arange(len(one))[None], [0, m], [k], 1 / math.sqrt(d))
            assert (np.abs(got[lo:lo + m] - want) <= bound).all()


@pytest.mark.parametrize("lens,h_q,h_kv,d", [
    ([(300 * i + 17, 1 + i % 3) for i in range(12)], 8, 2, 128), ([(128 * i, 1) for i in range(1, 40)], 4, 1, 64),
    ([(1279, 1)] * 19, 8, 8, 64), ([(127, 1), (20000, 2), (255, 1), (9, 3)], 2, 2, 128), ([(128 * 8 - 1, 1)] * 38, 4, 4, 64),
    ([(3, 1)] * 100, 2, 1, 64), ([(5000, 4), (6000, 0), (128, 128)], 2, 1, 128)])
def test_tiles_in_a_line(cuda, lens, h_q, h_kv, d):
    """Requests of one row block each: the tiles of all of them go to the CTAs in equal stretches, which begin and end
    anywhere, also with an item."""
    c = Case(lens, h_q, h_kv, d, seed=len(lens), spare=1)
    c.check(c.run(cuda))
    c = Case(lens, h_q, h_kv, d, seed=len(lens), integers=True)
    c.check(c.run(cuda, context(h_q, h_kv, d, sm_scale=math.log(2))), math.log(2), exact=True)


def test_infinities_in_a_line(cuda):
    """Rows that are formed again, in items that stretches cut and in whole ones."""
    lens = [(40 * i + 5, 2) for i in range(60)]
    c = Case(lens, 4, 2, 64, seed=9)
    for b in range(0, 60, 7):
        t = c.total[b] - 1                                   # seen by the second row alone
        c.pool[c.tables[b, t // P], :, 1, t % P, 7] = np.inf
    want, bound = chunk_oracle.extend(c.q, np.where(np.isfinite(c.pool), c.pool, 0.0), c.tables, c.start, c.total, 1 / 8)
    got = c.run(cuda).double().cpu().numpy()
    rows = [int(c.start[b + 1]) - 1 for b in range(0, 60, 7)]
    assert np.isposinf(got[rows, :, 7]).all()
    got[rows, :, 7] = want[rows, :, 7]
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("batch,new_hi,h_q,h_kv,d", [(200, 2, 4, 2, 64), (1100, 3, 2, 1, 64), (150, 40, 8, 2, 128), (3, 9000, 4, 1, 64)])
def test_many_requests_and_rows(cuda, batch, new_hi, h_q, h_kv, d):
    """More requests or row blocks than a loader plans for: the plan kernel, its lists in shared memory and outside."""
    r = np.random.default_rng(batch)
    lens = [(int(r.integers(0, 90)), int(r.integers(0, new_hi + 1))) for _ in range(batch)]
    c = Case(lens, h_q, h_kv, d, seed=batch, spare=2)
    out = c.run(cuda)
    got = out.double().cpu().numpy()
    assert (got[-2:] == 7).all()
    rows = np.unique(np.concatenate([r.integers(0, len(got) - 2, 60), c.start[1:][c.new > 0][:40] - 1]))
    for row in rows:                                         # single rows of the definition
        b = int(np.searchsorted(c.start, row, side="right")) - 1
        one = chunk_oracle.extend(c.q[row:row + 1], c.pool, c.tables[b:b + 1], [0, 1], [c.total[b] - (c.start[b + 1] - 1 - row)], 1 / math.sqrt(d))
        assert (np.abs(got[row] - one[0][0]) <= one[1][0]).all(), row


@pytest.mark.parametrize("batch", [30, 1500])
def test_starts_that_do_not_ascend(cuda, batch):
    """Requests that claim the same rows again and again touch nothing but those."""
    c = Case([(20, 300)] + [(5, 0)] * (batch - 1), 8, 1, 64, seed=batch, spare=4)
    start = np.where(np.arange(batch + 1) % 2, 300, 0)
    got = c.run(cuda, start=start)
    assert (got[300:] == 7).all()
    ordered = c.run(cuda)
    c.check(ordered)


def test_far_into_the_pool(cuda):
    """Pages whose bytes and elements lie past 32 bits, and query rows as far apart; also rows that are formed again."""
    c = Case([(70, 60), (300, 2)], 8, 8, 128, seed=11)
    pages = 140000                                           # 9.2 GB
    far = torch.empty(pages, 8, 2, P, 128, dtype=BF, device=cuda)
    used = len(c.pool)
    far[pages - used:] = torch.from_numpy(c.pool).to(BF).to(cuda)
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(cuda).to(dt)
    wide = torch.empty(len(c.q), 36 << 20, dtype=BF, device=cuda)        # 62 rows of 75 MB
    q = wide[:, -1024:].unflatten(1, (8, 128))
    q.copy_(torch.from_numpy(c.q).to(BF))
    ctx = context(8, 8, 128)
    ws = torch.empty(ctx.extend_bf16_workspace_size(2, len(c.q)), dtype=torch.uint8, device=cuda)
    for bad in (False, True):
        if bad:                                              # the last token of the first request
            c.pool[c.tables[0, 129 // P], :, 1, 129 % P, 3] = np.inf
            far[pages - used:] = torch.from_numpy(c.pool).to(BF).to(cuda)
        out = torch.full(q.shape, 7.0, dtype=BF, device=cuda)
        ctx.extend_bf16(q, far, t(c.tables + (pages - used), I32), t(c.start, I32), t(c.total, I32), out, ws)
        torch.cuda.synchronize()
        got = out.double().cpu().numpy()
        want, bound = chunk_oracle.extend(c.q, np.where(np.isfinite(c.pool), c.pool, 0.0), c.tables, c.start, c.total, 1 / math.sqrt(128))
        if bad:
            assert np.isposinf(got[59, :, 3]).all()
            got[59, :, 3] = want[59, :, 3]
        assert (np.abs(got - want) <= bound).all()


def test_two_graphs_of_one_workspace(cuda):
    """Captured calls that share a workspace and run one after the other; a workspace that serves a larger call too."""
    a, b = Case([(3000, 2), (100, 1)], 8, 2, 128, seed=12), Case([(0, 300), (50, 7)], 8, 2, 128, seed=13)
    ctx = context(8, 2, 128)
    t = lambda x, dt: torch.from_numpy(np.ascontiguousarray(x)).to(cuda).to(dt)
    ws = torch.full((ctx.extend_bf16_workspace_size(5, 400),), 255, dtype=torch.uint8, device=cuda)
    calls = []
    for c in (a, b):
        args = [t(c.q, BF), t(c.pool, BF), t(c.tables, I32), t(c.start, I32), t(c.total, I32), torch.zeros(c.q.shape, dtype=BF, device=cuda), ws]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ctx.extend_bf16(*args)
        calls.append((graph, args, c))
    for graph, args, c in calls * 3:
        args[5].zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, bound = chunk_oracle.extend(c.q, c.pool, c.tables, c.start, c.total, 1 / math.sqrt(128))
        assert (np.abs(args[5].double().cpu().numpy() - want) <= bound).all()


def test_calls_at_once(cuda):
    """Two calls with a workspace each on two streams."""
    cases = [Case([(2000, 3), (40, 90)], 4, 2, 64, seed=14), Case([(0, 260)], 4, 2, 64, seed=15)]
    ctx = context(4, 2, 64)
    t = lambda x, dt: torch.from_numpy(np.ascontiguousarray(x)).to(cuda).to(dt)
    ready = []
    for c in cases:
        ws = torch.empty(ctx.extend_bf16_workspace_size(len(c.total), len(c.q)), dtype=torch.uint8, device=cuda)
        ready.append([t(c.q, BF), t(c.pool, BF), t(c.tables, I32), t(c.start, I32), t(c.total, I32), torch.zeros(c.q.shape, dtype=BF, device=cuda), ws])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for args, stream in zip(ready, streams):
            ctx.extend_bf16(*args, stream=stream)
    torch.cuda.synchronize()
    for args, c in zip(ready, cases):
        want, bound = chunk_oracle.extend(c.q, c.pool, c.tables, c.start, c.total, 1 / 8)
        assert (np.abs(args[5].double().cpu().numpy() - want) <= bound).all()


def page_sums(q, pool):
    """Per query head and page: the sums of 2^(q.k) and of 2^(q.k) v over each number of its first tokens, 0 .. 16."""
    logits = torch.einsum("rd,ptd->rpt", q, pool[:, 0, 0].double())
    w = torch.exp2(logits)
    wv = torch.cumsum(w[..., None] * pool[:, 0, 1].double(), 2)
    pad = torch.nn.functional.pad
    return pad(torch.cumsum(w, 2), (1, 0)), pad(wv, (0, 0, 1, 0))


@pytest.mark.parametrize("d,new,length", [(64, 70, 4_000_003), (128, 1, 1_500_000), (128, 150, 700_013)])
def test_sums_of_millions(cuda, d, new, length):
    """Requests enough that none is cut: an item's sums pass what the tensor core's accumulator holds without loss. The
    logits are whole and rise by 12 on the way, so that what was added up before is scaled; the values are positive.

    Of 512 tiles an accumulator takes 8 steps each, off by at most 9 * 2^-23 of it at that time, half the last one on
    average: 512 * 8 * 9 / 2 * 2^-23 of the mean. The stretches' sums, and those of the weights, are rounded to nearest,
    under 1,100 additions: 2^-13. Weights are powers of two. The output is rounded once: 2^-8."""
    batch, h_q, pages = torch.cuda.get_device_properties(0).multi_processor_count, 2, 400
    r = np.random.default_rng(d + new)
    pool = r.integers(-3, 4, (pages, 1, 2, P, d)).astype(np.float64)
    pool[pages // 2:, 0, 0] += 12.0
    pool[:, 0, 1] = r.integers(128, 256, (pages, P, d)) / 128.0
    pool = torch.from_numpy(pool).to(BF).to(cuda)
    stride = -(-length // P)
    gen = torch.Generator(device=cuda).manual_seed(new)
    tables = torch.randint(0, pages // 2, (batch, stride), dtype=I32, device=cuda, generator=gen)
    tables[1::2, stride // 3:] += pages // 2                 # the later pages of every other request weigh 2^12 as much
    tables[0, 2 * stride // 3:] += pages // 2
    q = torch.zeros(batch * new, h_q, d, dtype=BF, device=cuda)
    q[:, 0, 5] = q[:, 1, d - 1] = 1.0
    start = torch.arange(0, batch * new + 1, new, dtype=I32, device=cuda)
    total = torch.full((batch,), length, dtype=I32, device=cuda)
    out = torch.empty_like(q)
    ctx = context(h_q, 1, d, sm_scale=math.log(2))
    ws = torch.full((ctx.extend_bf16_workspace_size(batch, batch * new),), 255, dtype=torch.uint8, device=cuda)
    ctx.extend_bf16(q, pool, tables, start, total, out, ws)
    torch.cuda.synchronize()
    assert ctx.debug_error()[0] == 0
    w, wv = page_sums(q[0].double(), pool)
    relative = 512 * 8 * 9 / 2 * 2.0 ** -23 + 2.0 ** -13
    for b in range(batch):
        for i in {0, new // 2, new - 1}:
            seen = length - new + i + 1
            count = torch.bincount(tables[b, :seen // P], minlength=pages).double()
            sums, values = w[:, :, P] @ count, torch.einsum("rpd,p->rd", wv[:, :, P], count)
            if seen % P:
                last = int(tables[b, seen // P])
                sums, values = sums + w[:, last, seen % P], values + wv[:, last, seen % P]
            want = values / sums[:, None]
            bound = relative * want + 2.0 ** -8 * want * (1 + relative)
            assert ((out[b * new + i].double() - want).abs() <= bound).all(), (b, i)


def test_items_of_more_than_a_second(cuda):
    """The longest wait of a CTA's warps without rows is for a whole item of the others: here 1.3 million tiles."""
    batch, d, pages = torch.cuda.get_device_properties(0).multi_processor_count, 64, 8
    pool = torch.randint(128, 256, (pages, 1, 2, P, d), device=cuda).to(BF) / 128
    stride = 10_500_000
    tables = torch.zeros(batch, stride, dtype=I32, device=cuda)           # 6.4 GB
    tables[:, ::2] = 3
    q = torch.zeros(batch, 1, d, dtype=BF, device=cuda)
    start = torch.arange(batch + 1, dtype=I32, device=cuda)
    total = torch.full((batch,), stride * P, dtype=I32, device=cuda)
    out = torch.empty_like(q)
    ctx = context(1, 1, d)
    ws = torch.empty(ctx.extend_bf16_workspace_size(batch, batch), dtype=torch.uint8, device=cuda)
    ctx.extend_bf16(q, pool, tables, start, total, out, ws)
    torch.cuda.synchronize()
    assert ctx.debug_error()[0] == 0
    want = pool[[0, 3], 0, 1].double().mean((0, 1))
    relative = 512 * 8 * 9 / 2 * 2.0 ** -23 + 2.0 ** -12      # as above, with more stretches
    assert ((out.double() - want).abs() <= (relative + 2.0 ** -8 * (1 + relative)) * want).all()


def test_a_long_row_formed_again(cuda):
    """A row that an infinity has reached, over more tokens than a sum of ones in fp32 counts to: 2^24 values of 1, then
    as many of 2. Sums of 32 tokens are exact, those of 2^20 such sums off by 2^20 * 2^-24 at most; halved, as the sum of
    weights is exact."""
    d, length = 64, 1 << 25
    pool = torch.zeros(3, 1, 2, P, d, dtype=BF, device=cuda)
    pool[0, 0, 1], pool[1, 0, 1], pool[2, 0, 1] = 1, 2, 2
    pool[2, 0, 1, 7, 5] = float("inf")
    tables = torch.zeros(1, length // P, dtype=I32, device=cuda)
    tables[0, length // P // 2:] = 1
    tables[0, -1] = 2
    q, start = torch.zeros(1, 1, d, dtype=BF, device=cuda), torch.tensor([0, 1], dtype=I32, device=cuda)
    out, ctx = torch.empty_like(q), context(1, 1, d)
    ws = torch.empty(ctx.extend_bf16_workspace_size(1, 1), dtype=torch.uint8, device=cuda)
    ctx.extend_bf16(q, pool, tables, start, torch.tensor([length], dtype=I32, device=cuda), out, ws)
    torch.cuda.synchronize()
    assert ctx.debug_error()[0] == 0
    got = out[0, 0].double()
    assert torch.isposinf(got[5])
    got[5] = 1.5
    assert ((got - 1.5).abs() <= 1.5 * (2.0 ** -4 + 2.0 ** -8)).all()


def test_largest_batch(cuda):
    """65,535 requests, and nearly as many rows as a call takes: as many items for the plan, sampled."""
    batch, new, d, pages = 65535, 256, 64, 512
    n = batch * new
    gen = torch.Generator(device=cuda).manual_seed(3)
    lens = torch.randint(0, 40, (batch,), generator=gen, device=cuda, dtype=I32)
    pool = torch.randn(pages, 1, 2, P, d, generator=gen, device=cuda).to(BF)
    tables = torch.randint(0, pages, (batch, 19), generator=gen, device=cuda, dtype=I32)
    q = torch.randn(n, 1, d, generator=gen, device=cuda, dtype=BF)
    start = torch.arange(0, n + 1, new, dtype=I32, device=cuda)
    out, ctx = torch.full_like(q, 7.0), context(1, 1, d)
    ws = torch.full((ctx.extend_bf16_workspace_size(batch, n),), 255, dtype=torch.uint8, device=cuda)
    ctx.extend_bf16(q, pool, tables, start, lens + new, out, ws)
    torch.cuda.synchronize()
    assert ctx.debug_error()[0] == 0
    for b in [0, 1, 777, 32768, 65000, batch - 1]:
        rows = slice(b * new, (b + 1) * new)
        want, bound = chunk_oracle.extend(q[rows].double().cpu().numpy(), pool.double().cpu().numpy(), tables[b:b + 1].cpu().numpy(),
                                          [0, new], [int(lens[b]) + new], 1 / 8)
        assert (np.abs(out[rows].double().cpu().numpy() - want) <= bound).all(), b
