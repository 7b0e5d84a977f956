"""oscar_norm_rope against its fp64 definition (rope_oracle.py, which derives the tolerance)."""

import numpy as np
import pytest
import torch

import rope_oracle
from bit_kv_cache_write_gb300 import oscar as O
from bit_kv_cache_write_gb300 import rope

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


def context(h_q, h_kv, d):
    return O.Oscar(n_layers=1, n_q_heads=h_q, n_kv_heads=h_kv, head_dim=d, group=32)


def rows(cuda, n, h_q, h_kv, d, seed, gap=0):
    """q, k as slices of projection rows [n][H_q + 2 H_kv][d], `gap` elements between rows."""
    gen = torch.Generator(device=cuda).manual_seed(seed)
    w = (h_q + 2 * h_kv) * d
    qkv = torch.randn(max(n, 1), w + gap, generator=gen, device=cuda).to(BF)[:n, :w].unflatten(1, (h_q + 2 * h_kv, d))
    return qkv[:, :h_q], qkv[:, h_q:h_q + h_kv]


def check(got, x, weight, eps, turns, layout, scale, positions):
    want, bound = rope_oracle.norm_rope(x.double().cpu().numpy(), None if weight is None else weight.cpu().numpy(), eps,
                                        np.asarray(turns).view(np.uint64).tolist(), layout == O.OSCAR_ROPE_INTERLEAVED,
                                        scale, positions)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("n,h_q,h_kv,d,rot,layout,norm,gap", [
    (1, 32, 8, 128, 128, 0, True, 0), (1, 4, 2, 64, 64, 1, True, 8), (3, 8, 8, 64, 16, 0, False, 0),
    (5, 2, 1, 128, 24, 0, True, 0), (5, 2, 1, 128, 24, 1, False, 16), (7, 1, 1, 64, 8, 1, True, 0),
    (257, 32, 8, 128, 64, 1, True, 0), (300, 64, 8, 64, 64, 0, False, 0), (2203, 16, 2, 128, 96, 0, True, 8),
    (2500, 4, 4, 64, 0, 0, True, 0),
])
def test_given_positions(cuda, n, h_q, h_kv, d, rot, layout, norm, gap):
    q, k = rows(cuda, n, h_q, h_kv, d, n, gap)
    r = np.random.default_rng(n)
    pos = r.integers(0, 1 << 20, n)
    turns, scale = (rope.rope_turns(rot, 1e6, dict(kind="yarn", factor=4, trained=32768)) if rot else
                    (np.zeros(0, np.int64), 1.0))
    weights = [torch.from_numpy(r.normal(1, 0.3, d)).float().to(cuda) if norm else None for _ in range(2)]
    qo, ko = torch.empty(n, h_q, d, dtype=BF, device=cuda), torch.empty(n, h_kv, d, dtype=BF, device=cuda)
    context(h_q, h_kv, d).norm_rope(q, k, qo, ko, torch.from_numpy(turns).to(cuda),
                                    positions=torch.from_numpy(pos).to(I32).to(cuda), q_weight=weights[0],
                                    k_weight=weights[1], layout=layout, scale=scale)
    for x, y, w in ((q, qo, weights[0]), (k, ko, weights[1])):
        check(y, x, w, 1e-6, turns, layout, scale, pos)


@pytest.mark.parametrize("lens", [[(0, 1)], [(100, 1)] * 70, [(5, 0), (0, 3), (7, 0), (9, 0), (2000, 33), (1, 0)],
                                  [(i % 7, i % 3) for i in range(1500)], [(3, 2), (40, 900), (0, 1)]])
def test_positions_of_the_plan(cuda, lens):
    """Rows of the requests turn by their place in the sequence; rows behind the last request stay."""
    h_q, h_kv, d, spare = 4, 2, 64, 5
    new = np.array([m for _, m in lens])
    start = np.concatenate([[0], np.cumsum(new)])
    n = int(start[-1])
    q, k = rows(cuda, n + spare, h_q, h_kv, d, n)
    pos = np.concatenate([np.arange(c, c + m) for c, m in lens])
    turns, _ = rope.rope_turns(d, 1e4)
    qo, ko = (torch.full((n + spare, h, d), 7.0, dtype=BF, device=cuda) for h in (h_q, h_kv))
    total = np.array([c + m for c, m in lens])
    context(h_q, h_kv, d).norm_rope(q, k, qo, ko, torch.from_numpy(turns).to(cuda),
                                    row_start=torch.from_numpy(start).to(I32).to(cuda),
                                    total_len=torch.from_numpy(total).to(I32).to(cuda))
    check(qo[:n], q[:n], None, 0, turns, 0, 1.0, pos)
    check(ko[:n], k[:n], None, 0, turns, 0, 1.0, pos)
    assert (qo[n:] == 7).all() and (ko[n:] == 7).all()


def test_no_request_leaves_every_row(cuda):
    q, k = rows(cuda, 3, 4, 2, 64, 1)
    qo, ko = torch.full((3, 4, 64), 7.0, dtype=BF, device=cuda), torch.full((3, 2, 64), 7.0, dtype=BF, device=cuda)
    turns, _ = rope.rope_turns(64)
    context(4, 2, 64).norm_rope(q, k, qo, ko, torch.from_numpy(turns).to(cuda),
                                row_start=torch.zeros(1, dtype=I32, device=cuda),
                                total_len=torch.empty(0, dtype=I32, device=cuda))
    assert (qo == 7).all() and (ko == 7).all()


@pytest.mark.parametrize("layout", [0, 1])
def test_far_and_negative_positions(cuda, layout):
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 24, (1 << 24) + 1])
    q, k = rows(cuda, len(pos), 4, 2, 64, 3)
    turns, _ = rope.rope_turns(64, 1e4)
    qo, ko = torch.empty(len(pos), 4, 64, dtype=BF, device=cuda), torch.empty(len(pos), 2, 64, dtype=BF, device=cuda)
    context(4, 2, 64).norm_rope(q, k, qo, ko, torch.from_numpy(turns).to(cuda),
                                positions=torch.from_numpy(pos).to(I32).to(cuda), layout=layout)
    check(qo, q, None, 0, turns, layout, 1.0, pos)
    check(ko, k, None, 0, turns, layout, 1.0, pos)


@pytest.mark.parametrize("n", [2, 700])
def test_in_place_and_one_of_both(cuda, n):
    q, k = rows(cuda, n, 32, 8, 128, n)
    turns, _ = rope.rope_turns(128, 1e4)
    t, pos = torch.from_numpy(turns).to(cuda), torch.arange(n, dtype=I32, device=cuda)
    w = torch.linspace(0.5, 2, 128, device=cuda)
    ctx = context(32, 8, 128)
    qo, ko = torch.empty(n, 32, 128, dtype=BF, device=cuda), torch.empty(n, 8, 128, dtype=BF, device=cuda)
    ctx.norm_rope(q, k, qo, ko, t, positions=pos, q_weight=w)
    only_q, only_k = torch.empty_like(qo), torch.empty_like(ko)
    ctx.norm_rope(q, None, only_q, None, t, positions=pos, q_weight=w)
    ctx.norm_rope(None, k, None, only_k, t, positions=pos, q_weight=w)
    check(qo, q, w, 1e-6, turns, 0, 1.0, range(n))
    check(ko, k, None, 1e-6, turns, 0, 1.0, range(n))
    ctx.norm_rope(q, k, q, k, t, positions=pos, q_weight=w)
    for a in (only_q, q):
        assert torch.equal(a, qo)
    for a in (only_k, k):
        assert torch.equal(a, ko)


def test_norm_of_extreme_rows(cuda):
    """Squares that pass fp32 do not lose the norm; a row that holds an infinity, NaN or zeros keeps that to itself."""
    d = 128
    x = torch.randn(6, 1, d, device=cuda).to(BF)
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -40
    x[3] = 0
    x[4, 0, 5] = float("inf")
    x[5, 0, 6] = float("nan")
    turns, _ = rope.rope_turns(d)
    out, w = torch.empty_like(x), torch.ones(d, device=cuda)
    context(1, 1, d).norm_rope(x, None, out, None, torch.from_numpy(turns).to(cuda), q_weight=w,
                               positions=torch.zeros(6, dtype=I32, device=cuda))
    check(out[:4], x[:4], w, 1e-6, turns, 0, 1.0, [0] * 4)
    assert (out[3] == 0).all() and torch.isnan(out[4, 0, [5, 69]]).all() and torch.isnan(out[5]).all()
    assert (out[4, 0, [0, 1, 2, 3, 4, 64, 65, 68]] == 0).all()


def test_captured_on_another_stream(cuda):
    """One graph: lengths that move on the device, outputs that another call made on the same stream reads."""
    h_q, h_kv, d, batch = 4, 2, 64, 3
    q, k = rows(cuda, batch, h_q, h_kv, d, 9)
    turns, _ = rope.rope_turns(d)
    t, start = torch.from_numpy(turns).to(cuda), torch.arange(batch + 1, dtype=I32, device=cuda)
    total = torch.tensor([1, 50, 3001], dtype=I32, device=cuda)
    qo, ko = torch.empty(batch, h_q, d, dtype=BF, device=cuda), torch.empty(batch, h_kv, d, dtype=BF, device=cuda)
    ctx, side = context(h_q, h_kv, d), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ctx.norm_rope(q, k, qo, ko, t, row_start=start, total_len=total)
        total += 1
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        pos = np.array([0, 49, 3000]) + step
        check(qo, q, None, 0, turns, 0, 1.0, pos)
        check(ko, k, None, 0, turns, 0, 1.0, pos)


def test_rows_far_apart(cuda):
    """Row offsets past 32 bits, in and out."""
    n, h, d = 70, 4, 64
    wide = torch.empty(n, 36 << 20, dtype=BF, device=cuda)               # 70 rows of 75 MB
    q, out = (wide[:, at:at + h * d].unflatten(1, (h, d)) for at in (0, 1 << 20))
    x = torch.randn(n, h, d, device=cuda).to(BF)
    q.copy_(x)
    turns, _ = rope.rope_turns(d)
    w = torch.linspace(0.5, 2, d, device=cuda)
    context(h, h, d).norm_rope(q, None, out, None, torch.from_numpy(turns).to(cuda), q_weight=w,
                               positions=torch.arange(n, dtype=I32, device=cuda))
    check(out, x, w, 1e-6, turns, 0, 1.0, range(n))
    assert torch.equal(q, x)


@pytest.mark.parametrize("layout", [0, 1])
def test_norm_of_the_smallest_and_largest(cuda, layout):
    """Squares above and below fp32: rows of the largest numbers, one of them, and with no eps (or hardly any) rows of the
    smallest. Rows of both kinds in one warp."""
    d, top = 64, torch.finfo(BF).max
    x = torch.randn(4, 4, d, device=cuda).double()
    sign = torch.sign(x)
    x[0] = sign[0] * top
    x[1] *= 2.0 ** 100
    x[1, :, 5] = top
    x[2, 0], x[2, 1], x[2, 2] = x[2, 0] * 2.0 ** -40, x[2, 1] * 2.0 ** -70, x[2, 2] * 2.0 ** -110
    x[3, :] = sign[3] * 2.0 ** -133                                      # bf16's smallest
    x[3, 1] = sign[3, 1] * top
    x = x.to(BF)
    turns, _ = rope.rope_turns(d)
    w, pos = torch.linspace(0.5, 2, d, device=cuda), [0, 1, 77, 1 << 20]
    for eps, rows_of in ((0.0, 4), (1e-30, 2), (1e-6, 3)):
        out = torch.empty_like(x)
        context(4, 4, d).norm_rope(x, None, out, None, torch.from_numpy(turns).to(cuda), q_weight=w, eps=eps, layout=layout,
                                   positions=torch.tensor(pos, dtype=I32, device=cuda))
        check(out[:rows_of], x[:rows_of], w, float(np.float32(eps)), turns, layout, 1.0, pos[:rows_of])
    # an eps between the squares of two heads: no root of either's alone
    x = (torch.randn(1, 4, d, device=cuda).double() * torch.tensor([2.0 ** -52, 2.0 ** -49, 2.0 ** -36, 1.0], device=cuda)[:, None]).to(BF)
    out = torch.empty_like(x)
    context(4, 4, d).norm_rope(x, None, out, None, torch.from_numpy(turns).to(cuda), q_weight=w, eps=2.0 ** -100, layout=layout,
                               positions=torch.zeros(1, dtype=I32, device=cuda))
    check(out, x, w, 2.0 ** -100, turns, layout, 1.0, [0])


def test_turns_formed_on_the_stream(cuda):
    """Turns that a kernel in front of the call writes, as when the context's scaling follows the length."""
    n, h, d = 3, 4, 64
    q, _ = rows(cuda, n, h, h, d, 5)
    tables = [torch.from_numpy(rope.rope_turns(d, base)[0]).to(cuda) for base in (1e4, 1e5, 1e6)]
    t, pos = torch.zeros_like(tables[0]), torch.tensor([3, 1000, 100000], dtype=I32, device=cuda)
    outs = [torch.empty(n, h, d, dtype=BF, device=cuda) for _ in tables]
    ctx, side = context(h, h, d), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for table, out in zip(tables, outs):
            torch.add(table, 0, out=t)
            ctx.norm_rope(q, None, out, None, t, positions=pos)
    for _ in range(3):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for table, out in zip(tables, outs):
            check(out, q, None, 0, table.cpu().numpy(), 0, 1.0, pos.tolist())
