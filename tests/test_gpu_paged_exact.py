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
