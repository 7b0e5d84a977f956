"""The BF16 paged-cache operators, as cases to measure: planning, appending, dense and sparse decode.

A case names one operator and its sizes. ``run`` makes one pass: with ``own`` false in elementary torch
operations, with ``own`` true through the library's calls. Pools are BF16 pages of 16 tokens,
[pages][H_kv][K, V][16][d]; lengths are a function of the case alone (log-spaced between two bounds),
their order, the page ids and all values come from the seed.
"""

import math

import numpy as np
import torch

own = False

_DEV = torch.device("cuda")
_P = 16                      # tokens per page
_SINK, _RECENT = 64, 256     # windows that the sparse decode always reads


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a serving batch: a token for each of 64 running requests
        dict(name="plan_step_b64", op="plan", batch=64, cached_lo=200, cached_hi=32768, new_lo=1, new_hi=1),
        # a chunk of ragged prefills next to running requests, 131k tokens at most in one plan
        dict(name="plan_prefill_b96", op="plan", batch=96, cached_lo=0, cached_hi=16384, new_lo=1, new_hi=8192),
        # the same decode step's K/V rows, 256 sequences, no key bounds kept
        dict(name="append_step_b256", op="append", batch=256, cached_lo=77, cached_hi=2048, new_lo=1, new_hi=1,
             h_kv=8, d=128, bounds=False),
        # a bulk prefill with key bounds: 131,072 tokens, the size of the bulk INT2 write
        dict(name="append_prefill_131k", op="append", batch=8, cached_lo=0, cached_hi=0, new_lo=16384, new_hi=16384,
             h_kv=8, d=128, bounds=True),
        # the smallest decode: the tiny configuration (latency)
        dict(name="dense_tiny", op="dense", batch=1, len_lo=1344, len_hi=1344, h_q=4, h_kv=2, d=64, out="float32"),
        # one user, 100,000 tokens of context
        dict(name="dense_bs1_100k", op="dense", batch=1, len_lo=100000, len_hi=100000, h_q=32, h_kv=8, d=128,
             out="float32"),
        # a large batch at 32k
        dict(name="dense_b64_32k", op="dense", batch=64, len_lo=32768, len_hi=32768, h_q=32, h_kv=8, d=128,
             out="bfloat16"),
        # a mixed batch, 4k to 131k, eight query heads to a KV head
        dict(name="dense_mixed16", op="dense", batch=16, len_lo=4096, len_hi=131072, h_q=64, h_kv=8, d=128,
             out="float32"),
        # sparse decode, smallest: the tiny configuration with an eighth of its pages
        dict(name="sparse_tiny", op="sparse", batch=1, len_lo=1344, len_hi=1344, h_q=4, h_kv=2, d=64, top=8,
             out="float32"),
        # one user at 100,000 tokens, 4,096 of them selected next to sink and recent window
        dict(name="sparse_bs1_100k", op="sparse", batch=1, len_lo=100000, len_hi=100000, h_q=32, h_kv=8, d=128,
             top=256, out="float32"),
        # the large batch at 32k, 2,048 tokens selected
        dict(name="sparse_b64_32k", op="sparse", batch=64, len_lo=32768, len_hi=32768, h_q=32, h_kv=8, d=128,
             top=128, out="bfloat16"),
        # the mixed batch: the shorter sequences are read almost whole
        dict(name="sparse_mixed16", op="sparse", batch=16, len_lo=4096, len_hi=131072, h_q=64, h_kv=8, d=128,
             top=256, out="float32"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["plan", "append", "dense", "dense", "sparse", "sparse"])
    if op == "plan":
        batch = log(1, 512)
        new_hi = log(1, min(8192, 131072 // batch))
        return dict(op=op, batch=batch, cached_lo=rng.choice([0, log(1, 300)]), cached_hi=log(301, 32768),
                    new_lo=rng.randint(0, 1), new_hi=new_hi)
    h_kv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "append":
        batch = log(1, 256)
        return dict(op=op, batch=batch, cached_lo=rng.choice([0, log(1, 300)]), cached_hi=log(301, 8192),
                    new_lo=rng.randint(0, 1), new_hi=log(1, min(16384, 131072 // batch)), h_kv=h_kv, d=d,
                    bounds=rng.random() < 0.7)
    g = rng.choice([1, 2, 4, 8])
    batch = log(1, 64)
    hi = log(17, min(131072, 1 << 21) // (1 if batch <= 16 else batch // 16 + 1))
    lo = min(hi, rng.choice([0, 1, log(1, hi), hi]))
    case = dict(op=op, batch=batch, len_lo=lo, len_hi=hi, h_q=g * h_kv, h_kv=h_kv, d=d,
                out=rng.choice(["float32", "bfloat16"]))
    if op == "sparse":
        case["top"] = log(1, 384)
    return case


def _spread(lo, hi, n):
    """n lengths, log-spaced from lo to hi (0 stands for an empty one)."""
    if n == 1 or lo == hi:
        return [hi] * n
    a = max(lo, 1)
    got = [int(round(a * (hi / a) ** (i / (n - 1)))) for i in range(n)]
    if lo == 0:
        got[0] = 0
    return got


def _pages(n):
    return (n + _P - 1) // _P


def _window(length, top):
    """(pages, kept sink pages, first kept recent page, selected pages) of a sequence in the sparse decode."""
    n = _pages(length)
    sink = min(n, _pages(_SINK))
    first = min(n, max(length - _RECENT, 0) // _P)
    return n, sink, first, min(top, max(first - sink, 0))


def _capacity(top):
    """Entries of a chosen list: sink pages, the pages that a recent window can touch, selected pages."""
    return _pages(_SINK) + _pages(_RECENT) + 1 + top


def work(case):
    if case["op"] == "plan":
        news = _spread(case["new_lo"], case["new_hi"], case["batch"])
        total = sum(news)
        # lengths in, totals and row starts out, one slot of 8 bytes per token, one page id in and out per page
        return dict(bytes=16 * case["batch"] + 8 * total + 8 * (total // _P + case["batch"]), flops=0)
    if case["op"] == "append":
        total = sum(_spread(case["new_lo"], case["new_hi"], case["batch"]))
        row = case["h_kv"] * case["d"]
        pages = total // _P + case["batch"]
        return dict(bytes=8 * total + 2 * total * row * 2 * 2 + (pages * 2 * row if case["bounds"] else 0),
                    flops=2 * total * row if case["bounds"] else 0)
    lens = _spread(case["len_lo"], case["len_hi"], case["batch"])
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    io = case["batch"] * h_q * d * (2 + (4 if case["out"] == "float32" else 2))
    if case["op"] == "dense":
        return dict(bytes=sum(lens) * h_kv * d * 4 + 4 * sum(map(_pages, lens)) + io, flops=4 * sum(lens) * h_q * d)
    read = scored = 0
    for n in lens:
        pages, sink, first, sel = _window(n, case["top"])
        scored += max(first - sink, 0)
        read += min(n, sink * _P) + sel * _P + max(n - max(first, sink) * _P, 0)
    return dict(bytes=read * h_kv * d * 4 + scored * h_kv * 2 * d + 4 * sum(map(_pages, lens)) + io,
                flops=4 * read * h_q * d + 4 * scored * h_q * d)


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device=_DEV, dtype=torch.float32)


def _order(values, gen):
    """The values as int32 on the GPU, in an order of the seed's."""
    t = torch.tensor(values, dtype=torch.int32).to(_DEV)
    return t[torch.randperm(len(values), generator=gen, device=_DEV)].contiguous()


def _tables(lens, extra, gen):
    """Block tables of shuffled page ids for the given lengths plus `extra` page ids that no table holds."""
    n = ((lens + _P - 1) // _P).long()
    used = int(n.sum())
    stride = max(1, int(n.max()))
    ids = torch.randperm(used + extra, generator=gen, device=_DEV).to(torch.int32)
    col = torch.arange(stride, device=_DEV)
    start = torch.cumsum(n, 0) - n
    inside = col[None] < n[:, None]
    at = (start[:, None] + col[None]).clamp(max=max(used - 1, 0))
    table = torch.where(inside, ids[at] if used else torch.zeros_like(at, dtype=torch.int32), torch.zeros((), dtype=torch.int32, device=_DEV))
    return table.to(torch.int32).contiguous(), ids[used:].contiguous(), used + extra


def _channel_scale(gen, h_kv, d):
    """Key scales per channel as real keys have them: log-normal, with a few outlier channels."""
    s = torch.exp(0.4 * _randn(gen, h_kv, d))
    s[:, torch.randperm(d, generator=gen, device=_DEV)[: max(1, d // 50)]] *= 4.0
    return s


def _steps(scale):
    """Power-of-two steps of the key bounds: 4.5 standard deviations reach 127 steps."""
    return torch.ceil(torch.log2(4.5 * scale / 127.0)).to(torch.int8).contiguous()


def _fill(pool, scale, gen, bounds=None, steps=None):
    """K and V rows of every page; keys of a page share a drift, so that pages differ for a query."""
    pages, h_kv, _, _, d = pool.shape
    chunk = max(1, (1 << 27) // (h_kv * 2 * _P * d))
    for p in range(0, pages, chunk):
        q = min(pages, p + chunk)
        x = torch.randn(q - p, h_kv, 2, _P, d, generator=gen, device=_DEV, dtype=torch.bfloat16)
        drift = _randn(gen, q - p, h_kv, 1, d) * 0.6
        x[:, :, 0] = ((x[:, :, 0].float() * 0.8 + drift) * scale[None, :, None]).to(torch.bfloat16)
        pool[p:q] = x
        if bounds is not None:
            c = _codes(x[:, :, 0], steps[None, :, None])
            bounds[p:q, :, 0], bounds[p:q, :, 1] = c.amin(2), c.amax(2)


def _codes(k, steps):
    c = torch.round(torch.ldexp(k.float(), -steps.int()))
    return torch.nan_to_num(c, nan=0.0, posinf=127.0, neginf=-127.0).clamp(-127, 127).to(torch.int8)


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] in ("plan", "append"):
        cached = _order(_spread(case["cached_lo"], case["cached_hi"], case["batch"]), gen)
        new = _order(_spread(case["new_lo"], case["new_hi"], case["batch"]), gen)
        total = int(new.sum())
        need = total // _P + 2 * case["batch"]
        tables, free, pages = _tables(cached, need + 5, gen)
        stride = _pages(case["cached_hi"] + case["new_hi"])
        wide = torch.zeros(case["batch"], stride, dtype=torch.int32, device=_DEV)
        wide[:, : min(stride, tables.shape[1])] = tables[:, :stride]
        i32 = dict(dtype=torch.int32, device=_DEV)
        s.update(seq_len=cached, new_len=new, tables=wide, free_pages=free, free_head=torch.full((1,), 3, **i32),
                 slots=torch.empty(total + 9, dtype=torch.int64, device=_DEV), row_start=torch.empty(case["batch"] + 1, **i32),
                 total_len=torch.empty(case["batch"], **i32), state=torch.empty(4, **i32))
        if case["op"] == "append":
            h_kv, d = case["h_kv"], case["d"]
            slots = _plan(s)["slots"][:total].clone()
            scale = _channel_scale(gen, h_kv, d)
            pool = torch.zeros(pages, h_kv, 2, _P, d, dtype=torch.bfloat16, device=_DEV)
            # K and V as a projection leaves them: two slices of one row
            kv = torch.randn(max(total, 1), 2, h_kv, d, generator=gen, device=_DEV, dtype=torch.bfloat16)[:total]
            kv[:, 0] = (kv[:, 0].float() * scale[None]).to(torch.bfloat16)
            s = dict(case=case, k=kv[:, 0], v=kv[:, 1], slots=slots, pool=pool, steps=None, bounds=None)
            if case["bounds"]:
                s["steps"] = _steps(scale)
                s["bounds"] = torch.randint(-20, 0, (pages, h_kv, 2, d), generator=gen, device=_DEV, dtype=torch.int8)
                s["bounds"][:, :, 1] += 30
        if own:      # the context that a serving loop keeps
            h_kv = case.get("h_kv", 8)
            s["ctx"] = _context(h_kv, h_kv, case.get("d", 128))
        return s
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    lens = _order(_spread(case["len_lo"], case["len_hi"], case["batch"]), gen)
    tables, _, pages = _tables(lens, 2, gen)
    scale = _channel_scale(gen, h_kv, d)
    pool = torch.empty(pages, h_kv, 2, _P, d, dtype=torch.bfloat16, device=_DEV)
    bounds = steps = None
    if case["op"] == "sparse":
        bounds = torch.empty(pages, h_kv, 2, d, dtype=torch.int8, device=_DEV)
        steps = _steps(scale)
    _fill(pool, scale, gen, bounds, steps)
    q = _randn(gen, case["batch"], h_q, d).to(torch.bfloat16)
    out = torch.empty(case["batch"], h_q, d, dtype=getattr(torch, case["out"]), device=_DEV)
    s.update(q=q, pool=pool, tables=tables, seq_len=lens, max_len=case["len_hi"], out=out)
    if case["op"] == "sparse":
        cap = _capacity(case["top"])
        s.update(bounds=bounds, steps=steps, top=case["top"],
                 chosen=torch.empty(case["batch"], h_kv, cap, dtype=torch.int32, device=_DEV),
                 n_chosen=torch.empty(case["batch"], h_kv, dtype=torch.int32, device=_DEV))
    if own:      # the context and workspace that a serving loop keeps
        s["ctx"] = ctx = _context(h_q, h_kv, d)
        size = (ctx.decode_bf16_sparse_workspace_size(case["batch"], s["max_len"], s["top"]) if case["op"] == "sparse"
                else ctx.decode_bf16_workspace_size(case["batch"], s["max_len"]))
        s["ws"] = torch.empty(max(size, 1), dtype=torch.uint8, device=_DEV)
    return s


def _context(h_q, h_kv, d):
    from bit_kv_cache_write_gb300 import oscar
    return oscar.Oscar(n_layers=1, n_q_heads=h_q, n_kv_heads=h_kv, head_dim=d, group=64, sink=_SINK, recent=_RECENT)


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        ctx = s["ctx"]
        if op == "plan":
            ctx.plan_append(s["seq_len"], s["new_len"], s["free_pages"], s["free_head"], s["tables"], s["slots"],
                            s["row_start"], s["total_len"], s["state"])
            return {k: s[k] for k in ("tables", "slots", "row_start", "total_len", "state")}
        if op == "append":
            ctx.append_bf16(s["k"], s["v"], s["slots"], s["pool"], s["steps"], s["bounds"])
            return {k: s[k] for k in ("pool", "bounds")}
        if op == "dense":
            ctx.decode_bf16(s["q"], s["pool"], s["tables"], s["seq_len"], s["max_len"], s["out"], s["ws"])
            return s["out"]
        ctx.decode_bf16_sparse(s["q"], s["pool"], s["steps"], s["bounds"], s["tables"], s["seq_len"], s["max_len"],
                               s["top"], s["chosen"], s["n_chosen"], s["out"], s["ws"])
        return {k: s[k] for k in ("out", "chosen", "n_chosen")}
    return {"plan": _plan, "append": _append, "dense": _dense, "sparse": _sparse}[op](s)


def _plan(s):
    """Block tables and slot maps: pages handed out in request order, tokens numbered request by request."""
    cached, new = s["seq_len"].long(), s["new_len"].long()
    tables, slots = s["tables"], s["slots"]
    batch, stride = tables.shape
    rows = torch.cumsum(new, 0)
    valid = (cached >= 0) & (new >= 0) & (cached + new <= stride * _P) & (rows <= slots.numel())
    old = (cached + _P - 1) // _P
    need = torch.where(valid, (cached + new + _P - 1) // _P - old, 0)
    upto = torch.cumsum(need, 0)
    head = s["free_head"].long()
    ok = valid & ((need == 0) | (upto <= s["free_pages"].numel() - head))
    taken = torch.where(ok, need, 0)
    col = torch.arange(stride, device=tables.device)[None]
    fresh = (col >= old[:, None]) & (col < (old + taken)[:, None])
    at = (head + (upto - need)[:, None] + col - old[:, None]).clamp(0, s["free_pages"].numel() - 1)
    out_tables = torch.where(fresh, s["free_pages"][at], tables)
    t = torch.arange(slots.numel(), device=tables.device)
    b = torch.searchsorted(rows, t, right=True)
    inside = b < batch
    b = b.clamp(max=batch - 1)
    pos = cached[b] + t - (rows - new)[b]
    page = out_tables[b, (pos // _P).clamp(0, stride - 1)].long()
    row_start = torch.cat([torch.zeros_like(rows[:1]), rows]).int()
    bad = ~ok
    first = torch.where(bad.any(), bad.int().argmax(), -1)
    return dict(tables=out_tables, slots=torch.where(inside & ok[b], page * _P + pos % _P, -1), row_start=row_start,
                total_len=torch.where(ok, cached + new, cached).int(),
                state=torch.stack([head[0] + taken.sum(), rows[-1], bad.sum(), first]).int())


def _append(s):
    """K and V rows into their slots; the key bounds of the pages that they touch."""
    pool, slots = s["pool"], s["slots"]
    page, row = slots // _P, slots % _P
    pool[page, :, 0, row] = s["k"]
    pool[page, :, 1, row] = s["v"]
    if s["bounds"] is None:
        return dict(pool=pool, bounds=None)
    bounds = s["bounds"]
    codes = _codes(s["k"], s["steps"][None])
    lo, hi = bounds[:, :, 0].float(), bounds[:, :, 1].float()
    started = torch.zeros(pool.shape[0], device=pool.device).index_add(0, page, (row == 0).float()) > 0
    lo = torch.where(started[:, None, None], 127.0, lo)
    hi = torch.where(started[:, None, None], -127.0, hi)
    at = page[:, None, None].expand(codes.shape)
    bounds[:, :, 0] = lo.scatter_reduce(0, at, codes.float(), "amin").to(torch.int8)
    bounds[:, :, 1] = hi.scatter_reduce(0, at, codes.float(), "amax").to(torch.int8)
    return dict(pool=pool, bounds=bounds)


def _softmax_av(q, k, v, valid):
    """q [B, H, g, d], k and v [B, H, n, d] in fp32, valid [B, 1 or H, 1, n]: attention, zeros where nothing is valid."""
    logits = (q @ k.transpose(-1, -2)) * q.shape[-1] ** -0.5
    logits = torch.where(valid, logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return (p @ torch.where(valid.transpose(-1, -2), v, 0.0)) / torch.where(total > 0, total, 1.0)


def _dense(s):
    q, pool, tables = s["q"], s["pool"], s["tables"].long()
    batch, h_q, d = q.shape
    h_kv = pool.shape[1]
    n = tables.shape[1] * _P
    kv = pool[tables]                                                 # [B, pages, H_kv, 2, 16, d]
    k = kv[:, :, :, 0].float().permute(0, 2, 1, 3, 4).reshape(batch, h_kv, n, d)
    v = kv[:, :, :, 1].float().permute(0, 2, 1, 3, 4).reshape(batch, h_kv, n, d)
    valid = torch.arange(n, device=q.device)[None] < s["seq_len"][:, None]
    out = _softmax_av(q.float().reshape(batch, h_kv, h_q // h_kv, d), k, v, valid[:, None, None])
    return out.reshape(batch, h_q, d).to(s["out"].dtype)


def _query_codes(q, steps):
    """Integer query codes and their exponents: q [B, H_kv, g, d] fp32 in the steps of the key bounds."""
    x = torch.ldexp(q, steps.int()[None, :, None])
    x = torch.where(torch.isfinite(x), x, 0.0)
    top = x.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 7).clamp(max=60)
    codes = torch.round(torch.ldexp(x, -e)).clamp(-127, 127)
    return torch.where(top < 2.0 ** -60, 0.0, codes), e


def _sparse(s):
    q, pool, tables, lens, top = s["q"], s["pool"], s["tables"].long(), s["seq_len"].long(), s["top"]
    batch, h_q, d = q.shape
    h_kv, g, pages = pool.shape[1], h_q // pool.shape[1], tables.shape[1]
    qf = q.float().reshape(batch, h_kv, g, d)
    codes, e = _query_codes(qf, s["steps"])
    b = s["bounds"][tables].float()                                   # [B, pages, H_kv, 2, d]
    lo, hi = b[:, :, :, 0].permute(0, 2, 3, 1), b[:, :, :, 1].permute(0, 2, 3, 1)
    dots = codes.clamp(max=0) @ lo + codes.clamp(min=0) @ hi         # integers below 2^24: exact in fp32
    score = torch.ldexp(dots, e).amax(2)                              # [B, H_kv, pages]
    idx = torch.arange(pages, device=q.device)[None]
    n = ((lens + _P - 1) // _P)[:, None]
    sink = n.clamp(max=_pages(_SINK))
    first = torch.minimum(n, ((lens - _RECENT).clamp(min=0) // _P)[:, None])
    kept = (idx < n) & ((idx < sink) | (idx >= first))
    cand = ((idx >= sink) & (idx < first))[:, None]
    order = torch.sort(torch.where(cand, score, -math.inf), dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(-1, order, idx[None].expand_as(order))
    take = kept[:, None] | (cand & (rank < top))
    cap = s["chosen"].shape[-1]
    chosen = torch.sort(torch.where(take, idx[None], pages), dim=-1)[0]
    chosen = torch.nn.functional.pad(chosen, (0, max(0, cap - pages)), value=pages)[..., :cap]
    real = chosen < pages
    chosen = torch.where(real, chosen, 0)
    phys = torch.gather(tables[:, None].expand(batch, h_kv, pages), 2, chosen)
    kv = pool[phys, torch.arange(h_kv, device=q.device)[None, :, None]]      # [B, H_kv, cap, 2, 16, d]
    k, v = (kv[:, :, :, i].float().reshape(batch, h_kv, cap * _P, d) for i in range(2))
    token = chosen[..., None] * _P + torch.arange(_P, device=q.device)
    valid = (real[..., None] & (token < lens[:, None, None, None])).reshape(batch, h_kv, 1, cap * _P)
    out = _softmax_av(qf, k, v, valid).reshape(batch, h_q, d)
    return dict(out=out.to(s["out"].dtype), chosen=torch.where(real, chosen, -1).int(), n_chosen=real.sum(-1).int())


# ---------------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                                      # whole numbers only
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_decode(s)


def _exact_append(s):
    pool = s["pool"].double()
    flat = pool.permute(0, 3, 1, 2, 4).reshape(-1, pool.shape[1], 2, pool.shape[4])       # one row per slot
    flat.index_copy_(0, s["slots"], torch.stack([s["k"], s["v"]], 2).double())
    pool = flat.reshape(pool.shape[0], _P, pool.shape[1], 2, pool.shape[4]).permute(0, 2, 3, 1, 4).contiguous()
    return dict(pool=pool, bounds=None)


def _exact_decode(s):
    case, lens = s["case"], s["seq_len"].tolist()
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    g = h_q // h_kv
    sparse = case["op"] == "sparse"
    out = torch.zeros(case["batch"], h_q, d, dtype=torch.float64, device=_DEV)
    for b, length in enumerate(lens):
        n = _pages(length)
        if n == 0:
            continue
        ids = s["tables"][b, :n].long()
        q = s["q"][b].double().reshape(h_kv, g, d)
        if not sparse:
            kv = s["pool"][ids].double().permute(2, 1, 0, 3, 4).reshape(2, h_kv, n * _P, d)[:, :, :length]
            out[b] = _exact_attention(q, kv[0], kv[1]).reshape(h_q, d)
            continue
        score = _exact_scores(q, s["steps"], s["bounds"][ids])
        _, sink, first, sel = _window(length, s["top"])
        for h in range(h_kv):
            cand = np.arange(sink, max(first, sink))
            best = cand[np.lexsort((cand, -score[h, cand]))[:sel]]
            take = np.sort(np.concatenate([np.arange(sink), best, np.arange(max(first, sink), n)]))
            kv = s["pool"][ids[torch.from_numpy(take).to(_DEV)], h].double()
            tok = (torch.from_numpy(take).to(_DEV)[:, None] * _P + torch.arange(_P, device=_DEV)).reshape(-1) < length
            k, v = kv[:, 0].reshape(-1, d)[tok], kv[:, 1].reshape(-1, d)[tok]
            out[b, h * g:(h + 1) * g] = _exact_attention(q[h][None], k[None], v[None])[0]
    return dict(out=out, chosen=None, n_chosen=None) if sparse else out


def _exact_attention(q, k, v):
    x = torch.einsum("hgd,hnd->hgn", q, k) / math.sqrt(q.shape[-1])
    w = torch.exp(x - x.max(-1, keepdim=True).values)
    return torch.einsum("hgn,hnd->hgd", w, v) / w.sum(-1, keepdim=True)


def _exact_scores(q, steps, bounds):
    """[H_kv, pages]: the largest of the heads' upper bounds, on the host in 64 bits."""
    x = q.cpu().numpy() * np.exp2(steps.cpu().numpy().astype(np.float64))[:, None]
    top = np.abs(x).max(-1, keepdims=True)
    e = np.frexp(top)[1] - 7
    code = np.clip(np.rint(x * np.exp2(-e.astype(np.float64))), -127, 127)
    b = bounds.cpu().numpy().astype(np.float64)                     # [pages, H_kv, 2, d]
    up = np.einsum("hgd,phd->hgp", np.maximum(code, 0), b[:, :, 1]) + np.einsum("hgd,phd->hgp", np.minimum(code, 0), b[:, :, 0])
    return (up * np.exp2(e.astype(np.float64))).max(1)
