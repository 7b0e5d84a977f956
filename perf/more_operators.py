"""What a prompt chunk needs before and around its paged cache, as cases to measure: the norm and rotation of
queries and keys, and the attention of new tokens over the cache that already holds them.

A case names one operator and its sizes. ``run`` makes one pass: with ``own`` false in elementary torch
operations, with ``own`` true through the library's calls. Pools are BF16 pages of 16 tokens,
[pages][H_kv][K, V][16][d]. Lengths are a function of the case alone (log-spaced between two bounds, the longest
caches with the fewest new tokens); the order of the requests, the page ids and all values come from the seed.
"""

import math

import torch

own = False

_DEV = torch.device("cuda")
_P = 16                      # tokens per page
_EPS = 1e-6
_BASE = 1000000.0            # rotation base
_TRAINED = 32768             # positions that the unscaled rotation was trained on


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # one token of one request, normed and rotated (latency)
        dict(name="rope_step_b1", op="rope", batch=1, cached_lo=100000, cached_hi=100000, new_lo=1, new_hi=1, h_q=32,
             h_kv=8, d=128, rot=128, layout="half", norm=True, factor=1.0, given=False, spare=0),
        # a decode step of 256 running requests, their positions from the plan's lengths
        dict(name="rope_step_b256", op="rope", batch=256, cached_lo=77, cached_hi=32768, new_lo=1, new_hi=1, h_q=32,
             h_kv=8, d=128, rot=128, layout="half", norm=True, factor=1.0, given=False, spare=0),
        # ragged prompts of a model that rotates half of each head, pairs side by side, scaled past its trained
        # positions and without norms; positions given by the caller
        dict(name="rope_far_partial", op="rope", batch=5, cached_lo=300, cached_hi=1000000, new_lo=301, new_hi=2203,
             h_q=64, h_kv=8, d=64, rot=32, layout="interleaved", norm=False, factor=32.0, given=True, spare=0),
        # a bulk prefill: 131,072 tokens, the size of the bulk cache write
        dict(name="rope_prefill_131k", op="rope", batch=8, cached_lo=0, cached_hi=0, new_lo=16384, new_hi=16384,
             h_q=32, h_kv=8, d=128, rot=128, layout="half", norm=True, factor=1.0, given=False, spare=0),
        # the smallest chunk: five tokens in the tiny configuration (latency)
        dict(name="chunk_tiny", op="chunk", batch=1, cached_lo=1339, cached_hi=1339, new_lo=5, new_hi=5, h_q=4,
             h_kv=2, d=64, spare=0),
        # one user at 100,000 tokens checks eight drafted tokens
        dict(name="chunk_draft_bs1_100k", op="chunk", batch=1, cached_lo=99992, cached_hi=99992, new_lo=8, new_hi=8,
             h_q=32, h_kv=8, d=128, spare=0),
        # a serving batch checks one to eight drafted tokens a request
        dict(name="chunk_draft_b32", op="chunk", batch=32, cached_lo=4096, cached_hi=32768, new_lo=1, new_hi=8,
             h_q=32, h_kv=8, d=128, spare=0),
        # short ragged prompts of a model with 64 channels a head and no shared heads
        dict(name="chunk_prompts_d64", op="chunk", batch=7, cached_lo=0, cached_hi=900, new_lo=333, new_hi=1501, h_q=8,
             h_kv=8, d=64, spare=3),
        # one prompt from an empty cache
        dict(name="chunk_prompt_8k", op="chunk", batch=1, cached_lo=0, cached_hi=0, new_lo=8192, new_hi=8192, h_q=32,
             h_kv=8, d=128, spare=0),
        # prefills of any length next to running requests, in one call
        dict(name="chunk_mixed16", op="chunk", batch=16, cached_lo=0, cached_hi=32768, new_lo=1, new_hi=4096, h_q=32,
             h_kv=8, d=128, spare=0),
        # the next 2,048 tokens of a long prompt that is taken in chunks
        dict(name="chunk_long_prompt", op="chunk", batch=1, cached_lo=97952, cached_hi=97952, new_lo=2048, new_hi=2048,
             h_q=64, h_kv=8, d=128, spare=0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    h_kv, d, g = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    if rng.random() < 0.4:
        batch = log(1, 256)
        new_hi = log(1, min(16384, max(1, 131072 // batch)))
        return dict(op="rope", batch=batch, cached_lo=rng.choice([0, log(1, 300)]), cached_hi=log(301, 1000000),
                    new_lo=rng.randint(0, 1), new_hi=new_hi, h_q=g * h_kv, h_kv=h_kv, d=d,
                    rot=rng.choice([d, d, d // 2, d // 4, 24]), layout=rng.choice(["half", "interleaved"]),
                    norm=rng.random() < 0.6, factor=rng.choice([1.0, 1.0, 4.0, 32.0]), given=rng.random() < 0.5,
                    spare=rng.choice([0, 5]))
    while True:
        batch = log(1, 48)
        cached_hi = log(1, 131072)
        case = dict(op="chunk", batch=batch, cached_lo=min(cached_hi, rng.choice([0, log(1, 4096)])),
                    cached_hi=cached_hi, new_lo=rng.randint(0, 1), new_hi=log(1, rng.choice([8, 300, 8192])),
                    h_q=g * h_kv, h_kv=h_kv, d=d, spare=rng.choice([0, 5]))
        w = work(case)
        if w["flops"] < 4e12 and w["bytes"] < 8e9:
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


def _lengths(case):
    """(cached, new) of each request: the longest caches with the fewest new tokens."""
    return list(zip(_spread(case["cached_lo"], case["cached_hi"], case["batch"])[::-1],
                    _spread(case["new_lo"], case["new_hi"], case["batch"])))


def work(case):
    pairs = _lengths(case)
    new = sum(n for _, n in pairs)
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    if case["op"] == "rope":
        # queries and keys in and out, positions; a multiply-add for the norm, two products and a sum a channel
        return dict(bytes=new * (h_q + h_kv) * d * 4 + (4 * new if case["given"] else 8 * case["batch"]),
                    flops=new * (h_q + h_kv) * ((4 * d if case["norm"] else 0) + 3 * case["rot"]))
    seen = sum(n * c + n * (n + 1) // 2 for c, n in pairs)          # (new token, token it sees) pairs
    total = sum(c + n for c, n in pairs if n)
    return dict(bytes=total * h_kv * d * 4 + total // _P * 4 + new * h_q * d * 4, flops=4 * seen * h_q * d)


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------

def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=_DEV, dtype=dtype)


def _frequencies(case):
    """Radians a position of each pair, and the factor on the rotated channels: beyond a factor of 1 the slow pairs
    turn slower by it, the fast ones as trained, with a ramp between them."""
    rot, factor = case["rot"], case["factor"]
    freq = [_BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    if factor == 1.0:
        return freq, 1.0

    def pair_of(turns):               # the pair that makes this many turns over the trained positions
        return rot * math.log(_TRAINED / (turns * 2 * math.pi)) / (2 * math.log(_BASE))

    low, high = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rot - 1)
    for i in range(rot // 2):
        slow = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
        freq[i] = freq[i] / factor * slow + freq[i] * (1.0 - slow)
    return freq, 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    gen = torch.Generator(device=_DEV)
    gen.manual_seed(int(seed))
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    pairs = _lengths(case)
    order = torch.randperm(len(pairs), generator=gen, device=_DEV).tolist()
    pairs = [pairs[i] for i in order]
    cached, new = (torch.tensor(x, dtype=torch.int32, device=_DEV) for x in zip(*pairs))
    n = sum(x for _, x in pairs)
    # what a plan of the step leaves on the GPU, and the lengths that the program knows itself
    s = dict(case=case, pairs=pairs, total_len=cached + new,
             row_start=torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0)).to(torch.int32))
    rows = n + case["spare"]
    if case["op"] == "rope":
        # queries, keys and values as a projection leaves them: slices of one row
        qkv = _randn(gen, max(rows, 1), h_q + 2 * h_kv, d, dtype=torch.bfloat16)[:rows]
        qkv *= torch.exp(0.5 * _randn(gen, h_q + 2 * h_kv, 1)).to(torch.bfloat16)
        s.update(q=qkv[:, :h_q], k=qkv[:, h_q:h_q + h_kv], positions=None, q_weight=None, k_weight=None,
                 q_out=torch.zeros(rows, h_q, d, dtype=torch.bfloat16, device=_DEV),
                 k_out=torch.zeros(rows, h_kv, d, dtype=torch.bfloat16, device=_DEV))
        s["freq"], s["scale"] = _frequencies(case)
        if case["norm"]:
            s["q_weight"], s["k_weight"] = 1 + 0.2 * _randn(gen, d), 1 + 0.2 * _randn(gen, d)
        if case["given"]:
            s["positions"] = torch.cat([torch.arange(c, c + m) for c, m in pairs] +
                                       [torch.zeros(case["spare"], dtype=torch.int64)]).to(torch.int32).to(_DEV)
        if own:      # the table and the context that a serving loop keeps
            from bit_kv_cache_write_gb300 import oscar, rope
            scaling = None if case["factor"] == 1.0 else dict(kind="yarn", factor=case["factor"], trained=_TRAINED)
            turns, s["scale"] = rope.rope_turns(case["rot"], _BASE, scaling)
            s["turns"] = torch.from_numpy(turns).to(_DEV)
            s["layout"] = dict(half=oscar.OSCAR_ROPE_HALF, interleaved=oscar.OSCAR_ROPE_INTERLEAVED)[case["layout"]]
            s["ctx"] = _context(h_q, h_kv, d)
        return s
    count = (s["total_len"].long() + _P - 1) // _P
    used, stride = int(count.sum()), max(1, int(count.max()))
    ids = torch.randperm(used + 3, generator=gen, device=_DEV).to(torch.int32)
    col = torch.arange(stride, device=_DEV)
    at = (torch.cumsum(count, 0) - count)[:, None] + col[None]
    s["tables"] = torch.where(col[None] < count[:, None], ids[at.clamp(max=used + 2)], 0).to(torch.int32).contiguous()
    # keys per channel as real ones are, log-normal with a few outlier channels
    scale = torch.exp(0.4 * _randn(gen, h_kv, d))
    scale[:, torch.randperm(d, generator=gen, device=_DEV)[: max(1, d // 50)]] *= 4.0
    s["pool"] = pool = torch.empty(used + 3, h_kv, 2, _P, d, dtype=torch.bfloat16, device=_DEV)
    step = max(1, (1 << 27) // (h_kv * 2 * _P * d))
    for p in range(0, used + 3, step):
        pool[p:p + step] = _randn(gen, min(step, used + 3 - p), h_kv, 2, _P, d, dtype=torch.bfloat16)
        pool[p:p + step, :, 0] *= scale[None, :, None].to(torch.bfloat16)
    s["q"] = _randn(gen, max(rows, 1), h_q, d).to(torch.bfloat16)[:rows]
    s["out"] = torch.zeros(rows, h_q, d, dtype=torch.bfloat16, device=_DEV)
    if own:          # the context and workspace that a serving loop keeps
        s["ctx"] = _context(h_q, h_kv, d)
        s["ws"] = torch.empty(s["ctx"].extend_bf16_workspace_size(case["batch"], rows), dtype=torch.uint8, device=_DEV)
    return s


def _context(h_q, h_kv, d):
    from bit_kv_cache_write_gb300 import oscar
    return oscar.Oscar(n_layers=1, n_q_heads=h_q, n_kv_heads=h_kv, head_dim=d, group=64)


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------

def run(s):
    if s["case"]["op"] == "rope":
        if own:
            s["ctx"].norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["turns"], positions=s["positions"],
                               row_start=s["row_start"], total_len=s["total_len"], q_weight=s["q_weight"],
                               k_weight=s["k_weight"], eps=_EPS, layout=s["layout"], scale=s["scale"])
            return s["q_out"], s["k_out"]
        return _rope(s)
    if own:
        s["ctx"].extend_bf16(s["q"], s["pool"], s["tables"], s["row_start"], s["total_len"], s["out"], s["ws"])
        return s["out"]
    return _chunk(s)


def _rope(s):
    """Each head's RMS norm, then the rotation of its first channels; rows behind the last request stay."""
    case, rot, rows = s["case"], s["case"]["rot"], s["q"].shape[0]
    start, total = s["row_start"].long(), s["total_len"].long()
    t = torch.arange(rows, device=_DEV)
    request = torch.searchsorted(start[1:].contiguous(), t, right=True)
    at = request.clamp(max=case["batch"] - 1)
    # a caller's positions cover every row, the plan's lengths the requests' rows only
    inside = torch.ones_like(t, dtype=torch.bool) if case["given"] else request < case["batch"]
    pos = s["positions"].long() if case["given"] else total[at] - start[at + 1] + t
    angle = pos.double()[:, None] * torch.tensor(s["freq"], dtype=torch.float64, device=_DEV)
    cos, sin = ((f(angle) * s["scale"]).float()[:, None] for f in (torch.cos, torch.sin))
    outs = []
    for x, weight, out in ((s["q"], s["q_weight"], s["q_out"]), (s["k"], s["k_weight"], s["k_out"])):
        y = x.float()
        if weight is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS) * weight
        if case["layout"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = [a * cos - b * sin, b * cos + a * sin]
        if case["layout"] == "half":
            turned = torch.cat(turned, -1)
        else:
            turned = torch.stack(turned, -1).flatten(-2)
        y = torch.cat([turned, y[..., rot:]], -1).to(out.dtype)
        outs.append(torch.where(inside[:, None, None], y, out))
    return tuple(outs)


def _chunk(s):
    """Each new token's attention over the tokens up to and with its own."""
    q, pool, out = s["q"], s["pool"], s["out"].clone()
    h_kv, d = pool.shape[1], pool.shape[4]
    g = q.shape[1] // h_kv
    row = 0
    for b, (cached, new) in enumerate(s["pairs"]):
        if new == 0:
            continue
        total = cached + new
        ids = s["tables"][b, :(total + _P - 1) // _P].long()
        step = max(1, (1 << 29) // (total * g))
        for h in range(h_kv):
            kv = pool[ids, h].float()
            k, v = (kv[:, i].reshape(-1, d)[:total] for i in (0, 1))
            for i in range(0, new, step):
                m = min(step, new - i)
                part = slice(row + i, row + i + m), slice(h * g, (h + 1) * g)
                x = (q[part].float().reshape(m * g, d) @ k.T) * d ** -0.5
                if cached + i + 1 < total:
                    seen = cached + i + torch.arange(m, device=_DEV).repeat_interleave(g)
                    x.masked_fill_(torch.arange(total, device=_DEV)[None] > seen[:, None], -math.inf)
                x = torch.exp(x - x.amax(-1, keepdim=True))
                out[part] = ((x @ v) / x.sum(-1, keepdim=True)).reshape(m, g, d).to(out.dtype)
        row += new
    return out


# ---------------------------------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    return _exact_chunk(s)


def _exact_rope(s):
    """Request by request, each pair of channels as a complex number."""
    case, rot = s["case"], s["case"]["rot"]
    freq, scale = _frequencies(case)
    freq = torch.tensor(freq, dtype=torch.float64, device=_DEV)
    outs = [s["q_out"].double(), s["k_out"].double()]
    row = 0
    for cached, new in s["pairs"] + ([(None, case["spare"])] if case["given"] and case["spare"] else []):
        if new == 0:
            continue
        pos = torch.arange(cached, cached + new, dtype=torch.float64, device=_DEV) if cached is not None else \
            torch.zeros(new, dtype=torch.float64, device=_DEV)
        phase = torch.polar(torch.full((), scale, dtype=torch.float64, device=_DEV), torch.outer(pos, freq))[:, None]
        for x, weight, out in zip((s["q"], s["k"]), (s["q_weight"], s["k_weight"]), outs):
            y = x[row:row + new].double()
            if case["norm"]:
                y = weight.double() * (y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["d"] + _EPS))
            got = out[row:row + new]
            got[..., rot:] = y[..., rot:]
            first = torch.arange(rot // 2, device=_DEV) * (1 if case["layout"] == "half" else 2)
            second = first + (rot // 2 if case["layout"] == "half" else 1)
            z = torch.complex(y[..., first], y[..., second]) * phase
            got[..., first], got[..., second] = z.real, z.imag
        row += new
    return tuple(outs)


def _exact_chunk(s):
    """Query head by query head, over rows of the cache gathered token by token."""
    q, pool, out = s["q"], s["pool"], s["out"].double()
    h_q, d = q.shape[1:]
    g = h_q // pool.shape[1]
    start = s["row_start"].tolist()
    for b, (cached, new) in enumerate(s["pairs"]):
        if new == 0:
            continue
        token = torch.arange(cached + new, device=_DEV)
        page, line = s["tables"][b].long()[token // _P], token % _P
        last = torch.arange(cached, cached + new, device=_DEV)
        step = max(1, (1 << 28) // (cached + new))
        for h in range(h_q):
            if h % g == 0:
                k, v = (pool[page, h // g, i, line].double() for i in (0, 1))
            for i in range(0, new, step):
                at = slice(i, min(new, i + step))
                x = torch.einsum("id,td->it", q[start[b] + i:start[b] + min(new, i + step), h].double(), k) / math.sqrt(d)
                x = x.masked_fill(token[None] > last[at, None], -math.inf)
                out[start[b] + i:start[b] + min(new, i + step), h] = torch.softmax(x, -1) @ v
    return out
