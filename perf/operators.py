"""The operators of a serving step around the weight stream, as cases that can be measured: block tables and slots
(plan), query/key norms with rotation and the 8-bit cache write (append), attention over the 8-bit cache (attend) and
the verification of drafted tokens (verify). `own` false computes them with elementary torch operations; true calls
this package."""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # one request, a verify pass of eight rows: the smallest call
        dict(name="plan-1x8", op="plan", requests=1, seq=4093, new=8, block=16),
        # prompts admitted beside running requests: lengths from zero to thousands
        dict(name="plan-384-mixed", op="plan", requests=384, seq=6001, new=2048, block=64),
        # one decoded token of the 27B-shape layer (24 query heads, 4 kv heads of 256, a quarter rotated)
        dict(name="append-1x1-d256", op="append", requests=1, new=1, q_heads=24, kv_heads=4, dim=256, rot=64,
             block=64, seq=1000, interleaved=False, far=0),
        # a verify batch: 48 requests of 1 to 5 rows that start inside a block, far positions
        dict(name="append-48x5-d128", op="append", requests=48, new=5, q_heads=32, kv_heads=8, dim=128, rot=128,
             block=16, seq=77, interleaved=False, far=900001),
        # a prompt chunk written at once: whole blocks and ragged ends, adjacent pairs rotated
        dict(name="append-chunk-d64", op="append", requests=7, new=1999, q_heads=16, kv_heads=16, dim=64, rot=32,
             block=32, seq=45, interleaved=True, far=0),
        # batch 1, one row, short context: latency
        dict(name="attend-1x1-777-d256", op="attend", requests=1, rows=1, q_heads=24, kv_heads=4, dim=256, block=64,
             kv=777, ragged=False),
        # batch 1, one row, a long context
        dict(name="attend-1x1-131071-d256", op="attend", requests=1, rows=1, q_heads=24, kv_heads=4, dim=256,
             block=64, kv=131071, ragged=False),
        # batch 1, the eight rows of a verify pass over a long context
        dict(name="attend-1x8-100001-d256", op="attend", requests=1, rows=8, q_heads=24, kv_heads=4, dim=256,
             block=64, kv=100001, ragged=False),
        # a decode batch with lengths from one to the longest, small blocks
        dict(name="attend-80x1-ragged-d128", op="attend", requests=80, rows=1, q_heads=32, kv_heads=8, dim=128,
             block=16, kv=9001, ragged=True),
        # a verify batch of 1 to 5 rows with a kv head for every query head
        dict(name="attend-24x5-ragged-d64", op="attend", requests=24, rows=5, q_heads=16, kv_heads=16, dim=64,
             block=32, kv=5003, ragged=True),
        # one request, seven drafts, the 27B-shape vocabulary
        dict(name="verify-1x8-248320", op="verify", requests=1, rows=8, vocab=248320, draft=True),
        # a batch, up to four drafts each, the other vocabulary
        dict(name="verify-64x5-157184", op="verify", requests=64, rows=5, vocab=157184, draft=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "append", "attend", "attend", "attend", "attend", "verify"])
    block = rng.choice([16, 32, 64, 128])
    q, kv, dim = rng.choice([(24, 4, 256), (32, 8, 128), (16, 16, 64), (40, 8, 128), (16, 2, 256), (16, 1, 128), (7, 7, 128)])
    if op == "plan":
        return dict(op="plan", requests=_log(rng, 1, 384), seq=_log(rng, 1, 6000), new=_log(rng, 1, 2047), block=block)
    if op == "append":
        requests = _log(rng, 1, 64)
        rot = dim if rng.random() < 0.6 else dim // 2
        most = max(2, 13000 * 1024 // (q * dim + 2 * kv * dim) // requests)
        return dict(op="append", requests=requests, new=_log(rng, 1, min(2000, most)), q_heads=q,
                    kv_heads=kv, dim=dim, rot=rot, block=block, seq=_log(rng, 1, 200),
                    interleaved=rng.random() < 0.3, far=rng.choice([0, _log(rng, 1000, 1000000)]))
    if op == "attend":
        requests, rows = _log(rng, 1, 96), rng.choice([1, 1, 2, 3, 5, 8])
        # the cache's bytes and the products stay below the largest listed cases'
        most = min(2.6e8 / (2 * kv * dim), 1.9e10 / (4 * q * dim * rows)) / requests
        return dict(op="attend", requests=requests, rows=rows, q_heads=q, kv_heads=kv, dim=dim, block=block,
                    kv=_log(rng, 16, max(17, min(131071, int(most)))), ragged=requests > 1 or rng.random() < 0.3)
    return dict(op="verify", requests=_log(rng, 1, 64), rows=rng.randint(1, 8) if rng.random() < 0.3 else rng.randint(2, 5),
                vocab=_log(rng, 1001, 150001), draft=rng.random() < 0.7)


def work(case):
    c = case
    if c["op"] == "plan":
        seq, new = _plan_lens(c)
        blocks = sum(-(-(s + n) // c["block"]) - -(-s // c["block"]) for s, n in zip(seq, new))
        return {"bytes": 8 * sum(new) + 8 * blocks + 16 * c["requests"], "flops": 4 * sum(new)}
    if c["op"] == "append":
        rows, q, kv = sum(_lens(c["requests"], c["new"])), c["q_heads"] * c["dim"], c["kv_heads"] * c["dim"]
        return {"bytes": rows * (4 * q + 6 * kv), "flops": rows * 8 * (q + kv)}
    if c["op"] == "attend":
        keys, heads = _kv_lens(c), c["kv_heads"] * c["dim"]
        rows = _lens(c["requests"], c["rows"])
        flops = sum(4 * c["q_heads"] * c["dim"] * k * n for k, n in zip(keys, rows))
        return {"bytes": 2 * heads * sum(keys) + 8 * c["kv_heads"] * sum(-(-k // c["block"]) for k in keys)
                + 4 * c["q_heads"] * c["dim"] * sum(rows), "flops": flops}
    # one target row a request, and a draft row for the requests that stop at a refused draft (about seven in ten)
    return {"bytes": c["requests"] * c["vocab"] * 4 * (1.7 if c["draft"] and c["rows"] > 1 else 1), "flops": 2 * c["requests"] * c["vocab"]}


def _lens(requests, longest):
    """Row counts of the requests: the longest first, then a fixed ragged pattern from one up."""
    return [longest if r == 0 else 1 + (r * 7919) % longest for r in range(requests)]


def _kv_lens(c):
    rows = _lens(c["requests"], c["rows"])
    if not c["ragged"]:
        return [max(n, c["kv"]) for n in rows]
    return [max(n, c["kv"] if r == 0 else 1 + (r * 104729 + 17) % c["kv"]) for r, n in enumerate(rows)]


def _plan_lens(c):
    r = range(c["requests"])
    new = [c["new"] if i == 0 else 1 + (i * 7919) % c["new"] for i in r]
    seq = [c["seq"] if i == 0 else (0 if i % 3 == 1 else (i * 104729) % c["seq"]) for i in r]
    return seq, new


# ---- inputs -------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(lens):
    t = [0]
    for n in lens:
        t.append(t[-1] + n)
    return _ints(t)


def _rows_of(held, pool, wide):
    """Table rows [len(held), wide]: the first held[r] entries of row r from `pool` in order, -1 after them."""
    t = torch.tensor(held, device="cuda")
    col = torch.arange(wide, device="cuda")[None, :]
    at = col + (torch.cumsum(t, 0) - t)[:, None]
    return torch.where(col < t[:, None], pool[at.clamp(max=pool.numel() - 1)], -1).contiguous()


def _tables(kv_lens, block, g):
    """Block tables over a shuffled pool, and the pool's size."""
    need = [-(-k // block) for k in kv_lens]
    pool = torch.randperm(sum(need) + 3, generator=g, device="cuda").to(torch.int32)
    return _rows_of(need, pool, max(max(need), 1)), pool.numel()


def _filled(n_blocks, heads, block, dim, g, spread):
    """Codes and scales of a filled side of the cache; `spread`: how unlike the blocks' magnitudes are, in octaves."""
    codes = torch.empty((n_blocks, heads, block, dim), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n_blocks, heads), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (heads * block * dim))
    for a in range(0, n_blocks, step):
        n = min(step, n_blocks - a)
        x = torch.randn((n, heads, block, dim), generator=g, device="cuda")
        x *= torch.exp2(spread * torch.randn((n, heads, 1, 1), generator=g, device="cuda"))
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / E4M3_MAX)))
        codes[a:a + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[a:a + n] = s
    return codes, scale


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    if c["op"] == "plan":
        seq, new = _plan_lens(c)
        held = [-(-s // c["block"]) for s in seq]
        total = sum(-(-(s + n) // c["block"]) for s, n in zip(seq, new)) + 5
        pool = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        used = sum(held)
        c.update(seq_lens=_ints(seq), new_lens=_ints(new), table=_rows_of(held, pool, -(-(c["seq"] + c["new"]) // c["block"])),
                 free=pool[used:].contiguous(), n_free=_ints([total - used]), n_rows=sum(new) + 3)
        return c
    if c["op"] == "append":
        lens, D, B = _lens(c["requests"], c["new"]), c["dim"], c["block"]
        seqs = [c["seq"] if r == 0 else (r * 31) % (c["seq"] + 1) for r in range(len(lens))]
        table, n_blocks = _tables([s + n for s, n in zip(seqs, lens)], B, g)
        pos = torch.cat([torch.arange(s, s + n) for s, n in zip(seqs, lens)]).cuda()
        req = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()
        slots = (table[req, pos // B] * B + (pos % B).to(torch.int32)).to(torch.int32)
        T, H, K = sum(lens), c["q_heads"], c["kv_heads"]
        # one projection's output, as the layer makes it: query, key and value heads of a row side by side
        qkv = (2.5 * torch.randn((T, H + 2 * K, D), generator=g, device="cuda")).to(torch.bfloat16)
        k, ks = _filled(n_blocks, K, B, D, g, 0.0)
        v, vs = _filled(n_blocks, K, B, D, g, 0.0)
        c.update(q=qkv[:, :H], k=qkv[:, H:H + K], v=qkv[:, H + K:], positions=(pos + c["far"]).to(torch.int32), slots=slots,
                 qw=1 + 0.2 * torch.randn(D, generator=g, device="cuda"), kw=1 + 0.2 * torch.randn(D, generator=g, device="cuda"),
                 inv_freq=(1e6 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])).float(),
                 cache_k=k, cache_v=v, k_scale=ks, v_scale=vs)
        c["cache"] = _handle(c)
        return c
    if c["op"] == "attend":
        rows, kv = _lens(c["requests"], c["rows"]), _kv_lens(c)
        table, n_blocks = _tables(kv, c["block"], g)
        k, ks = _filled(n_blocks, c["kv_heads"], c["block"], c["dim"], g, 0.3)
        v, vs = _filled(n_blocks, c["kv_heads"], c["block"], c["dim"], g, 1.0)
        q = (1.5 * torch.randn((sum(rows), c["q_heads"], c["dim"]), generator=g, device="cuda")).to(torch.bfloat16)
        c.update(q=q, table=table, row_start=_starts(rows), kv_lens=_ints(kv), cache_k=k, cache_v=v, k_scale=ks, v_scale=vs)
        c["cache"] = _handle(c)
        return c
    rows, V = _lens(c["requests"], c["rows"]), c["vocab"]
    T = sum(rows)
    logits = 2.5 * torch.randn((T, V), generator=g, device="cuda")
    q = torch.softmax(logits + 0.8 * torch.randn((T, V), generator=g, device="cuda"), -1)
    cum = torch.cumsum(q, -1, dtype=torch.float64)
    u = torch.rand((T, 1), generator=g, device="cuda", dtype=torch.float64) * cum[:, -1:]
    tokens = torch.searchsorted(cum, u, right=True)[:, 0].clamp(max=V - 1).to(torch.int32)
    c.update(p=torch.softmax(logits, -1), q_draft=q if c["draft"] else None, tokens=tokens, row_start=_starts(rows),
             accept_u=torch.rand(T, generator=g, device="cuda"), sample_u=torch.rand(c["requests"], generator=g, device="cuda"))
    return c


def _handle(c):
    """The cache's handle, where the package has one."""
    if not own:
        return None
    import bit_weight_streaming_gb300 as bws
    return bws.KvCache(c["cache_k"], c["cache_v"], c["k_scale"], c["v_scale"]), bws.Workspace()


# ---- one pass -----------------------------------------------------------------

def run(state):
    s = state
    if own:
        import bit_weight_streaming_gb300 as bws
        if s["op"] == "plan":
            p = bws.kv_plan(s["seq_lens"], s["new_lens"], s["block"], s["table"], s["free"], s["n_free"], s["n_rows"])
            return [s["table"], p.slots, p.positions, p.row_start, p.kv_lens, p.n_free]
        if s["op"] == "append":
            q = bws.qk_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cache"][0], s["inv_freq"],
                                        s["qw"], s["kw"], eps=1e-6, interleaved=s["interleaved"])
            return [q] + _held(s)
        if s["op"] == "attend":
            out, lse = bws.kv_attention(s["q"], s["cache"][0], s["table"], s["row_start"], s["kv_lens"], s["rows"],
                                        lse=True, ws=s["cache"][1])
            return [out, lse]
        tokens, n = bws.draft_verify(s["p"], s["tokens"], s["row_start"], s["accept_u"], s["sample_u"], s["rows"],
                                     draft=s["q_draft"])
        return [tokens, n]
    return {"plan": _plan, "append": _append, "attend": _attend, "verify": _verify}[s["op"]](s)


def _held(s):
    """The cache as it stands: the 8-bit values and the scales of the blocks."""
    return [s["cache_k"].view(torch.float8_e4m3fn), s["cache_v"].view(torch.float8_e4m3fn), s["k_scale"], s["v_scale"]]


def _plan(s):
    B, seq, new, table = s["block"], s["seq_lens"].long(), s["new_lens"].long(), s["table"]
    have, need = (seq + B - 1) // B, (seq + new + B - 1) // B
    more = need - have
    first = torch.cumsum(more, 0) - more
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    at = s["n_free"].long() - 1 - (first[:, None] + col - have[:, None])
    got = torch.where(at >= 0, s["free"][at.clamp(0, s["free"].numel() - 1)], -1)
    table.copy_(torch.where((col >= have[:, None]) & (col < need[:, None]), got, table))
    start = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    row = torch.arange(s["n_rows"], device="cuda")
    r = torch.searchsorted(start[1:].contiguous(), row, right=True).clamp(max=seq.numel() - 1)
    pos = seq[r] + row - start[r]
    block = table[r, (pos // B).clamp(max=table.shape[1] - 1)].long()
    live = row < start[-1]
    slots = torch.where(live & (block >= 0), block * B + pos % B, -1)
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return [table, i32(slots), i32(torch.where(live, pos, -1)), i32(start), i32(seq + new),
            i32((s["n_free"].long() - more.sum()).clamp(min=0))]


def _rotated(x, w, cos, sin, rot, interleaved, eps=1e-6):
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _append(s):
    # the angles in 64 bits: a far position times a frequency loses its turn in 32
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotated(s["q"].float(), s["qw"], cos, sin, s["rot"], s["interleaved"])
    k = _rotated(s["k"].float(), s["kw"], cos, sin, s["rot"], s["interleaved"])
    _store(s["cache_k"], s["k_scale"], k, s["slots"].long())
    _store(s["cache_v"], s["v_scale"], s["v"].float(), s["slots"].long())
    return [q.to(torch.bfloat16)] + _held(s)


def _store(codes, scale, x, slots):
    """Writes rows x [T, heads, dim] at `slots`: a block's scale grows to what its new rows need, its older codes are
    rounded again under a grown scale, and a block that is entered at its first slot starts anew."""
    n_blocks, heads, B, dim = codes.shape
    block, at = slots // B, slots % B
    amax = torch.zeros((n_blocks, heads), device="cuda").index_reduce_(0, block, x.abs().amax(-1), "amax")
    first = torch.full((n_blocks,), B, device="cuda").index_reduce_(0, block, at, "amin")
    need = torch.exp2(_exponent(amax).to(amax.dtype))
    new = torch.where((first > 0)[:, None], torch.maximum(scale, need), need)
    new = torch.where((first < B)[:, None], new, scale)
    ids = torch.unique(block)
    old = codes[ids].view(torch.float8_e4m3fn).float() * (scale[ids] / new[ids])[:, :, None, None]
    keep = torch.arange(B, device="cuda")[None, :] < first[ids][:, None]
    again = old.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[ids] = torch.where(keep[:, None, :, None], again, codes[ids])
    scale.copy_(new)
    codes[block, :, at] = (x / new[block][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _exponent(amax):
    """e of the smallest 2^e with amax <= 448 * 2^e, 448 = 0.875 * 2^9; in whole numbers, since a quotient would round."""
    m, x = torch.frexp(amax)
    return torch.where(amax == 0, -60, x - 9 + (m > 0.875)).clamp(-60, 60)


def _attend(s):
    """All requests at once, padded to the widest table row and the most query rows."""
    R, n, D, B, K = s["requests"], s["rows"], s["dim"], s["block"], s["kv_heads"]
    G = s["q_heads"] // K
    start, kv = s["row_start"].long(), s["kv_lens"].long()
    lens = start[1:] - start[:-1]
    j = torch.arange(n, device="cuda")
    q = s["q"][(start[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)].float()                     # [R, n, H, D]
    q = q.view(R, n, K, G, D).permute(0, 2, 1, 3, 4).reshape(R, K, n * G, D)
    last = (kv - lens)[:, None] + j                                                                # [R, n]
    ids = s["table"].long().clamp(min=0)

    def side(codes, scale):
        x = codes.view(torch.float8_e4m3fn)[ids].float() * scale[ids][..., None, None]             # [R, W, K, B, D]
        return x.permute(0, 2, 1, 3, 4).reshape(R, K, -1, D)

    z = (q @ side(s["cache_k"], s["k_scale"]).transpose(-1, -2)) * D ** -0.5
    pos = torch.arange(ids.shape[1] * B, device="cuda")
    hide = (pos > last[:, :, None])[:, None, :, None, :]
    z = z.view(R, K, n, G, -1).masked_fill(hide, -math.inf).view(R, K, n * G, -1)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    o = torch.where(total > 0, (e @ side(s["cache_v"], s["v_scale"])) / total, torch.zeros_like(total))
    row = torch.arange(s["q"].shape[0], device="cuda")
    r = torch.searchsorted(start[1:].contiguous(), row, right=True)
    at = r * n + row - start[r]

    def back(t):
        return t.view(R, K, n, G, -1).permute(0, 2, 1, 3, 4).reshape(R * n, K * G, -1)[at]

    return [back(o).to(torch.bfloat16), back(top + torch.log(total))[..., 0]]


def _verify(s):
    p, q, V, n = s["p"], s["q_draft"], s["vocab"], s["rows"]
    start = s["row_start"].long()
    drafts = start[1:] - start[:-1] - 1
    row = torch.arange(p.shape[0], device="cuda")
    x = s["tokens"].long()
    px = p[row, x].double()
    qx = q[row, x].double() if q is not None else torch.ones_like(px)
    ok = s["accept_u"].double() * qx < px
    j = torch.arange(n, device="cuda")
    at = (start[:-1, None] + j).clamp(max=p.shape[0] - 1)                       # [R, n]
    a = torch.cumprod((ok[at] & (j < drafts[:, None])).long(), 1).sum(1)
    here = start[:-1] + a
    base = p[here]
    # what is left of the target where the draft was refused, in the inputs' own 32 bits; summed in 64
    left = (base - q[here]).clamp(min=0) if q is not None else base.scatter(1, x[here][:, None], 0.0)
    left = torch.where(left.double().sum(1, keepdim=True) > 0, left, base)
    w = torch.where((a < drafts)[:, None], left, base)
    cum = torch.cumsum(w.double(), 1)
    tok = torch.searchsorted(cum, s["sample_u"].double()[:, None] * cum[:, -1:], right=True)[:, 0]
    last = V - 1 - torch.argmax((w > 0).to(torch.int32).flip(1), 1)
    tok = torch.minimum(tok, last)
    out = torch.where(j < a[:, None], x[at], torch.where(j == a[:, None], tok[:, None], -1))
    return [out.to(torch.int32), (a + 1).to(torch.int32)]


# ---- 64 bits ------------------------------------------------------------------

def exact(case, seed):
    """The outputs that are computed numbers, in 64 bits and from the definitions: request by request."""
    if case["op"] in ("plan", "verify"):
        return None      # whole numbers
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_append(s):
    turn = torch.outer(s["positions"].double(), s["inv_freq"].double())
    half, B = s["rot"] // 2, s["block"]
    dims = torch.arange(half, device="cuda")
    lo, hi = (2 * dims, 2 * dims + 1) if s["interleaved"] else (dims, dims + half)
    slots = s["slots"].long()
    blocks = torch.unique(slots // B).tolist()

    def heads(x, w):
        y = x.double()
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / s["dim"] + 1e-6) * w.double()
        z = y.clone()
        c, d = turn.cos()[:, None, :], turn.sin()[:, None, :]
        z[..., lo] = y[..., lo] * c - y[..., hi] * d
        z[..., hi] = y[..., hi] * c + y[..., lo] * d
        return z

    def held(codes, scale, x):
        codes, scale = codes.view(torch.float8_e4m3fn).double(), scale.double()
        for blk in blocks:
            rows = ((slots // B) == blk).nonzero()[:, 0]
            at = slots[rows] % B
            o = int(at.min())
            top = x[rows].abs().amax((0, 2))
            e = torch.ceil(torch.log2(top / E4M3_MAX))
            # the quotient rounds: whether 448 * 2^(e - 1) already holds the largest value is asked of the value itself
            e = torch.where(top <= E4M3_MAX * torch.pow(2.0, e - 1), e - 1, e)
            new = torch.pow(2.0, torch.where(top == 0, -60.0, e).clamp(-60, 60))
            if o:
                new = torch.maximum(new, scale[blk])
                codes[blk, :, :o] = _e4m3(codes[blk, :, :o] * (scale[blk] / new)[:, None, None])
            codes[blk, :, at] = _e4m3(x[rows] / new[None, :, None]).transpose(0, 1)
            scale[blk] = new
        return codes, scale

    if len(blocks) > 3000:
        return None
    ck, ks = held(s["cache_k"], s["k_scale"], heads(s["k"], s["kw"]))
    cv, vs = held(s["cache_v"], s["v_scale"], s["v"].double())
    return [heads(s["q"], s["qw"]), ck, cv, ks, vs]


def _e4m3(x):
    """Round to nearest, ties to even, on the grid of four significant bits down to 2^-9, within +-448."""
    a = x.abs().clamp(min=2.0 ** -6)
    step = torch.pow(2.0, torch.floor(torch.log2(a)) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_attend(s):
    start, kv, D, K = s["row_start"].tolist(), s["kv_lens"].tolist(), s["dim"], s["kv_heads"]
    G, B = s["q_heads"] // K, s["block"]
    out = torch.zeros((start[-1], s["q_heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((start[-1], s["q_heads"]), dtype=torch.float64, device="cuda")
    for r, length in enumerate(kv):
        ids = s["table"][r, :-(-length // B)].long()
        a, b = start[r], start[r + 1]
        seen = torch.arange(length, device="cuda")[None, :] <= (length - (b - a) + torch.arange(b - a, device="cuda"))[:, None]
        seen = seen.repeat_interleave(G, 0)
        for h in range(K):
            k = (s["cache_k"][ids, h].view(torch.float8_e4m3fn).double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:length]
            v = (s["cache_v"][ids, h].view(torch.float8_e4m3fn).double() * s["v_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:length]
            q = s["q"][a:b, h * G:(h + 1) * G].double().reshape((b - a) * G, D)
            z = (q @ k.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
            l = torch.logsumexp(z, -1)
            out[a:b, h * G:(h + 1) * G] = (torch.exp(z - l[:, None]) @ v).reshape(b - a, G, D)
            lse[a:b, h * G:(h + 1) * G] = l.reshape(b - a, G)
    return [out, lse]
