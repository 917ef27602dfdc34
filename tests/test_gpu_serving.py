"""The serving entry points on the GPU against the FP64 oracle: block tables,
cache writes, attention over the 8-bit cache, draft verification."""
import numpy as np
import pytest
import torch

from gpu_util import bws, device, f64, np_
from oracle import formats as F, serving as S, tolerance as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return bws()


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int64).tolist(), dtype=torch.int32, device=device())


def gen(seed):
    return torch.Generator(device=device()).manual_seed(seed)


# ---- block tables and slots ------------------------------------------------------

def check_plan(m, seq, new, B, wide, n_free, n_rows, seed=0, total=None):
    rng = np.random.RandomState(seed)
    R = len(seq)
    pool = rng.permutation((total or 20000))
    table = np.full((R, wide), -1)
    at = 0
    for r in range(R):
        have = min(-(-max(seq[r], 0) // B), wide)
        table[r, :have] = pool[at:at + have]
        at += have
    free = pool[at:at + max(n_free, 1) + 4]
    tab, free_t, nf = ints(table), ints(free), ints([n_free])
    want = S.kv_plan(seq, new, B, table, free, n_free, n_rows)
    for _ in range(2):   # a second call on the first one's table gives the same
        got = m.kv_plan(ints(seq), ints(new), B, tab, free_t, nf, n_rows)
        torch.cuda.synchronize()
        have = (tab, got.slots, got.positions, got.row_start, got.kv_lens)
        for g, w in zip(have, want):
            assert np.array_equal(np_(g), np.asarray(w)), (np_(g), w)
        assert got.n_free.item() == want[5] and got.status.item() == want[6]
        assert nf.item() == n_free


@pytest.mark.parametrize("seq,new,B", [
    ([0], [1], 16), ([15], [1], 16), ([15], [2], 16), ([16], [1], 16), ([4093], [8], 16), ([0], [5000], 64),
    ([7, 0, 33, 64], [0, 3, 1, 130], 32), ([0, 0], [0, 0], 256), ([255, 256, 257], [2, 2, 2], 256)])
def test_plan_small(m, seq, new, B):
    check_plan(m, seq, new, B, -(-(max(s + n for s, n in zip(seq, new))) // B) + 1, 2000, sum(new) + 3)


@pytest.mark.parametrize("R,B,longest", [(257, 16, 40), (1000, 48, 9), (4096, 16, 3)])
def test_plan_many(m, R, B, longest):
    rng = np.random.RandomState(R)
    seq, new = rng.randint(0, 100, R).tolist(), rng.randint(0, longest, R).tolist()
    check_plan(m, seq, new, B, 10, 19000 if R < 4096 else 9000, sum(new), total=50000)


def test_plan_limits(m):
    check_plan(m, [3, 20], [40, 40], 16, 8, 2, 80)            # the free list runs out
    check_plan(m, [3, 20], [40, 40], 16, 8, 0, 80)
    check_plan(m, [3, 20], [40, 40], 16, 3, 30, 80)           # rows wider than the table
    check_plan(m, [3, 20], [40, 40], 16, 8, 30, 50)           # more tokens than rows
    check_plan(m, [3, 20], [40, 40], 16, 8, 30, 0)
    check_plan(m, [-5, 20], [4, -3], 16, 8, 30, 9)            # negative lengths count as zero
    p = m.kv_plan(ints([]), ints([]), 16, torch.empty((0, 4), dtype=torch.int32, device=device()), ints([1]), ints([1]), 3)
    assert p.slots.tolist() == [-1] * 3 and p.row_start.tolist() == [0] and p.n_free.item() == 1


# ---- norm, rotation, cache write -------------------------------------------------

def make_cache(m, n_blocks, heads, B, D, layout="block"):
    """A cache whose unwritten memory holds NaN codes; by block, by head, or with keys and values side by side."""
    dev = device()
    if layout == "block":
        t = torch.full((2, n_blocks, heads, B, D), 0x7F, dtype=torch.uint8, device=dev)
        k, v = t[0], t[1]
    elif layout == "head":
        t = torch.full((2, heads, n_blocks, B, D), 0x7F, dtype=torch.uint8, device=dev)
        k, v = t[0].transpose(0, 1), t[1].transpose(0, 1)
    else:
        t = torch.full((n_blocks, 2, heads, B, D), 0x7F, dtype=torch.uint8, device=dev)
        k, v = t[:, 0], t[:, 1]
    s = torch.full((2, n_blocks, heads), 0.25, dtype=torch.float32, device=dev)
    return m.KvCache(k, v, s[0], s[1])


def held(c):
    return [np_(c.k).copy(), np_(c.v).copy(), np_(c.k_scale).copy(), np_(c.v_scale).copy()]


# FP32 error of a normed and rotated value, relative to |a| + |b| of its pair: the sum of squares (at most 13
# roundings of 2^-24), the reciprocal root, three products, the angle's turn (a few 2^-24 of a turn: 2 pi of that) and
# sincospi: below 2^-18 in all.
ROT_ERR = 2.0 ** -18


def check_append(m, cache, state, q, k, v, positions, slots, inv_freq, qw, kw, inter=False, eps=1e-6):
    """One append against the oracle, from the cache's state before it; returns the state after."""
    got_q = m.qk_norm_rope_append(q, k, v, ints(positions), ints(slots), cache, inv_freq, qw, kw, eps, inter)
    torch.cuda.synchronize()
    f = np_(inv_freq) if inv_freq is not None else np.zeros(0)
    w = lambda t: None if t is None else f64(t)  # noqa: E731
    yq, size = S.norm_rotate(f64(q), w(qw), positions, f, eps, inter)
    ok, worst, at = T.check(yq, f64(got_q), size, rel=ROT_ERR)
    assert ok, (worst, at)
    yk, size = S.norm_rotate(f64(k), w(kw), positions, f, eps, inter)
    want = [a.copy() for a in state]
    S.cache_append(want[0], want[2], yk, slots)
    S.cache_append(want[1], want[3], f64(v), slots)
    got = held(cache)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[3], want[3])      # values: bit for bit
    assert np.array_equal(got[2], want[2])
    # keys: FP32 against FP64 may fall on either side of a midpoint; half a step and that error bound them
    n_blocks, heads, B, D = cache.k.shape
    new = np.zeros((n_blocks, heads, B, D), dtype=bool)
    for t, s in enumerate(slots):
        if not 0 <= s < n_blocks * B:
            continue
        blk, off = s // B, s % B
        new[blk, :, off] = True
        sc = got[2][blk].astype(np.float64)[:, None]
        y = yk[t]
        held_y = F.e4m3_decode(got[0][blk, :, off]) * sc
        lim = np.maximum(np.abs(y) * 2.0 ** -4, sc * 2.0 ** -10) + ROT_ERR * size[t]
        fine = np.isfinite(y)
        assert (np.abs(held_y - y)[fine] <= lim[fine]).all()
        assert np.isnan(held_y[np.isnan(y)]).all()
    assert np.array_equal(got[0][~new], want[0][~new])
    return got


def rows(n, heads, D, g, std=1.0):
    return (std * torch.randn((n, heads, D), generator=g, device=device())).to(torch.bfloat16)


def freqs(rot, base=1e6):
    i = torch.arange(0, rot, 2, device=device(), dtype=torch.float64)
    return (base ** (-i / max(rot, 1))).float()


@pytest.mark.parametrize("D,H,K,B,rot,inter,norm", [
    (64, 4, 4, 16, 64, False, True), (64, 3, 1, 32, 32, True, True), (128, 8, 2, 16, 128, False, True),
    (128, 5, 5, 48, 20, False, False), (128, 8, 1, 64, 0, False, True), (256, 24, 4, 64, 64, False, True),
    (256, 2, 1, 256, 256, True, True), (256, 2, 2, 16, 254, False, True)])
def test_append(m, D, H, K, B, rot, inter, norm):
    g = gen(D + H + B + rot)
    cache = make_cache(m, 9, K, B, D)
    state = held(cache)
    qw = 1 + 0.2 * torch.randn(D, generator=g, device=device()) if norm else None
    kw = 1 + 0.2 * torch.randn(D, generator=g, device=device()) if norm else None
    f = freqs(rot) if rot else None
    # a prompt of 1.5 blocks and two rows in blocks 4 and 2, then single and verify steps with growing values
    at = 0
    table = [4, 2, 7, 0]
    for n, std in [(B + B // 2 + 2, 1.0), (1, 0.5), (1, 30.0), (5, 4.0), (8, 300.0), (1, 1e-3), (3, 1e4)]:
        slots = [table[p // B] * B + p % B for p in range(at, at + n)]
        pos = list(range(at, at + n))
        state = check_append(m, cache, state, rows(n, H, D, g, std), rows(n, K, D, g, std), rows(n, K, D, g, std), pos,
                             slots, f, qw, kw, inter)
        at += n
    # three drafts did not stand: their slots are written again
    at -= 3
    slots = [table[p // B] * B + p % B for p in range(at, at + 2)]
    check_append(m, cache, state, rows(2, H, D, g), rows(2, K, D, g), rows(2, K, D, g), [at, at + 1], slots, f, qw, kw, inter)


@pytest.mark.parametrize("layout", ["head", "pair"])
def test_append_strided_batch(m, layout):
    """Rows of one projection, padding and out-of-range slots among them, a strided cache, far positions."""
    D, H, K, B = 128, 6, 2, 16
    g = gen(5)
    cache = make_cache(m, 12, K, B, D, layout)
    state = held(cache)
    x = rows(40, H + 2 * K + 1, D, g)
    slots = [16 * 3 + i for i in range(5)] + [-1, 12 * 16, 2 ** 31 - 1] + [16 * 5 + 9 + i for i in range(7)] \
        + [16 * 1 + i for i in range(16)] + [16 * 2 + i for i in range(3)] + [16 * 9 + 15] + [-1] * 5
    pos = [900001 + 7 * i for i in range(35)] + [2 ** 24 + 1, 2 ** 30 + 3, 2 ** 31 - 1, 0, 65536]
    kw = torch.ones(D, device=device())
    check_append(m, cache, state, x[:, :H], x[:, H:H + K], x[:, H + K:H + 2 * K], pos, slots, freqs(D), kw, kw)


def test_append_long_runs(m):
    """More rows than the shared buffer holds, many spans, a run that starts inside a block."""
    D, H, K, B = 256, 1, 1, 256
    g = gen(6)
    cache = make_cache(m, 8, K, B, D)
    n = 700
    slots = [100 + i if 100 + i < 256 else 512 + (100 + i - 256) for i in range(n)]
    w = torch.ones(D, device=device())
    check_append(m, cache, held(cache), rows(n, H, D, g), rows(n, K, D, g), rows(n, K, D, g), list(range(n)), slots,
                 freqs(64), w, w)
    cache = make_cache(m, 700, 2, 16, 64)
    n = 5000
    slots = [3 + i for i in range(n)]
    check_append(m, cache, held(cache), rows(n, 1, 64, g), rows(n, 2, 64, g), rows(n, 2, 64, g), list(range(n)), slots,
                 freqs(64), None, None)


@pytest.mark.parametrize("D,K,B,longest,R", [(128, 8, 16, 5, 48), (128, 8, 16, 16, 40), (64, 4, 32, 12, 60),
                                             (256, 4, 16, 3, 50), (256, 2, 64, 20, 64), (64, 16, 16, 9, 400)])
def test_append_short_and_long_runs_side_by_side(m, D, K, B, longest, R):
    """Spans that hold runs of one warp's and of the whole CTA's, next to each other."""
    for seed in range(3):
        rng = np.random.RandomState(seed)
        lens = [longest] + rng.randint(1, longest + 1, R - 1).tolist()
        seqs = rng.randint(0, 3 * B, R)
        table, n_blocks = tables([s + n for s, n in zip(seqs, lens)], B, seed=seed)
        slots = [int(table[r, p // B]) * B + p % B for r in range(R) for p in range(seqs[r], seqs[r] + lens[r])]
        pos = [p for r in range(R) for p in range(seqs[r], seqs[r] + lens[r])]
        g = gen(seed)
        cache = make_cache(m, n_blocks, K, B, D)
        fill(cache, g)
        n, w = len(pos), torch.ones(D, device=device())
        check_append(m, cache, held(cache), rows(n, 2, D, g, 3.0), rows(n, K, D, g, 3.0), rows(n, K, D, g, 3.0), pos, slots,
                     freqs(D), w, w)


def test_append_special_values(m):
    """Zero rows, infinities and NaN: they set no scale, NaN stays, infinity saturates."""
    D, K, B = 64, 1, 16
    g = gen(7)
    cache = make_cache(m, 2, K, B, D)
    state = held(cache)
    v = rows(4, K, D, g)
    v[0] = 0
    v[1, 0, 3], v[1, 0, 4], v[2, 0, 5] = float("nan"), float("inf"), -float("inf")
    v[3] = float("nan")
    k = rows(4, K, D, g)
    k[0] = 0
    state = check_append(m, cache, state, rows(4, 1, D, g), k, v, [0, 1, 2, 3], [0, 1, 2, 3], None, None, None)
    z = torch.zeros((1, K, D), dtype=torch.bfloat16, device=device())
    state = check_append(m, cache, state, z, z, z, [0], [16], None, None, None)     # a block of zeros: the least scale
    assert state[2][1, 0] == 2.0 ** -60
    big = torch.full((1, K, D), 3e38, dtype=torch.bfloat16, device=device())
    state = check_append(m, cache, state, z, z, big, [1], [17], None, None, None)
    assert state[3][1, 0] == 2.0 ** 60 and (F.e4m3_decode(state[1][1, 0, 1]) == 448).all()


# ---- attention -------------------------------------------------------------------

def fill(cache, g, spread=1.0, std=1.0):
    for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = std * torch.randn(codes.shape, generator=g, device=device())
        x *= torch.exp2(spread * torch.randn(codes.shape[:2], generator=g, device=device()).round())[:, :, None, None]
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448.0)))
        codes.copy_((x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8))
        scale.copy_(s)


def blank_unused(cache, table, kv):
    """NaN codes wherever no request has a token."""
    used = torch.zeros(cache.k.shape[0], cache.k.shape[2], dtype=torch.bool)
    for r, n in enumerate(kv):
        for t in range(n):
            b = int(table[r][t // cache.block_tokens])
            if 0 <= b < used.shape[0]:
                used[b, t % cache.block_tokens] = True
    dead = ~used.to(device())[:, None, :, None].expand(cache.k.shape)
    cache.k[dead] = 0x7F
    cache.v[dead] = 0xFF


def tables(kv, B, extra=0, seed=0):
    need = [-(-n // B) for n in kv]
    pool = np.random.RandomState(seed).permutation(sum(need) + 3)
    table = np.full((len(kv), max(max(need), 1) + extra), -1)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = pool[at:at + n]
        at += n
    return table, len(pool)


def check_attention(m, cache, q, table, start, kv, max_rows, scale=None, **kw):
    """Against FP64. The bound per output: the weights' rounding to f16 (2^-11 of sum p |v|, and half of f16's least
    step, 2^-25 of the largest p vs 448 per token), the scores' FP32 sums (D roundings of 2^-24 of the absolute sum,
    twice: weight and total), exponent arguments and remaining sums (2^-14), and half a BF16 step."""
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, lse = m.kv_attention(q, cache, ints(table), ints(start), ints(kv), max_rows, scale, lse=True, **kw)
    torch.cuda.synchronize()
    want, want_lse, (size, score, top, seen) = S.attention(
        f64(q), np_(cache.k), np_(cache.v), np_(cache.k_scale), np_(cache.v_scale), np.asarray(table), start, kv, scale)
    delta = D * 2.0 ** -24 * score
    # spread blocks keep the argument of the exponential below about 64 + 60: 2^-24 of that, rounded twice
    rel = 2.0 ** -11 + 2.0 ** -14 + 2 * delta
    extra = (seen * 448 * 2.0 ** -25 * top)[..., None]
    got = f64(out)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    big = np.where(nan, 0, np.maximum(np.abs(want), np.abs(got)))
    lim = rel[..., None] * size + extra + 0.5 * F.bf16_ulp(big)
    bad = (np.abs(got - want) > lim) & ~nan
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], lim[bad][:4])
    gl = f64(lse)
    assert np.array_equal(np.isfinite(gl), np.isfinite(want_lse))
    fin = np.isfinite(want_lse)
    assert (np.abs(gl - want_lse)[fin] <= (delta + 2.0 ** -18 * (1 + np.abs(want_lse)))[fin]).all()
    return out, lse


def attention_case(m, D, H, K, B, rows_of, kv, seed=0, layout="block", std=1.0, spread=1.0, extra=0):
    g = gen(seed)
    table, n_blocks = tables(kv, B, extra, seed)
    cache = make_cache(m, n_blocks, K, B, D, layout)
    fill(cache, g, spread)
    blank_unused(cache, table, kv)
    start = np.concatenate([[0], np.cumsum(rows_of)])
    q = rows(int(start[-1]), H, D, g, std)
    return cache, q, table, start, max(max(rows_of), 1)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 127, 128, 129, 700])
def test_attention_lengths(m, D, kv):
    c, q, t, s, n = attention_case(m, D, 4, 2, 16, [1], [kv], seed=kv)
    check_attention(m, c, q, t, s, [kv], n)


@pytest.mark.parametrize("D,H,K,B", [(64, 2, 2, 32), (64, 16, 1, 16), (128, 8, 1, 64), (128, 7, 7, 16), (128, 40, 8, 48),
                                     (256, 6, 1, 256), (256, 24, 4, 64), (256, 16, 1, 16), (64, 64, 4, 16), (128, 32, 2, 16)])
@pytest.mark.parametrize("n", [1, 2, 5, 8])
def test_attention_heads_and_rows(m, D, H, K, B, n):
    kv = [333, n, 61]
    c, q, t, s, mx = attention_case(m, D, H, K, B, [n, n, 1], kv, seed=n)
    check_attention(m, c, q, t, s, kv, mx)


@pytest.mark.parametrize("D,H,K", [(64, 8, 2), (128, 4, 2), (256, 4, 1)])
def test_attention_ragged_batch(m, D, H, K):
    """Lengths from none up, requests without rows, rows that see no token."""
    kv = [0, 5, 0, 1, 400, 3, 90, 16, 33, 700, 2, 0, 1, 47]
    rw = [1, 3, 0, 2, 8, 8, 0, 1, 5, 4, 2, 8, 1, 1]
    c, q, t, s, n = attention_case(m, D, H, K, 16, rw, kv, seed=3)
    out, lse = check_attention(m, c, q, t, s, kv, n)
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all()


def test_attention_many_requests(m):
    """More requests than threads, more segments than CTAs."""
    rng = np.random.RandomState(4)
    kv = rng.randint(0, 60, 700).tolist()
    rw = rng.randint(0, 3, 700).tolist()
    c, q, t, s, n = attention_case(m, 64, 2, 1, 16, rw, kv, seed=4)
    check_attention(m, c, q, t, s, kv, n)


@pytest.mark.parametrize("layout", ["head", "pair"])
def test_attention_layouts_and_strides(m, layout):
    kv = [77, 200]
    c, q, t, s, n = attention_case(m, 128, 6, 2, 32, [3, 2], kv, seed=8, layout=layout, extra=5)
    wide = torch.zeros((5, 9, 136), dtype=torch.bfloat16, device=device())
    wide[:, 1:7, :128] = q
    check_attention(m, c, wide[:, 1:7, :128], t, s, kv, n, scale=0.3)
    out = torch.empty_like(q)
    got, _ = check_attention(m, c, q, t, s, kv, 8, out=out, ws=m.Workspace())      # max_rows above what is there
    assert got.data_ptr() == out.data_ptr()


def test_attention_extreme_scales(m):
    """Blocks whose value scales lie 2^60 apart, sharp scores, and a tiny cache beside them."""
    kv = [200]
    c, q, t, s, n = attention_case(m, 128, 4, 2, 16, [2], kv, seed=9, std=3.0)
    e = torch.randint(-30, 31, c.v_scale.shape, generator=gen(10), device=device()).float()
    c.v_scale.copy_(torch.exp2(e))
    check_attention(m, c, q, t, s, kv, n)
    c.k_scale.mul_(16.0)                      # scores in the hundreds: one token takes all
    check_attention(m, c, q, t, s, kv, n)
    c.v_scale.fill_(2.0 ** -60)
    check_attention(m, c, q, t, s, kv, n)


def test_attention_wide_queries(m):
    """Query rows whose magnitudes f16 does not hold."""
    kv = [150]
    c, q, t, s, n = attention_case(m, 64, 4, 1, 16, [3], kv, seed=11)
    q[0] *= 2.0 ** 100
    q[1] *= 2.0 ** -100
    check_attention(m, c, q[:, :1].expand(3, 4, 64).contiguous(), t, s, kv, n, scale=2.0 ** -103)


def test_attention_bad_pages(m):
    """Table entries outside the cache: their tokens are not there."""
    kv = [100, 40, 20]
    c, q, t, s, n = attention_case(m, 128, 4, 1, 16, [2, 1, 1], kv, seed=12)
    t[0, 1], t[0, 6], t[2, :2] = -1, 2 ** 31 - 1, 1000
    t[1, 2] = -7
    out, lse = check_attention(m, c, q, t, s, kv, n)
    assert (out[3] == 0).all() and (lse[3] == -float("inf")).all()


def test_attention_nan_in_masked_places(m):
    """A NaN among the rows' own tokens reaches the rows that see it, and no other."""
    kv, n = [70], 4
    c, q, t, s, mx = attention_case(m, 128, 4, 2, 16, [n], kv, seed=13)
    B = 16
    tok = kv[0] - 2                                     # seen by rows 2 and 3
    c.v[int(t[0, tok // B]), 1, tok % B, 5] = 0x7F
    c.v[int(t[0, tok // B]), 1, tok % B, 90] = 0xFF

    # the oracle drops unseen tokens before its products, so its NaN are where they belong
    check_attention(m, c, q, t, s, kv, mx)
    c, q, t, s, mx = attention_case(m, 128, 4, 2, 16, [n], kv, seed=14)
    tok = kv[0] - 1                                     # a key only row 3 sees
    c.k[int(t[0, tok // B]), 0, tok % B, 3] = 0x7F
    out, lse = m.kv_attention(q, c, ints(t), ints(s), ints(kv), mx, lse=True)
    torch.cuda.synchronize()
    bad = torch.isnan(out).any(-1)
    assert bad[3, :2].all() and not bad[:3].any() and not bad[3, 2:].any()
    q[1, 2, 7] = float("nan")                           # a query row's NaN stays in its row
    out = m.kv_attention(q, c, ints(t), ints(s), ints(kv), mx)
    bad = torch.isnan(out).any(-1)
    assert bad[1, 2] and bad.sum().item() == 3


# ---- wide row groups (more rows than a warp holds: the kernel on the tensor cores) ----

@pytest.mark.parametrize("D,H,K,n,kv", [(256, 24, 4, 8, 9001), (256, 24, 4, 5, 4097), (256, 16, 1, 2, 3000),
                                        (256, 16, 1, 8, 1500), (128, 48, 3, 3, 5003), (128, 8, 1, 8, 2049),
                                        (128, 16, 1, 8, 800)])
def test_attention_wide_long(m, D, H, K, n, kv):
    """Many tiles a share, shares that cut segments, row groups that go round the rings several times."""
    c, q, t, s, mx = attention_case(m, D, H, K, 32, [n], [kv], seed=kv)
    ws = m.Workspace()
    a = check_attention(m, c, q, t, s, [kv], mx, ws=ws)
    b = m.kv_attention(q, c, ints(t), ints(s), ints([kv]), mx, lse=True, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and m.status_word(ws) == 0


@pytest.mark.parametrize("D,H,K", [(256, 12, 2), (128, 16, 2)])
def test_attention_wide_batch(m, D, H, K):
    """Ragged lengths and rows, requests without either, tiles whose blocks are not all there."""
    kv = [0, 5, 0, 129, 400, 3, 90, 16, 33, 1700, 128, 0, 1, 47, 256]
    rw = [1, 3, 0, 2, 8, 8, 0, 1, 5, 8, 7, 8, 1, 1, 6]
    c, q, t, s, n = attention_case(m, D, H, K, 16, rw, kv, seed=23)
    t[4, 3], t[9, 0], t[9, 8:17], t[10, :7] = -1, 2 ** 31 - 1, 10 ** 6, -3
    ws = m.Workspace()
    check_attention(m, c, q, t, s, kv, n, ws=ws)
    assert m.status_word(ws) == 0


def test_attention_wide_special_values(m):
    """NaN among the rows' own tokens, in keys and queries; infinite queries; spread value scales."""
    D, H, K, n, kv, B = 256, 24, 4, 8, [300], 16
    c, q, t, s, mx = attention_case(m, D, H, K, B, [n], kv, seed=24)
    c.v_scale.copy_(torch.exp2(torch.randint(-30, 31, c.v_scale.shape, generator=gen(25), device=device()).float()))
    check_attention(m, c, q, t, s, kv, mx)
    tok = kv[0] - 3                                     # seen by rows 5, 6 and 7
    c.v[int(t[0, tok // B]), 2, tok % B, 200] = 0x7F
    check_attention(m, c, q, t, s, kv, mx)
    tok = kv[0] - 1
    c.k[int(t[0, tok // B]), 0, tok % B, 3] = 0x7F      # seen by row 7
    q[2, 13, 7], q[3, 20, 9] = float("nan"), float("inf")
    out = m.kv_attention(q, c, ints(t), ints(s), ints(kv), mx)
    torch.cuda.synchronize()
    bad = torch.isnan(out).any(-1)
    want = torch.zeros_like(bad)
    want[7, :6] = True
    want[5:, 12:18] = True                              # the value's NaN, in kv head 2
    want[2, 13] = want[3, 20] = True
    assert torch.equal(bad, want)


def test_attention_wide_uneven_queries(m):
    """Query values far below their row's largest: held to 2^-22 of it (half the low part's least step)."""
    D, H, K, n, kv = 256, 16, 1, 4, [500]
    c, q, t, s, mx = attention_case(m, D, H, K, 16, [n], kv, seed=26)
    q[:, :, 0] = 2.0 ** 12
    c.k[:, :, :, 0] = 0                                 # the largest meets nothing
    out, lse = m.kv_attention(q, c, ints(t), ints(s), ints(kv), mx, lse=True)
    torch.cuda.synchronize()
    _, want, (_, score, _, _) = S.attention(f64(q), np_(c.k), np_(c.v), np_(c.k_scale), np_(c.v_scale), t, s, kv, D ** -0.5)
    keys = np.abs(F.e4m3_decode(np_(c.k)[t[0]][:, 0]) * np_(c.k_scale)[t[0]][:, :1, None])
    lost = 2.0 ** -22 * 2.0 ** 12 * np.nanmax(keys.sum(-1)) * D ** -0.5
    assert (np.abs(f64(lse) - want) <= lost + D * 2.0 ** -24 * score + 2.0 ** -18 * (1 + np.abs(want))).all()


def test_attention_split_is_deterministic(m):
    """A long request is cut into shares; the same bits every time, alone and among others."""
    kv = [20001]
    c, q, t, s, n = attention_case(m, 128, 8, 2, 64, [2], kv, seed=15)
    a = check_attention(m, c, q, t, s, kv, n)
    b = m.kv_attention(q, c, ints(t), ints(s), ints(kv), n, lse=True, ws=m.Workspace())
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_far_block(m):
    """Codes beyond 2^32 bytes of the cache's start."""
    D, B, K = 256, 256, 16
    n_blocks = 4400                                     # 4400 blocks of 1 MiB a side
    k = torch.empty((2, n_blocks, K, B, D), dtype=torch.uint8, device=device())
    sc = torch.ones((2, n_blocks, K), device=device())
    far = m.KvCache(k[0], k[1], sc[0], sc[1])
    near = make_cache(m, 2, K, B, D)
    fill(near, gen(16))
    for i, b in enumerate((4399, 4097)):
        far.k[b], far.v[b] = near.k[i], near.v[i]
        far.k_scale[b], far.v_scale[b] = near.k_scale[i], near.v_scale[i]
    q = rows(1, K, D, gen(17))
    a = m.kv_attention(q, near, ints([[0, 1]]), ints([0, 1]), ints([500]), 1)
    b = m.kv_attention(q, far, ints([[4399, 4097]]), ints([0, 1]), ints([500]), 1)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    # and a write there
    x = rows(1, K, D, gen(18))
    m.qk_norm_rope_append(x, x, x, ints([9]), ints([4399 * B + 3]), far, freqs(64))
    m.qk_norm_rope_append(x, x, x, ints([9]), ints([3]), near, freqs(64))
    torch.cuda.synchronize()
    assert torch.equal(far.k[4399], near.k[0]) and torch.equal(far.v[4399], near.v[0])


def test_attention_graph_follows_lengths(m):
    """A captured step reads its lengths, tables and slots when it is replayed; on a stream of its own."""
    D, H, K, B, wide = 128, 8, 2, 16, 40
    g = gen(19)
    cache = make_cache(m, 64, K, B, D)
    fill(cache, g)
    seq, new, table = ints([0, 0]), ints([0, 0]), torch.full((2, wide), -1, dtype=torch.int32, device=device())
    free, n_free = ints(list(range(64))), ints([64])
    x = rows(6, H + 2 * K, D, g)
    w, f, ws = torch.ones(D, device=device()), freqs(D), m.Workspace()
    state = {}

    def step():
        p = m.kv_plan(seq, new, B, table, free, n_free, 6)
        q = m.qk_norm_rope_append(x[:, :H], x[:, H:H + K], x[:, H + K:], p.positions, p.slots, cache, f, w, w)
        out, lse = m.kv_attention(q, cache, table, p.row_start, p.kv_lens, 4, lse=True, ws=ws)
        n_free.copy_(p.n_free)
        state.update(plan=p, q=q, out=out, lse=lse)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step()
    torch.cuda.synchronize()
    lens = [0, 0]
    for n in ([4, 1], [2, 4], [1, 1], [0, 3]):
        seq.copy_(ints(lens))
        new.copy_(ints(n))
        x.copy_(rows(6, H + 2 * K, D, g))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        lens = [a + b for a, b in zip(lens, n)]
        p = state["plan"]
        assert p.kv_lens.tolist() == lens and p.status.item() == 0
        t, q = sum(n), state["q"]
        want, want_lse, (size, score, top, seen) = S.attention(
            f64(q)[:t], np_(cache.k), np_(cache.v), np_(cache.k_scale), np_(cache.v_scale), np_(table),
            [0, n[0], t], lens, D ** -0.5)
        lim = (2.0 ** -11 + 2.0 ** -14 + 2 * D * 2.0 ** -24 * score)[..., None] * size \
            + (seen * 448 * 2.0 ** -25 * top)[..., None] + 0.5 * F.bf16_ulp(np.maximum(np.abs(want), np.abs(f64(state["out"])[:t])))
        assert (np.abs(f64(state["out"])[:t] - want) <= lim).all()
    assert m.status_word(ws) == 0


def test_attention_python_refusals(m):
    c, q, t, s, n = attention_case(m, 64, 4, 2, 16, [1], [20], seed=20)
    with pytest.raises(m.BwsError):
        m.kv_attention(q.float(), c, ints(t), ints(s), ints([20]), 1)
    with pytest.raises(m.BwsError):
        m.kv_attention(q, c, ints(t), ints([0, 1, 1]), ints([20]), 1)
    with pytest.raises(m.BwsError):
        m.kv_attention(q, c, ints(t), ints(s), ints([20]), 9)
    with pytest.raises(m.BwsError):
        m.kv_attention(q[:, :3], c, ints(t), ints(s), ints([20]), 1)
    with pytest.raises(m.BwsError):
        m.KvCache(c.k, c.v[:, :, :, ::2], c.k_scale, c.v_scale)
    with pytest.raises(m.BwsError):
        m.qk_norm_rope_append(q, q[:, :1], q[:, :2], ints([0]), ints([0]), c)


# ---- draft verification ----------------------------------------------------------

def verify_case(rows_of, V, seed, sharp=2.0, noise=0.7):
    g = gen(seed)
    n = sum(rows_of)
    z = sharp * torch.randn((n, V), generator=g, device=device())
    p = torch.softmax(z, -1)
    q = torch.softmax(z + noise * torch.randn((n, V), generator=g, device=device()), -1)
    tok = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32) if V > 1 else torch.zeros(n, dtype=torch.int32, device=device())
    start = np.concatenate([[0], np.cumsum(rows_of)])
    return p, q, tok, start, torch.rand(n, generator=g, device=device()), torch.rand(len(rows_of), generator=g, device=device())


def check_verify(m, p, q, tok, start, au, su, max_rows):
    out, n = m.draft_verify(p, tok, ints(start), au, su, max_rows, draft=q)
    torch.cuda.synchronize()
    want, want_n = S.draft_verify(np_(p), np_(tok), start, np_(au), np_(su), max_rows, None if q is None else np_(q))
    assert np.array_equal(np_(n), want_n), (np_(n), want_n)
    assert np.array_equal(np_(out), want), (np_(out), want)
    return out, n


@pytest.mark.parametrize("V", [1, 2, 3, 127, 1000, 4097, 32000, 100032])
@pytest.mark.parametrize("rows_of", [[1], [8], [3, 1, 0, 5, 2, 4]])
@pytest.mark.parametrize("draft", [True, False])
def test_verify(m, V, rows_of, draft):
    p, q, tok, start, au, su = verify_case(rows_of, V, V + len(rows_of))
    check_verify(m, p, q if draft else None, tok, start, au, su, 8)


def test_verify_batch(m):
    rng = np.random.RandomState(1)
    rows_of = rng.randint(0, 6, 400).tolist()
    for V in (3001, 32):
        p, q, tok, start, au, su = verify_case(rows_of, V, 77)
        check_verify(m, p, q, tok, start, au, su, 5)


def test_verify_many_rows(m):
    """All 31 drafts of a request stand, or all but the last."""
    p, _, tok, start, au, su = verify_case([32, 32], 257, 9)
    au.zero_()
    check_verify(m, p, p.clone(), tok, start, au, su, 32)
    au[30], p[30, int(tok[30])] = 0.99, 0.0
    q = p.clone()
    q[30, int(tok[30])] = 0.5
    check_verify(m, p, q, tok, start, au, su, 32)


def test_verify_edges(m):
    V = 513
    p, q, tok, start, au, su = verify_case([3, 2, 2, 2, 2, 1, 2], V, 5)
    au.fill_(0.999)
    q[3] = p[3]                                  # nothing left of the target: drawn from the target
    au[3] = 1.0                                  # u q < p fails at equality
    tok[5] = V                                   # outside the vocabulary
    tok[7] = -1
    p[9] = 0
    q[9] = 0                                     # a row without weight
    p[11, :100] = float("nan")
    p[11, 100] = -1.0
    su[:] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.0, 0.5, 0.5, 0.25, 1 - 2.0 ** -24], device=device())
    out, n = check_verify(m, p, q, tok, start, au, su, 4)
    check_verify(m, p, None, tok, start, au, su, 4)
    # strided rows off 16 bytes, and a whole table of them
    wide_p, wide_q = torch.zeros((14, V + 5), device=device()), torch.zeros((14, V + 2), device=device())
    wide_p[:, 1:V + 1], wide_q[:, 2:V + 2] = p, q
    check_verify(m, wide_p[:, 1:V + 1], wide_q[:, 2:V + 2], tok, start, au, su, 4)
    assert m.draft_verify(p[:0], tok[:0], ints([0, 0]), au[:0], su[:1], 3)[1].tolist() == [0]


# ---- the calls together ------------------------------------------------------------

def test_serving_step_example(m, monkeypatch):
    """The example serves: every step yields between one token and all of its rows', of the vocabulary."""
    import importlib.util
    import os
    import sys
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_step.py")
    spec = importlib.util.spec_from_file_location("serving_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    monkeypatch.setattr(sys, "argv", ["serving_step.py", "--steps", "12", "--drafts", "7"])
    text = ex.main()
    assert 12 <= len(text) - 1 <= 12 * 8 and all(0 <= t < ex.VOCAB for t in text)
