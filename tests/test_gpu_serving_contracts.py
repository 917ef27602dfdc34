"""The serving entry points on the GPU at the edges of their contracts: lists and tables that run short, rows beyond
what a call takes, tokens far apart in weight, lengths near 2^31."""
import numpy as np
import pytest
import torch

from gpu_util import bws, device, f64, np_
from oracle import formats as F, serving as S
from test_gpu_serving import attention_case, check_append, check_attention, check_plan, check_verify, freqs, gen, held, \
    ints, make_cache, rows, verify_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return bws()


# ---- block tables ----------------------------------------------------------------

def test_plan_free_count_past_its_list(m):
    """A count of free blocks that the list does not have is held to the list and reported."""
    new, table = [40, 100], ints([[-1] * 8, [-1] * 8])
    free = [5, 9, 2, 7]
    p = m.kv_plan(ints([0, 0]), ints(new), 16, table, ints(free), ints([5000]), sum(new))
    torch.cuda.synchronize()
    want = S.kv_plan([0, 0], new, 16, [[-1] * 8, [-1] * 8], free, 4, sum(new))
    for g, w in zip((table, p.slots, p.positions, p.row_start, p.kv_lens), want):
        assert np.array_equal(np_(g), np.asarray(w))
    assert p.n_free.item() == 0 and p.status.item() == want[6] | 8
    p = m.kv_plan(ints([0, 0]), ints([16, 16]), 16, table, ints(free), ints([5]), 32)
    torch.cuda.synchronize()
    assert p.n_free.item() == 2 and p.status.item() == 8


def test_plan_empty_free_list(m):
    """Nothing is free and no list is there: rows that fit into held blocks get their slots."""
    table = ints([[7, -1, -1], [4, -1, -1]])
    p = m.kv_plan(ints([3, 15]), ints([20, 1]), 16, table, ints([]), ints([0]), 22)
    torch.cuda.synchronize()
    want = S.kv_plan([3, 15], [20, 1], 16, [[7, -1, -1], [4, -1, -1]], [], 0, 22)
    for g, w in zip((table, p.slots, p.positions, p.row_start, p.kv_lens), want):
        assert np.array_equal(np_(g), np.asarray(w))
    assert p.n_free.item() == 0 and p.status.item() == want[6] == 1
    assert p.slots.tolist()[:13] == [7 * 16 + 3 + i for i in range(13)] and p.slots.tolist()[13:] == [-1] * 7 + [4 * 16 + 15, -1]


@pytest.mark.parametrize("seq,new,wide,n_free", [
    ([0, 0], [80, 16], 2, 8), ([0, 0], [80, 16], 2, 3), ([20, 3], [40, 40], 3, 5), ([70, 0], [16, 16], 2, 4),
    ([15, 0, 100], [100, 33, 1], 4, 9)])
def test_plan_takes_only_what_tables_hold(m, seq, new, wide, n_free):
    """A request longer than its table row takes no block that the row cannot hold, and none from those behind it."""
    check_plan(m, seq, new, 16, wide, n_free, sum(new))
    table = torch.full((len(seq), wide), -1, dtype=torch.int32, device=device())
    for r, s in enumerate(seq):
        have = min(-(-s // 16), wide)
        table[r, :have] = 900 + torch.arange(have, dtype=torch.int32, device=device())
    before = table.clone()
    p = m.kv_plan(ints(seq), ints(new), 16, table, ints(list(range(n_free))), ints([n_free]), sum(new))
    torch.cuda.synchronize()
    stored = ((table != before) & (table >= 0)).sum().item()
    wanted = sum(min(-(-(s + n) // 16), wide) - min(-(-s // 16), wide) for s, n in zip(seq, new))
    assert n_free - p.n_free.item() == stored == min(wanted, n_free)
    assert p.status.item() & 2 and bool(p.status.item() & 1) == (wanted > n_free)


# ---- norm, rotation, cache write ---------------------------------------------------

@pytest.mark.parametrize("D,rot,inter", [(64, 48, False), (64, 48, True), (128, 96, False), (128, 80, True), (256, 192, False),
                                         (256, 144, False), (256, 160, True), (256, 128, False)])
def test_append_more_than_half_rotated(m, D, rot, inter):
    """Most of a head turns but not all of it: short runs, long runs, a prompt of many spans."""
    H, K, B = 3, 2, 32
    g = gen(D + rot)
    w = [1 + 0.2 * torch.randn(D, generator=g, device=device()) for _ in range(2)]
    cache = make_cache(m, 70, K, B, D)
    state = held(cache)
    at = 0
    for n in (1, 5, 70, 2000):
        pos = list(range(at, at + n))
        slots = [(p // B * 7 % 67) * B + p % B for p in pos]
        state = check_append(m, cache, state, rows(n, H, D, g), rows(n, K, D, g), rows(n, K, D, g), pos, slots, freqs(rot),
                             w[0], w[1], inter)
        at += n


# ---- attention -----------------------------------------------------------------------

def check_result(got, gl, want, want_lse, size, score, D):
    """The bound per output: weights in f16 (2^-11), the scores' FP32 sums (D roundings of 2^-24 of the absolute sum, in
    weight and total), the exponents' arguments and remaining sums (2^-14), each of sum p |v|, and half a BF16 step.
    Nothing of it grows with the tokens."""
    delta = D * 2.0 ** -24 * score
    lim = (2.0 ** -11 + 2.0 ** -14 + 2 * delta)[..., None] * size + 0.5 * F.bf16_ulp(np.maximum(np.abs(want), np.abs(got)))
    err = np.abs(got - want)
    assert (err <= lim).all(), ((err > lim).sum(), (err / np.maximum(lim, 1e-300)).max())
    fin = np.isfinite(want_lse)
    assert np.array_equal(np.isfinite(gl), fin)
    assert (np.abs(gl[fin] - want_lse[fin]) <= delta[fin] + 2.0 ** -18 * (1 + np.abs(want_lse[fin]))).all()


def check_rows(q, c, table, start, kv, scale, out, lse, which):
    """Rows `which` of a result against the oracle."""
    want, want_lse, (size, score, _, _) = S.attention(f64(q), np_(c.k), np_(c.v), np_(c.k_scale), np_(c.v_scale),
                                                      np.asarray(table), start, kv, scale)
    check_result(*(x[which] for x in (f64(out), f64(lse), want, want_lse, size, score)), q.shape[2])


@pytest.mark.parametrize("D,H,K,first", [(64, 8, 2, 0), (128, 8, 2, 37), (256, 24, 4, 100)])
def test_attention_prompt_in_eights(m, D, H, K, first):
    """A prompt's 45 rows behind `first` cached tokens in one call: a request for every eight, over the same blocks."""
    n, B = 45, 16
    kv = first + n
    c, q, t, _, _ = attention_case(m, D, H, K, B, [n], [kv], seed=first)
    start = list(range(0, n, 8)) + [n]
    lens = [first + e for e in start[1:]]
    out, lse = m.kv_attention(q, c, ints(np.repeat(t, len(lens), 0)), ints(start), ints(lens), 8, lse=True)
    torch.cuda.synchronize()
    check_rows(q, c, t, [0, n], [kv], D ** -0.5, out, lse, slice(None))


@pytest.mark.parametrize("D,H,K,n", [(64, 4, 2, 4), (128, 4, 2, 4), (256, 4, 1, 4), (256, 24, 4, 8), (128, 32, 2, 8)])
@pytest.mark.parametrize("past", [1, 3, 9, 100, 2 ** 31 - 1])
def test_attention_longer_than_its_table(m, D, H, K, n, past):
    """Tokens past the table row are not there; the rows' sight goes by the request's length all the same."""
    B, held_tokens = 16, 160
    c, q, t, s, mx = attention_case(m, D, H, K, B, [n, 1], [held_tokens, 40], seed=n + D)
    kv = [min(held_tokens + past, 2 ** 31 - 1), 40]
    out, lse = m.kv_attention(q, c, ints(t), ints(s), ints(kv), mx, lse=True)
    torch.cuda.synchronize()
    for j in range(n):   # each row as a request of its own, of as many tokens as it sees
        sees = min(kv[0] - n + j + 1, held_tokens)
        check_rows(q[j:j + 1], c, t[:1], [0, 1], [sees], D ** -0.5, out[j:j + 1], lse[j:j + 1], slice(None))
    check_rows(q[n:], c, t[1:], [0, 1], [40], D ** -0.5, out[n:], lse[n:], slice(None))


@pytest.mark.parametrize("D,H,K", [(64, 4, 2), (128, 8, 2), (256, 24, 4), (256, 16, 1)])
def test_attention_more_rows_than_allowed(m, D, H, K):
    """A request with more rows than max_rows: the first max_rows by their own sight, zeros for the rest, and a status."""
    kv, rw, mx = [200, 90, 50], [2, 7, 1], 3
    c, q, t, s, _ = attention_case(m, D, H, K, 16, rw, kv, seed=31)
    ws = m.Workspace()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=device())
    m.kv_attention(q, c, ints(t), ints(s), ints(kv), mx, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    live = np.ones(10, dtype=bool)
    live[5:9] = False
    check_rows(q, c, t, s, kv, D ** -0.5, out, lse, live)
    assert (out[5:9] == 0).all() and (lse[5:9] == -float("inf")).all()
    assert m.status_word(ws) == 0x10
    m.kv_attention(q, c, ints(t), ints(s), ints(kv), 7, out=out, lse=lse, ws=ws)      # enough rows: none of it
    torch.cuda.synchronize()
    check_rows(q, c, t, s, kv, D ** -0.5, out, lse, slice(None))
    assert m.status_word(ws) == 0


# ---- draft verification -------------------------------------------------------------------

def test_verify_more_rows_than_allowed(m):
    """A request with more rows than max_rows is refused on the device; its neighbours are not touched by it."""
    p, q, tok, start, au, su = verify_case([2, 5, 3, 33], 1001, 36)
    out, n = m.draft_verify(p, tok, ints(start), au, su, 3, draft=q)
    torch.cuda.synchronize()
    assert n.tolist()[1] == -1 and n.tolist()[3] == -1 and (out[1] == -1).all() and (out[3] == -1).all()
    check_verify(m, p, q, tok, start, au, su, 3)
    for r in (0, 2):
        a, b = start[r], start[r + 1]
        want, want_n = S.draft_verify(np_(p[a:b]), np_(tok[a:b]), [0, b - a], np_(au[a:b]), np_(su[r:r + 1]), 3, np_(q[a:b]))
        assert n[r].item() == want_n[0] and np.array_equal(np_(out[r]), want[0])


@pytest.mark.parametrize("D,H,K,pad", [(64, 4, 2, 1), (128, 8, 2, 6), (256, 24, 4, 700)])
def test_attention_rows_of_no_request(m, D, H, K, pad):
    """Rows before the first request's and past the last one's, as the padding of a captured step, are zero."""
    kv, rw = [200, 0, 50], [2, 0, 1]
    c, q, t, s, mx = attention_case(m, D, H, K, 16, rw, kv, seed=32)
    for before in (0, 2):
        x = torch.full((before + 3 + pad, H, D), float("nan"), dtype=torch.bfloat16, device=device())
        x[before:before + 3] = q
        out, lse = torch.full_like(x, float("nan")), torch.full(x.shape[:2], float("nan"), device=device())
        m.kv_attention(x, c, ints(t), ints(s + before), ints(kv), mx, out=out, lse=lse)
        torch.cuda.synchronize()
        mine = slice(before, before + 3)
        check_rows(q, c, t, s, kv, D ** -0.5, out[mine], lse[mine], slice(None))
        out[mine], lse[mine] = 0, -float("inf")
        assert (out == 0).all() and (lse == -float("inf")).all()


def test_attention_without_requests(m):
    """No request at all: every row is one of no request."""
    c, q, t, _, _ = attention_case(m, 64, 4, 2, 16, [3], [20], seed=33)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=device())
    m.kv_attention(q, c, ints(t)[:0], ints([0]), ints([]), 3, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("D,H,K,n", [(128, 2, 2, 1), (256, 24, 4, 8)])
def test_attention_length_near_2_31(m, D, H, K, n):
    """A table row of 2^31 - 16 tokens whose last blocks alone are there."""
    B, wide = 16, 2 ** 27 - 1
    tail = 109                                    # seven blocks but three tokens
    kv = wide * B - 3
    c, q, t, s, mx = attention_case(m, D, H, K, B, [n], [tail], seed=34)
    last = -(-tail // B)
    table = torch.full((1, wide), -1, dtype=torch.int32, device=device())
    table[0, wide - last:] = ints(t[0, :last])
    out, lse = m.kv_attention(q, c, table, ints([0, n]), ints([kv]), mx, lse=True)
    torch.cuda.synchronize()
    check_rows(q, c, t, s, [tail], D ** -0.5, out, lse, slice(None))


def attend64(q, c, kv, scale):
    """One request over blocks 0, 1, ... in FP64: output, log-sum-exp, sum p |v|, the largest score's absolute sum."""
    n, H, D = q.shape
    K = c.kv_heads
    side = lambda s: c.dequantize(s).transpose(0, 1).reshape(K, -1, D)[:, :kv].double()  # noqa: E731
    k, v = side("k"), side("v")
    x = q.double().view(n, K, H // K, D).permute(1, 0, 2, 3)                     # [K, n, G, D]
    hide = torch.arange(kv, device=q.device) > (kv - n + torch.arange(n, device=q.device))[:, None]
    z = (torch.einsum("kngd,ktd->kngt", x, k) * scale).masked_fill(hide[None, :, None], -float("inf"))
    score = (torch.einsum("kngd,ktd->kngt", x.abs(), k.abs()) * scale).masked_fill(hide[None, :, None], 0).amax(-1)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - lse[..., None])
    back = lambda t: t.permute(1, 0, 2, *range(3, t.dim())).reshape(n, H, *t.shape[3:]).cpu().numpy()  # noqa: E731
    return (back(torch.einsum("kngt,ktd->kngd", p, v)), back(lse), back(torch.einsum("kngt,ktd->kngd", p, v.abs())),
            back(score))


SINK_FORMS = [(64, 16, 4, 1), (64, 16, 4, 8), (128, 8, 4, 1), (128, 16, 4, 3), (256, 24, 4, 1), (256, 24, 4, 8), (256, 16, 1, 8),
              (128, 32, 2, 8), (256, 16, 1, 2)]


def sink_case(m, D, H, K, n, kv, gap, where):
    """Tokens whose scores differ by half a nat and carry values about 1, behind one that lies `gap` nats above them and
    carries none."""
    B, g = 64, gen(gap + D)
    n_blocks = -(-kv // B)
    k = torch.randn((n_blocks, K, B, D), generator=g, device=device())
    v = 1 + 0.25 * torch.randn((n_blocks, K, B, D), generator=g, device=device())
    k[..., 0] = 0
    k[where // B, :, where % B] = 0
    v[where // B, :, where % B] = 0
    code = min(gap, 16)                       # E4M3 has no 17
    k[where // B, :, where % B, 0] = code
    e4 = lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    s = torch.ones((2, n_blocks, K), device=device())
    c = m.KvCache(e4(k), e4(v), s[0], s[1])
    q = 0.5 * D ** -0.5 * torch.randn((n, H, D), generator=g, device=device())
    q[..., 0] = gap / code
    return c, q.to(torch.bfloat16)


@pytest.mark.parametrize("gap", [12, 13, 14, 15, 16, 17])
@pytest.mark.parametrize("D,H,K,n", SINK_FORMS)
def test_attention_dominant_token(m, D, H, K, n, gap):
    """A token that takes most of the weight and carries no value leaves the others their precision: whole segments (many
    requests over the same blocks) and one that is cut."""
    kv = 9001
    c, q = sink_case(m, D, H, K, n, kv, gap, 3)
    want = attend64(q, c, kv, 1.0)
    t = [list(range(c.n_blocks))]
    R = 320 // K
    out, lse = m.kv_attention(q.repeat(R, 1, 1), c, ints(t * R), ints([n * r for r in range(R + 1)]), ints([kv] * R), n, 1.0,
                              lse=True)
    torch.cuda.synchronize()
    for r in (0, 1, R // 2, R - 1):
        check_result(f64(out[r * n:(r + 1) * n]), f64(lse[r * n:(r + 1) * n]), *want, D)
    out, lse = m.kv_attention(q, c, ints(t), ints([0, n]), ints([kv]), n, 1.0, lse=True)
    torch.cuda.synchronize()
    check_result(f64(out), f64(lse), *want, D)


@pytest.mark.parametrize("D,H,K,n,kv", [(64, 4, 2, 1, 1), (64, 4, 2, 2, 2), (128, 4, 2, 1, 1), (128, 8, 2, 2, 2),
                                        (128, 40, 8, 5, 5), (256, 6, 1, 1, 2), (256, 24, 4, 8, 8), (256, 24, 4, 2, 600)])
def test_attention_infinite_queries(m, D, H, K, n, kv):
    """A query row with an infinity has no score that is a number: NaN, of one or two tokens too, whose keys may all be of
    the other sign there. Other rows keep their results."""
    c, q, t, s, mx = attention_case(m, D, H, K, 16, [n], [kv], seed=D + n)
    c.k[..., D // 2] = 0x38                             # 1
    check_attention(m, c, q, t, s, [kv], mx)
    bad = np.zeros((n, H), dtype=bool)
    for j, h, x in ((0, 0, "inf"), (0, H - 1, "-inf"), (n - 1, H // 2, "inf"), (n - 1, 1, "-inf")):
        q[j, h, D // 2], bad[j, h] = float(x), True
    out, lse = check_attention(m, c, q, t, s, [kv], mx)
    assert np.array_equal(np_(torch.isnan(out).all(-1)), bad) and np.array_equal(np_(torch.isnan(lse)), bad)


# ---- arguments -------------------------------------------------------------------------

def test_attention_refuses_host_workspace(m):
    c, q, t, s, n = attention_case(m, 64, 4, 2, 16, [1], [20], seed=37)
    for ws in (m.Workspace("cpu"), torch.zeros(1 << 24, dtype=torch.uint8), torch.zeros(1 << 24, device=device())):
        with pytest.raises(m.BwsError, match="workspace"):
            m.kv_attention(q, c, ints(t), ints(s), ints([20]), n, ws=ws)


def test_single_row_and_head_strides(m):
    """A dimension of one entry has no stride of its own: whatever stands there is not looked at."""
    D, B = 64, 16
    g = gen(35)
    c = make_cache(m, 4, 1, B, D)
    flat = rows(1, 1, 8 * D, g).view(-1)
    q = flat.as_strided((1, 4, D), (4 * D + 3, D, 1))
    k = flat[4 * D:].as_strided((1, 1, D), (D + 1, 5, 1))
    v = flat[5 * D:].as_strided((1, 1, D), (1, 1, 1))
    w = torch.ones(D, device=device())
    state = held(c)
    check_append(m, c, state, q, k, v, [0], [16], freqs(D), w, w)
    a = m.kv_attention(q, c, ints([[1]]), ints([0, 1]), ints([1]), 1)
    b = m.kv_attention(q.contiguous(), c, ints([[1]]), ints([0, 1]), ints([1]), 1)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
