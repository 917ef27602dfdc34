"""The 4-bit cache's entry points on the GPU at the edges of their contracts: dimensions that do not turn beside ones that
are not finite, infinite queries, tokens far apart in weight, truncated requests of many rows, prompts in eights, other
devices."""
import numpy as np
import pytest
import torch

from gpu_util import bws, device, f64, np_
from oracle import serving as S
from test_gpu_kv4 import case4, check4, check_long, check_result, check_rope, long_table, make_cache4, sides
from test_gpu_serving import attention_case, freqs, gen, ints, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    return bws()


# ---- norm and rotation: dimensions that do not turn ---------------------------------------

# rotated dimensions in and off whole lanes, none, and a pair that ends inside a lane of adjacent pairs
PARTIAL = [(64, 0, False), (64, 16, False), (64, 20, False), (64, 0, True), (64, 6, True), (64, 18, True), (128, 64, False),
           (128, 8, False), (128, 30, False), (128, 122, True), (256, 64, False), (256, 64, True), (256, 254, False)]


@pytest.mark.parametrize("D,rot,inter", PARTIAL)
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_rope_unturned_dimensions_pass(m, D, rot, inter, bad):
    """Without a norm a dimension that does not turn is copied bit for bit, a negative zero too, and no other result knows
    of it: one value that is not finite, in every place that does not turn."""
    n, H, K = D - rot, 3, 2
    f = freqs(rot) if rot else None
    q, k, pos = rows(n, H, D, gen(D + rot)), rows(n, K, D, gen(D)), ints(1000 + np.arange(n))
    q[:, 0, rot:] = -0.0
    k[0, 1, rot:] = -0.0
    clean = m.qk_norm_rope(q, k, pos, f, interleaved=inter)
    for x in (q, k):
        for t in range(n):
            x[t, t % x.shape[1], rot + t] = bad
    got = m.qk_norm_rope(q, k, pos, f, interleaved=inter)
    torch.cuda.synchronize()
    bits = lambda x: x.contiguous().view(torch.int16)  # noqa: E731
    for x, a, y in zip((q, k), clean, got):
        there = torch.zeros(x.shape, dtype=torch.bool, device=device())
        for t in range(n):
            there[t, t % x.shape[1], rot + t] = True
        assert torch.equal(bits(y)[~there], bits(a)[~there])
        assert torch.equal(bits(y)[..., rot:][~there[..., rot:]], bits(x)[..., rot:][~there[..., rot:]])
        assert torch.isnan(y[there]).all() if bad != bad else (y[there] == bad).all()


@pytest.mark.parametrize("D,rot,inter", PARTIAL)
def test_rope_unturned_dimensions_under_the_norm(m, D, rot, inter):
    """With a norm an infinity makes its own place NaN and the rest of its head zero, as x / sqrt(mean x^2) has it; a NaN
    the whole head."""
    n, H, K = D - rot, 3, 2
    f = freqs(rot) if rot else None
    w = 1 + 0.2 * torch.randn(D, generator=gen(2), device=device())
    q, k = rows(n, H, D, gen(D + rot)), rows(n, K, D, gen(D))
    for x in (q, k):
        for t in range(n):
            x[t, t % x.shape[1], rot + t] = float("inf") if t % 3 else float("nan")
    p = 1000 + np.arange(n)
    got = m.qk_norm_rope(q, k, ints(p), f, q_weight=w, k_weight=w, interleaved=inter)
    torch.cuda.synchronize()
    for x, y in zip((q, k), got):
        with np.errstate(invalid="ignore"):
            want, _ = S.norm_rotate(f64(x), f64(w), p, np_(f) if rot else np.zeros(0), 1e-6, inter)
        y = f64(y)
        assert np.array_equal(np.isnan(y), np.isnan(want))
        for t in range(n):
            if t % 3:
                h = t % x.shape[1]
                assert np.isnan(y[t, h]).sum() == 1 and (np.delete(y[t, h], rot + t) == 0).all()


@pytest.mark.parametrize("D,rot,n,H,K", [(64, 20, 5, 3, 1), (64, 62, 70, 5, 2), (64, 36, 3001, 24, 8), (128, 28, 2000, 32, 8),
                                         (256, 100, 900, 24, 4)])
def test_rope_pairs_off_whole_lanes(m, D, rot, n, H, K):
    """Halves that are no multiple of four: 64 dimensions, many heads a warp, in place, far positions."""
    g = gen(D + rot)
    w = 1 + 0.2 * torch.randn(D, generator=g, device=device())
    pos = np.stack([np.arange(n) - 3, 2 ** 24 - 2 + np.arange(n), np.random.RandomState(n).randint(-2 ** 31, 2 ** 31, n)])
    axis = np.arange(rot // 2) % 3
    q, k = rows(n, H, D, g), rows(n, K, D, g)
    a = check_rope(m, q, k, pos, freqs(rot), axis, w, None)
    b = m.qk_norm_rope(q, k, ints(pos), freqs(rot), ints(axis), w, None, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert b[0] is q and torch.equal(q, a[0]) and torch.equal(k, a[1])


# ---- attention: queries that are not finite -------------------------------------------------

@pytest.mark.parametrize("D,H,K,n,kv,wide", [
    (64, 4, 2, 1, 1, 0), (64, 4, 2, 2, 2, 0), (128, 4, 2, 1, 1, 0), (128, 40, 8, 5, 5, 0), (256, 6, 1, 1, 2, 0), (256, 24, 4, 8, 8, 0),
    (256, 24, 4, 1, 1, 4000), (128, 8, 2, 1, 2, 3000), (64, 8, 8, 2, 2, 200000), (256, 24, 4, 1, 1, 200000), (256, 24, 4, 8, 8, 200000),
    (128, 40, 8, 8, 8, 200000)])
def test_attention4_infinite_queries(m, D, H, K, n, kv, wide):
    """A query row with an infinity has no score that is a number, so its result and log-sum-exp are NaN, of one or two
    tokens too, whose keys may all be of the other sign there; in whole segments, clusters, on the line and of many rows (by
    tables of `wide` tokens). Other rows keep their results."""
    c, q, t, s, mx = case4(m, D, H, K, 16, [n], [kv], seed=D + n)
    t = np.pad(t, ((0, 0), (0, max(wide // 16 - t.shape[1], 0))), constant_values=-1)
    c.k[..., D // 4] = 0x11 if D == 64 else 0x99       # no zero code: 0.5 or -0.5 everywhere, in dimensions D / 2 and the next
    many = (D, n * H // K) in ((256, 48), (128, 40)) and wide
    (check_long if many else check4)(m, c, q, t, s, [kv], mx)
    bad = np.zeros((n, H), dtype=bool)
    for i, (j, h, x) in enumerate([(0, 0, "inf"), (0, H - 1, "-inf"), (n - 1, H // 2, "inf"), (n - 1, 1, "-inf")]):
        q[j, h, D // 2 + i % 2] = float(x)
        bad[j, h] = True
    out, lse = m.kv4_attention(q, c, ints(t), ints(s), ints([kv]), mx, lse=True)
    torch.cuda.synchronize()
    assert np.array_equal(np_(torch.isnan(out).all(-1)), bad) and np.array_equal(np_(torch.isnan(out).any(-1)), bad)
    assert np.array_equal(np_(torch.isnan(lse)), bad)
    if not many:
        check4(m, c, q, t, s, [kv], mx)


def test_attention4_infinite_query_without_tokens(m):
    """A row that sees no token gives zero whatever its query holds."""
    c, q, t, s, mx = case4(m, 128, 4, 2, 16, [3], [1], seed=3)
    q[0] = float("inf")
    q[1, 0, 0] = float("nan")
    out, lse = m.kv4_attention(q, c, ints(t), ints(s), ints([1]), mx, lse=True)
    torch.cuda.synchronize()
    assert (out[:2] == 0).all() and (lse[:2] == -float("inf")).all() and torch.isfinite(out[2]).all()


# ---- attention: many rows a kv head --------------------------------------------------------

@pytest.mark.parametrize("D,H,K,n", [(256, 24, 4, 3), (256, 24, 4, 8), (128, 40, 8, 8), (64, 8, 4, 4), (128, 8, 4, 2)])
def test_attention4_tail_behind_a_dominant_token(m, D, H, K, n):
    """A first token without a value, 23 to 30 octaves above some hundred others that are all alike, so that their weights'
    roundings add up: held to half of f16's least step under a largest weight of 2^9, 2^-34 of it a token, by tables for
    either kernel. (A query of one dimension has one score for all of these tokens, so that its own rounding is no part.)"""
    R, B, tokens = 160 // K, 16, 600
    t = np.random.RandomState(D).permutation(R * 38).reshape(R, 38)
    c = make_cache4(m, R * 38, K, B, D)
    c.k.zero_()
    c.k_scale.fill_(0x38)                    # 1
    c.v.fill_(0x22)                          # 1, 1
    c.v_scale.fill_(0x38)
    first = torch.tensor(t[:, 0].tolist(), device=device())
    c.k[first, :, 0, 4] = 0x07               # 6 in dimension 8
    c.k_scale[first, :, 0, 0] = 0x48         # 4
    c.v_scale[first, :, 0] = 0
    q = torch.zeros((R * n, H, D), dtype=torch.bfloat16, device=device())
    q[..., 8] = 1 + torch.arange(R * n, device=device())[:, None] % 9 / 32 + torch.arange(H, device=device()) % 4 / 64
    start = np.arange(R + 1) * n
    check4(m, c, q, long_table(t, K, B, D), start, [tokens] * R, n, scale=23 * np.log(2.0) / 24)


@pytest.mark.parametrize("D,H,K", [(128, 16, 2), (256, 24, 4), (128, 40, 8)])
def test_attention4_long_table_truncated_requests(m, D, H, K):
    """More rows than max_rows: the first of them within the bound of every output, each with the sight that it has by all
    of its request's rows (check_long's bound, but for weights held to 2^-34 of the largest)."""
    kv, rw, mx = [200, 90, 350], [2, 8, 1], 5
    c, q, t, s, _ = case4(m, D, H, K, 16, rw, kv, seed=32)
    wide = long_table(t, K, 16, D)
    ws = m.Workspace()
    out, lse = m.kv4_attention(q, c, ints(wide), ints(s), ints(kv), mx, lse=True, ws=ws)
    torch.cuda.synchronize()
    assert m.status_word(ws) == 0x10
    assert (out[2 + mx:10] == 0).all() and (lse[2 + mx:10] == -float("inf")).all()
    live = [0, 1, *range(2, 2 + mx), 10]
    cut_s, cut_kv = [0, 2, 2 + mx, 3 + mx], [200, 90 - (8 - mx), 350]     # the same sight
    x, (k, v) = f64(q[live]), sides(c)
    most = np.abs(x).reshape(*x.shape[:2], D // 16, 16).max(-1)
    off = 2.0 ** -14.9 * np.repeat(most, 16, -1) + 2.0 ** -21 * most.max(-1)[..., None]
    ref, ref_lse, (size, score, total) = S.attention4(x, k, v, wide, cut_s, cut_kv, D ** -0.5)
    planes = S.attention4(off, np.abs(k), v, wide, cut_s, cut_kv, D ** -0.5)[2][1]
    check_result(f64(out[live]), f64(lse[live]), ref, ref_lse, size, score + planes * 2.0 ** 24 / D, total, D)


@pytest.mark.parametrize("D,H,K,first,wide", [(64, 8, 4, 0, 0), (128, 8, 2, 300, 0), (256, 24, 4, 0, 0), (256, 24, 4, 700, 0),
                                              (256, 24, 4, 700, 1), (128, 40, 8, 130, 1), (128, 40, 8, 0, 0)])
def test_attention4_prompt_in_eights(m, D, H, K, first, wide):
    """A prompt's 45 rows behind `first` cached tokens in one call: a request for every eight, over the same blocks; by
    tables for either kernel."""
    n, B = 45, 16
    c, q, t, _, _ = case4(m, D, H, K, B, [n], [first + n], seed=first + 1)
    start = [*range(0, n, 8), n]
    lens = [first + e for e in start[1:]]
    t = np.repeat(t, len(lens), 0)
    if wide:
        check_long(m, c, q, t, start, lens, 8)
    else:
        check4(m, c, q, t, start, lens, 8)


# ---- devices -------------------------------------------------------------------------------

@pytest.mark.parametrize("bits", [8, 4])
def test_workspace_size_of_the_tensors_device(m, monkeypatch, bits):
    """The size that a handle keeps is that of its tensors' device, whichever is current at the first call."""
    from bit_weight_streaming_gb300 import serving
    if bits == 4:
        c, q, t, s, n = case4(m, 64, 4, 2, 16, [1], [20], seed=6)
    else:
        c, q, t, s, n = attention_case(m, 64, 4, 2, 16, [1], [20], seed=6)
    name, entered, asked = "kv4_attention_workspace_size" if bits == 4 else "kv_attention_workspace_size", [], []
    size = getattr(serving, name)

    class Guard(torch.cuda.device):
        def __enter__(self):
            entered.append(self.idx)
            return super().__enter__()

        def __exit__(self, *a):
            entered.pop()
            return super().__exit__(*a)

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(serving, "_current_device", lambda: q.get_device() + 1, raising=False)
    monkeypatch.setattr(serving, name, lambda *a: asked.append(list(entered)) or size(*a))
    f = m.kv4_attention if bits == 4 else m.kv_attention
    out = [f(q, c, ints(t), ints(s), ints([20]), n) for _ in range(2)]
    torch.cuda.synchronize()
    assert asked == [[q.get_device()]] and torch.equal(*out)
