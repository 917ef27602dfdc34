"""The 4-bit cache's entry points on the GPU at the edges of their contracts: dimensions that do not turn beside ones that
are not finite."""
import numpy as np
import pytest
import torch

from gpu_util import bws, device, f64, np_
from oracle import serving as S
from test_gpu_serving import freqs, gen, ints, rows

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
