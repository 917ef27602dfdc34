"""The 4-bit cache's entry points on the CPU: their refusals, and the oracle's pieces against hand-worked values (no
GPU)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import formats as F, quant as Q, serving as S


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    import bit_weight_streaming_gb300 as bws
    return bws.lib()


def cache(**kw):
    from bit_weight_streaming_gb300.serving import _Kv4Cache
    v = dict(n_blocks=4, n_kv_heads=2, block_tokens=16, head_dim=64, k=4096, v=8192, k_scale=64, v_scale=128, k_global=None,
             v_global=16, block_stride=1024, head_stride=512, scale_block_stride=128, scale_head_stride=64)
    v.update(kw)
    return _Kv4Cache(*v.values())


@pytest.mark.parametrize("bad,code", [
    (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(block_tokens=8), 2), (dict(block_tokens=40), 2),
    (dict(block_tokens=512), 2), (dict(n_kv_heads=0), 2), (dict(n_kv_heads=129), 2), (dict(n_blocks=0), 2),
    (dict(n_blocks=1 << 28), 2), (dict(k=None), 1), (dict(v_scale=None), 1), (dict(k=4104), 3), (dict(k_scale=72), 3),
    (dict(v_global=18), 3), (dict(block_stride=1032), 3), (dict(scale_head_stride=72), 3), (dict(head_stride=256), 2),
    (dict(block_stride=512), 2), (dict(scale_block_stride=64), 2), (dict(scale_head_stride=32), 2), (dict(block_stride=1 << 41), 2)])
def test_cache_refusals(lib, bad, code):
    held = cache(**bad)
    c = ctypes.addressof(held)
    assert lib.bws_kv4_append(16, 128, 64, 16, 128, 64, 16, 1, c, None) == code
    assert lib.bws_kv4_read(c, 16, 4, 1, 16, 16, 1, 16, 16, None) == code
    assert lib.bws_kv4_attention(16, 256, 64, 1, 4, c, 16, 4, 1, 16, 16, 1, 0.1, 16, None, 256, 1 << 40, None) == code


def test_append_refusals(lib):
    held = cache()
    c = ctypes.addressof(held)

    def call(k=16, kr=128, kh=64, v=16, vr=128, vh=64, slots=16, n=1, at=c):
        return lib.bws_kv4_append(k, kr, kh, v, vr, vh, slots, n, at, None)

    assert call(at=None) == 1 and call(n=-1) == 1
    assert call(n=0, k=None) == 0                      # nothing to do
    assert call(k=None) == 1 and call(v=None) == 1 and call(slots=None) == 1 and b"null" in lib.bws_last_error()
    assert call(k=24) == 3 and call(v=8) == 3 and call(slots=18) == 3
    assert call(kr=132) == 3 and call(vh=60) == 3 and b"strides" in lib.bws_last_error()


def test_read_refusals(lib):
    held = cache()
    c = ctypes.addressof(held)

    def call(at=c, table=16, wide=4, R=1, first=16, start=16, n=1, k=16, v=16):
        return lib.bws_kv4_read(at, table, wide, R, first, start, n, k, v, None)

    assert call(at=None) == 1 and call(n=-1) == 1 and call(R=-1) == 1 and call(wide=-1) == 1 and call(R=(1 << 20) + 1) == 1
    assert call(wide=1 << 27) == 2
    assert call(n=0, k=None) == 0 and call(R=0, first=None) == 0
    assert call(table=None) == 1 and call(first=None) == 1 and call(start=None) == 1 and call(k=None) == 1 and call(v=None) == 1
    assert call(k=24) == 3 and call(v=8) == 3 and call(table=17) == 3 and call(first=18) == 3 and call(start=2) == 3


def test_attention_refusals(lib):
    held = cache()
    c = ctypes.addressof(held)
    size = lib.bws_kv4_attention_workspace_size(4, 2, 64, 1)
    assert size > 0

    def call(q=16, qr=256, qh=64, n=1, H=4, at=c, table=16, wide=4, R=1, start=16, kv=16, most=1, scale=0.1, out=16, lse=None,
             ws=256, nbytes=1 << 40):
        return lib.bws_kv4_attention(q, qr, qh, n, H, at, table, wide, R, start, kv, most, scale, out, lse, ws, nbytes, None)

    assert call(at=None) == 1 and call(most=0) == 1 and call(most=9) == 1 and call(n=-1) == 1 and call(R=-1) == 1
    assert call(H=3) == 2 and call(H=34) == 2 and call(H=0) == 2 and call(wide=1 << 27) == 2
    assert call(n=0, q=None) == 0 and call(R=0, kv=None) == 0
    assert call(q=None) == 1 and call(out=None) == 1 and call(start=None) == 1 and call(kv=None) == 1 and call(table=None) == 1
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(q=24) == 3 and call(out=8) == 3 and call(qr=252) == 3 and call(qh=60) == 3 and call(lse=18) == 3
    assert call(ws=None) == 7 and call(nbytes=size - 1) == 7 and call(ws=128) == 3
    for bad in ((4, 3, 64, 1), (4, 2, 96, 1), (4, 2, 64, 0), (4, 2, 64, 9), (34, 2, 64, 1), (0, 0, 64, 1)):
        assert lib.bws_kv4_attention_workspace_size(*bad) == 0


def test_rope_refusals(lib):
    from bit_weight_streaming_gb300.serving import _Qk

    def call(q_out=16, k_out=16, **kw):
        v = dict(q=16, qr=256, qh=64, k=16, kr=128, kh=64, n=1, H=4, K=2, D=64, pos=16, axes=1, axis=None, qw=None, kw=None,
                 f=16, rot=64, inter=0, eps=1e-6)
        v.update(kw)
        a = _Qk(*v.values())
        return lib.bws_qk_norm_rope(ctypes.addressof(a), q_out, k_out, None)

    assert lib.bws_qk_norm_rope(None, 16, 16, None) == 1
    assert call(n=0, q=None) == 0 and call(H=0, K=0, q=None) == 0
    assert call(D=96) == 2 and call(rot=63) == 2 and call(rot=66) == 2 and call(rot=-2) == 2
    assert call(n=-1) == 1 and call(H=-1) == 1 and call(K=1025) == 1
    assert call(axes=0) == 1 and call(axes=5, axis=16) == 1 and call(axes=2) == 1 and b"axis" in lib.bws_last_error()
    assert call(q=None) == 1 and call(k=None) == 1 and call(pos=None) == 1 and call(f=None) == 1
    assert call(q_out=None) == 1 and call(k_out=None) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(q=24) == 3 and call(k_out=8) == 3 and call(pos=18) == 3 and call(axis=2) == 3 and call(qw=6) == 3
    assert call(qr=252) == 3 and call(kh=60) == 3


def test_quantize4_by_hand():
    """Scale 1 for a largest magnitude of 6; middles go to the even code; zero, infinite and NaN 16s."""
    x = np.zeros((1, 80), dtype=np.float32)
    x[0, :16] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6]
    x[0, 33], x[0, 50], x[0, 64:] = np.inf, np.nan, 3e-4
    codes, scale = S.quantize4(x, np.ones(1))
    assert scale.tolist() == [[0x38, 0, 0x7E, 0x7F, 0]]      # 1, 0, 448, NaN, and 5e-5 below half of 2^-9
    got = F.e2m1_decode(Q.unpack_nibbles(codes))[0]
    assert got[:16].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -1, -2, -2, -4, -4, -6]
    assert got[33] == 6 and (got[np.arange(80) > 47] == 0).all()


def test_quantize4_scales_by_the_heads_number():
    """The nearest E4M3 number to amax / 6 / g; codes to the nearest of the grid."""
    rng = np.random.RandomState(1)
    x = rng.standard_normal((300, 2, 32)).astype(np.float32)
    g = np.array([0.37, 5.0], dtype=np.float32)
    codes, scale = S.quantize4(x, np.broadcast_to(g, (300, 2)))
    v = F.e2m1_decode(Q.unpack_nibbles(codes)) * np.repeat(F.e4m3_decode(scale), 16, -1) * g[None, :, None]
    d = np.repeat(F.e4m3_decode(scale), 16, -1) * g[None, :, None]
    # half the widest step (4 to 6), and what a largest value past 6 d is cut by: the scale is off by up to 2^-4
    assert (np.abs(v - x) <= d + 2.0 ** -4 * np.abs(x)).all()
    amax = np.abs(x.reshape(300, 2, 2, 16)).max(-1)
    assert (np.abs(F.e4m3_decode(scale) - amax / 6 / g[:, None]) <= np.maximum(2.0 ** -4 * F.e4m3_decode(scale), 2.0 ** -10)).all()


def test_attention4_by_hand():
    """Two tokens, one of them in a block that is not there for the second request."""
    k, v = np.zeros((2, 1, 16, 4)), np.zeros((2, 1, 16, 4))
    k[1, 0, 0, 0], v[1, 0, 0], v[1, 0, 1] = np.log(3.0), 1.0, 5.0
    q = np.zeros((3, 1, 4))
    q[..., 0] = 1.0
    out, lse, _ = S.attention4(q, k, v, np.array([[1], [7]]), [0, 2, 3], [2, 1], 1.0)
    assert np.allclose(out[0], 1.0) and np.allclose(out[1], 0.75 * 1 + 0.25 * 5) and (out[2] == 0).all()
    assert np.allclose(lse[:2, 0], [np.log(3.0), np.log(4.0)]) and lse[2, 0] == -np.inf


def test_norm_rotate_axes_by_hand():
    """A quarter turn by one axis, none by the other; and one axis as the plain rotation."""
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    y, _ = S.norm_rotate_axes(x, None, [[1], [0]], [0, 1, 0, 1], [np.pi / 2] * 4, 0.0, False)
    assert np.allclose(y[0, 0], [-5, 2, -7, 4, 1, 6, 3, 8])
    a, _ = S.norm_rotate_axes(x, np.ones(8), [[3]], None, [0.3, 0.2], 1e-6, True)
    b, _ = S.norm_rotate(x, np.ones(8), [3], [0.3, 0.2], 1e-6, True)
    assert np.array_equal(a, b)


def test_read4_by_hand():
    v = np.arange(2 * 16).reshape(2, 1, 16, 1) + 1.0
    out = S.read4(v, np.array([[1, -1], [0, 1]]), [15, 14], [1, 3, 7], 8)
    assert out[:, 0, 0].tolist() == [0, 32, 0, 15, 16, 17, 18, 0]


COUNTS_MODEL = r"""
#include <cstdio>
#include "device_counts.h"
static bws::DeviceCounts<4, 9> counts;
int main() {
  int bad = 0, asked = 0;
  auto ask = [&](int n) { return [&asked, n]() { ++asked; return n; }; };
  bad += counts.get(0, 8, ask(18)) != 18 || asked != 1;
  bad += counts.get(0, 8, ask(5)) != 18 || asked != 1;    // known
  bad += counts.get(1, 8, ask(7)) != 7 || asked != 2;     // another device's own
  bad += counts.get(0, 4, ask(36)) != 36 || asked != 3;   // another index
  bad += counts.get(0, 8, ask(5)) != 18 || counts.get(1, 8, ask(5)) != 7 || asked != 3;
  bad += counts.get(3, 2, ask(-1)) != 0 || asked != 4;    // failed: none, and asked again
  bad += counts.get(3, 2, ask(0)) != 0 || asked != 5;
  bad += counts.get(3, 2, ask(9)) != 0 || asked != 5;     // none is an answer too
  std::printf("%d\n", bad);
  return bad != 0;
}
"""


def test_counts_are_each_devices_own(tmp_path):
    """How many clusters run at once is asked for on every device, and again where the question failed."""
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_streaming_gb300", "csrc")
    (tmp_path / "counts.cpp").write_text(COUNTS_MODEL)
    subprocess.run(["g++", "-std=c++17", "-I", src, "-o", str(tmp_path / "counts"), str(tmp_path / "counts.cpp")], check=True)
    r = subprocess.run([str(tmp_path / "counts")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


SIXTH_MODEL = r"""
#include <cstdio>
#include <cstdint>
#include <cstring>
#include "kv4_cache.cuh"
int main() {
  int bad = 0;
  for (uint32_t b = 0; b < 0x7F80u; ++b) {   // every finite BF16 magnitude
    const uint32_t w = b << 16;
    float a;
    std::memcpy(&a, &w, 4);
    bad += bws::sixth_of(a) != a / 6.0f;
  }
  std::printf("%d\n", bad);
  return bad != 0;
}
"""


def test_sixth_is_the_quotients_rounding(tmp_path):
    """The write's product in place of a division by 6 gives the quotient's FP32 rounding of every BF16 magnitude."""
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_streaming_gb300", "csrc")
    (tmp_path / "sixth.cu").write_text(SIXTH_MODEL)
    r = subprocess.run([nvcc, "-std=c++17", "-O2", "-I", src, "-o", str(tmp_path / "sixth"), str(tmp_path / "sixth.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(tmp_path / "sixth")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
