"""The serving entry points on the CPU: their refusals, and the oracle's pieces
against hand-worked values (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import formats as F, serving as S


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    import bit_weight_streaming_gb300 as bws
    return bws.lib()


def cache(**kw):
    from bit_weight_streaming_gb300.serving import _KvCache
    v = dict(n_blocks=4, n_kv_heads=2, block_tokens=16, head_dim=64, k=4096, v=8192, k_scale=64, v_scale=128,
             block_stride=2048, head_stride=1024)
    v.update(kw)
    return _KvCache(*v.values())


def test_plan_refuses_lengths_in_place(lib):
    """CTAs read the lengths while another writes kv_lens."""
    def call(seq, new, kv):
        return lib.bws_kv_plan(seq, new, 1, 16, 16, 4, 16, 16, 8, 16, 16, 16, kv, 32, 16, None)

    for lens in ((64, 128, 64), (64, 128, 128)):
        assert call(*lens) == 1 and b"kv_lens" in lib.bws_last_error()


def test_plan_refusals(lib):
    f = lib.bws_kv_plan

    def call(seq=16, new=16, R=1, B=16, table=16, wide=4, free=16, n_free=16, rows=8, slots=16, pos=16, start=16, kv=16,
             out=32, status=16):
        return f(seq, new, R, B, table, wide, free, n_free, rows, slots, pos, start, kv, out, status, None)

    assert call(R=-1) == 1 and call(R=4097) == 1 and call(rows=-1) == 1 and call(wide=-1) == 1
    assert call(B=8) == 2 and call(B=24) == 2 and call(B=272) == 2 and call(B=0) == 2
    assert call(seq=None) == 1 and call(table=None) == 1 and call(slots=None) == 1 and call(status=None) == 1
    assert b"null" in lib.bws_last_error()
    assert call(out=16) == 1 and b"n_free_out" in lib.bws_last_error()
    assert call(seq=18) == 3 and call(status=17) == 3
    assert lib.bws_kv_plan_bounded(16, 16, 1, 16, 16, 4, 16, -1, 16, 8, 16, 16, 16, 16, 32, 16, None) == 1
    assert b"n_list" in lib.bws_last_error()


@pytest.mark.parametrize("bad,code", [
    (dict(head_dim=96), 2), (dict(head_dim=0), 2), (dict(block_tokens=8), 2), (dict(block_tokens=40), 2),
    (dict(block_tokens=512), 2), (dict(n_kv_heads=0), 2), (dict(n_kv_heads=129), 2), (dict(n_blocks=0), 2),
    (dict(n_blocks=1 << 28), 2), (dict(k=None), 1), (dict(v_scale=None), 1), (dict(k=4104), 3),
    (dict(k_scale=66), 3), (dict(block_stride=2056), 3), (dict(head_stride=512), 2), (dict(block_stride=1024), 2),
    (dict(block_stride=1 << 41), 2)])
def test_cache_refusals(lib, bad, code):
    from bit_weight_streaming_gb300.serving import _Qkv
    c = cache(**bad)
    a = _Qkv(16, 256, 64, 16, 128, 64, 16, 128, 64, 1, 4, 16, 16, None, None, 16, 64, 0, 1e-6)
    assert lib.bws_qk_norm_rope_append(ctypes.addressof(a), ctypes.addressof(c), 16, None) == code
    assert lib.bws_kv_attention(16, 256, 64, 1, 4, ctypes.addressof(c), 16, 4, 1, 16, 16, 1, 0.1, 16, None, 256,
                                1 << 40, None) == code


def test_append_refusals(lib):
    from bit_weight_streaming_gb300.serving import _Qkv
    c = cache()

    def call(out=16, **kw):
        v = dict(q=16, qr=256, qh=64, k=16, kr=128, kh=64, v=16, vr=128, vh=64, n=1, H=4, pos=16, slots=16, qw=None,
                 kw=None, f=16, rot=64, inter=0, eps=1e-6)
        v.update(kw)
        a = _Qkv(*v.values())
        return lib.bws_qk_norm_rope_append(ctypes.addressof(a), ctypes.addressof(c), out, None)

    assert lib.bws_qk_norm_rope_append(None, ctypes.addressof(c), 16, None) == 1
    assert call(n=0, q=None) == 0                      # nothing to do
    assert call(n=-1) == 1 and call(H=0) == 1 and call(H=2000) == 1
    assert call(rot=66) == 2 and call(rot=63) == 2 and call(rot=-2) == 2
    assert call(q=None) == 1 and call(slots=None) == 1 and call(f=None) == 1 and call(out=None) == 1
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(q=24) == 3 and call(kr=132) == 3 and call(pos=18) == 3 and call(qw=2) == 3 and call(out=8) == 3


def test_attention_refusals(lib):
    c = cache()

    def call(q=16, qr=256, qh=64, T=1, H=4, table=16, wide=4, R=1, start=16, kv=16, rows=1, scale=0.1, out=16, lse=None,
             ws=256, nbytes=1 << 40, at=None):
        return lib.bws_kv_attention(q, qr, qh, T, H, at or ctypes.addressof(c), table, wide, R, start, kv, rows, scale,
                                    out, lse, ws, nbytes, None)

    assert call(T=0, q=None) == 0 and call(R=0, kv=None) == 0
    assert call(rows=0) == 1 and call(rows=9) == 1 and call(T=-1) == 1 and call(R=-1) == 1 and call(wide=-1) == 1
    assert call(H=5) == 2 and call(H=34) == 2 and call(H=0) == 2
    assert call(wide=1 << 28) == 2
    assert call(q=None) == 1 and call(out=None) == 1 and call(table=None) == 1 and call(kv=None) == 1
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(q=8) == 3 and call(qr=260) == 3 and call(lse=2) == 3 and call(ws=272) == 3
    assert call(nbytes=1024) == 7 and call(ws=None) == 7
    size = lib.bws_kv_attention_workspace_size
    assert size(5, 2, 64, 1) == 0 and size(4, 2, 96, 1) == 0 and size(4, 2, 64, 9) == 0 and size(64, 2, 64, 1) == 0
    assert 0 < size(4, 4, 64, 1) <= size(64, 4, 64, 8)


def test_verify_refusals(lib):
    f = lib.bws_draft_verify

    def call(p=16, ps=64, q=None, qs=0, tok=16, T=2, V=64, start=16, R=1, au=16, su=16, rows=2, out=16, n=16):
        return f(p, ps, q, qs, tok, T, V, start, R, au, su, rows, out, n, None)

    assert call(R=0, p=None) == 0
    assert call(R=-1) == 1 and call(T=-1) == 1 and call(rows=0) == 1 and call(rows=33) == 1
    assert call(V=0) == 2 and call(V=1 << 29) == 2
    assert call(p=None) == 1 and call(su=None) == 1 and call(n=None) == 1
    assert call(ps=63) == 1 and call(q=16, qs=63) == 1
    assert call(p=18) == 3 and call(n=17) == 3


RING_MODEL = r"""
#include <cstdio>
#include "copy_ring.h"
using namespace bws;
// A barrier per stage counts the phases its landed uses completed; a wait on a parity passes when the phase of that
// parity is the last one completed.
int main() {
  int bad = 0;
  for (uint32_t n = 2; n <= 4; ++n)
    for (uint32_t started = 1; started < 40; ++started)
      for (uint32_t late = ring_oldest(started, n); late <= started; ++late) {   // the use that has not landed, if any
        uint32_t phase[4] = {0, 0, 0, 0};
        for (uint32_t it = 0; it < started; ++it)
          if (it != late) ++phase[ring_stage(it, n)];
        bool waited = false, seen[4] = {false, false, false, false};
        for (uint32_t it = ring_oldest(started, n); it < started; ++it) {
          const uint32_t s = ring_stage(it, n);
          const bool passes = (phase[s] & 1u) != ring_parity(it, n);
          bad += seen[s];                       // a stage is waited for once
          seen[s] = true;
          bad += passes != (it != late);        // what has landed passes, what has not is waited for
          waited |= !passes;
        }
        bad += waited != (late < started);
      }
  std::printf("%d\n", bad);
  return bad != 0;
}
"""


def test_copies_on_their_way(tmp_path):
    """A kernel that gives up a wait leaves only when its own copies have landed: it waits for the right phases."""
    import os
    import subprocess
    src = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_streaming_gb300", "csrc")
    (tmp_path / "ring.cpp").write_text(RING_MODEL)
    subprocess.run(["g++", "-std=c++17", "-I", src, "-o", str(tmp_path / "ring"), str(tmp_path / "ring.cpp")], check=True)
    r = subprocess.run([str(tmp_path / "ring")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_python_refuses_cpu_tensors():
    import torch
    import bit_weight_streaming_gb300 as bws
    k = torch.zeros((2, 1, 16, 64), dtype=torch.uint8)
    s = torch.ones((2, 1))
    with pytest.raises(bws.BwsError):
        bws.KvCache(k, k, s, s)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(bws.BwsError):
        bws.kv_plan(i, i, 16, torch.zeros((1, 4), dtype=torch.int32), i, i, 4)


def test_python_refuses_overlapping_rows():
    """A broadcast matrix is one row of memory: taken for a row each, its rows would be read past the end of it."""
    import torch
    import bit_weight_streaming_gb300 as bws
    p, one = torch.zeros((5, 100)), torch.zeros((1, 100))
    i, u = torch.zeros(5, dtype=torch.int32), torch.zeros(5)
    start = torch.tensor([0, 5], dtype=torch.int32)
    for target, draft in ((p, one.expand(5, 100)), (one.expand(5, 100), None), (p.view(-1).as_strided((5, 100), (60, 1)), p)):
        with pytest.raises(bws.BwsError, match="lie (0|60) apart"):
            bws.draft_verify(target, i, start, u, u[:1], 5, draft=draft)
    with pytest.raises(bws.BwsError, match="last dimension"):
        bws.draft_verify(torch.zeros((100, 5)).t(), i, start, u, u[:1], 5)
    from bit_weight_streaming_gb300.serving import _row_stride
    assert _row_stride("p", p) == 100 and _row_stride("p", p[::2]) == 200 and _row_stride("p", p[:, 3:90]) == 100
    assert _row_stride("p", one.expand(1, 100)) == 100 and _row_stride("p", one.as_strided((1, 100), (7, 1))) == 100
    assert _row_stride("p", torch.zeros((0, 100))) == 100 and _row_stride("p", torch.zeros((5, 1))) == 1
    with pytest.raises(bws.BwsError):
        _row_stride("p", torch.zeros((1, 1)).expand(5, 1))


def test_oracle_scale():
    assert S.scale_for(448.0) == 1.0 and S.scale_for(448.5) == 2.0 and S.scale_for(224.0) == 0.5
    assert S.scale_for(0.0) == 2.0 ** -60 and S.scale_for(1e30) == 2.0 ** 60


def test_oracle_plan_by_hand():
    # 16-token blocks; one request at 15 tokens gains 2: its second block, the list's last
    t, slots, pos, start, kv, n, st = S.kv_plan([15, 0], [2, 1], 16, [[7, -1], [-1, -1]], [3, 4, 5], 3, 4)
    assert t.tolist() == [[7, 5], [4, -1]]
    assert slots.tolist() == [7 * 16 + 15, 5 * 16, 4 * 16, -1] and pos.tolist() == [15, 16, 0, -1]
    assert start.tolist() == [0, 2, 3] and kv.tolist() == [17, 1] and n == 1 and st == 0


def test_oracle_plan_loses_no_block():
    # the first request's row holds two of the five blocks it needs: three stay free, and the second gets its own
    t, slots, _, _, kv, n, st = S.kv_plan([0, 0], [80, 16], 16, [[-1, -1], [-1, -1]], list(range(8)), 8, 96)
    assert t.tolist() == [[7, 6], [5, -1]] and n == 5 and st == 2 and kv.tolist() == [80, 16]
    assert (slots[:32] >= 0).all() and (slots[32:80] == -1).all() and slots[80:].tolist() == list(range(80, 96))


def test_oracle_append_grows_and_rounds_again():
    codes = np.zeros((1, 1, 16, 64), dtype=np.uint8)
    scale = np.ones((1, 1), dtype=np.float32)
    x = np.zeros((1, 1, 64))
    x[0, 0, 0], x[0, 0, 1] = 448.0, 2.0 ** -9
    S.cache_append(codes, scale, x, [0])
    assert scale[0, 0] == 1.0 and F.e4m3_decode(codes[0, 0, 0])[:2].tolist() == [448.0, 2.0 ** -9]
    S.cache_append(codes, scale, 4 * x, [1])
    assert scale[0, 0] == 4.0
    assert (F.e4m3_decode(codes[0, 0, 0])[:2] * 4).tolist() == [448.0, 0.0]     # the smallest is rounded away
    S.cache_append(codes, scale, x / 8, [0])                                    # the block starts anew
    assert scale[0, 0] == 0.125


def test_oracle_attention_closed_form():
    # equal scores: the mean of the values seen; an empty request gives zeros
    k = np.zeros((2, 1, 16, 64), dtype=np.uint8)
    v = np.zeros((2, 1, 16, 64), dtype=np.uint8)
    v[1, 0, :3] = F.e4m3_encode(np.array([1.0, 2.0, 4.0]))[:, None]
    s = np.ones((2, 1), dtype=np.float32)
    out, lse, _ = S.attention(np.ones((3, 1, 64)), k, v, s, s, np.array([[1], [0]]), [0, 2, 3], [3, 0], 0.125)
    assert np.allclose(out[0], 1.5) and np.allclose(out[1], 7 / 3) and (out[2] == 0).all()
    assert np.allclose(lse[:2, 0], [np.log(2), np.log(3)]) and lse[2, 0] == -np.inf


def test_oracle_attention_longer_than_its_table():
    # 40 tokens of which the table holds 32: both rows see all 32, the last token's value among equal scores too
    k = np.zeros((2, 1, 16, 64), dtype=np.uint8)
    v = np.zeros((2, 1, 16, 64), dtype=np.uint8)
    v[1, 0, 15] = F.e4m3_encode(np.array([448.0]))
    s = np.ones((2, 1), dtype=np.float32)
    out, lse, _ = S.attention(np.ones((2, 1, 64)), k, v, s, s, np.array([[0, 1]]), [0, 2], [40], 0.125)
    assert np.allclose(out, 14.0) and np.allclose(lse, np.log(32))


def test_oracle_verify_draws_the_target():
    """Speculative sampling leaves the target's distribution: counted over a grid of uniform numbers."""
    p = np.array([[0.5, 0.25, 0.25], [1, 0, 0]], dtype=np.float32)
    q = np.array([[0.125, 0.625, 0.25], [1, 0, 0]], dtype=np.float32)
    got = np.zeros(3)
    n = 32
    for x in range(3):
        for a in range(n):
            for b in range(n):
                out, k = S.draft_verify(p, [x, 0], [0, 2], [(a + 0.5) / n, 0], [(b + 0.5) / n], 2, q)
                got[out[0, 0]] += q[0, x] / (n * n)
    # counting a threshold on n points is off by at most half a point: of the acceptance, and of the draw
    assert np.abs(got - p[0]).max() <= q[0].sum() * 0.5 / n + 1e-6
