"""Python names of the serving step's entry points around the weight stream:
the 8-bit key/value cache, its block tables and writes, attention over it, and
the verification of drafted tokens (argument marshalling only; the contracts
are in include/bws.h)."""
import collections
import ctypes as C

import torch

from ._lib import BwsError, check, lib
from .api import _ptr, _stream, _ws


class _KvCache(C.Structure):
    """Mirror of struct bws_kv_cache."""
    _fields_ = [("n_blocks", C.c_int), ("n_kv_heads", C.c_int), ("block_tokens", C.c_int), ("head_dim", C.c_int),
                ("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("block_stride", C.c_size_t), ("head_stride", C.c_size_t)]


class _Qkv(C.Structure):
    """Mirror of struct bws_qkv."""
    _fields_ = [("q", C.c_void_p), ("q_row_stride", C.c_int64), ("q_head_stride", C.c_int64),
                ("k", C.c_void_p), ("k_row_stride", C.c_int64), ("k_head_stride", C.c_int64),
                ("v", C.c_void_p), ("v_row_stride", C.c_int64), ("v_head_stride", C.c_int64),
                ("n_rows", C.c_int), ("n_q_heads", C.c_int),
                ("positions", C.c_void_p), ("slots", C.c_void_p),
                ("q_weight", C.c_void_p), ("k_weight", C.c_void_p),
                ("inv_freq", C.c_void_p), ("rot", C.c_int), ("interleaved", C.c_int), ("eps", C.c_float)]


def _check(name, t, dtype, shape=None):
    """A contiguous CUDA tensor of `dtype` (and of `shape`, None = any size)."""
    if t is None or not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise BwsError(f"{name} must be a contiguous CUDA tensor of {dtype}")
    if shape is not None and (t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape))):
        raise BwsError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _check_heads(name, t, dim, rows=None):
    if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 3 or t.shape[2] != dim or t.stride(2) != 1:
        raise BwsError(f"{name} must be a CUDA bfloat16 tensor [rows, heads, {dim}] with a contiguous last dimension")
    if rows is not None and t.shape[0] != rows:
        raise BwsError(f"{name} has {t.shape[0]} rows, expected {rows}")


class KvCache:
    """A key/value cache in blocks of tokens, E4M3 codes with one power-of-two
    scale per (block, kv head) and side. k, v: uint8 [n_blocks, kv_heads,
    block_tokens, head_dim], a (block, head) contiguous, blocks and heads at
    any common strides (multiples of 16 bytes); k_scale, v_scale: fp32
    [n_blocks, kv_heads]. The tensors stay the caller's."""

    def __init__(self, k, v, k_scale, v_scale):
        if k.dtype != torch.uint8 or v.dtype != torch.uint8 or k.dim() != 4 or k.shape != v.shape or not k.is_cuda \
                or not v.is_cuda or k.stride() != v.stride():
            raise BwsError("k and v must be CUDA uint8 tensors [n_blocks, kv_heads, block_tokens, head_dim] of one "
                           "shape and one set of strides")
        n, h, b, d = k.shape
        if k.stride(3) != 1 or k.stride(2) != d:
            raise BwsError("the tokens of a (block, head) must be contiguous rows")
        _check("k_scale", k_scale, torch.float32, (n, h))
        _check("v_scale", v_scale, torch.float32, (n, h))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_blocks, self.kv_heads, self.block_tokens, self.head_dim = n, h, b, d
        # a dimension of one entry has no stride of its own
        head = k.stride(1) if h > 1 else b * d
        block = k.stride(0) if n > 1 else head * h
        self._struct = _KvCache(n, h, b, d, k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                block, head)
        self._at = C.addressof(self._struct)

    @classmethod
    def empty(cls, n_blocks, kv_heads, head_dim, block_tokens=64, device="cuda"):
        """A cache of its own memory: zero codes under scale 1."""
        k = torch.zeros((2, n_blocks, kv_heads, block_tokens, head_dim), dtype=torch.uint8, device=device)
        s = torch.ones((2, n_blocks, kv_heads), dtype=torch.float32, device=device)
        return cls(k[0], k[1], s[0], s[1])

    def dequantize(self, side):
        """The held values of 'k' or 'v' as fp32 (for inspection)."""
        codes, scale = (self.k, self.k_scale) if side == "k" else (self.v, self.v_scale)
        return codes.view(torch.float8_e4m3fn).float() * scale[:, :, None, None]


KvPlan = collections.namedtuple("KvPlan", "slots positions row_start kv_lens n_free status")


def kv_plan(seq_lens, new_lens, block_tokens, block_table, free_blocks, n_free, n_rows):
    """Block tables and slots of a step from request lengths (int32 CUDA
    tensors): block_table [requests, max_blocks] gains the blocks the new
    tokens need, from the end of free_blocks[:n_free]. Returns KvPlan(slots
    [n_rows], positions [n_rows], row_start [requests + 1], kv_lens
    [requests], n_free [1], status [1]: bits of bws_kv_plan_status)."""
    R = seq_lens.shape[0]
    i32 = torch.int32
    _check("seq_lens", seq_lens, i32, (R,))
    _check("new_lens", new_lens, i32, (R,))
    _check("block_table", block_table, i32, (R, None))
    _check("free_blocks", free_blocks, i32, (None,))
    _check("n_free", n_free, i32, (1,))
    if n_rows < 0:
        raise BwsError("n_rows must not be negative")
    # one allocation; each part starts on a 16-byte boundary
    a, b = (n_rows + 3) & ~3, (R + 4) & ~3
    buf = torch.empty(2 * a + 2 * b + 8, dtype=i32, device=seq_lens.device)
    at = buf.data_ptr()
    out = KvPlan(buf[:n_rows], buf[a:a + n_rows], buf[2 * a:2 * a + R + 1], buf[2 * a + b:2 * a + b + R],
                 buf[2 * a + 2 * b:2 * a + 2 * b + 1], buf[2 * a + 2 * b + 4:2 * a + 2 * b + 5])
    check(lib().bws_kv_plan(seq_lens.data_ptr(), new_lens.data_ptr(), R, block_tokens, block_table.data_ptr(),
                            block_table.shape[1], free_blocks.data_ptr(), n_free.data_ptr(), n_rows, at, at + 4 * a,
                            at + 8 * a, at + 8 * a + 4 * b, at + 8 * (a + b), at + 8 * (a + b) + 16,
                            _stream(seq_lens.device)), "bws_kv_plan")
    return out


def qk_norm_rope_append(q, k, v, positions, slots, cache, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
                        interleaved=False, q_out=None):
    """Per-head RMS norm (where a weight is given) and rotation of q and k by
    position, and the 8-bit write of k and v into the cache's slots. q bf16
    [rows, q_heads, dim], k, v bf16 [rows, kv_heads, dim], strided; inv_freq
    fp32 [rot / 2] or None (no rotation). Returns the queries, bf16 [rows,
    q_heads, dim]; the cache changes in place."""
    T, H, D = q.shape
    _check_heads("q", q, cache.head_dim)
    _check_heads("k", k, cache.head_dim, T)
    _check_heads("v", v, cache.head_dim, T)
    if k.shape[1] != cache.kv_heads or v.shape[1] != cache.kv_heads:
        raise BwsError(f"k and v must have the cache's {cache.kv_heads} heads")
    _check("positions", positions, torch.int32, (T,))
    _check("slots", slots, torch.int32, (T,))
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _check(name, w, torch.float32, (D,))
    if inv_freq is not None:
        _check("inv_freq", inv_freq, torch.float32, (None,))
    if q_out is None:
        q_out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
    else:
        _check("q_out", q_out, torch.bfloat16, (T, H, D))
    a = _Qkv(q.data_ptr(), q.stride(0), q.stride(1), k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
             v.stride(1), T, H, positions.data_ptr(), slots.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(inv_freq),
             0 if inv_freq is None else 2 * inv_freq.shape[0], int(interleaved), eps)
    check(lib().bws_qk_norm_rope_append(C.addressof(a), cache._at, q_out.data_ptr(), _stream(q.device)),
          "bws_qk_norm_rope_append")
    return q_out


def kv_attention_workspace_size(q_heads, kv_heads, head_dim, max_rows):
    return int(lib().bws_kv_attention_workspace_size(q_heads, kv_heads, head_dim, max_rows))


def kv_attention(q, cache, block_table, row_start, kv_lens, max_rows, scale=None, out=None, lse=False, ws=None):
    """Attention of each request's last row_start[r+1] - row_start[r] <=
    max_rows <= 8 tokens over the cache, causal among them. q bf16 [rows,
    q_heads, dim], strided; block_table int32 [requests, max_blocks],
    row_start int32 [requests + 1], kv_lens int32 [requests]; scale defaults
    to dim ** -0.5. Returns out bf16 [rows, q_heads, dim], and with lse=True
    also the fp32 [rows, q_heads] log-sum-exp of the scores."""
    T, H, D = q.shape
    _check_heads("q", q, cache.head_dim)
    R = kv_lens.shape[0]
    _check("block_table", block_table, torch.int32, (R, None))
    _check("row_start", row_start, torch.int32, (R + 1,))
    _check("kv_lens", kv_lens, torch.int32, (R,))
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
    else:
        _check("out", out, torch.bfloat16, (T, H, D))
    if lse is True:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    elif lse is not False:
        _check("lse", lse, torch.float32, (T, H))
    L = lib()
    buf = _ws(ws, L.bws_kv_attention_workspace_size(H, cache.kv_heads, D, max_rows), q.device)
    check(L.bws_kv_attention(q.data_ptr(), q.stride(0), q.stride(1), T, H, cache._at, block_table.data_ptr(),
                             block_table.shape[1], R, row_start.data_ptr(), kv_lens.data_ptr(), max_rows,
                             D ** -0.5 if scale is None else scale, out.data_ptr(),
                             None if lse is False else lse.data_ptr(), buf.data_ptr(), buf.numel(),
                             _stream(q.device)), "bws_kv_attention")
    return out if lse is False else (out, lse)


def draft_verify(target, tokens, row_start, accept_u, sample_u, max_rows, draft=None):
    """Which drafted tokens stand against the target's probabilities, and the
    token drawn after them, from given uniform numbers. target fp32 [rows,
    vocab]; draft fp32 [rows, vocab] or None (each draft was certain); tokens
    int32 [rows] (the last row of a request has no draft), accept_u fp32
    [rows], row_start int32 [requests + 1], sample_u fp32 [requests]. Returns
    (out int32 [requests, max_rows]: the drafts that stand, the drawn token,
    then -1; n_out int32 [requests])."""
    T, V = target.shape
    R = sample_u.shape[0]
    for name, t in (("target", target), ("draft", draft)):
        if t is not None and (not t.is_cuda or t.dtype != torch.float32 or tuple(t.shape) != (T, V)
                              or (t.stride(1) != 1 and V > 1)):
            raise BwsError(f"{name} must be a CUDA fp32 tensor [{T}, {V}] with a contiguous last dimension")
    _check("tokens", tokens, torch.int32, (T,))
    _check("accept_u", accept_u, torch.float32, (T,))
    _check("sample_u", sample_u, torch.float32, (R,))
    _check("row_start", row_start, torch.int32, (R + 1,))
    out = torch.empty((R, max_rows), dtype=torch.int32, device=target.device)
    n_out = torch.empty((R,), dtype=torch.int32, device=target.device)
    check(lib().bws_draft_verify(target.data_ptr(), max(target.stride(0), V), _ptr(draft),
                                 max(draft.stride(0), V) if draft is not None else 0, tokens.data_ptr(), T, V,
                                 row_start.data_ptr(), R, accept_u.data_ptr(), sample_u.data_ptr(), max_rows,
                                 out.data_ptr(), n_out.data_ptr(), _stream(target.device)), "bws_draft_verify")
    return out, n_out
