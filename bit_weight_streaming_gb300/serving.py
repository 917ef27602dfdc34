"""Python names of the serving step's entry points around the weight stream:
the 8-bit and the 4-bit key/value cache, their block tables and writes, attention
over them, and the verification of drafted tokens (argument marshalling only;
the contracts are in include/bws.h)."""
import collections
import ctypes as C
import math

import torch

from ._lib import BwsError, check, lib
from .api import _ws


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


class _Qk(C.Structure):
    """Mirror of struct bws_qk."""
    _fields_ = [("q", C.c_void_p), ("q_row_stride", C.c_int64), ("q_head_stride", C.c_int64),
                ("k", C.c_void_p), ("k_row_stride", C.c_int64), ("k_head_stride", C.c_int64),
                ("n_rows", C.c_int), ("n_q_heads", C.c_int), ("n_k_heads", C.c_int), ("head_dim", C.c_int),
                ("positions", C.c_void_p), ("n_axes", C.c_int), ("axis", C.c_void_p),
                ("q_weight", C.c_void_p), ("k_weight", C.c_void_p),
                ("inv_freq", C.c_void_p), ("rot", C.c_int), ("interleaved", C.c_int), ("eps", C.c_float)]


class _Kv4Cache(C.Structure):
    """Mirror of struct bws_kv4_cache."""
    _fields_ = [("n_blocks", C.c_int), ("n_kv_heads", C.c_int), ("block_tokens", C.c_int), ("head_dim", C.c_int),
                ("k", C.c_void_p), ("v", C.c_void_p), ("k_scale", C.c_void_p), ("v_scale", C.c_void_p),
                ("k_global", C.c_void_p), ("v_global", C.c_void_p),
                ("block_stride", C.c_size_t), ("head_stride", C.c_size_t),
                ("scale_block_stride", C.c_size_t), ("scale_head_stride", C.c_size_t)]


# The current stream's handle from a device index, without the stream object
# torch.cuda.current_stream builds (2 us of a call's 10).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)

_I32, _F32, _BF16, _U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8


def _check(name, t, dtype, shape):
    """A contiguous CUDA tensor of `dtype` and `shape`."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        raise BwsError(f"{name} must be a contiguous CUDA tensor of {dtype}, shape {tuple(shape)}; it is {t.dtype}, "
                       f"{tuple(t.shape)} on {t.device}")


def _check_heads(name, t, rows, heads, dim):
    if t.dtype is not _BF16 or t.shape != (rows, heads, dim) or not t.is_cuda:
        raise BwsError(f"{name} must be a CUDA bfloat16 tensor [{rows}, {heads}, {dim}]; it is {t.dtype}, "
                       f"{tuple(t.shape)} on {t.device}")
    row, head, one = t.stride()
    if one != 1:
        raise BwsError(f"{name} must be contiguous in its last dimension")
    # a dimension of one entry has no stride of its own
    return row if rows > 1 else 0, head if heads > 1 else 0


def _row_stride(name, t):
    """Elements from row to row of a matrix whose rows may lie apart but not on each other (as expand() makes them)."""
    rows, wide = t.shape
    if t.stride(1) != 1 and wide > 1:
        raise BwsError(f"{name} must be contiguous in its last dimension")
    if rows <= 1:
        return wide               # one row has no stride of its own
    if t.stride(0) < wide:
        raise BwsError(f"{name}'s rows of {wide} lie {t.stride(0)} apart: they must not overlap (a broadcast matrix "
                       "needs contiguous())")
    return t.stride(0)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(device, f, *args):
    """f(*args) with the CUDA device of index `device` current."""
    if _current_device() == device:
        return f(*args)
    with torch.cuda.device(device):
        return f(*args)


def _fail(rc, what):
    if rc:
        check(rc, what)


class KvCache:
    """A key/value cache in blocks of tokens, E4M3 codes with one power-of-two
    scale per (block, kv head) and side. k, v: uint8 [n_blocks, kv_heads,
    block_tokens, head_dim], a (block, head) contiguous, blocks and heads at
    any common strides (multiples of 16 bytes); k_scale, v_scale: fp32
    [n_blocks, kv_heads]. The tensors stay the caller's."""

    def __init__(self, k, v, k_scale, v_scale):
        if k.dtype != _U8 or v.dtype != _U8 or k.dim() != 4 or k.shape != v.shape or not k.is_cuda \
                or not v.is_cuda or k.stride() != v.stride():
            raise BwsError("k and v must be CUDA uint8 tensors [n_blocks, kv_heads, block_tokens, head_dim] of one "
                           "shape and one set of strides")
        n, h, b, d = k.shape
        if k.stride(3) != 1 or k.stride(2) != d:
            raise BwsError("the tokens of a (block, head) must be contiguous rows")
        _check("k_scale", k_scale, _F32, (n, h))
        _check("v_scale", v_scale, _F32, (n, h))
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_blocks, self.kv_heads, self.block_tokens, self.head_dim = n, h, b, d
        # a dimension of one entry has no stride of its own
        head = k.stride(1) if h > 1 else b * d
        block = k.stride(0) if n > 1 else head * h
        self._struct = _KvCache(n, h, b, d, k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                block, head)
        self._at = C.addressof(self._struct)
        self._attn_ws = {}      # workspace bytes by (query heads, rows)

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
    R, wide = block_table.shape
    one = (R,)
    _check("seq_lens", seq_lens, _I32, one)
    _check("new_lens", new_lens, _I32, one)
    _check("block_table", block_table, _I32, (R, wide))
    _check("free_blocks", free_blocks, _I32, (free_blocks.numel(),))
    _check("n_free", n_free, _I32, (1,))
    if n_rows < 0:
        raise BwsError("n_rows must not be negative")
    # a tensor each: views of one cost more than the allocator
    dev = seq_lens.device
    slots = torch.empty(n_rows, dtype=_I32, device=dev)
    positions = torch.empty_like(slots)
    row_start = torch.empty(R + 1, dtype=_I32, device=dev)
    kv_lens = torch.empty_like(seq_lens)
    n_out = torch.empty_like(n_free)
    status = torch.empty_like(n_free)
    _fail(lib().bws_kv_plan_bounded(seq_lens.data_ptr(), new_lens.data_ptr(), R, block_tokens, block_table.data_ptr(),
                                    wide, free_blocks.data_ptr(), free_blocks.numel(), n_free.data_ptr(), n_rows,
                                    slots.data_ptr(), positions.data_ptr(), row_start.data_ptr(), kv_lens.data_ptr(),
                                    n_out.data_ptr(), status.data_ptr(), _raw_stream(seq_lens.get_device())),
          "bws_kv_plan")
    return KvPlan(slots, positions, row_start, kv_lens, n_out, status)


def qk_norm_rope_append(q, k, v, positions, slots, cache, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
                        interleaved=False, q_out=None):
    """Per-head RMS norm (where a weight is given) and rotation of q and k by
    position, and the 8-bit write of k and v into the cache's slots. q bf16
    [rows, q_heads, dim], k, v bf16 [rows, kv_heads, dim], strided; inv_freq
    fp32 [rot / 2] or None (no rotation). Returns the queries, bf16 [rows,
    q_heads, dim]; the cache changes in place."""
    T, H, D = q.shape
    K = cache.kv_heads
    q_row, q_head = _check_heads("q", q, T, H, cache.head_dim)
    k_row, k_head = _check_heads("k", k, T, K, D)
    v_row, v_head = _check_heads("v", v, T, K, D)
    one = (T,)
    _check("positions", positions, _I32, one)
    _check("slots", slots, _I32, one)
    qw = kw = f = None
    rot = 0
    if q_weight is not None:
        _check("q_weight", q_weight, _F32, (D,))
        qw = q_weight.data_ptr()
    if k_weight is not None:
        _check("k_weight", k_weight, _F32, (D,))
        kw = k_weight.data_ptr()
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        _check("inv_freq", inv_freq, _F32, (rot // 2,))
        f = inv_freq.data_ptr()
    if q_out is None:
        q_out = torch.empty((T, H, D), dtype=_BF16, device=q.device)
    else:
        _check("q_out", q_out, _BF16, (T, H, D))
    a = _Qkv(q.data_ptr(), q_row, q_head, k.data_ptr(), k_row, k_head, v.data_ptr(), v_row, v_head, T, H,
             positions.data_ptr(), slots.data_ptr(), qw, kw, f, rot, interleaved, eps)
    _fail(lib().bws_qk_norm_rope_append(C.addressof(a), cache._at, q_out.data_ptr(), _raw_stream(q.get_device())),
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
    also the fp32 [rows, q_heads] log-sum-exp of the scores. Rows of no request
    are zero (-inf), as are a request's past max_rows, which the workspace's
    status word reports."""
    T, H, D = q.shape
    row, head = _check_heads("q", q, T, H, cache.head_dim)
    R, wide = block_table.shape
    _check("block_table", block_table, _I32, (R, wide))
    _check("row_start", row_start, _I32, (R + 1,))
    _check("kv_lens", kv_lens, _I32, (R,))
    if out is None:
        out = torch.empty((T, H, D), dtype=_BF16, device=q.device)
    else:
        _check("out", out, _BF16, (T, H, D))
    if lse is False:
        lse_at = None
    else:
        if lse is True:
            lse = torch.empty((T, H), dtype=_F32, device=q.device)
        else:
            _check("lse", lse, _F32, (T, H))
        lse_at = lse.data_ptr()
    if R == 0:     # every row is one of no request
        out.zero_()
        if lse_at is not None:
            lse.fill_(-math.inf)
        return out if lse_at is None else (out, lse)
    so = lib()
    size = cache._attn_ws.get((H, max_rows))
    if size is None:
        size = cache._attn_ws[H, max_rows] = _on(q.get_device(), kv_attention_workspace_size, H, cache.kv_heads, D, max_rows)
    buf = _ws(ws, size, q.device)
    if not buf.is_cuda or buf.dtype is not _U8:
        raise BwsError(f"the workspace must be CUDA uint8 memory; it is {buf.dtype} on {buf.device}")
    _fail(so.bws_kv_attention(q.data_ptr(), row, head, T, H, cache._at, block_table.data_ptr(), wide, R,
                              row_start.data_ptr(), kv_lens.data_ptr(), max_rows, D ** -0.5 if scale is None else scale,
                              out.data_ptr(), lse_at, buf.data_ptr(), buf.numel(), _raw_stream(q.get_device())),
          "bws_kv_attention")
    return out if lse_at is None else (out, lse)


# ---- the 4-bit cache ---------------------------------------------------------------

def _call(what, device, f, *args):
    """f(*args, stream) on the tensors' device, whichever is current."""
    rc = _on(device, f, *args, _raw_stream(device))
    if rc:
        check(rc, what)


def _need(name, t, dtype, shape, device):
    """The address of a contiguous tensor of `dtype` and `shape` on the CUDA device of index `device`."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise BwsError(f"{name} must be a contiguous tensor of {dtype}, shape {tuple(shape)}, on cuda:{device}; it is "
                       f"{t.dtype}, {tuple(t.shape)}, strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _need_heads(name, t, shape, device):
    """Row and head strides of BF16 heads of `shape` on the device."""
    if t.dtype is not _BF16 or t.shape != shape or t.get_device() != device:
        raise BwsError(f"{name} must be a bfloat16 tensor {list(shape)} on cuda:{device}; it is {t.dtype}, "
                       f"{tuple(t.shape)} on {t.device}")
    row, head, one = t.stride()
    if one != 1:
        raise BwsError(f"{name} must be contiguous in its last dimension")
    # a dimension of one entry has no stride of its own
    return row if shape[0] > 1 else 0, head if shape[1] > 1 else 0


def _side_strides(name, t, wide):
    """Bytes from block to block and from head to head of an array whose (block, head)s are rows of `wide` bytes."""
    n, h, b, _ = t.shape
    if t.stride(3) != 1 or t.stride(2) != wide:
        raise BwsError(f"{name}: the tokens of a (block, head) must be contiguous rows")
    head = t.stride(1) if h > 1 else b * wide     # a dimension of one entry has no stride of its own
    return t.stride(0) if n > 1 else head * h, head


class Kv4Cache:
    """A key/value cache in blocks of tokens held in 4 bits: E2M1 codes, two a
    byte, an E4M3 scale for every 16 dimensions of a token's head, an fp32 number
    for every head and side. k, v: uint8 [n_blocks, kv_heads, block_tokens,
    head_dim / 2]; k_scale, v_scale: uint8 [n_blocks, kv_heads, block_tokens,
    head_dim / 16]; a (block, head) contiguous, blocks and heads at any strides
    common to k and v (multiples of 16 bytes); k_global, v_global: fp32 [kv_heads],
    positive, or None (1). The tensors stay the caller's."""

    def __init__(self, k, v, k_scale, v_scale, k_global=None, v_global=None):
        for a, b, name in ((k, v, "k and v"), (k_scale, v_scale, "k_scale and v_scale")):
            if a.dtype is not _U8 or b.dtype is not _U8 or a.dim() != 4 or a.shape != b.shape or not a.is_cuda \
                    or not b.is_cuda or a.stride() != b.stride():
                raise BwsError(f"{name} must be CUDA uint8 tensors of four dimensions, one shape and one set of strides")
        n, h, b, half = k.shape
        if k_scale.shape != (n, h, b, half // 8):
            raise BwsError(f"k_scale and v_scale must be [{n}, {h}, {b}, {half // 8}]: a scale for every 8 bytes of codes")
        self.device_index = k.get_device()
        for name, t in (("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if t.get_device() != self.device_index:
                raise BwsError(f"{name} is on {t.device}, k on {k.device}")
        at = lambda name, t: None if t is None else _need(name, t, _F32, (h,), self.device_index)  # noqa: E731
        k_at, v_at = at("k_global", k_global), at("v_global", v_global)
        self.k, self.v, self.k_scale, self.v_scale, self.k_global, self.v_global = k, v, k_scale, v_scale, k_global, v_global
        self.n_blocks, self.kv_heads, self.block_tokens, self.head_dim = n, h, b, 2 * half
        block, head = _side_strides("k and v", k, half)
        scale_block, scale_head = _side_strides("k_scale and v_scale", k_scale, half // 8)
        self._struct = _Kv4Cache(n, h, b, 2 * half, k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                 k_at, v_at, block, head, scale_block, scale_head)
        self._at = C.addressof(self._struct)
        self._attn_ws = {}      # workspace bytes by (query heads, rows)

    @classmethod
    def empty(cls, n_blocks, kv_heads, head_dim, block_tokens=64, device="cuda", k_global=None, v_global=None):
        """A cache of its own memory: zero codes under zero scales."""
        k = torch.zeros((2, n_blocks, kv_heads, block_tokens, head_dim // 2), dtype=torch.uint8, device=device)
        s = torch.zeros((2, n_blocks, kv_heads, block_tokens, head_dim // 16), dtype=torch.uint8, device=device)
        return cls(k[0], k[1], s[0], s[1], k_global, v_global)

    def dequantize(self, side):
        """The held values of 'k' or 'v' as fp32 [n_blocks, kv_heads, block_tokens, head_dim] (for inspection)."""
        codes, scale, g = (self.k, self.k_scale, self.k_global) if side == "k" else (self.v, self.v_scale, self.v_global)
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        x = torch.cat((grid, -grid))[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
        x = (x.unflatten(-1, (-1, 16)) * scale.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)
        return x if g is None else x * g[:, None, None]


def qk_norm_rope(q, k, positions, inv_freq=None, axis=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                 q_out=None, k_out=None):
    """Per-head RMS norm (where a weight is given) of q and k and their rotation
    by positions of several axes, apart from any cache. q bf16 [rows, q_heads,
    dim], k bf16 [rows, k_heads, dim], strided; positions int32 [rows], or [axes,
    rows] (up to four) with axis int32 [rot / 2], the axis by which each pair
    turns; inv_freq fp32 [rot / 2] or None (no rotation). Returns (q, k) as bf16
    [rows, heads, dim]; q_out and k_out may be contiguous q and k themselves."""
    T, H, D = shape = q.shape
    device = q.get_device()
    if device < 0 or k.dim() != 3:
        raise BwsError(f"q and k must be CUDA tensors [rows, heads, dim]; they are on {q.device} and of {k.dim()} dimensions")
    q_row, q_head = _need_heads("q", q, shape, device)
    K = k.shape[1]
    k_shape = (T, K, D)
    k_row, k_head = _need_heads("k", k, k_shape, device)
    rot, axes, f, ax, pos, qw, kw = 0, 1, None, None, None, None, None
    if inv_freq is not None:
        half = inv_freq.numel()
        f = _need("inv_freq", inv_freq, _F32, (half,), device)
        rot = 2 * half
        if positions.dim() == 2:
            axes = positions.shape[0]
            pos = _need("positions", positions, _I32, (axes, T), device)
        else:
            pos = _need("positions", positions, _I32, (T,), device)
        if axis is not None:
            ax = _need("axis", axis, _I32, (half,), device)
    if q_weight is not None:
        qw = _need("q_weight", q_weight, _F32, (D,), device)
    if k_weight is not None:
        kw = _need("k_weight", k_weight, _F32, (D,), device)
    if q_out is None:
        q_out = torch.empty(shape, dtype=_BF16, device=q.device)
    else:
        _need("q_out", q_out, _BF16, shape, device)
    if k_out is None:
        k_out = torch.empty(k_shape, dtype=_BF16, device=q.device)
    else:
        _need("k_out", k_out, _BF16, k_shape, device)
    a = _Qk(q.data_ptr(), q_row, q_head, k.data_ptr(), k_row, k_head, T, H, K, D, pos, axes, ax, qw, kw, f, rot,
            interleaved, eps)
    _call("bws_qk_norm_rope", device, lib().bws_qk_norm_rope, C.addressof(a), q_out.data_ptr(), k_out.data_ptr())
    return q_out, k_out


def kv4_append(k, v, slots, cache):
    """Writes k and v, bf16 [rows, kv_heads, dim], strided, into the slots (int32
    [rows], as kv_plan gives them) of a Kv4Cache, which changes in place. Every
    token's head gets scales of its own, so rows may come in any order, each with a
    slot of its own; a slot < 0 or past the cache is skipped."""
    device = cache.device_index
    shape = (slots.shape[0], cache.kv_heads, cache.head_dim)
    k_row, k_head = _need_heads("k", k, shape, device)
    v_row, v_head = _need_heads("v", v, shape, device)
    at = _need("slots", slots, _I32, shape[:1], device)
    _call("bws_kv4_append", device, lib().bws_kv4_append, k.data_ptr(), k_row, k_head, v.data_ptr(), v_row, v_head, at,
          shape[0], cache._at)


def kv4_read(cache, block_table, first, row_start, n_rows, k_out=None, v_out=None):
    """Reads tokens back from a Kv4Cache: row row_start[r] + j becomes token
    first[r] + j of request r. block_table int32 [requests, max_blocks], first
    int32 [requests], row_start int32 [requests + 1]. Returns (k, v), bf16
    [n_rows, kv_heads, dim]; tokens that no block holds and rows of no request are
    zero."""
    device = cache.device_index
    R, wide = block_table.shape
    table = _need("block_table", block_table, _I32, (R, wide), device)
    first_at = _need("first", first, _I32, (R,), device)
    start = _need("row_start", row_start, _I32, (R + 1,), device)
    if n_rows < 0:
        raise BwsError("n_rows must not be negative")
    shape = (n_rows, cache.kv_heads, cache.head_dim)
    if k_out is None:
        k_out = torch.empty(shape, dtype=_BF16, device=block_table.device)
    else:
        _need("k_out", k_out, _BF16, shape, device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=_BF16, device=block_table.device)
    else:
        _need("v_out", v_out, _BF16, shape, device)
    if R == 0:     # every row is one of no request
        return k_out.zero_(), v_out.zero_()
    _call("bws_kv4_read", device, lib().bws_kv4_read, cache._at, table, wide, R, first_at, start, n_rows,
          k_out.data_ptr(), v_out.data_ptr())
    return k_out, v_out


def kv4_attention_workspace_size(q_heads, kv_heads, head_dim, max_rows):
    return int(lib().bws_kv4_attention_workspace_size(q_heads, kv_heads, head_dim, max_rows))


def kv4_attention(q, cache, block_table, row_start, kv_lens, max_rows, scale=None, out=None, lse=False, ws=None):
    """kv_attention over a Kv4Cache: the same arguments, results and status."""
    T, H, D = shape = q.shape
    device = cache.device_index
    if D != cache.head_dim:
        raise BwsError(f"q's heads are of {D} dimensions, the cache's of {cache.head_dim}")
    row, head = _need_heads("q", q, shape, device)
    R, wide = block_table.shape
    table = _need("block_table", block_table, _I32, (R, wide), device)
    start = _need("row_start", row_start, _I32, (R + 1,), device)
    lens = _need("kv_lens", kv_lens, _I32, (R,), device)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=q.device)
    else:
        _need("out", out, _BF16, shape, device)
    lse_at = None
    if lse is True:
        lse = torch.empty((T, H), dtype=_F32, device=q.device)
        lse_at = lse.data_ptr()
    elif lse is not False:
        lse_at = _need("lse", lse, _F32, (T, H), device)
    if R == 0:     # every row is one of no request
        out.zero_()
        if lse_at is not None:
            lse.fill_(-math.inf)
        return out if lse_at is None else (out, lse)
    so = lib()
    size = cache._attn_ws.get((H, max_rows))
    if size is None:
        size = cache._attn_ws[H, max_rows] = _on(device, kv4_attention_workspace_size, H, cache.kv_heads, D, max_rows)
    buf = _ws(ws, size, q.device)
    if buf.dtype is not _U8 or buf.get_device() != device:
        raise BwsError(f"the workspace must be uint8 memory on cuda:{device}; it is {buf.dtype} on {buf.device}")
    _call("bws_kv4_attention", device, so.bws_kv4_attention, q.data_ptr(), row, head, T, H, cache._at, table, wide, R,
          start, lens, max_rows, D ** -0.5 if scale is None else scale, out.data_ptr(), lse_at, buf.data_ptr(),
          buf.numel())
    return out if lse_at is None else (out, lse)


def draft_verify(target, tokens, row_start, accept_u, sample_u, max_rows, draft=None):
    """Which drafted tokens stand against the target's probabilities, and the
    token drawn after them, from given uniform numbers. target fp32 [rows,
    vocab]; draft fp32 [rows, vocab] or None (each draft was certain), rows of
    both at any stride of vocab or more; tokens int32 [rows] (the last row of
    a request has no draft), accept_u fp32 [rows], row_start int32
    [requests + 1], sample_u fp32 [requests]. Returns (out int32 [requests,
    max_rows]: the drafts that stand, the drawn token, then -1; n_out int32
    [requests], -1 for a request of more than max_rows rows)."""
    T, V = target.shape
    R = sample_u.shape[0]
    target_stride = _row_stride("target", target)
    draft_stride = 0
    if draft is not None:
        if draft.shape != (T, V):
            raise BwsError(f"draft must have target's shape [{T}, {V}]; it is {tuple(draft.shape)}")
        draft_stride = _row_stride("draft", draft)
    for t in (target, draft):
        if t is not None and (t.dtype is not _F32 or not t.is_cuda):
            raise BwsError(f"target and draft must be CUDA fp32 tensors; one is {t.dtype} on {t.device}")
    rows = (T,)
    _check("tokens", tokens, _I32, rows)
    _check("accept_u", accept_u, _F32, rows)
    _check("sample_u", sample_u, _F32, (R,))
    _check("row_start", row_start, _I32, (R + 1,))
    if max_rows < 1:
        raise BwsError("max_rows must be positive")
    out = torch.empty((R, max_rows), dtype=_I32, device=target.device)
    n_out = torch.empty_like(sample_u, dtype=_I32)
    _fail(lib().bws_draft_verify(target.data_ptr(), target_stride, None if draft is None else draft.data_ptr(),
                                 draft_stride, tokens.data_ptr(), T, V, row_start.data_ptr(), R, accept_u.data_ptr(),
                                 sample_u.data_ptr(), max_rows, out.data_ptr(), n_out.data_ptr(),
                                 _raw_stream(target.get_device())), "bws_draft_verify")
    return out, n_out
