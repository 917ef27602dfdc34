"""The serving step around the weight stream in FP64 and plain loops: block
tables and slots, norm and rotation, the E4M3 cache, attention over it, and
the verification of drafted tokens."""
import numpy as np

from . import formats as F


def kv_plan(seq_lens, new_lens, block_tokens, table, free_blocks, n_free, n_rows):
    """(table, slots, positions, row_start, kv_lens, n_free, status) of a step."""
    table = np.array(table, dtype=np.int64)
    B, wide = block_tokens, table.shape[1]
    slots, positions = np.full(n_rows, -1), np.full(n_rows, -1)
    row_start, kv_lens, status, taken, t = [0], [], 0, 0, 0
    for r, (seq, new) in enumerate(zip(seq_lens, new_lens)):
        seq, new = max(int(seq), 0), max(int(new), 0)
        have, need = -(-seq // B), -(-(seq + new) // B)
        got = {}
        for c in range(have, min(need, wide)):   # a block that the table row cannot hold is not taken
            got[c] = int(free_blocks[n_free - 1 - taken]) if taken < n_free else -1
            if taken >= n_free:
                status |= 1
            taken += 1
            table[r, c] = got[c]
        if need > wide:
            status |= 2
        for j in range(new):
            pos = seq + j
            c = pos // B
            block = -1 if c >= wide else got.get(c, int(table[r, c]))
            if t < n_rows:
                positions[t] = pos
                slots[t] = block * B + pos % B if block >= 0 else -1
            else:
                status |= 4
            t += 1
        row_start.append(t)
        kv_lens.append(seq + new)
    return table, slots, positions, np.array(row_start), np.array(kv_lens), max(n_free - taken, 0), status


def norm_rotate(x, weight, positions, inv_freq, eps, interleaved):
    """Heads x [rows, heads, dim] normed (weight not None) and rotated; also
    |a| + |b| of each value's pair, the size its rounding errors go by."""
    y = np.array(x, dtype=np.float64)
    dim = y.shape[-1]
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    size = np.abs(y)
    half = len(inv_freq)
    i = np.arange(half)
    a_at, b_at = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    assert 2 * half <= dim
    turn = np.outer(np.asarray(positions, dtype=np.float64), np.asarray(inv_freq, dtype=np.float64))
    c, s = np.cos(turn)[:, None, :], np.sin(turn)[:, None, :]
    a, b = y[..., a_at].copy(), y[..., b_at].copy()
    y[..., a_at] = a * c - b * s
    y[..., b_at] = b * c + a * s
    size[..., a_at] = size[..., b_at] = np.abs(a) + np.abs(b)
    return y, size


def scale_for(amax):
    """The smallest 2^e, e in [-60, 60], with amax <= 448 * 2^e."""
    e = -60
    while e < 60 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def cache_append(codes, scale, rows, slots):
    """Writes rows [n, heads, dim] (FP64) into one side of a cache, in place:
    codes uint8 [blocks, heads, tokens, dim], scale fp32 [blocks, heads]."""
    n_blocks, heads, B, _ = codes.shape
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if s < 0 or s >= n_blocks * B:
            t += 1
            continue
        m = 1
        while t + m < len(slots) and (s % B) + m < B and slots[t + m] == s + m:
            m += 1
        blk, off = s // B, s % B
        for h in range(heads):
            x = rows[t:t + m, h]
            fin = np.abs(x[np.isfinite(x)])
            need = scale_for(fin.max() if fin.size else 0.0)
            old = float(scale[blk, h])
            new = need if off == 0 else max(old, need)
            if off and new != old:
                codes[blk, h, :off] = encode(F.e4m3_decode(codes[blk, h, :off]) * (old / new))
            codes[blk, h, off:off + m] = encode(x / new)
            scale[blk, h] = new
        t += m


def encode(v):
    """E4M3 codes, nearest even, saturating; NaN stays NaN."""
    v = np.asarray(v, dtype=np.float64)
    return np.where(np.isnan(v), np.uint8(0x7F), F.e4m3_encode(np.where(np.isnan(v), 0.0, v)))


def attention(q, k_codes, v_codes, k_scale, v_scale, table, row_start, kv_lens, scale):
    """(out, lse, terms): attention of each request's last rows, and per output
    the sizes its error is bounded by: sum p |v|, the largest score's absolute
    sum, the largest p * v_scale, and the tokens seen."""
    T, H, D = q.shape
    n_blocks, K, B, _ = k_codes.shape
    G = H // K
    out = np.zeros((T, H, D))
    lse = np.full((T, H), -np.inf)
    size = np.zeros((T, H, D))
    score = np.zeros((T, H))
    top = np.zeros((T, H))
    seen = np.zeros((T, H))
    for r, length in enumerate(kv_lens):
        a, b = int(row_start[r]), int(row_start[r + 1])
        length = max(int(length), 0)
        if b <= a:
            continue
        # what the table cannot hold is not there; the rows' sight goes by the length all the same
        toks = [t for t in range(min(length, table.shape[1] * B)) if 0 <= table[r, t // B] < n_blocks]
        blk = np.array([table[r, t // B] for t in toks], dtype=np.int64)
        at = np.array([t % B for t in toks], dtype=np.int64)
        toks = np.array(toks, dtype=np.int64)
        for h in range(K):
            k = F.e4m3_decode(k_codes[blk, h, at]) * k_scale[blk, h].astype(np.float64)[:, None]
            v = F.e4m3_decode(v_codes[blk, h, at]) * v_scale[blk, h].astype(np.float64)[:, None]
            vs = v_scale[blk, h].astype(np.float64)
            for j in range(b - a):
                ok = toks <= length - (b - a) + j
                if not ok.any():
                    continue
                for g in range(G):
                    x = q[a + j, h * G + g].astype(np.float64)
                    z = (k[ok] @ x) * scale
                    m = z.max()
                    e = np.exp(z - m)
                    p = e / e.sum()
                    i = (a + j, h * G + g)
                    out[i] = p @ v[ok]
                    lse[i] = m + np.log(e.sum())
                    size[i] = p @ np.abs(v[ok])
                    score[i] = (np.abs(k[ok]) @ np.abs(x)).max() * abs(scale)
                    top[i] = (p * vs[ok]).max()
                    seen[i] = ok.sum()
    return out, lse, (size, score, top, seen)


def draft_verify(target, tokens, row_start, accept_u, sample_u, max_rows, draft=None):
    """(out, n_out): the drafts that stand and the drawn token, request by request."""
    V = target.shape[1]
    out = np.full((len(sample_u), max_rows), -1, dtype=np.int64)
    n_out = np.zeros(len(sample_u), dtype=np.int64)
    for r, u in enumerate(sample_u):
        a, b = int(row_start[r]), int(row_start[r + 1])
        if b <= a:
            continue
        if b - a > max_rows:
            n_out[r] = -1
            continue
        i = a
        while i < b - 1:
            x = int(tokens[i])
            if not 0 <= x < V:
                break
            qx = 1.0 if draft is None else float(draft[i, x])
            if not float(accept_u[i]) * qx < float(target[i, x]):
                break
            out[r, i - a] = x
            i += 1
        def clean(w):
            return np.where(w > 0, w, np.float32(0))   # negative and NaN count as 0
        w = clean(target[i])
        if i < b - 1:
            if draft is not None:
                left = clean(target[i] - draft[i])     # both fp32: the difference rounds to fp32
            else:
                left = w.copy()
                if 0 <= tokens[i] < V:
                    left[int(tokens[i])] = 0
            if left.any():
                w = left
        c = np.cumsum(w.astype(np.float64))
        if c[-1] > 0:
            v = int(np.searchsorted(c, float(u) * c[-1], side="right"))
            out[r, i - a] = min(v, int(np.nonzero(w)[0][-1]))
        n_out[r] = i - a + 1
    return out, n_out
