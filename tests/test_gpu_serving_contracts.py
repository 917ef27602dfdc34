"""The serving entry points on the GPU at the edges of their contracts: lists and tables that run short, rows beyond
what a call takes, tokens far apart in weight, lengths near 2^31."""
import numpy as np
import pytest
import torch

from gpu_util import bws, device, f64, np_
from oracle import formats as F, serving as S
from test_gpu_serving import attention_case, check_append, check_plan, check_verify, freqs, gen, held, ints, make_cache, \
    rows, verify_case

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
