"""Attention over 4-bit caches when tokens past a query's position, but inside
the sequence's length, were never written: their tiles may hold any bytes."""

import numpy as np
import pytest
import torch

import q4_reference as R
from test_gpu_q4 import Case, ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bound", [0, 5000])
@pytest.mark.parametrize("nq,nkv,d", [(8, 2, 64), (16, 2, 128), (5, 1, 128), (12, 2, 64)])
@pytest.mark.parametrize("new", [1, 2, 40])
def test_unwritten_tokens_between_a_position_and_the_length(nq, nkv, d, bound, new):
    c = Case([(new, 100 + new), (new, 64 + new), (new, 700 + new), (1, 33)], nq, nkv, d, seed=41, bound=bound)
    back = [50, 1, 300, 0]
    for b, n in enumerate(back):
        t0, t1 = c.qsl[b], c.qsl[b + 1]
        total = c.seqs[b][1]
        c.pos[t0:t1] -= n
        slots = np.array([c.table[b][j // 16] * 16 + j % 16 for j in range(total - n, total)], dtype=np.int64)
        for tiles, is_v in ((c.tiles[0], False), (c.tiles[1], True)):  # codes of 6, scales that are NaN
            R.pack_rows(tiles, slots, np.full((len(slots), nkv, d), 7, np.uint8),
                        np.full((len(slots), nkv, d // 16), 0x7F, np.uint8), d, is_v)
    c.batch.positions.copy_(torch.from_numpy(c.pos))
    c.kc, c.vc = (torch.from_numpy(t).cuda() for t in c.tiles)
    c.run()
    ok()
    c.check()
