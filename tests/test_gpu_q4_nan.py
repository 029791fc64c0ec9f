"""Query rows with a NaN or an infinity in the attention over 4-bit caches: the
formula's answer for such a row is NaN, on every path, and the other rows keep
theirs."""

import numpy as np
import pytest
import torch

import q4_reference as R
from test_gpu_q4 import Case, f64, ok

pytestmark = pytest.mark.gpu

# decode whole and cut, 16 query rows, prompts on either prefill kernel with their keys whole and split over CTAs
PATHS = {
    "whole": ([(1, 40), (1, 300)], 8, 2, 64, 0),
    "cut": ([(1, 3000), (1, 17)], 32, 4, 128, 5000),
    "rows16": ([(2, 700), (2, 33)], 16, 2, 128, 5000),
    "prompt_tc": ([(40, 77), (1, 5)], 8, 2, 128, 0),
    "prompt": ([(40, 77), (1, 5)], 8, 2, 64, 0),
    "split": ([(70, 900), (1, 60)], 8, 2, 64, 0),
    "split_odd": ([(33, 1300), (1, 60)], 5, 1, 128, 0),
    "split_tc": ([(20, 5000), (1, 60)], 8, 2, 128, 0),
}


def check_with_nan_rows(c, rows):
    """c's output: NaN exactly in the (token, head) rows, the others as they should be."""
    got = f64(c.out).reshape(-1, c.nq, c.d)
    want, spread, flat = R.attention(f64(c.q), c.pos, c.qsl, c.table, c.tiles[0], c.tiles[1], c.kg, c.vg)
    poisoned = np.zeros(got.shape, bool)
    for t, h in rows:
        poisoned[t, h] = True
    assert np.array_equal(np.isnan(want), poisoned)  # the formula's own
    assert np.array_equal(np.isnan(got), poisoned), np.argwhere(np.isnan(got) != poisoned)[:3].tolist()
    tol = 2.0 ** -8 * np.abs(want) + 2 * (2.0 ** -8 + 2.0 ** -12) * spread + 2.0 ** -31 * flat
    assert np.all((np.abs(got - want) <= tol)[~poisoned])


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("x", [np.nan, np.inf, -np.inf])
def test_a_query_row_that_is_not_finite(path, x):
    seqs, nq, nkv, d, bound = PATHS[path]
    c = Case(seqs, nq, nkv, d, seed=31, bound=bound)
    n = seqs[0][0]
    rows = {(0, 1), (n - 1, nq - 1), (n, 0)}
    for t, h in rows:
        c.q[t, h, 5] = x
    c.qd = c.q.cuda()
    c.run()
    ok()
    check_with_nan_rows(c, rows)


@pytest.mark.parametrize("path", PATHS)
def test_a_query_row_all_of_whose_scores_are_minus_infinity(path):
    # softmax of nothing but -inf: NaN by the formula
    seqs, nq, nkv, d, bound = PATHS[path]
    c = Case(seqs, nq, nkv, d, seed=32, bound=bound)
    for k in range(16):  # element 0 of every key: positive (code 7)
        c.tiles[0][..., R.code_place(d, k, 0, False)] &= 0xF0
        c.tiles[0][..., R.code_place(d, k, 0, False)] |= 7
    c.kc = torch.from_numpy(c.tiles[0]).cuda()
    n = seqs[0][0]
    rows = {(0, 1), (n - 1, nq - 1), (n, 0)}
    for t, h in rows:
        c.q[t, h, 0] = -np.inf
    c.qd = c.q.cuda()
    c.run()
    ok()
    check_with_nan_rows(c, rows)
