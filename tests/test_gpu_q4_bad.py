"""Sequences of one new token that the attention over 4-bit caches reports: their
rows are left, whole and cut over CTAs, and the others are right."""

import numpy as np
import pytest

import q4_reference as R
from test_gpu_q4 import Case, f64, guard

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,bound", [((40, 100, 60), 0), ((40, 100, 60), 5000), ((3000, 4000, 2500), 0),
                                        ((40, 4000, 60), 9000)])
@pytest.mark.parametrize("nq,nkv,d", [(8, 2, 128), (12, 2, 64)])
@pytest.mark.parametrize("what", ["past", "negative", "long"])
def test_rows_of_a_reported_sequence_are_left(lens, bound, nq, nkv, d, what):
    c = Case([(1, n) for n in lens], nq, nkv, d, seed=61, bound=bound)
    if what == "past":
        c.batch.positions[1] = lens[1]
    elif what == "negative":
        c.batch.positions[1] = -1
    else:
        c.batch.seq_lens[1] = 100000
        c.batch.positions[1] = 99999
    c.run()
    guard()
    got = f64(c.out).reshape(-1, nq, d)
    want, spread, flat = R.attention(f64(c.q), c.pos, c.qsl, c.table, c.tiles[0], c.tiles[1], 1.0, 1.0)
    assert np.all(got[1] == 5.0)
    tol = 2.0 ** -8 * np.abs(want) + 2 * (2.0 ** -11 + 2.0 ** -12) * spread + 2.0 ** -31 * flat
    assert np.all((np.abs(got - want) <= tol)[[0, 2]])
