"""Rows of the 4-bit cache whose warps hold several tokens, at sizes where the
writing CTAs go round more than once and their last tokens end inside a warp."""

import pytest

from test_gpu_q4 import test_write_and_read_bit_for_bit as write_and_read

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,nkv,d", [(3649, 2, 64), (3650, 2, 64), (3655, 1, 128), (7299, 1, 64), (609, 5, 128),
                                     (1217, 3, 128), (1219, 3, 128), (4001, 3, 64)])
def test_the_last_tokens_end_inside_a_warp(T, nkv, d):
    write_and_read(d, T, nkv, 0, -3)


@pytest.mark.parametrize("T", [1, 40, 3001])
@pytest.mark.parametrize("nkv", [17, 23, 31])
def test_heads_that_no_number_of_whole_rows_makes_warps_of(T, nkv):
    write_and_read(64, T, nkv, 2, 0)
