"""A row's norm does not depend on how many rows are normed with it, bit for bit, whatever
the number of threads that a row is given."""

import pytest
import torch

import mx_reference as R
from llama_decoder_layer_gb300 import binding as lb

pytestmark = pytest.mark.gpu

DEV = "cuda"


# fewer rows than two a multiprocessor, and more; row lengths on both sides of every choice of threads
@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP8])
@pytest.mark.parametrize("H", [32, 256, 288, 512, 544, 1024, 1056, 2048, 2080, 4096, 4128, 8192, 8224, 12320, 16384])
@pytest.mark.parametrize("res", [False, True])
def test_a_row_among_few_and_many(fmt, H, res):
    rows, part = 6000, 300
    g = torch.Generator(device=DEV).manual_seed(H)
    x, r = ((3 * torch.randn(rows, H, device=DEV, generator=g)).bfloat16() for _ in range(2))
    gamma = (1 + 0.3 * torch.randn(H, device=DEV, generator=g)).bfloat16()
    scale = 2.0 ** -6 if fmt == R.NVFP4 else 1.0

    def norm(a, b):
        m = lb.MxMatrix.empty(fmt, b - a, H, scale)
        lb.fused_add_rmsnorm_mx(x[a:b], r[a:b] if res else None, None, m, gamma, 1e-5)
        out = torch.empty(b - a, H, dtype=torch.bfloat16, device=DEV)
        lb.dequantize_mx(m, out)
        assert lb.get_device_error()[0] == lb.LLAMA_OK
        return m.codes, out

    codes, out = norm(0, rows)
    for a in range(0, rows, part):
        few = norm(a, a + part)
        assert torch.equal(few[0], codes[a:a + part]) and torch.equal(few[1], out[a:a + part])
    one = norm(rows - 1, rows)
    assert torch.equal(one[0], codes[-1:]) and torch.equal(one[1], out[-1:])
