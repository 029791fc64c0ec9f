"""Finite values are stored as finite codes: no fp8 code is NaN and no scale is, whoever wrote
them (bounds that compare codes with numbers let a NaN pass)."""

import numpy as np
import pytest
import torch

import mx_reference as R
from llama_decoder_layer_gb300 import binding as lb

pytestmark = pytest.mark.gpu

DEV = "cuda"


def finite(m):
    assert lb.get_device_error()[0] == lb.LLAMA_OK
    b = m.scales.cpu().numpy()[R.scale_places(m.rows, m.cols // R.GROUP[m.format])]
    return bool(np.isfinite(R.scale_value(b, m.format)).all() and np.isfinite(R.code_values(m.codes.cpu().numpy(), m.format)).all())


def rows(n, cols, seed):
    """Values from bf16's smallest to near its largest, a binade a group."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(n, cols, device=DEV, generator=g)
    e = torch.randint(-140, 120, (n, cols // 32), device=DEV, generator=g).repeat_interleave(32, 1)
    return torch.ldexp(x, e).bfloat16()


@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4, R.FP8])
@pytest.mark.parametrize("n", [3, 700])
def test_rows_and_norms(fmt, n):
    g = 2.0 ** -6 if fmt == R.NVFP4 else 1.0
    m = lb.MxMatrix.empty(fmt, n, 1056, g)
    lb.quantize_mx(rows(n, 1056, n), m)
    assert finite(m)
    x = torch.ldexp(rows(n, 1056, n), torch.tensor(-60, device=DEV)).bfloat16()  # (squares within fp32)
    lb.fused_add_rmsnorm_mx(x, None, None, m, torch.ones(1056, dtype=torch.bfloat16, device=DEV), 1e-6)
    assert finite(m)


@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4, R.FP8])
@pytest.mark.parametrize("out_fmt", [R.NVFP4, R.FP4, R.FP8])
@pytest.mark.parametrize("M,I", [(5, 160), (70, 4128), (2600, 1376)])
def test_gate_up(fmt, out_fmt, M, I):  # noqa: E741
    def mat(n, seed):
        m = lb.MxMatrix.empty(fmt, n, 288, 2.0 ** -4 if fmt == R.NVFP4 else 1.0)
        lb.quantize_mx(torch.randn(n, 288, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)).bfloat16(), m)
        return m

    x, gate, up = mat(M, 1), mat(I, 2), mat(I, 3)
    for alpha in (1e-30, 0.05, 1e4, 1e30):
        out = lb.MxMatrix.empty(out_fmt, M, I)
        lb.gate_up_silu_mx(x, gate, up, out, min(alpha, 1e4), alpha)
        assert finite(out)
