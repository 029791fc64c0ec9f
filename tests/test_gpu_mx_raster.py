"""SM pairs take a product's tiles in groups of as many rows of x as 32 MB of codes
hold: sizes with several groups, the last of which is not full, every result against
64 bits and the tolerances of test_gpu_mx."""

import pytest
import torch

import mx_reference as R
import test_gpu_mx as T
from llama_decoder_layer_gb300 import binding as lb

pytestmark = pytest.mark.gpu

# rows of tiles and of them a group: 18 and 16, 35 and 16 (three groups), 39 and 32
SIZES = [(R.FP8, 4400, 1544, 8192), (R.FP8, 8900, 776, 8192), (R.NVFP4, 9900, 1288, 8192), (R.FP4, 9900, 1288, 8192)]


def operand(fmt, rows, cols, seed):
    """A random matrix and its values in 64 bits, made and kept on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = lb.MxMatrix.empty(fmt, rows, cols, 2.0 ** -6 if fmt == R.NVFP4 else 1.0)
    lb.quantize_mx(torch.randn(rows, cols, device="cuda", generator=g).bfloat16(), m)
    v = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    lb.dequantize_mx(m, v)
    return m, v.double()


@pytest.mark.parametrize("fmt,M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear(fmt, M, N, K, dtype):
    (x, xv), (w, wv) = operand(fmt, M, K, 1), operand(fmt, N, K, 2)
    out = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    lb.linear_mx(x, w, out)
    T.ok()
    y = xv @ wv.T
    bar = T.sum_slack(xv.abs() @ wv.abs().T, K) + y.abs() * ((T.BF16 if dtype is torch.bfloat16 else T.FP32) + T.FP32)
    assert bool(((out.double() - y).abs() <= bar).all())


@pytest.mark.parametrize("fmt,M,N,K", SIZES)
@pytest.mark.parametrize("out_fmt", [0, R.NVFP4, R.FP8])
def test_gate_up_silu(fmt, M, N, K, out_fmt):
    I = N // 32 * 32  # noqa: E741
    (x, xv), (gate, gv), (up, uv) = operand(fmt, M, K, 1), operand(fmt, I, K, 2), operand(fmt, I, K, 3)
    og = 2.0 ** -7 if out_fmt == R.NVFP4 else 1.0
    alpha = K ** -0.5
    out = T.empty(out_fmt, M, I, og) if out_fmt else torch.full((M, I), 7.0, dtype=torch.bfloat16, device="cuda")
    lb.gate_up_silu_mx(x, gate, up, out, alpha, alpha)
    T.ok()
    xa = xv.abs()
    g, u = xv @ gv.T * alpha, xv @ uv.T * alpha
    dg = T.sum_slack(xa @ gv.abs().T, K) * alpha + g.abs() * 2 * T.FP32  # (alpha: rounded to fp32)
    du = T.sum_slack(xa @ uv.abs().T, K) * alpha + u.abs() * 2 * T.FP32
    silu = g * torch.sigmoid(g)
    want = silu * u
    slack = 1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du + want.abs() * 2.0 ** -18
    if out_fmt:
        R.check_quantised(out.codes.cpu().numpy(), out.scales.cpu().numpy(), want.cpu().numpy(), slack.cpu().numpy(), out_fmt, og)
    else:
        assert bool(((out.double() - want).abs() <= slack + want.abs() * T.BF16).all())
