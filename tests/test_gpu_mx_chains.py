"""Sums of several chains: K a stage below, at and past the chains' lengths, last
chains and stages that are not full, with every kind of result, against 64 bits.  The
tolerances are those of test_gpu_mx; a chain that is left out, added twice or taken from
another row or column is off by far more than they allow."""

import pytest
import torch

import mx_reference as R
import test_gpu_mx as T
from llama_decoder_layer_gb300 import binding as lb
from test_gpu_mx_raster import operand

pytestmark = pytest.mark.gpu

STAGE = {R.NVFP4: 256, R.FP4: 256, R.FP8: 128}
DEV = "cuda"


def check_linear(fmt, M, N, K):
    (x, xv), (w, wv) = operand(fmt, M, K, 1), operand(fmt, N, K, 2)
    y, size = xv @ wv.T, xv.abs() @ wv.abs().T
    for dtype, half in ((torch.float32, T.FP32), (torch.bfloat16, T.BF16)):
        out = torch.full((M, N), 7.0, dtype=dtype, device=DEV)
        lb.linear_mx(x, w, out)
        T.ok()
        assert bool(((out.double() - y).abs() <= T.sum_slack(size, K) + y.abs() * (half + T.FP32)).all())
        again = torch.empty_like(out)
        lb.linear_mx(x, w, again)
        assert torch.equal(out, again)


def check_gate_up(fmt, M, I, K, outs):  # noqa: E741
    (x, xv), (gate, gv), (up, uv) = operand(fmt, M, K, 1), operand(fmt, I, K, 2), operand(fmt, I, K, 3)
    alpha, xa = K ** -0.5, xv.abs()
    g, u = xv @ gv.T * alpha, xv @ uv.T * alpha
    dg = T.sum_slack(xa @ gv.abs().T, K) * alpha + g.abs() * 2 * T.FP32  # (alpha: rounded to fp32)
    du = T.sum_slack(xa @ uv.abs().T, K) * alpha + u.abs() * 2 * T.FP32
    silu = g * torch.sigmoid(g)
    want = silu * u
    slack = 1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du + want.abs() * 2.0 ** -18
    for out_fmt in outs:
        og = 2.0 ** -7 if out_fmt == R.NVFP4 else 1.0
        out = T.empty(out_fmt, M, I, og) if out_fmt else torch.full((M, I), 7.0, dtype=torch.bfloat16, device=DEV)
        lb.gate_up_silu_mx(x, gate, up, out, alpha, alpha)
        T.ok()
        if out_fmt:
            R.check_quantised(out.codes.cpu().numpy(), out.scales.cpu().numpy(), want.cpu().numpy(), slack.cpu().numpy(), out_fmt, og)
        else:
            assert bool(((out.double() - want).abs() <= slack + want.abs() * T.BF16).all())


# stages and an odd rest, on SM pairs; not split; split in eight (of the stages a block has)
@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4, R.FP8])
@pytest.mark.parametrize("stages", [15, 16, 32, 33, 64, 97])
def test_linear_on_pairs(fmt, stages):
    check_linear(fmt, 2600, 2056, stages * STAGE[fmt] + 32)


@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4, R.FP8])
@pytest.mark.parametrize("stages", [11, 12, 24, 31, 32, 33, 65, 97])
def test_linear_of_few_tiles(fmt, stages):
    check_linear(fmt, 37, 9864, stages * STAGE[fmt] + 32)


@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4, R.FP8])
@pytest.mark.parametrize("M", [1, 100, 130])
def test_linear_split(fmt, M):
    check_linear(fmt, M, 392, (8 * 33 + 5) * STAGE[fmt] + 32)


@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4, R.FP8])
@pytest.mark.parametrize("stages", [16, 33, 65])
def test_gate_up_on_pairs(fmt, stages):
    check_gate_up(fmt, 2500, 1120, stages * STAGE[fmt] + 32, [0, R.NVFP4, R.FP4, R.FP8])


@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4, R.FP8])
@pytest.mark.parametrize("stages", [12, 32, 33, 66])
def test_gate_up_of_few_tiles(fmt, stages):
    check_gate_up(fmt, 37, 4960, stages * STAGE[fmt] + 32, [0, R.NVFP4, R.FP4, R.FP8])


@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4, R.FP8])
def test_gate_up_split(fmt):
    check_gate_up(fmt, 100, 224, (8 * 33 + 5) * STAGE[fmt] + 32, [0, R.NVFP4, R.FP4, R.FP8])


# bf16 results of 4-bit products have chains of 256 stages.  Against fp32 results of the same sums, which have shorter ones: the
# cuts of 1040 steps are 2^-24 of the sums' rms each in the mean, all on one side at the worst: d = 2^-14 rms.
@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4])
def test_bf16_chains_of_linear(fmt):
    K, N = 260 * 256 + 32, 9864
    x, w = operand(fmt, 40, K, 1)[0], operand(fmt, N, K, 2)[0]
    y, z = torch.empty(40, N, device=DEV), torch.empty(40, N, dtype=torch.bfloat16, device=DEV)
    lb.linear_mx(x, w, y, K ** -0.5)
    lb.linear_mx(x, w, z, K ** -0.5)
    T.ok()
    y = y.double()
    assert bool(((z.double() - y).abs() <= y.abs() * T.BF16 + 2.0 ** -14 * y.square().mean().sqrt()).all())


@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4])
def test_bf16_chains_of_gate_up(fmt):
    K, I = 260 * 256 + 32, 4960  # noqa: E741
    x, a, b = operand(fmt, 40, K, 1)[0], operand(fmt, I, K, 2)[0], operand(fmt, I, K, 3)[0]
    g, u = (torch.empty(40, I, device=DEV) for _ in range(2))
    lb.linear_mx(x, a, g, K ** -0.5)
    lb.linear_mx(x, b, u, K ** -0.5)
    out = torch.empty(40, I, dtype=torch.bfloat16, device=DEV)
    lb.gate_up_silu_mx(x, a, b, out, K ** -0.5, K ** -0.5)
    T.ok()
    g, u = g.double(), u.double()
    silu, dg, du = g * torch.sigmoid(g), 2.0 ** -14 * g.square().mean().sqrt(), 2.0 ** -14 * u.square().mean().sqrt()
    bar = (silu * u).abs() * (T.BF16 + 2.0 ** -18) + 1.1 * dg * u.abs() + (silu.abs() + 1.1 * dg) * du
    assert bool(((out.double() - silu * u).abs() <= bar).all())
