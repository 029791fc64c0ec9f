"""How near the sums of microscaled products come to 64 bits, whatever K is.

An instruction adds a K step of 32 (fp8) or 64 (4 bits) elements to the accumulator,
and the tensor cores cut the sum to 24 bits.  Results in fp32, and those that are quantised
from it, are to be as near as sums in 32 bits are, relative to the results' rms:
* Independent terms of both signs.  A sum that is rounded to nearest once a step is off by at
  most 2^-24 |s_k| there, 2^-24 / sqrt(3) |s_k| in the rms of a uniform error; s_k^2 is k / n of
  the last one in the mean, so that n steps make 2^-24 / sqrt(3) sqrt(n / 2) = 2^-24 sqrt(n / 6).
  (A chain without an end is beyond it: cuts fall to one side, and their sum grows as n.)
* Terms of one sign, where every cut is on the same side: half a unit in the last place in
  the mean, the unit at most 2^-23 |s_k|, and s_k = k / n of the last.  A chain of n steps
  is off by 2^-24 (n + 1) / 2.  Chains have at most 64 steps (fp8) or 128 (4 bits); their
  c sums are added to nearest: 2^-24 sqrt(c / 3) more.
* Behind silu(g) u, quantised: with g and u off by dg and du (the first bar times their
  rms) a result is off by d = 1.1 dg |u| + |silu(g)| du, and by 2^-20 of itself for the
  epilogue's own roundings; it falls on the other side of a border of codes that are `step` apart
  with a chance of d / step.  Twice the sum of these chances, and ten more, may differ.
"""

import numpy as np
import pytest
import torch

import mx_reference as R
from llama_decoder_layer_gb300 import binding as lb

pytestmark = pytest.mark.gpu

DEV = "cuda"
CHAIN = {R.NVFP4: 128, R.FP4: 128, R.FP8: 64}  # steps
# K split over a cluster, not split, and SM pairs
SIZES = [(64, 512), (64, 9728), (100, 19456), (2600, 2048)]


def matrix(fmt, rows, cols, seed, positive=False):
    """A quantised random matrix and its values in 64 bits."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(rows, cols, device=DEV, generator=g)
    m = lb.MxMatrix.empty(fmt, rows, cols, 2.0 ** -6 if fmt == R.NVFP4 else 1.0)
    lb.quantize_mx((x.abs() if positive else x).bfloat16(), m)
    v = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    lb.dequantize_mx(m, v)  # exact
    return m, v.double()


def rms(t):
    return float(t.square().mean().sqrt())


def off(fmt, M, N, K, positive):
    """rms of an fp32 product's errors over the rms of the results."""
    (a, av), (b, bv) = matrix(fmt, M, K, 1, positive), matrix(fmt, N, K, 2, positive)
    y = torch.empty(M, N, device=DEV)
    lb.linear_mx(a, b, y)
    assert lb.get_device_error()[0] == lb.LLAMA_OK
    want = av @ bv.T
    return rms(y.double() - want) / rms(want)


@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("K", [512, 2048, 4096, 8192, 14368, 28672])
def test_fp8_sums_of_both_signs(M, N, K):
    got, bar = off(R.FP8, M, N, K, False), 2.0 ** -24 * (K / 32 / 6) ** 0.5
    assert got <= bar, (got, bar)


@pytest.mark.parametrize("fmt", [R.NVFP4, R.FP4, R.FP8])
@pytest.mark.parametrize("M,N", SIZES)
@pytest.mark.parametrize("K", [2048, 8192, 28672])
def test_sums_of_one_sign(fmt, M, N, K):
    steps = K // R.STEP[fmt]
    chain = min(steps, CHAIN[fmt])
    bar = 2.0 ** -24 * ((chain + 1) / 2 + (steps / chain / 3) ** 0.5)
    got = off(fmt, M, N, K, True)
    assert got <= bar, (got, bar)


@pytest.mark.parametrize("fmt,M,N,K", [(R.FP8, 520, 264, 70016), (R.FP4, 520, 264, 200064), (R.FP8, 2600, 1032, 131072),
                                       (R.FP8, 2600, 1032, 131104)])
def test_bf16_results_of_very_long_sums(fmt, M, N, K):
    """Against fp32 results of the same sums: a rounding to bf16, half a step of 2^-7, and a sixteenth of that for the cuts of
    a chain of up to 1024 stages (4096 steps, half a unit each in the mean, all on one side: 4097 / 2 2^-24 = 2^-13)."""
    (a, _), (b, _) = matrix(fmt, M, K, 1, True), matrix(fmt, N, K, 2, True)
    y, z = (torch.empty(M, N, dtype=t, device=DEV) for t in (torch.float32, torch.bfloat16))
    lb.linear_mx(a, b, y)
    lb.linear_mx(a, b, z)
    assert lb.get_device_error()[0] == lb.LLAMA_OK
    assert float(((z.double() - y.double()).abs() / y.double()).max()) <= 2.0 ** -8 + 2.0 ** -12


@pytest.mark.parametrize("M,I", [(64, 2048), (2600, 1024)])
@pytest.mark.parametrize("K", [2048, 28672])
def test_fp8_codes_behind_gate_up(M, I, K):
    (x, xv), (gate, gv), (up, uv) = matrix(R.FP8, M, K, 1), matrix(R.FP8, I, K, 2), matrix(R.FP8, I, K, 3)
    out = lb.MxMatrix.empty(R.FP8, M, I)
    alpha = K ** -0.5
    lb.gate_up_silu_mx(x, gate, up, out, alpha, alpha)
    assert lb.get_device_error()[0] == lb.LLAMA_OK
    g, u = xv @ gv.T * alpha, xv @ uv.T * alpha
    silu, bar = g * torch.sigmoid(g), 2.0 ** -24 * (K / 32 / 6) ** 0.5
    h = silu * u
    d = (1.1 * bar * rms(g) * u.abs() + silu.abs() * bar * rms(u) + 2.0 ** -20 * h.abs()).cpu().numpy()
    q, b = R.quantise(h.cpu().numpy(), R.FP8, 1.0)
    got = out.scales.cpu().numpy()[R.scale_places(M, I // 32)]
    assert (got != b).sum() <= 10
    same = np.repeat(got == b, 32, 1)
    step = np.repeat(R.scale_value(b, R.FP8), 32, 1) * 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -9))), -6) - 3)
    differ = int((R.code_values(out.codes.cpu().numpy(), R.FP8) != q)[same].sum())
    bound = 2 * float((d / step).clip(max=1).sum()) + 10
    assert differ <= bound, (differ, bound)
