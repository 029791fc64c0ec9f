"""Microscaled matrices on the GPU, against their 64-bit forms.

Tolerances.
* Quantised bf16 rows: bit for bit (a zero may carry either sign).
* The norm: fp32 arithmetic before the rounding to codes.  The sum of H <= 16384
  squares is taken by 256 threads of at most 64 elements, five steps within a
  warp and eight over the warps: 77 additions of relative error 2^-24 each, and
  half of that remains after the root; with the quotient, the root (2^-22) and
  two products the result is off by less than 2^-18 of itself.
* A product's fp32 sums: the products themselves are exact in fp32 (at most 4 + 4
  bits of codes and 4 + 4 of scales); each instruction adds its K step to the
  accumulator, and aligning its addends and the accumulator to the largest and
  cutting them there is off by no more than 2^-23 of the largest of them for each
  addend, none of which is beyond sum |x w|, so a sum is off by at most
  (K + K / 32) 2^-23 sum |x w|.  Then one rounding to bf16 (2^-8) or fp32
  (2^-24), after the factor's (2^-24).
* silu(g) u with sums off by dg and du: silu' is at most 1.1, so it is off by
  1.1 dg |u| + (|silu(g)| + 1.1 dg) du, and by 2^-18 of itself for exp, the
  quotient and the products (exp's argument adds |g| 2^-23, |g| < 2^5 wherever
  silu(g) matters).
"""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import mx_reference as R
from llama_decoder_layer_gb300 import binding as lb

pytestmark = pytest.mark.gpu

DEV = "cuda"
FORMATS = [R.NVFP4, R.FP4, R.FP8]
BF16, FP32 = 2.0 ** -8, 2.0 ** -24


def ok():
    st, detail = lb.get_device_error()
    assert st == lb.LLAMA_OK, (lb.status_string(st), detail)


def f64(t):
    return t.detach().double().cpu().numpy()


def empty(fmt, rows, cols, g=1.0, fill=0xAB):
    m = lb.MxMatrix.empty(fmt, rows, cols, g)
    m.codes.fill_(fill)
    m.scales.fill_(fill)
    return m


def hard_rows(rows, cols, fmt, g, seed, bad=True):
    """bf16 rows that meet the borders of a format: ties, equal values, tiny and huge groups, zeros, both signs, and
    (bad) infinities and NaN."""
    r = np.random.default_rng(seed)
    G = R.GROUP[fmt]
    x = r.standard_normal((rows, cols // G, G)) * 2.0 ** r.integers(-14, 12, (rows, cols // G, 1))
    kind = r.integers(0, 10, (rows, cols // G))[..., None]
    grid = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 1.0625, 1.1875, 27.0, 31.0, 416.0, 432.0])
    tie = grid[r.integers(0, 11 if fmt != R.FP8 else 17, x.shape)] * np.where(r.random(x.shape) < 0.5, -1, 1)
    tie[..., 0] = R.TOP[fmt]
    x = np.where(kind == 0, tie * 2.0 ** r.integers(-6, 8, kind.shape), x)
    x = np.where(kind == 1, 0.0, x)
    x = np.where(kind == 2, x[..., :1], x)
    x = np.where(kind == 5, x * 2.0 ** -12, x)
    x = np.where(kind == 6, x * 2.0 ** -120, x)
    x = np.where(kind == 7, x * 2.0 ** 100, x)
    if bad:
        odd = r.random(x.shape) < 0.05
        x = np.where((kind == 3) & odd, np.inf, x)
        x = np.where((kind == 4) & odd, np.nan, x)
    return (torch.from_numpy(x.reshape(rows, cols)) * g).to(torch.bfloat16)


def same_codes(codes, want, fmt):
    return np.array_equal(R.code_values(codes, fmt), R.code_values(want, fmt))  # -0 == 0


# ---------------------------------------------------------------------------
# quantising and reading back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 64), (3, 96), (5, 160), (128, 128), (129, 2080), (300, 1376),
                                       (1000, 4096), (40, 14336)])
@pytest.mark.parametrize("gexp", [0, -5])
def test_quantise_and_read_bit_for_bit(fmt, rows, cols, gexp):
    g = 2.0 ** gexp if fmt == R.NVFP4 else 1.0
    x = hard_rows(rows, cols, fmt, g, rows + cols)
    q, b = R.quantise(f64(x), fmt, g)
    m = empty(fmt, rows, cols, g)
    lb.quantize_mx(x.to(DEV), m)
    ok()
    codes, scales = R.pack(q, b, fmt, fill=0xAB)
    assert np.array_equal(m.scales.cpu().numpy(), scales)  # rows past the last as they were, groups past it zero
    fine = np.repeat(np.isfinite(R.scale_value(b, fmt)), R.GROUP[fmt], 1)
    got = R.code_values(m.codes.cpu().numpy(), fmt)
    assert np.array_equal(got[fine], q[fine])
    out = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    lb.dequantize_mx(m, out)
    ok()
    want = torch.from_numpy(R.values(q, b, fmt, g)).to(torch.bfloat16)
    assert torch.equal(torch.nan_to_num(out.cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0))
    assert np.array_equal(np.isnan(f64(out)), ~fine)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("wide", [8, 1032])
def test_columns_of_wider_rows(fmt, wide):
    rows, cols = 133, 480
    x = torch.randn(rows, cols + wide, device=DEV).bfloat16()
    a, b = empty(fmt, rows, cols), empty(fmt, rows, cols)
    lb.quantize_mx(x[:, 8:8 + cols], a)
    lb.quantize_mx(x[:, 8:8 + cols].contiguous(), b)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    out = torch.full((rows, cols + wide), 3.0, dtype=torch.bfloat16, device=DEV)
    flat = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    lb.dequantize_mx(a, out[:, 8:8 + cols])
    lb.dequantize_mx(a, flat)
    ok()
    assert torch.equal(out[:, 8:8 + cols], flat)
    assert bool((out[:, :8] == 3.0).all()) and bool((out[:, 8 + cols:] == 3.0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_code_and_scale_reads_back(fmt):
    """Every byte of codes with scales that give normal bf16 numbers, and the scales' ends."""
    rows, cols = 256, 32 * 8
    codes = torch.arange(rows * (cols if fmt == R.FP8 else cols // 2), dtype=torch.int64).remainder(256).to(torch.uint8)
    codes = codes.view(rows, -1)
    groups = cols // R.GROUP[fmt]
    b = np.random.default_rng(0).integers(0, 127 if fmt == R.NVFP4 else 255, (rows, groups))
    b[0, :2] = [0, 126 if fmt == R.NVFP4 else 254]
    _, scales = R.pack(np.zeros((rows, cols)), b, fmt)
    m = lb.MxMatrix(fmt, cols, codes.to(DEV), torch.from_numpy(scales).to(DEV), 0.25 if fmt == R.NVFP4 else 1.0)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    lb.dequantize_mx(m, out)
    ok()
    with np.errstate(over="ignore"):
        # as fp32 (448 * 2^127 is beyond it), then bf16
        v = torch.from_numpy(R.values(R.code_values(codes.numpy(), fmt), b, fmt, m.scale).astype(np.float32)).to(torch.bfloat16)
    assert torch.equal(torch.nan_to_num(out.cpu(), nan=1.25), torch.nan_to_num(v, nan=1.25))


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,H,res", [(1, 32, True), (3, 96, False), (130, 1376, True), (7, 2048, True),
                                        (64, 4096, True), (300, 8192, False), (2, 16384, True), (5, 12320, True),
                                        (403, 224, True), (331, 480, False), (345, 992, True), (309, 1056, True),
                                        (310, 4064, True), (307, 8160, True), (306, 16352, True)])
def test_norm(fmt, rows, H, res):
    gen = torch.Generator().manual_seed(rows + H)
    x = (torch.randn(rows, H, generator=gen) * 3).bfloat16()
    r = torch.randn(rows, H, generator=gen).bfloat16() if res else None
    gamma = (1 + 0.3 * torch.randn(H, generator=gen)).bfloat16()
    eps, g = 1e-5, 2.0 ** -6 if fmt == R.NVFP4 else 1.0
    m = empty(fmt, rows, H, g)
    res_out = torch.empty(rows, H, dtype=torch.bfloat16, device=DEV)
    lb.fused_add_rmsnorm_mx(x.to(DEV), None if r is None else r.to(DEV), res_out, m, gamma.to(DEV), eps)
    ok()
    s = x if r is None else (x.float() + r.float()).bfloat16()
    assert torch.equal(res_out.cpu(), s)
    v = f64(s)
    h = v / np.sqrt((v * v).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * f64(gamma)
    scales = m.scales.cpu().numpy()
    R.check_quantised(m.codes.cpu().numpy(), scales, h, np.abs(h) * 2.0 ** -18, fmt, g)
    # rows past the last as they were, groups past it zero
    groups = H // R.GROUP[fmt]
    rest = scales.copy()
    rest[R.scale_places(rows, groups)] = 0
    _, expect = R.pack(np.zeros((rows, H)), np.zeros((rows, groups), int), fmt, fill=0xAB)
    assert np.array_equal(rest, expect)


def test_norm_in_place_and_without_residual_out():
    rows, H = 37, 512
    x, r = (torch.randn(rows, H, device=DEV).bfloat16() for _ in range(2))
    gamma = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    a, b, c = (empty(R.FP8, rows, H) for _ in range(3))
    out = torch.empty_like(x)
    lb.fused_add_rmsnorm_mx(x, r, out, a, gamma, 1e-6)
    lb.fused_add_rmsnorm_mx(x, r, None, b, gamma, 1e-6)
    x2, r2 = x.clone(), r.clone()
    lb.fused_add_rmsnorm_mx(x2, r2, r2, c, gamma, 1e-6)
    ok()
    assert torch.equal(a.codes, b.codes) and torch.equal(a.codes, c.codes) and torch.equal(r2, out)
    lb.fused_add_rmsnorm_mx(x2, r, x2, c, gamma, 1e-6)
    ok()
    assert torch.equal(x2, out) and torch.equal(a.codes, c.codes) and torch.equal(a.scales, c.scales)


def test_norm_rows_with_nan_and_zero():
    H = 256
    x = torch.randn(5, H).bfloat16()
    x[1, 40] = float("nan")
    x[2, 3] = float("inf")
    x[3] = 0
    gamma = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    m = empty(R.FP8, 5, H)
    out = torch.empty(5, H, dtype=torch.bfloat16, device=DEV)
    lb.fused_add_rmsnorm_mx(x.to(DEV), None, None, m, gamma, 1e-6)
    lb.dequantize_mx(m, out)
    ok()
    o = f64(out)
    assert np.isnan(o[1]).all()  # its sum of squares is NaN
    assert np.isnan(o[2, :32]).all() and (o[2, 32:] == 0).all()  # inf / inf, and finite / inf
    assert (o[3] == 0).all() and np.isfinite(o[0]).all() and np.isfinite(o[4]).all()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def random_matrix(rows, cols, fmt, g, seed, spread=2):
    """Any codes and scales of a few binades, as (matrix on the GPU, values in 64 bits)."""
    r = np.random.default_rng(seed)
    if fmt == R.FP8:
        codes = r.integers(0, 256, (rows, cols))
        codes = np.where(codes % 128 == 127, 0, codes).astype(np.uint8)
    else:
        codes = r.integers(0, 256, (rows, cols // 2)).astype(np.uint8)
    groups = cols // R.GROUP[fmt]
    b = r.integers(40, 72, (rows, groups)) if fmt == R.NVFP4 else 127 + r.integers(-spread, spread + 1, (rows, groups))
    _, scales = R.pack(np.zeros((rows, cols)), b, fmt, fill=0xFF)  # rows past the last: NaN scales
    q = R.code_values(codes, fmt)
    m = lb.MxMatrix(fmt, cols, torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), g)
    return m, R.values(q, b, fmt, g)


def dot(x, w):
    """x w^T and |x| |w|^T in 64 bits, on the GPU."""
    x, w = torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV)
    return (x @ w.T).cpu().numpy(), (x.abs() @ w.abs().T).cpu().numpy()


def sum_slack(size, K):
    return size * (K + K // 32) * 2.0 ** -23


SIZES = [(1, 8, 32), (1, 256, 64), (3, 264, 96), (17, 520, 160), (128, 256, 256), (129, 392, 288), (130, 128, 512),
         (64, 4096, 4096), (300, 1384, 2080), (513, 768, 1024), (5, 8, 14336), (1021, 520, 1376),
         (2500, 2056, 288), (4000, 1288, 1056)]  # more tiles than SMs: SM pairs


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear(fmt, M, N, K, dtype):
    gx, gw = (2.0 ** -3, 2.0 ** -9) if fmt == R.NVFP4 else (1.0, 1.0)
    x, xv = random_matrix(M, K, fmt, gx, M)
    w, wv = random_matrix(N, K, fmt, gw, N + 1)
    out = torch.full((M, N), 7.0, dtype=dtype, device=DEV)
    lb.linear_mx(x, w, out, alpha=1.5)
    ok()
    y, size = dot(xv, wv)
    bar = 1.5 * sum_slack(size, K) + np.abs(1.5 * y) * ((BF16 if dtype is torch.bfloat16 else FP32) + FP32)
    err = np.abs(f64(out) - 1.5 * y)
    assert (err <= bar).all(), (err.max(), bar[err > bar][:5], np.argwhere(err > bar)[:5])


# K of a block from 15 to 17 stages of 128 elements on, where fp8 sums are of two
# accumulators: not split with one block an SM and with two, split in two, in eight
@pytest.mark.parametrize("M,N,K", [(40, 9864, 1920), (40, 9864, 2048), (33, 9864, 2112), (64, 19464, 2080), (130, 4864, 4160),
                                   (1, 424, 16544), (65, 424, 16416), (128, 1032, 16384), (128, 136, 32800)])
def test_linear_long_sums(M, N, K):
    test_linear(R.FP8, M, N, K, torch.float32)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,I,K,out_fmt", [(1, 32, 32, 0), (1, 128, 64, 3), (3, 136, 96, 0), (64, 1376, 512, 3),
                                           (130, 160, 288, 1), (77, 416, 2080, 2), (300, 1376, 512, 0),
                                           (129, 352, 1024, 3), (64, 14336, 256, 1), (2500, 1096, 160, 0),
                                           (2500, 1120, 544, 3), (4000, 800, 96, 1)])
def test_gate_up_silu(fmt, M, I, K, out_fmt):
    gx, gg, gu = (2.0 ** -3, 2.0 ** -9, 2.0 ** -8) if fmt == R.NVFP4 else (1.0, 1.0, 1.0)
    (x, xv), (gate, gv), (up, uv) = (random_matrix(M, K, fmt, gx, 1), random_matrix(I, K, fmt, gg, 2),
                                     random_matrix(I, K, fmt, gu, 3))
    (g, gs), (u, us) = dot(xv, gv), dot(xv, uv)
    ag, au = 3.0 / np.abs(g).max() * 4, 1.0 / np.abs(u).std()  # silu's curved part
    ag, au = float(np.float32(ag)), float(np.float32(au))
    og = 2.0 ** -7 if out_fmt == R.NVFP4 else 1.0
    out = empty(out_fmt, M, I, og) if out_fmt else torch.full((M, I), 7.0, dtype=torch.bfloat16, device=DEV)
    lb.gate_up_silu_mx(x, gate, up, out, alpha_gate=ag, alpha_up=au)
    ok()
    g, u, dg, du = g * ag, u * au, ag * sum_slack(gs, K) + np.abs(g * ag) * FP32, au * sum_slack(us, K) + np.abs(u * au) * FP32
    silu = g / (1 + np.exp(-g))
    want = silu * u
    slack = 1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + np.abs(want) * 2.0 ** -18
    if out_fmt:
        scales = out.scales.cpu().numpy()
        R.check_quantised(out.codes.cpu().numpy(), scales, want, slack, out_fmt, og)
        groups = I // R.GROUP[out_fmt]
        scales[R.scale_places(M, groups)] = 0
        _, expect = R.pack(np.zeros((M, I)), np.zeros((M, groups), int), out_fmt, fill=0xAB)
        assert np.array_equal(scales, expect)
    else:
        err = np.abs(f64(out) - want)
        assert (err <= slack + np.abs(want) * BF16).all(), err.max()


@pytest.mark.parametrize("M,I,K,out_fmt", [(33, 5152, 2080, 3), (70, 5136, 2112, 0), (64, 9792, 2080, 1), (96, 1376, 12416, 2),
                                           (17, 72, 16544, 0)])
def test_gate_up_silu_long_sums(M, I, K, out_fmt):
    test_gate_up_silu(R.FP8, M, I, K, out_fmt)


def to_matrix(x, fmt, g=1.0):
    m = empty(fmt, *x.shape, g if fmt == R.NVFP4 else 1.0)
    lb.quantize_mx(x, m)
    return m


def values(m):
    """What a matrix on the GPU stands for, in 64 bits."""
    b = m.scales.cpu().numpy()[R.scale_places(m.rows, m.cols // R.GROUP[m.format])]
    return R.values(R.code_values(m.codes.cpu().numpy(), m.format), b, m.format, m.scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(5, 136, 96), (64, 4096, 4096), (2600, 2056, 160)])
def test_a_bad_row_stays_by_itself(fmt, M, N, K):
    gen = torch.Generator(device=DEV).manual_seed(M)
    x, w = (torch.randn(r, K, generator=gen, device=DEV).bfloat16() for r in (M, N))
    good, bad = torch.empty(M, N, dtype=torch.bfloat16, device=DEV), torch.empty(M, N, dtype=torch.bfloat16, device=DEV)
    lb.linear_mx(to_matrix(x, fmt, 2.0 ** -6), to_matrix(w, fmt, 2.0 ** -6), good)
    x[2, 40], x[3, K - 1], w[7, 0] = float("nan"), float("inf"), float("-inf")
    lb.linear_mx(to_matrix(x, fmt, 2.0 ** -6), to_matrix(w, fmt, 2.0 ** -6), bad)
    ok()
    assert bool(bad[2:4].isnan().all()) and bool(bad[:, 7].isnan().all())
    keep_m, keep_n = (torch.ones(n, dtype=torch.bool, device=DEV) for n in (M, N))
    keep_m[2:4], keep_n[7] = False, False
    assert torch.equal(bad[keep_m][:, keep_n], good[keep_m][:, keep_n])


def test_a_matrix_with_itself():
    m, v = random_matrix(200, 512, R.FP8, 1.0, 5)
    out = torch.empty(200, 200, device=DEV)
    lb.linear_mx(m, m, out)
    ok()
    y, size = dot(v, v)
    assert (np.abs(f64(out) - y) <= sum_slack(size, 512) + np.abs(y) * 2 * FP32).all()
    assert torch.equal(out, out.T)


def test_no_rows():
    for fmt in FORMATS:
        x, w = lb.MxMatrix.empty(fmt, 0, 64), to_matrix(torch.randn(32, 64, device=DEV).bfloat16(), fmt)
        rows = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
        lb.quantize_mx(rows, x)
        lb.dequantize_mx(x, rows)
        lb.fused_add_rmsnorm_mx(rows, None, rows, x, torch.ones(64, dtype=torch.bfloat16, device=DEV), 1e-5)
        lb.linear_mx(x, w, torch.empty(0, 32, device=DEV))
        lb.gate_up_silu_mx(x, w, w, lb.MxMatrix.empty(fmt, 0, 32))
    ok()


@pytest.mark.parametrize("M,I", [(3, 64), (2600, 2080)])
@pytest.mark.parametrize("out_fmt", [0, R.FP8])
def test_silu_far_out(M, I, out_fmt):
    """Gate sums from -3e38 to 3e38, and zero: silu is g or 0 there, and never a NaN; a sum beyond fp32 is an infinity."""
    K = 32
    xv, gv, uv = np.zeros((M, K)), np.zeros((I, K)), np.zeros((I, K))
    xv[:, 0], uv[:, 0] = 1.0, 0.5
    powers = np.array([-384.0, -3.0, -0.875, 0.0, 0.75, 3.0, 416.0, 0.25])
    gv[:, 0] = powers[np.arange(I) % 8]
    one = lambda v: lb.MxMatrix(R.FP8, K, *(torch.from_numpy(t).to(DEV) for t in R.pack(  # noqa: E731
        v, np.full((len(v), 1), 127), R.FP8)))
    for alpha in (1.0, 100.0, 1e20, 2.0 ** 119):  # 2^119: 384 gives 2.6e38, 416 2.8e38
        out = empty(out_fmt, M, I) if out_fmt else torch.empty(M, I, dtype=torch.bfloat16, device=DEV)
        lb.gate_up_silu_mx(one(xv), one(gv), one(uv), out, alpha_gate=alpha)
        ok()
        g = (xv @ gv.T) * np.float64(np.float32(alpha))
        want = np.where(g < -700, 0.0, g / (1 + np.exp(np.minimum(-g, 700)))) * 0.5
        slack = np.abs(want) * 2.0 ** -18 + 2.0 ** -110  # (silu(-87) is below 2^-118)
        if out_fmt:
            R.check_quantised(out.codes.cpu().numpy(), out.scales.cpu().numpy(), want, slack, out_fmt, 1.0)
        else:
            assert (np.abs(f64(out) - want) <= slack + np.abs(want) * BF16).all()
    out = torch.empty(M, I, dtype=torch.bfloat16, device=DEV)
    lb.gate_up_silu_mx(one(xv), one(gv), one(uv), out, alpha_gate=3e38)  # 416 * 3e38: infinite
    ok()
    o = f64(out)
    assert (o[:, 6::8] == np.inf).all() and (np.abs(o[:, 0::8]) <= 2.0 ** -110).all() and (o[:, 3::8] == 0).all()


FIRST_UNDER_CAPTURE = """
import torch
from llama_decoder_layer_gb300 import binding as lb
F = lb.LLAMA_MX_NVFP4
x, w = (torch.randn(n, 512, device="cuda").bfloat16() for n in (M, 2056))
mx, mw = lb.MxMatrix.empty(F, M, 512, 2.0 ** -6), lb.MxMatrix.empty(F, 2056, 512, 2.0 ** -6)
res, g = torch.empty_like(x), torch.ones(512, dtype=torch.bfloat16, device="cuda")
out, eager = torch.empty(M, 2056, device="cuda"), torch.empty(M, 2056, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    lb.quantize_mx(w, mw)
    lb.fused_add_rmsnorm_mx(x, None, res, mx, g, 1e-5)
    lb.linear_mx(mx, mw, out)
graph.replay()
torch.cuda.synchronize()
lb.linear_mx(mx, mw, eager)
torch.cuda.synchronize()
assert lb.get_device_error()[0] == 0 and torch.equal(out, eager) and bool(out.abs().sum() > 0)
print("same")
"""


@pytest.mark.parametrize("M", [2, 3000])
def test_the_first_calls_of_a_process_may_be_captured(M):
    r = subprocess.run([sys.executable, "-c", f"M = {M}\n" + FIRST_UNDER_CAPTURE], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


class Mlp:
    """A norm, gate_up and down in one format, as a layer's second half calls them."""

    def __init__(self, fmt, M, H, I, seed):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
        self.x, self.res = rand(M, H).bfloat16(), rand(M, H).bfloat16()
        self.gamma = (1 + 0.2 * rand(H)).bfloat16()
        self.gate, self.up = (to_matrix((rand(I, H) * H ** -0.5).bfloat16(), fmt, 2.0 ** -12) for _ in range(2))
        self.down = to_matrix((rand(H, I) * I ** -0.5).bfloat16(), fmt, 2.0 ** -12)
        self.h, self.a = empty(fmt, M, H, 2.0 ** -6 if fmt == R.NVFP4 else 1.0), empty(fmt, M, I, 2.0 ** -8 if fmt == R.NVFP4 else 1.0)
        self.res_out, self.out = torch.empty_like(self.x), torch.empty_like(self.x)

    def run(self, stream=None):
        lb.fused_add_rmsnorm_mx(self.x, self.res, self.res_out, self.h, self.gamma, 1e-5, stream=stream)
        lb.gate_up_silu_mx(self.h, self.gate, self.up, self.a, stream=stream)
        lb.linear_mx(self.a, self.down, self.out, stream=stream)

    def results(self):
        return [t.clone() for t in (self.res_out, self.h.codes, self.h.scales, self.a.codes, self.a.scales, self.out)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,H,I", [(3, 512, 1376), (130, 1024, 2048), (1500, 2080, 4128)])
def test_mlp_of_a_layer(fmt, M, H, I):
    m = Mlp(fmt, M, H, I, 1)
    m.run()
    ok()
    s = f64((m.x.float() + m.res.float()).bfloat16())
    h = s / np.sqrt((s * s).mean(-1, keepdims=True) + np.float64(np.float32(1e-5))) * f64(m.gamma)
    R.check_quantised(m.h.codes.cpu().numpy(), m.h.scales.cpu().numpy(), h, np.abs(h) * 2.0 ** -18, fmt, m.h.scale)
    hv = values(m.h)
    (g, gs), (u, us) = dot(hv, values(m.gate)), dot(hv, values(m.up))
    dg, du = sum_slack(gs, H) + np.abs(g) * FP32, sum_slack(us, H) + np.abs(u) * FP32
    silu = g / (1 + np.exp(-g))
    slack = 1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + np.abs(silu * u) * 2.0 ** -18
    R.check_quantised(m.a.codes.cpu().numpy(), m.a.scales.cpu().numpy(), silu * u, slack, fmt, m.a.scale)
    y, size = dot(values(m.a), values(m.down))
    assert (np.abs(f64(m.out) - y) <= sum_slack(size, I) + np.abs(y) * (BF16 + FP32)).all()


@pytest.mark.parametrize("fmt,M,H,I", [(R.NVFP4, 1, 512, 1376), (R.FP8, 64, 2048, 8192), (R.FP4, 1500, 2080, 4128)])
def test_graph_replays_and_streams_give_the_same(fmt, M, H, I):
    m, other = Mlp(fmt, M, H, I, 2), Mlp(fmt, M, H, I, 3)
    m.run()
    other.run()
    ok()
    want, want_other = m.results(), other.results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        m.run()
        m.run()
    for t in (m.res_out, m.h.codes, m.a.codes, m.out):
        t.zero_()
    graph.replay()
    other.out.zero_()
    graph.replay()
    ok()
    assert all(torch.equal(a, b) for a, b in zip(m.results(), want))
    # two streams at once, one given as the stream of the call, one the current stream
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        m.run(stream=s1)
        with torch.cuda.stream(s2):
            other.run()
    torch.cuda.synchronize()
    ok()
    assert all(torch.equal(a, b) for a, b in zip(m.results(), want))
    assert all(torch.equal(a, b) for a, b in zip(other.results(), want_other))


def test_offsets_beyond_32_bits():
    """Codes, rows and results of more than 2^32 bytes: the last rows are those of a small call."""
    rows, cols, last = 300_000, 16384, 300
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[:1000].normal_()
    x[1000:-last] = 0.5
    x[-last:].normal_()
    m = lb.MxMatrix.empty(R.FP8, rows, cols)
    lb.quantize_mx(x, m)
    tail = to_matrix(x[-last:].contiguous(), R.FP8)
    assert torch.equal(m.codes[-last:], tail.codes)
    back = torch.empty_like(x)
    lb.dequantize_mx(m, back)
    small = torch.empty(last, cols, dtype=torch.bfloat16, device=DEV)
    lb.dequantize_mx(tail, small)
    assert torch.equal(back[-last:], small)
    lb.fused_add_rmsnorm_mx(x, None, back, m, torch.ones(cols, dtype=torch.bfloat16, device=DEV), 1e-5)
    lb.fused_add_rmsnorm_mx(x[-last:], None, small, tail, torch.ones(cols, dtype=torch.bfloat16, device=DEV), 1e-5)
    assert torch.equal(m.codes[-last:], tail.codes) and torch.equal(back[-last:], small)
    del x, back
    w = to_matrix(torch.randn(64, cols, device=DEV).bfloat16(), R.FP8)
    # the weight is the large matrix: its last rows are the last results
    out = torch.empty(64, rows, device=DEV)
    lb.linear_mx(w, m, out)
    ok()
    y, size = dot(values(w), values(tail))
    assert (np.abs(f64(out[:, -last:]) - y) <= sum_slack(size, cols) + np.abs(y) * 2 * FP32).all()
    del m, out
    # more than 2^32 bytes of results
    a, b = to_matrix(torch.randn(9000, 64, device=DEV).bfloat16(), R.FP8), to_matrix(
        torch.randn(262_144, 64, device=DEV).bfloat16(), R.FP8)
    out = torch.empty(9000, 262_144, dtype=torch.bfloat16, device=DEV)
    lb.linear_mx(a, b, out)
    ok()
    y = (torch.from_numpy(values(a)[-200:]).to(DEV) @ torch.from_numpy(values(b)).to(DEV).T)
    assert float((out[-200:].double() - y).abs().max()) <= float(y.abs().max()) * 2 * BF16
