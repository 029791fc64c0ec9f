"""Microscaled matrices without a GPU: the layout, the 64-bit reference on
hand-worked rows, and every refusal on the host."""

import ctypes
import math

import numpy as np
import pytest
import torch

import mx_reference as R
from llama_decoder_layer_gb300 import binding as lb
from llama_decoder_layer_gb300 import build as lbuild

FAKE = 256  # an aligned address nothing reads: every call here is refused before a launch
ARG, UNSUP = lb.LLAMA_ERR_ARG, lb.LLAMA_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    lbuild.build()
    return lb.lib()


@pytest.mark.parametrize("rows,groups", [(1, 1), (127, 4), (128, 5), (129, 8), (300, 43)])
def test_every_scale_has_a_place_of_its_own(rows, groups):
    at = R.scale_places(rows, groups)
    assert len(set(at.reshape(-1).tolist())) == rows * groups
    assert at.min() >= 0 and at.max() < -(-rows // 128) * -(-groups // 4) * 512


def test_reference_on_hand_worked_rows():
    x = np.zeros((1, 32))
    x[0, :8] = [6.0, -3.0, 0.25, 0.75, 2.5, 5.0, -0.2, 0.26]
    for fmt in (R.NVFP4, R.FP4):  # ties to the even code
        q, b = R.quantise(x, fmt, 1.0)
        assert list(R.values(q, b, fmt, 1.0)[0, :8]) == [6.0, -3.0, 0.0, 1.0, 2.0, 4.0, 0.0, 0.5]
        assert R.scale_value(b, fmt)[0, 0] == 1.0
    # the power of two is the least that holds the largest element: 6 and 7 differ, 448 and 449 too
    assert R.E8M0[R.scale_bytes(np.array([6.0, 6.03, 12.0, 0.0, 2.0 ** -140]), R.FP4, 1.0)].tolist() == \
        [1.0, 2.0, 2.0, 2.0 ** -127, 2.0 ** -127]
    assert R.E8M0[R.scale_bytes(np.array([448.0, 450.0, 2.0 ** 127 * 1.75]), R.FP8, 1.0)].tolist() == [1, 2, 2.0 ** 119]
    # nvfp4 saturates, and a scale that underflows stores zeros
    assert R.values(*R.quantise(np.full((1, 16), 1e30), R.NVFP4, 1.0), R.NVFP4, 1.0).max() == 6 * 448
    assert R.values(*R.quantise(np.full((1, 16), 2.0 ** -9), R.NVFP4, 1.0), R.NVFP4, 1.0).max() == 0
    # a NaN or an infinity takes its group with it
    x[0, 20] = np.inf
    assert np.isnan(R.values(*R.quantise(x, R.NVFP4, 1.0), R.NVFP4, 1.0)).tolist() == [[False] * 16 + [True] * 16]


def test_pack_and_read_back():
    r = np.random.default_rng(0)
    for fmt in (R.NVFP4, R.FP4, R.FP8):
        x = r.standard_normal((130, 96))
        q, b = R.quantise(x, fmt, 1.0)
        codes, scales = R.pack(q, b, fmt)
        assert np.array_equal(R.code_values(codes, fmt), q)
        assert np.array_equal(scales[R.scale_places(130, b.shape[1])], b)
        R.check_quantised(codes, scales, x, 0.0, fmt, 1.0)
        bad = codes.copy()
        bad[7, 5] ^= 0x11
        with pytest.raises(AssertionError):
            R.check_quantised(bad, scales, x, 0.0, fmt, 1.0)


def test_sizes(lib):
    assert lib.llama_mx_code_bytes(R.NVFP4, 3, 96) == 3 * 48 and lib.llama_mx_code_bytes(R.FP8, 3, 96) == 3 * 96
    assert lib.llama_mx_scale_bytes(R.NVFP4, 129, 96) == 2 * 2 * 512
    assert lib.llama_mx_scale_bytes(R.FP4, 128, 96) == 512 and lib.llama_mx_scale_bytes(R.FP8, 1, 160) == 1024
    assert lib.llama_mx_scale_bytes(R.FP8, 0, 160) == 0
    for fmt, rows, cols in ((0, 4, 64), (4, 4, 64), (1, -1, 64), (1, 4, 0), (1, 4, 48), (3, 4, 100), (1, 1 << 30, 64),
                            (2, 1, (1 << 26) + 32)):
        assert lib.llama_mx_code_bytes(fmt, rows, cols) == 0 and lib.llama_mx_scale_bytes(fmt, rows, cols) == 0


def matrix(fmt=R.NVFP4, rows=4, cols=64, g=1.0, codes=FAKE, scales=FAKE):
    return ctypes.byref(lb.LlamaMxMatrix(fmt, rows, cols, g, codes, scales))


BAD_MATRICES = (dict(fmt=0), dict(fmt=4), dict(rows=-1), dict(cols=0), dict(codes=None), dict(scales=None),
                dict(g=0.0), dict(g=-1.0), dict(g=3.0), dict(g=math.inf), dict(g=math.nan), dict(g=2.0 ** 33),
                dict(g=2.0 ** -33), dict(fmt=R.FP4, g=2.0), dict(fmt=R.FP8, g=0.5))
UNSUPPORTED_MATRICES = (dict(cols=48), dict(cols=8), dict(codes=FAKE + 4), dict(scales=FAKE + 8), dict(rows=1 << 30))


@pytest.mark.parametrize("write", [True, False])
def test_quantise_and_read_back_are_refused_on_the_host(lib, write):
    def call(x=FAKE, stride=64, m=None, **kw):
        m = matrix(**kw) if m is None else m
        return lib.llama_quantize_mx(x, stride, m, None) if write else lib.llama_dequantize_mx(m, x, stride, None)
    for kw in BAD_MATRICES + (dict(x=None), dict(stride=56), dict(stride=-64)):
        assert call(**kw) == ARG, kw
    for kw in UNSUPPORTED_MATRICES[2:4] + (dict(cols=48), dict(stride=68), dict(x=FAKE + 8)):
        assert call(**kw) == UNSUP, kw
    null = ctypes.POINTER(lb.LlamaMxMatrix)()
    assert call(m=null) == ARG
    assert call(rows=0, x=None, codes=None, scales=None) == lb.LLAMA_OK


def test_norm_is_refused_on_the_host(lib):
    def call(x=FAKE, res=FAKE, out=FAKE, gamma=FAKE, eps=1e-5, **kw):
        return lib.llama_fused_add_rmsnorm_mx(x, res, out, matrix(**kw), gamma, eps, None)
    for kw in BAD_MATRICES + (dict(x=None), dict(gamma=None), dict(eps=-1.0), dict(eps=math.nan)):
        assert call(**kw) == ARG, kw
    for kw in UNSUPPORTED_MATRICES + (dict(cols=16416), dict(x=FAKE + 2), dict(res=FAKE + 8), dict(out=FAKE + 8),
                                      dict(gamma=FAKE + 8)):
        assert call(**kw) == UNSUP, kw
    assert call(rows=0, x=None, codes=None, scales=None, gamma=None) == lb.LLAMA_OK


def test_products_are_refused_on_the_host(lib):
    def linear(x={}, w={}, alpha=1.0, y=FAKE):
        return lib.llama_linear_mx(matrix(**x), matrix(**{"rows": 8, **w}), alpha, y, 0, None)

    def silu(x={}, w={}, alpha=1.0, y=FAKE, up={}, beta=1.0, out=None):
        size = {"rows": 8, "cols": w.get("cols", 64), **{k: w[k] for k in ("rows", "fmt") if k in w}}
        out = None if out is None else matrix(**{"fmt": R.FP8, "rows": 4, "cols": 8, **out})
        return lib.llama_gate_up_silu_mx(matrix(**x), matrix(**{"rows": 8, **w}), matrix(**{**size, **up}), alpha, beta, y,
                                         out, None)
    for call in (linear, silu):
        for kw in BAD_MATRICES:
            assert call(x=kw) == ARG and call(w=kw) == ARG, kw
        for kw in (dict(x=dict(cols=96)), dict(w=dict(fmt=R.FP4)), dict(w=dict(rows=0)), dict(alpha=math.nan),
                   dict(alpha=math.inf), dict(alpha=3e38, x=dict(g=4.0)), dict(y=None)):
            assert call(**kw) == ARG, kw
        for kw in UNSUPPORTED_MATRICES:
            assert call(x=kw) == UNSUP and call(w=kw) == UNSUP, kw
        for kw in (dict(w=dict(rows=12)), dict(y=FAKE + 8)):
            assert call(**kw) == UNSUP, kw
        assert call(x=dict(rows=0, codes=None, scales=None), y=None) == lb.LLAMA_OK
    for kw in BAD_MATRICES + (dict(fmt=R.FP8), dict(rows=16), dict(cols=96)):
        assert silu(up=kw) == ARG, kw
    assert silu(beta=math.nan) == ARG
    w32 = dict(rows=32)
    for kw in (dict(fmt=0), dict(rows=5), dict(cols=64), dict(g=2.0), dict(codes=None)):
        assert silu(w=w32, y=None, out={"cols": 32, **kw}) == ARG, kw
    assert silu(w=w32, out=dict(cols=32)) == ARG  # y and out
    for kw in (dict(codes=FAKE + 8), dict(scales=FAKE + 8)):
        assert silu(w=w32, y=None, out={"cols": 32, **kw}) == UNSUP, kw
    assert silu(w=dict(rows=40), y=None, out=dict(cols=40)) == UNSUP


def test_binding_refuses_what_is_not_a_matrix():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    lb.MxMatrix(R.NVFP4, 64, u8(3, 32), u8(512))
    for fmt, cols, codes, scales in ((R.NVFP4, 64, u8(3, 64), u8(512)), (R.NVFP4, 64, u8(3, 32), u8(511)),
                                     (R.FP8, 64, u8(3, 64).char(), u8(512)), (R.FP8, 64, u8(3, 64), u8(512).int()),
                                     (R.FP8, 64, u8(3, 128)[:, ::2], u8(512)), (R.FP8, 64, u8(192), u8(512)),
                                     (5, 64, u8(3, 64), u8(512)), (R.FP8, 48, u8(3, 48), u8(512))):
        with pytest.raises(lb.LlamaError):
            lb.MxMatrix(fmt, cols, codes, scales)
    for fmt, rows, cols in ((0, 3, 64), (R.FP4, -1, 64), (R.FP4, 3, 40)):
        with pytest.raises(lb.LlamaError):
            lb.MxMatrix.empty(fmt, rows, cols, device="cpu")


def test_a_matrix_cannot_be_changed():
    m = lb.MxMatrix.empty(R.NVFP4, 3, 64, 0.5, device="cpu")
    assert (m.c.format, m.c.rows, m.c.cols, m.c.g, m.c.codes) == (R.NVFP4, 3, 64, 0.5, m.codes.data_ptr())
    for name in ("scale", "codes", "rows"):
        with pytest.raises(AttributeError):
            setattr(m, name, getattr(m, name))


def test_binding_refuses_tensors_of_another_kind():
    m = lb.MxMatrix.empty(R.FP8, 4, 64, device="cpu")
    other = lb.MxMatrix.empty(R.FP4, 4, 64, device="cpu")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    y = torch.zeros(4, 4, dtype=torch.bfloat16)
    gamma = torch.ones(64, dtype=torch.bfloat16)
    for call in (
            lambda: lb.quantize_mx(x.float(), m, stream=0), lambda: lb.quantize_mx(x[:3], m, stream=0),
            lambda: lb.quantize_mx(torch.zeros(64, 4, dtype=torch.bfloat16).T, m, stream=0),
            lambda: lb.dequantize_mx(m, x.half(), stream=0), lambda: lb.dequantize_mx(m, x[:, :32], stream=0),
            lambda: lb.fused_add_rmsnorm_mx(x.float(), None, None, m, gamma, 1e-5, stream=0),
            lambda: lb.fused_add_rmsnorm_mx(x, x[:3], None, m, gamma, 1e-5, stream=0),
            lambda: lb.fused_add_rmsnorm_mx(x, None, x.float(), m, gamma, 1e-5, stream=0),
            lambda: lb.fused_add_rmsnorm_mx(x, None, None, m, gamma[:32], 1e-5, stream=0),
            lambda: lb.linear_mx(m, other, y, stream=0), lambda: lb.linear_mx(m, m, y.half(), stream=0),
            lambda: lb.linear_mx(m, m, y[:3], stream=0), lambda: lb.linear_mx(m, m, y.T[:, :3].T, stream=0),
            lambda: lb.gate_up_silu_mx(m, m, other, y, stream=0),
            lambda: lb.gate_up_silu_mx(m, m, lb.MxMatrix.empty(R.FP8, 5, 64, device="cpu"), y, stream=0),
            lambda: lb.gate_up_silu_mx(m, m, m, y.float(), stream=0),
            lambda: lb.gate_up_silu_mx(m, m, m, m, stream=0)):
        with pytest.raises(lb.LlamaError):
            call()
    # of the right kind, but not where the call runs
    for call in (lambda: lb.quantize_mx(x, m, stream=0), lambda: lb.dequantize_mx(m, x, stream=0),
                 lambda: lb.fused_add_rmsnorm_mx(x, None, None, m, gamma, 1e-5, stream=0),
                 lambda: lb.linear_mx(m, m, y, stream=0), lambda: lb.gate_up_silu_mx(m, m, m, y, stream=0)):
        with pytest.raises(lb.LlamaError):
            call()
