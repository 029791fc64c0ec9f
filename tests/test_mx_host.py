"""Microscaled matrices without a GPU: the layout, the 64-bit reference on
hand-worked rows, and every refusal on the host."""

import math

import numpy as np
import pytest
import torch

import mx_reference as R
from llama_decoder_layer_gb300 import binding as lb
from llama_decoder_layer_gb300 import build as lbuild

FAKE = 256  # an aligned address nothing reads: every call here is refused before a launch
ARG, UNSUP, WS = lb.LLAMA_ERR_ARG, lb.LLAMA_ERR_UNSUPPORTED, lb.LLAMA_ERR_WORKSPACE


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
    for fmt, rows, cols in ((0, 4, 64), (4, 4, 64), (1, -1, 64), (1, 4, 0), (1, 4, 48), (3, 4, 100), (1, 1 << 30, 64)):
        assert lib.llama_mx_code_bytes(fmt, rows, cols) == 0 and lib.llama_mx_scale_bytes(fmt, rows, cols) == 0
    assert lb.linear_mx_workspace_size() > 0


def _rows_call(lib, write, **kw):
    a = dict(fmt=R.NVFP4, x=FAKE, stride=64, rows=4, cols=64, g=1.0, codes=FAKE, scales=FAKE)
    a.update(kw)
    if write:
        return lib.llama_quantize_mx(a["fmt"], a["x"], a["stride"], a["rows"], a["cols"], a["g"], a["codes"],
                                     a["scales"], None)
    return lib.llama_dequantize_mx(a["fmt"], a["codes"], a["scales"], a["rows"], a["cols"], a["g"], a["x"],
                                   a["stride"], None)


@pytest.mark.parametrize("write", [True, False])
def test_quantise_and_read_back_are_refused_on_the_host(lib, write):
    for kw in (dict(fmt=0), dict(fmt=4), dict(x=None), dict(codes=None), dict(scales=None), dict(rows=-1), dict(cols=0),
               dict(stride=56), dict(stride=-64), dict(g=0.0), dict(g=-1.0), dict(g=3.0), dict(g=math.inf),
               dict(g=math.nan), dict(g=2.0 ** 33), dict(g=2.0 ** -33), dict(fmt=R.FP4, g=2.0), dict(fmt=R.FP8, g=0.5)):
        assert _rows_call(lib, write, **kw) == ARG, kw
    for kw in (dict(cols=48), dict(cols=8), dict(stride=68), dict(x=FAKE + 8), dict(codes=FAKE + 4),
               dict(scales=FAKE + 8), dict(rows=1 << 30)):
        assert _rows_call(lib, write, **kw) == UNSUP, kw
    assert _rows_call(lib, write, rows=0, x=None, codes=None, scales=None) == lb.LLAMA_OK


def test_norm_is_refused_on_the_host(lib):
    def call(**kw):
        a = dict(fmt=R.FP8, x=FAKE, res=FAKE, out=FAKE, codes=FAKE, scales=FAKE, g=1.0, gamma=FAKE, rows=4, H=64, eps=1e-5)
        a.update(kw)
        return lib.llama_fused_add_rmsnorm_mx(a["fmt"], a["x"], a["res"], a["out"], a["codes"], a["scales"], a["g"],
                                              a["gamma"], a["rows"], a["H"], a["eps"], None)
    for kw in (dict(fmt=0), dict(fmt=7), dict(x=None), dict(codes=None), dict(scales=None), dict(gamma=None),
               dict(rows=-1), dict(H=0), dict(eps=-1.0), dict(eps=math.nan), dict(g=2.0), dict(fmt=R.NVFP4, g=5.0)):
        assert call(**kw) == ARG, kw
    for kw in (dict(H=48), dict(H=16416), dict(x=FAKE + 2), dict(res=FAKE + 8), dict(out=FAKE + 8),
               dict(codes=FAKE + 8), dict(scales=FAKE + 4), dict(gamma=FAKE + 8)):
        assert call(**kw) == UNSUP, kw
    assert call(rows=0, x=None, codes=None, scales=None, gamma=None) == lb.LLAMA_OK


def test_products_are_refused_on_the_host(lib):
    def linear(**kw):
        a = dict(fmt=R.NVFP4, xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, M=4, N=64, K=64, alpha=1.0, y=FAKE, f32=0, work=FAKE,
                 n=1 << 40)
        a.update(kw)
        return lib.llama_linear_mx(a["fmt"], a["xc"], a["xs"], a["wc"], a["ws"], a["M"], a["N"], a["K"], a["alpha"],
                                   a["y"], a["f32"], a["work"], a["n"], None)

    def silu(**kw):
        a = dict(fmt=R.NVFP4, xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, uc=FAKE, us=FAKE, M=4, N=64, K=64, alpha=1.0, beta=1.0,
                 of=0, og=1.0, y=FAKE, os=None, work=FAKE, n=1 << 40)
        a.update(kw)
        return lib.llama_gate_up_silu_mx(a["fmt"], a["xc"], a["xs"], a["wc"], a["ws"], a["uc"], a["us"], a["M"], a["N"],
                                         a["K"], a["alpha"], a["beta"], a["of"], a["og"], a["y"], a["os"], a["work"],
                                         a["n"], None)
    for call in (linear, silu):
        for kw in (dict(fmt=0), dict(fmt=4), dict(xc=None), dict(xs=None), dict(wc=None), dict(ws=None), dict(M=-1),
                   dict(N=0), dict(K=0), dict(alpha=math.nan), dict(alpha=math.inf), dict(y=None)):
            assert call(**kw) == ARG, kw
        for kw in (dict(K=48), dict(N=60), dict(xc=FAKE + 8), dict(xs=FAKE + 8), dict(wc=FAKE + 8), dict(ws=FAKE + 4),
                   dict(y=FAKE + 8)):
            assert call(**kw) == UNSUP, kw
        assert call(work=None) == WS and call(n=16) == WS
        assert call(M=0, xc=None, xs=None, wc=None, ws=None, y=None, work=None) == lb.LLAMA_OK
    for kw in (dict(uc=None), dict(us=None), dict(beta=math.nan), dict(of=-1), dict(of=4), dict(os=FAKE),
               dict(of=R.FP8), dict(of=R.FP8, os=FAKE, og=2.0), dict(of=R.NVFP4, os=FAKE, og=3.0)):
        assert silu(**kw) == ARG, kw
    for kw in (dict(uc=FAKE + 8), dict(us=FAKE + 8), dict(of=R.FP8, os=FAKE, N=72), dict(of=R.FP8, os=FAKE + 8)):
        assert silu(**kw) == UNSUP, kw


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


def test_binding_refuses_tensors_of_another_kind():
    m = lb.MxMatrix.empty(R.FP8, 4, 64, device="cpu")
    other = lb.MxMatrix.empty(R.FP4, 4, 64, device="cpu")
    x, ws = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.uint8)
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
            lambda: lb.linear_mx(m, other, y, ws, stream=0), lambda: lb.linear_mx(m, m, y.half(), ws, stream=0),
            lambda: lb.linear_mx(m, m, y[:3], ws, stream=0), lambda: lb.linear_mx(m, m, y.T[:, :3].T, ws, stream=0),
            lambda: lb.linear_mx(m, m, y, ws.float(), stream=0),
            lambda: lb.gate_up_silu_mx(m, m, other, y, ws, stream=0),
            lambda: lb.gate_up_silu_mx(m, m, lb.MxMatrix.empty(R.FP8, 5, 64, device="cpu"), y, ws, stream=0),
            lambda: lb.gate_up_silu_mx(m, m, m, y.float(), ws, stream=0),
            lambda: lb.gate_up_silu_mx(m, m, m, m, ws, stream=0)):
        with pytest.raises(lb.LlamaError):
            call()
    # of the right kind, but not where the call runs
    for call in (lambda: lb.quantize_mx(x, m, stream=0), lambda: lb.dequantize_mx(m, x, stream=0),
                 lambda: lb.fused_add_rmsnorm_mx(x, None, None, m, gamma, 1e-5, stream=0),
                 lambda: lb.linear_mx(m, m, y, ws, stream=0), lambda: lb.gate_up_silu_mx(m, m, m, y, ws, stream=0)):
        with pytest.raises(lb.LlamaError):
            call()
