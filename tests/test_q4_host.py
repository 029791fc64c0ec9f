"""The 4-bit cache and the head norm with rotation without a GPU: the format's
layout, the quantisation reference, and every refusal on the host."""

import ctypes
import math

import numpy as np
import pytest
import torch

import q4_reference as R
from llama_decoder_layer_gb300 import binding as lb
from llama_decoder_layer_gb300 import build as lbuild

FAKE = 256  # an aligned address nothing reads: every call here is refused before a launch


@pytest.fixture(scope="module")
def lib():
    lbuild.build()
    return lb.lib()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_every_code_and_scale_has_a_place_of_its_own(d, is_v):
    codes = {(R.code_place(d, k, e, is_v), e % 2) for k in range(16) for e in range(d)}
    scales = {R.scale_place(d, k, s, is_v) for k in range(16) for s in range(d // 16)}
    assert codes == {(b, i) for b in range(8 * d) for i in (0, 1)}
    assert scales == set(range(8 * d, 9 * d))
    # tokens share no byte
    owner = {}
    for k in range(16):
        for e in range(d):
            assert owner.setdefault(R.code_place(d, k, e, is_v), k) == k


def test_reference_quantisation_on_hand_worked_rows():
    x = np.zeros((1, 16))
    x[0, :8] = [6.0, -3.0, 0.25, 0.75, 2.5, 5.0, -0.2, 0.26]
    code, s8 = R.quantise(x, 1.0)
    assert R.E4M3[s8[0, 0]] == 1.0
    # ties: 0.25 -> 0, 0.75 -> 1, 2.5 -> 2, 5 -> 4
    assert list(R.value(code, s8, 1.0)[0, :8]) == [6.0, -3.0, 0.0, 1.0, 2.0, 4.0, 0.0, 0.5]
    # a scale that underflows stores zeros, one that overflows saturates
    assert R.value(*R.quantise(np.full((1, 16), 2.0 ** -9), 1.0), 1.0).max() == 0.0
    assert R.value(*R.quantise(np.full((1, 16), 1e30), 1.0), 1.0).max() == 6 * 448


def test_tile_bytes(lib):
    assert lb.kv_cache_q4_tile_bytes(64) == 576 and lb.kv_cache_q4_tile_bytes(128) == 1152
    for d in (0, 32, 96, 256, -64):
        with pytest.raises(lb.LlamaError):
            lb.kv_cache_q4_tile_bytes(d)


def _cache_call(lib, write, **kw):
    a = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, slots=FAKE, T=4, nkv=8, d=128, bs=16, nb=10, kg=1.0, vg=1.0, kc=FAKE,
             vc=FAKE)
    a.update(kw)
    if write:
        return lib.kv_cache_write_q4(a["k"], a["ks"], a["v"], a["vs"], a["slots"], a["T"], a["nkv"], a["d"], a["bs"],
                                     a["nb"], a["kg"], a["vg"], a["kc"], a["vc"], None)
    return lib.kv_cache_read_q4(a["kc"], a["vc"], a["slots"], a["T"], a["nkv"], a["d"], a["bs"], a["nb"], a["kg"],
                                a["vg"], a["k"], a["ks"], a["v"], a["vs"], None)


@pytest.mark.parametrize("write", [True, False])
def test_cache_calls_are_refused_on_the_host(lib, write):
    ARG, UNSUP = lb.LLAMA_ERR_ARG, lb.LLAMA_ERR_UNSUPPORTED
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None), dict(T=-1), dict(nkv=0),
               dict(nb=0), dict(d=0), dict(bs=0), dict(ks=1016), dict(vs=0), dict(ks=-1024), dict(nb=1 << 28),
               dict(kg=0.0), dict(kg=-1.0), dict(kg=3.0), dict(vg=math.inf), dict(vg=math.nan), dict(vg=2.0 ** -33),
               dict(kg=2.0 ** 33)):
        assert _cache_call(lib, write, **kw) == ARG, kw
    for kw in (dict(d=96), dict(bs=32), dict(ks=1028), dict(vs=1025), dict(k=FAKE + 8), dict(v=FAKE + 2),
               dict(kc=FAKE + 4), dict(vc=FAKE + 8)):
        assert _cache_call(lib, write, **kw) == UNSUP, kw
    # no tokens: nothing to do, whatever the pointers
    assert _cache_call(lib, write, T=0, k=None, v=None, slots=None, kc=None, vc=None) == lb.LLAMA_OK


def test_binding_refuses_tensors_of_another_kind(lib):
    kc, vc = torch.zeros(4, 2, 576, dtype=torch.uint8), torch.zeros(4, 2, 576, dtype=torch.uint8)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    bad = [dict(k=k.float()), dict(k=k[:, :, ::2]), dict(k=torch.zeros(3, 4, 64, dtype=torch.bfloat16)[:, ::2]),
           dict(v=k[:2]), dict(slots=slots.long()), dict(slots=slots[:2]), dict(kc=kc.int()), dict(kc=kc[:, :1]),
           dict(vc=torch.zeros(4, 2, 1152, dtype=torch.uint8)), dict(vc=vc[:3])]
    for b in bad:
        a = {"k": k, "v": k, "slots": slots, "kc": kc, "vc": vc, **b}
        with pytest.raises(lb.LlamaError):
            lb.kv_cache_write_q4(a["k"], a["v"], a["slots"], a["kc"], a["vc"], stream=0)
        with pytest.raises(lb.LlamaError):
            lb.kv_cache_read_q4(a["kc"], a["vc"], a["slots"], a["k"], a["v"], stream=0)


def _attn_call(lib, cfg=None, batch=None, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, kg=1.0, vg=1.0, pre=0, out=FAKE, ws=FAKE, n=1 << 40)
    a.update(kw)
    c = (cfg or lb.LayerConfig(512, 8, 2, 64, 1376, 1e-5, 1e4)).c()
    b = lb.LlamaBatch(4, 4, 8, 40, 1, 100, FAKE, FAKE, FAKE, FAKE, None)
    for name, x in (batch or {}).items():
        setattr(b, name, x)
    return lib.llama_paged_attention_q4(ctypes.byref(c), ctypes.byref(b), a["q"], a["kc"], a["vc"], a["kg"], a["vg"],
                                        a["pre"], a["out"], a["ws"], a["n"], None)


def test_attention_is_refused_on_the_host(lib):
    ARG, UNSUP = lb.LLAMA_ERR_ARG, lb.LLAMA_ERR_UNSUPPORTED
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(out=None), dict(kg=1.5), dict(vg=0.0),
               dict(kg=math.nan), dict(pre=-1), dict(pre=1 << 27)):
        assert _attn_call(lib, **kw) == ARG, kw
    for kw in (dict(q=FAKE + 8), dict(kc=FAKE + 4), dict(vc=FAKE + 8), dict(out=FAKE + 2)):
        assert _attn_call(lib, **kw) == UNSUP, kw
    assert _attn_call(lib, ws=None) == lb.LLAMA_ERR_WORKSPACE
    assert _attn_call(lib, n=16) == lb.LLAMA_ERR_WORKSPACE
    # the batch's and the configuration's checks are those of llama_paged_attention
    for b in (dict(num_seqs=0), dict(num_seqs=5), dict(positions=None), dict(max_query_len=0), dict(max_seq_len=0),
              dict(num_blocks=0), dict(max_query_len=5)):
        assert _attn_call(lib, batch=b) == ARG, b
    assert _attn_call(lib, batch=dict(num_tokens=0), q=None, out=None, ws=None) == lb.LLAMA_OK
    assert _attn_call(lib, cfg=lb.LayerConfig(512, 8, 2, 96, 1376, 1e-5, 1e4)) == UNSUP
    assert _attn_call(lib, cfg=lb.LayerConfig(4096, 32, 1, 128, 1376, 1e-5, 1e4)) == UNSUP
    assert lib.llama_paged_attention_q4(None, None, None, None, None, 1.0, 1.0, 0, None, None, 0, None) == ARG


def test_attention_workspace_sizes(lib):
    cfg = lb.LayerConfig(512, 8, 2, 64, 1376, 1e-5, 1e4)
    sizes = [lb.paged_attention_q4_workspace_size(cfg, 64, 4, 4096, n) for n in (0, 1, 100, 100000)]
    assert all(n > 0 for n in sizes) and sizes == sorted(sizes)
    for bad in ((-1, 4, 4096, 0), (64, -1, 4096, 0), (64, 4, -1, 0), (64, 4, 4096, -1)):
        with pytest.raises(lb.LlamaError):
            lb.paged_attention_q4_workspace_size(cfg, *bad)
    assert lb.prefill_blocks([1, 2, 3, 40, 0], [100, 33, 17, 40, 9], 8) == 2 + 3
    assert lb.prefill_blocks([1, 1], [100, 100], 16) == 0


def _qk_call(lib, cfg=None, **kw):
    c = dict(n_heads=8, n_kv_heads=2, head_dim=64, rotary_dim=64, interleaved=0, rms_eps=1e-6, rope_theta=1e4,
             rope_scaling=0, rs_factor=1.0, rs_low_freq_factor=1.0, rs_high_freq_factor=4.0, rs_original_max_pos=8192,
             rs_attention_factor=1.0)
    c.update(cfg or {})
    s = lb.LlamaQkNormRopeConfig(**c)
    a = dict(qw=FAKE, kw=FAKE, pos=FAKE, T=4, q=FAKE, qs=512, k=FAKE, ks=128, qo=FAKE, qos=512, ko=FAKE, kos=128)
    a.update(kw)
    return lib.llama_qk_norm_rope(ctypes.byref(s), a["qw"], a["kw"], a["pos"], a["T"], a["q"], a["qs"], a["k"], a["ks"],
                                  a["qo"], a["qos"], a["ko"], a["kos"], None)


def test_norm_rope_is_refused_on_the_host(lib):
    ARG, UNSUP = lb.LLAMA_ERR_ARG, lb.LLAMA_ERR_UNSUPPORTED
    for c in (dict(n_heads=0), dict(n_kv_heads=0), dict(head_dim=0), dict(rotary_dim=-16), dict(rotary_dim=80),
              dict(rms_eps=-1.0), dict(rms_eps=math.nan), dict(interleaved=2), dict(rope_theta=0.0),
              dict(rope_theta=math.inf), dict(rope_scaling=4), dict(rope_scaling=-1),
              dict(rope_scaling=2, rs_factor=0.0), dict(rope_scaling=1, rs_high_freq_factor=1.0),
              dict(rope_scaling=1, rs_original_max_pos=0), dict(rope_scaling=3, rope_theta=1.0),
              dict(rope_scaling=3, rs_attention_factor=0.0), dict(rope_scaling=3, rs_low_freq_factor=0.0)):
        assert _qk_call(lib, cfg=c) == ARG, c
    for c in (dict(head_dim=96), dict(rotary_dim=24), dict(head_dim=128, rotary_dim=104)):
        assert _qk_call(lib, cfg=c) == UNSUP, c
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(T=-1), dict(qs=504),
               dict(ks=0), dict(qos=8), dict(kos=120)):
        assert _qk_call(lib, **kw) == ARG, kw
    for kw in (dict(q=FAKE + 8), dict(k=FAKE + 2), dict(qo=FAKE + 4), dict(ko=FAKE + 8), dict(qw=FAKE + 2),
               dict(kw=FAKE + 8), dict(qs=516), dict(kos=132)):
        assert _qk_call(lib, **kw) == UNSUP, kw
    assert _qk_call(lib, T=0, q=None, k=None, qo=None, ko=None, pos=None) == lb.LLAMA_OK
    assert lib.llama_qk_norm_rope(None, *([None] * 3), 4, *([None, 0] * 4), None) == ARG


def test_norm_rope_binding_refusals(lib):
    cfg = lb.QkNormRopeConfig(8, 2, 64)
    q, k = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    w, pos = torch.ones(64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    good = dict(qn=w, kn=w, pos=pos, q=q, k=k, qo=q, ko=k)
    for bad in (dict(q=k), dict(k=q), dict(qo=q[:2]), dict(ko=k.float()), dict(pos=pos.long()), dict(pos=pos[:2]),
                dict(qn=w.float()), dict(kn=w[:32]), dict(k=k[:2], ko=k[:2]), dict(q=q.transpose(1, 2))):
        a = {**good, **bad}
        with pytest.raises(lb.LlamaError):
            lb.qk_norm_rope(cfg, a["qn"], a["kn"], a["pos"], a["q"], a["k"], a["qo"], a["ko"], stream=0)
    with pytest.raises(lb.LlamaError):
        lb.QkNormRopeConfig(8, 2, 64, rope_scaling={"rope_type": "longrope"}).c()
