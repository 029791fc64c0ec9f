"""How the 4-bit cache's row kernels share tokens among threads, walked on the
host over the header that the kernels are compiled from."""

import ctypes
import os
import shutil
import subprocess

import pytest

from llama_decoder_layer_gb300 import build as lbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rows") / "cache_rows_host.so")
    cxx = shutil.which("g++") or shutil.which("c++")
    subprocess.run([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", lbuild.CSRC, "-o", so,
                    os.path.join(HERE, "cache_rows_host.cpp")], check=True)
    lib = ctypes.CDLL(so)

    def run(n_kv, d, T, sms=152, loops=True):
        out = (ctypes.c_longlong * 8)()
        lib.walk(n_kv, d, T, sms, int(loops), out)
        names = ("uneven", "missed", "twice", "out_of_range", "u", "steps", "whole", "strangers")
        return dict(zip(names, out))

    return run


# (KV heads, head_dim, tokens from which a CTA of 152 SMs goes round again with rows that are no whole warps)
LOOPS = [(2, 64, 3649), (1, 128, 3649), (1, 64, 7297), (3, 128, 1217), (5, 128, 609), (3, 64, 4000), (7, 64, 2000)]


@pytest.mark.parametrize("n_kv,d,T", LOOPS)
@pytest.mark.parametrize("more", [0, 1, 2, 3, 5, 17, 611])
def test_the_lanes_of_a_warp_go_round_together(walk, n_kv, d, T, more):
    # the loop's body exchanges values over whole warps
    r = walk(n_kv, d, T + more)
    assert not r["whole"] and r["steps"] > 1
    assert r["uneven"] == 0 and r["strangers"] == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_kv", list(range(1, 36)) + [48, 63, 64, 65, 70])
@pytest.mark.parametrize("T", [1, 5, 40, 700])
@pytest.mark.parametrize("loops", [False, True])
def test_every_chunk_of_every_token_has_one_thread(walk, n_kv, d, T, loops):
    for sms in (152, 4):  # (few SMs: four tokens a thread, and steps)
        r = walk(n_kv, d, T, sms, loops)
        assert r["missed"] == 0 and r["twice"] == 0 and r["out_of_range"] == 0, (sms, r)
        assert r["uneven"] == 0 and r["strangers"] == 0, (sms, r)
