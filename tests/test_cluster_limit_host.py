"""How many clusters a device holds, as launches ask for it, without a GPU: once
on every device, and an error is neither kept nor taken for an answer."""

import ctypes
import os
import shutil
import subprocess

import pytest

from llama_decoder_layer_gb300 import build as lbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("clusters") / "cluster_limit_host.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(lbuild.nvcc()))), "include")
    subprocess.run([shutil.which("g++") or shutil.which("c++"), "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic",
                    "-I", lbuild.CSRC, "-I", cuda, "-o", so, os.path.join(HERE, "cluster_limit_host.cpp")], check=True)
    lib = ctypes.CDLL(so)

    def run(device, answer=30, get_error=0, error=0):
        out = (ctypes.c_int * 2)()
        return lib.ask(device, get_error, error, answer, out), out[0], out[1]

    return run


def test_it_is_asked_once_on_every_device(ask):
    assert ask(0, 30) == (0, 30, 1) and ask(0, 31) == (0, 30, 1)
    assert ask(1, 40) == (0, 40, 2) and ask(0, 41) == (0, 30, 2)
    # an error is returned, and the next call asks again
    assert ask(2, 50, error=2) == (2, -1, 3) and ask(2, 50, error=2) == (2, -1, 4)
    assert ask(2, 51) == (0, 51, 5) and ask(2, 52, error=2) == (0, 51, 5)
    assert ask(3, 60, get_error=100) == (100, -1, 5) and ask(3, 61) == (0, 61, 6)
    # none is an answer
    assert ask(4, 0) == (0, 0, 7) and ask(4, 9) == (0, 0, 7)
    # devices past the table: every time
    assert ask(70, 5) == (0, 5, 8) and ask(70, 6) == (0, 6, 9)


def test_microscaled_products_ask_it():
    """Nothing else keeps an answer: a failed one would change the order of sums for the life of the process."""
    with open(os.path.join(lbuild.CSRC, "gemm_mx.cu")) as src:
        assert "cudaOccupancyMaxActiveClusters" not in src.read()
