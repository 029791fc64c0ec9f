"""What a launch prepares on the host, without a GPU: kernels' shared-memory
limits are raised on every device, and a failure is not kept."""

import ctypes
import glob
import os
import shutil
import subprocess

import pytest

from llama_decoder_layer_gb300 import build as lbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def raise_on(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("smem") / "smem_limits_host.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(lbuild.nvcc()))), "include")
    subprocess.run([shutil.which("g++") or shutil.which("c++"), "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic",
                    "-I", lbuild.CSRC, "-I", cuda, "-o", so, os.path.join(HERE, "smem_limits_host.cpp")], check=True)
    lib = ctypes.CDLL(so)

    def run(device, get_error=0, set_error=0):
        calls = ctypes.c_int()
        return lib.raise_on(device, get_error, set_error, ctypes.byref(calls)), calls.value

    return run


def test_limits_are_raised_once_on_every_device(raise_on):
    assert raise_on(0) == (0, 2) and raise_on(0) == (0, 2)
    assert raise_on(1) == (0, 2) and raise_on(1) == (0, 2) and raise_on(0) == (0, 2)
    # an error is returned and the next call tries again
    assert raise_on(2, set_error=98) == (98, 1) and raise_on(2, set_error=98) == (98, 2)
    assert raise_on(2) == (0, 4) and raise_on(2) == (0, 4)
    assert raise_on(3, get_error=100) == (100, 0) and raise_on(3) == (0, 2)
    # devices past the table: every time
    assert raise_on(70) == (0, 2) and raise_on(70) == (0, 4)


def test_no_other_code_raises_them():
    for f in glob.glob(os.path.join(lbuild.CSRC, "*")):
        with open(f) as src:
            assert ("cudaFuncSetAttribute" in src.read()) == f.endswith("launch.cuh"), f
