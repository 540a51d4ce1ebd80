"""The bounded wait of the score kernel's warps: all lanes get one answer, whether the phase ends,
the limit runs out, or both fall together, and a wait that gives up sets the status word.

No lane's limit is longer than a few ms, and the arrival does not wait for anything."""
import ctypes
import os
import subprocess

import pytest

from conftest import ROOT
from row_wise_topk_b200 import build as B
from test_abi import header_define

ALL = 0xFFFFFFFF
MS = 1_000_000


def compile_probe(folder):
    lib = os.path.join(folder, "libwait_probe.so")
    subprocess.run([B.nvcc(), *B.ARCH, "-O3", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "-I", B.CSRC, "-o", lib,
                    os.path.join(ROOT, "tests", "warp_wait_probe.cu")], check=True)
    return lib


def test_probe_compiles(tmp_path):
    assert hasattr(ctypes.CDLL(compile_probe(str(tmp_path))), "wait_probe")


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    f = ctypes.CDLL(compile_probe(str(tmp_path_factory.mktemp("probe")))).wait_probe
    f.argtypes = [ctypes.c_uint64] * 3 + [ctypes.POINTER(ctypes.c_uint32)]

    def run(delay, limit, skew):
        out = (ctypes.c_uint32 * 3)()
        assert f(delay, limit, skew, out) == 0
        return out[0], out[1], ctypes.c_int32(out[2]).value
    return run


@pytest.mark.gpu
def test_a_phase_that_ends(probe):
    assert probe(1, 1000 * MS, 0) == (ALL, ALL, 0)
    assert probe(2 * MS, 1000 * MS, 0) == (ALL, ALL, 0)


@pytest.mark.gpu
def test_a_phase_that_never_ends(probe):
    assert probe(0, 2 * MS, 0) == (0, 0, header_define("DSEL_ERR_DEVICE_TIMEOUT"))


@pytest.mark.gpu
def test_lanes_whose_limits_run_out_at_different_times(probe):
    # lane 0's limit is 1 ms, lane 31's 32 ms; the phase ends between the two, then around lane 0's
    assert probe(8 * MS, 1 * MS, 1 * MS)[0] == 0
    assert probe(0, 1 * MS, 1 * MS) == (0, 0, header_define("DSEL_ERR_DEVICE_TIMEOUT"))
    for us in range(900, 1100, 10):
        first, second, status = probe(us * 1000, 1 * MS, 20_000)
        assert first in (0, ALL) and second in (0, ALL)
        assert (status == 0) == (first == second == ALL)
