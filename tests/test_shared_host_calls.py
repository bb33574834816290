"""What mla_shared_fwd's host side does in a call, counted on the CPU against stand-ins of the descriptors and launches:
keys in a row need TMA descriptors, keys by a page table none, and each failure is the call's error."""
import ctypes
import os
import shutil
import subprocess

import pytest

from mla_decode_attention_08_gb300 import binding

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "mla_decode_attention_08_gb300", "csrc")
CUDA_ERROR = 4


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    include = "/usr/local/cuda/include"
    if cxx is None or not os.path.exists(os.path.join(include, "cuda.h")):
        pytest.skip("no host C++ compiler or CUDA headers")
    out = str(tmp_path_factory.mktemp("host") / "libhost.so")
    # (-Bsymbolic: the stand-ins are the ones called, whatever else the process has loaded)
    subprocess.check_call([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", include, "-I", CSRC, "-x", "c++",
                           os.path.join(CSRC, "api_long.cu"), os.path.join(HERE, "shared_host_fakes.cpp"), "-o", out])
    lib = ctypes.CDLL(out)
    for name in ("mla_shared_plan", "mla_shared_fwd"):
        getattr(lib, name).restype, getattr(lib, name).argtypes = binding.SIGNATURES[name]
    return lib


class Counts:
    def __init__(self, lib):
        self.at = {n: ctypes.c_int.in_dll(lib, "fake_" + n) for n in ("maps", "launches", "joins", "maps_fail", "launch_fail")}
        for v in self.at.values():
            v.value = 0

    def set(self, name):
        self.at[name].value = 1

    def __call__(self):
        return tuple(self.at[n].value for n in ("maps", "launches", "joins"))


def call(lib, paged, batch=1, total=64, kv=8192):
    """A call whose pointers the stand-ins never follow."""
    plan, p = binding.mla_shared_plan_t(), lambda: ctypes.c_void_p(1 << 20)
    assert lib.mla_shared_plan(batch, total, kv, 152, ctypes.byref(plan)) == 0
    return plan, lib.mla_shared_fwd(p(), p(), p(), p(), p(), p(), None, None, ctypes.byref(plan), p() if paged else None,
                                    kv if paged else 0, 4096, p(), plan.ws_bytes)


@pytest.mark.parametrize("batch,total,kv,joins", [(1, 64, 8192, 1), (2000, 2000, 300, 0)])
def test_a_page_table_needs_no_descriptors(host, batch, total, kv, joins):
    counts = Counts(host)
    plan, status = call(host, True, batch, total, kv)
    assert status == 0 and plan.split == joins and counts() == (0, 1, joins)
    plan, status = call(host, False, batch, total, kv)
    assert status == 0 and counts() == (1, 2, 2 * joins)


def test_a_descriptor_that_cannot_be_made_fails_calls_that_need_it(host):
    counts = Counts(host)
    counts.set("maps_fail")
    assert call(host, True)[1] == 0 and counts() == (0, 1, 1)
    assert call(host, False)[1] == CUDA_ERROR and counts() == (1, 1, 1)


@pytest.mark.parametrize("paged", [False, True])
def test_nothing_is_joined_behind_a_launch_that_failed(host, paged):
    counts = Counts(host)
    counts.set("launch_fail")
    assert call(host, paged)[1] == CUDA_ERROR and counts()[1:] == (1, 0)
