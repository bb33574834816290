"""When the parts of cut keys are joined by threads that are all on the GPU at once (ops.h, compiled for the
host): four values a thread, two blocks of 256 threads an SM of the plan, on any number of SMs."""
import ctypes
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mla_decode_attention_08_gb300", "csrc")


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if cxx is None or not os.path.exists(nvcc):
        pytest.skip("no host C++ compiler or CUDA headers")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    out = str(tmp_path_factory.mktemp("rule") / "librule.so")
    subprocess.check_call([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-I", cuda,
                           os.path.join(HERE, "merge_rule.cpp"), "-o", out])
    fn = ctypes.CDLL(out).merges_at_once
    fn.restype, fn.argtypes = ctypes.c_bool, [ctypes.c_int64, ctypes.c_int32]
    return fn


@pytest.mark.parametrize("sms", [1, 19, 76, 148, 152, 160])
def test_the_limit_follows_the_plans_sms(rule, sms):
    rows = sms * 2 * 256 // (128 // 4)
    assert rule(rows, sms) and not rule(rows + 1, sms)
