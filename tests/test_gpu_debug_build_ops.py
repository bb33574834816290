"""The debug build's bounds checks in the operators around the decode step: present in every kernel file, and
none fails over the operators' shapes (an error word other than the expected one fails a run's own check)."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["stage1", "stage2", "page_map", "kv_append", "attn_merge", "prefill"])
def test_kernels_check_their_accesses(name):
    with open(os.path.join(ROOT, "mla_decode_attention_08_gb300", "csrc", name + ".cu")) as f:
        assert "MLA_DCHECK(" in f.read()


@pytest.mark.gpu
def test_no_check_fails():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_build_ops_check.py")],
                       capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    done = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(done) == len(set(done)) == 33
    assert any("cut" in name and "parts=1" not in name for name in done)
