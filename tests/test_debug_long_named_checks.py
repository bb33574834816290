"""Which accesses the debug build checks in the operators of decode steps over long contexts: every load and store whose
place comes from device data is named here with the condition that guards it; and no check fails over shapes that the first
run of the debug build does not have."""
import json
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ACCESSES = [
    ("shared", "offsets of a group that a job is looked for in", r"r\.at \+ 1 < p\.batch"),
    ("shared", "keys by TMA", r"key >= 0 && key < p\.kv_rows"),
    ("shared", "entries of the page table", r"job\.k0 >= 0 && job\.keys > 0 && static_cast<int64_t>\(job\.k0\) \+ job\.keys <= p\.kv_limit"),
    ("shared", "rows of the cache by a page table", r"row >= 0 && row < p\.kv_rows"),
    ("shared", "queries", r"job\.q0 >= 0 && job\.q0 \+ g < p\.total_q"),
    ("shared", "outputs, parts and their log-sum-exps", r"parts \? job\.slot < 2 \* p\.workers && p\.split\s+: job\.q0 >= 0 && job\.q0 \+ g < p\.total_q"),
    ("shared", "parts that are joined, and the output", r"token < p\.total_q && w0 >= 0 && w1 < p\.workers && place >= 0 && place < kTokens"),
    ("block_means", "the list of ended pages", r"at < kThreads"),
    ("block_means", "rows of the cache", r"first >= 0 && first \+ rows <= p\.kv_rows && rows > 0"),
    ("block_means", "means", r"now\.page >= 0 && static_cast<int64_t>\(now\.page\) \* p\.page_size < p\.limit"),
    ("block_scores", "entries of the block table", r"j < p\.max_pages"),
    ("block_scores", "means", r"id < p\.num_pages"),
    ("block_scores", "queries", r"qs >= 0 && qs \+ t0 \+ row / kNumHeads < p\.total_q"),
    ("block_scores", "scores", r"j >= 0 && j < p\.max_pages"),
    ("block_select", "scores and entries of the block table", r"row\.pages <= p\.max_pages && hi <= row\.pages"),
    ("block_select", "counts of the steps", r"step >= 0 && step < kSteps"),
    ("block_select", "counts of the steps of the bits", r"step < kSteps"),
    ("block_select", "the list that is ranked", r"to < inside && to < kListed"),
    ("block_select", "chosen pages", r"place >= 0 && j >= 0 && j < row\.pages"),
    ("block_select", "cache rows of chosen pages", r"at < static_cast<uint32_t>\(row\.taken\) && before \+ t < p\.indices_len"),
]


@pytest.mark.parametrize("name,access,condition", ACCESSES, ids=[f"{a}-{b}" for a, b, _ in ACCESSES])
def test_an_access_is_checked(name, access, condition):
    with open(os.path.join(ROOT, "mla_decode_attention_08_gb300", "csrc", name + ".cu")) as f:
        assert re.search(r"MLA_DCHECK\((!here \|\| \()?" + condition, f.read()), access


@pytest.mark.gpu
def test_no_check_fails():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "debug_build_uneven_check.py")],
                       capture_output=True, text=True, timeout=900, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    done = json.loads(r.stdout.strip().splitlines()[-1])
    assert len(done) == len(set(done)) == 31
