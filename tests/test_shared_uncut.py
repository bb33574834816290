"""Blocks of query tokens over shared keys that are not cut (schedule.h, compiled for the host): each is one worker's,
and workers have about as many key tiles each, however unlike the groups are."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from mla_decode_attention_08_gb300 import binding

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mla_decode_attention_08_gb300", "csrc")
i64, i32 = ctypes.c_int64, ctypes.c_int32


@pytest.fixture(scope="module")
def pieces(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("uncut") / "libuncut.so")
    subprocess.check_call([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC,
                           os.path.join(HERE, "shared_uncut.cpp"), "-o", out])
    so = ctypes.CDLL(out)
    so.share_begin.restype, so.share_begin.argtypes = i64, [i64] * 3
    so.uncut_piece_of.restype, so.uncut_piece_of.argtypes = None, [i64, i32, i64, ctypes.POINTER(i32)]
    return so


def loads(lib, blocks, workers, start):
    """Units of each worker's blocks, for blocks of so many key tiles; every block is whole and had once."""
    size = start + np.maximum(1, blocks)
    first = np.concatenate([[0], np.cumsum(size)]).astype(int)
    all_ = int(first[-1])
    workers = min(workers, all_)
    had, load, out = np.zeros(len(blocks), dtype=int), np.zeros(workers, dtype=int), (i32 * 3)()
    for c in range(workers):
        u, stop = lib.share_begin(all_, workers, c), lib.share_begin(all_, workers, c + 1)
        while u < stop:
            b = int(np.searchsorted(first, u, side="right")) - 1
            lib.uncut_piece_of(int(first[b]), int(blocks[b]), u, out)
            j0, j1, whole = out
            if whole:
                assert (j0, j1) == (0, blocks[b])
                had[b] += 1
                load[c] += size[b]
            else:
                assert j0 == j1
            u = int(first[b + 1])
    assert (had == 1).all()
    return load, size


@pytest.mark.parametrize("start", [1, 4])
@pytest.mark.parametrize("workers", [1, 2, 19, 152])
def test_every_block_is_one_workers(pieces, workers, start):
    rng = np.random.default_rng(workers * 8 + start)
    few = [[1], [0], [0, 0, 0], [1000], [64] * 16, [1] * 300, [0, 700, 0, 1, 3]]
    for blocks in few + [rng.integers(0, 1 + int(rng.integers(1, 400)), size=int(rng.integers(1, 900))) for _ in range(40)]:
        load, size = loads(pieces, np.array(blocks), workers, start)
        # (a worker's blocks begin in its share, the last of them may end behind it)
        assert load.max() <= -(-size.sum() // len(load)) + size.max()


def test_one_long_group_among_many(pieces, built_library):
    """256 queries over 32768 keys among 1100 groups of one over 130: no worker has two of the long blocks."""
    binding.load_library(built_library)
    plan = binding.mla_shared_plan(1101, 1100 + 256, 32768, 152)
    assert plan.split == 0 and plan.workers == 152 and plan.start > 0
    blocks = np.array([2] * 550 + [256] * 64 + [2] * 550)
    load, size = loads(pieces, blocks, 152, plan.start)
    assert load.max() < 2 * 256


@pytest.mark.parametrize("batch,total,kv,start", [(2000, 100, 9000, 0), (1, 100, 64, 0), (2000, 2000, 9000, 4),
                                                  (2000, 2000, 128, 0), (300, 300, 100, 0), (1025, 1025, 129, 4)])
def test_blocks_are_weighed_where_groups_cannot_be_cut(built_library, batch, total, kv, start):
    binding.load_library(built_library)
    plan = binding.mla_shared_plan(batch, total, kv, 152)
    assert plan.split == 0 and plan.start == start and plan.ws_bytes == 256
