"""How blocks of query tokens over shared keys are cut into shares (schedule.h, compiled for the host): every key
tile of every block is one worker's, no two pieces share a slot, and the join finds the slots the workers used."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mla_decode_attention_08_gb300", "csrc")
i64, i32 = ctypes.c_int64, ctypes.c_int32


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    out = str(tmp_path_factory.mktemp("pieces") / "libpieces.so")
    subprocess.check_call([cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC,
                           os.path.join(HERE, "shared_pieces.cpp"), "-o", out])
    so = ctypes.CDLL(out)
    for name in ("share_begin", "share_owner"):
        getattr(so, name).restype, getattr(so, name).argtypes = i64, [i64] * 3
    so.piece_slot.restype, so.piece_slot.argtypes = i64, [i64, ctypes.c_bool]
    so.piece_of.restype, so.piece_of.argtypes = None, [i64, i32, i32, i64, i64, ctypes.POINTER(i32)]
    return so


@pytest.mark.parametrize("all_,workers", [(1, 1), (7, 7), (152, 152), (1000, 152), (2**48, 152), (2**49 + 12345, 8191), (3, 2)])
def test_shares_are_whole_equal_and_owned(lib, all_, workers):
    begins = [lib.share_begin(all_, workers, c) for c in range(workers + 1)]
    assert begins == [c * all_ // workers for c in range(workers + 1)]
    assert begins[-1] == all_ and min(np.diff(begins)) >= 1 and np.ptp(np.diff(begins)) <= 1
    for c in range(workers):
        for u in {begins[c], begins[c + 1] - 1}:
            assert lib.share_owner(all_, workers, u) == c


def check(lib, blocks, workers, start):
    """blocks: the key tiles of each."""
    size = [start + max(1, n) for n in blocks]
    first = np.concatenate([[0], np.cumsum(size)]).astype(int)
    all_ = int(first[-1])
    workers = min(workers, all_)
    had = [np.zeros(max(1, n), dtype=int) for n in blocks]
    used, out = {}, (i32 * 3)()
    for c in range(workers):
        u, stop = lib.share_begin(all_, workers, c), lib.share_begin(all_, workers, c + 1)
        jobs = 0
        while u < stop:
            b = int(np.searchsorted(first, u, side="right")) - 1
            lib.piece_of(int(first[b]), blocks[b], start, u, stop, out)
            j0, j1, whole = out
            assert 0 <= j0 <= blocks[b] and 0 <= j1 <= blocks[b]
            if whole:
                had[b] += 1
            elif j1 > j0:
                had[b][j0:j1] += 1
                # a worker's first piece continues a block or it is the last it has
                slot = lib.piece_slot(c, j0 == 0)
                assert slot not in used and 0 <= slot < 2 * workers
                used[slot] = (b, j0, j1)
            u, jobs = int(first[b + 1]), jobs + 1
    for b, n in enumerate(blocks):
        assert (had[b] == 1).all(), (b, had[b])
        tile0 = int(first[b]) + start
        w0 = lib.share_owner(all_, workers, tile0)
        w1 = lib.share_owner(all_, workers, tile0 + n - 1) if n > 0 else w0
        mine = {s for s, (of, _, _) in used.items() if of == b}
        joined = {lib.piece_slot(w, w == w0) for w in range(w0, w1 + 1)} if w1 > w0 else set()
        assert mine == joined, (b, mine, joined)
        at = 0
        for w in range(w0, w1 + 1) if w1 > w0 else ():
            _, j0, j1 = used[lib.piece_slot(w, w == w0)]
            assert j0 == at and j1 > j0
            at = j1
        assert w1 == w0 or at == n


@pytest.mark.parametrize("start", [0, 1, 4])
@pytest.mark.parametrize("workers", [1, 2, 19, 152])
def test_every_key_tile_is_one_workers(lib, workers, start):
    rng = np.random.default_rng(workers * 8 + start)
    for blocks in ([1], [0], [0, 0, 0], [1000], [64] * 16, [1] * 300, [0, 700, 0, 1, 3], [151], [152], [153]):
        check(lib, blocks, workers, start)
    for _ in range(60):
        n = int(rng.integers(1, 40))
        check(lib, [int(x) for x in rng.integers(0, 1 + int(rng.integers(1, 400)), size=n)], workers, start)
