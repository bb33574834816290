"""The operators for decode steps over long contexts on the CPU: host-side refusals of their C
entry points and of the binding, the shared plan, and pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.attention import mla_decode_ref
from oracle.fp8 import e4m3fn_decode
from oracle.long_context import (attend_ref, block_means_ref, block_scores_ref, block_select_ref, shared_ref,
                                 written_pages)

INVALID, WS_SMALL = 1, 3


@pytest.fixture(scope="module")
def lib(built_library):
    return binding.load_library(built_library)


def ptr(offset=0):
    """A pointer that is never dereferenced: the checks fail first."""
    return ctypes.c_void_p((1 << 20) + offset)


def shared_args(made, **change):
    args = dict(q=ptr(), kv=ptr(), scale=ptr(), qo=ptr(), kvi=ptr(), out=ptr(), lse=None, stream=None,
                plan=ctypes.byref(made), indices=None, indices_len=0, rows=4096, ws=ptr(), ws_bytes=made.ws_bytes)
    return {**args, **change}.values()


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(q=ptr(8)), INVALID), (dict(kv=None), INVALID), (dict(kv=ptr(4)), INVALID),
    (dict(scale=None), INVALID), (dict(scale=ptr(2)), INVALID), (dict(qo=None), INVALID), (dict(qo=ptr(1)), INVALID),
    (dict(kvi=None), INVALID), (dict(kvi=ptr(2)), INVALID), (dict(out=None), INVALID), (dict(out=ptr(8)), INVALID),
    (dict(lse=ptr(2)), INVALID), (dict(plan=None), INVALID), (dict(indices=ptr(2), indices_len=4), INVALID),
    (dict(indices=ptr(), indices_len=-1), INVALID), (dict(indices=ptr(), indices_len=2**31), INVALID),
    (dict(rows=0), INVALID), (dict(rows=2**31), INVALID), (dict(ws=None), INVALID), (dict(ws=ptr(128)), INVALID),
    (dict(ws_bytes=0), WS_SMALL)])
def test_shared_refusals(lib, change, status):
    plan = binding.mla_shared_plan(1, 64, 8192, 152)
    assert plan.split == 1
    assert lib.mla_shared_fwd(*shared_args(plan, **change)) == status
    assert lib.mla_shared_fwd_stall_stream(*shared_args(plan, **change)) == status


def test_shared_refuses_a_changed_plan(lib):
    for field, value in [("workers", 0), ("workers", 3), ("workers", 4097), ("split", 0), ("split", 2),
                         ("abi_version", 4), ("start", -1), ("start", 65), ("ws_lse_offset", 0), ("batch", 0), ("batch", 65537),
                         ("batch", 1025), ("total_q", -1), ("max_kv_len", -1), ("num_sms", 0)]:
        plan = binding.mla_shared_plan(1, 64, 8192, 152)
        setattr(plan, field, value)
        assert lib.mla_shared_fwd(*shared_args(plan)) == INVALID, (field, value)


def test_shared_of_no_queries_launches_nothing(lib):
    plan = binding.mla_shared_plan(2, 0, 8192, 152)
    assert lib.mla_shared_fwd(*shared_args(plan, q=None, out=None)) == 0


@pytest.mark.parametrize("batch,total,kv,sms", [(1, 1, 1, 152), (1, 8, 1000, 152), (1, 64, 8192, 152), (5, 200, 6001, 152),
                                                (1, 256, 32768, 152), (12, 40, 3000, 7), (1, 4, 0, 152), (2000, 2000, 9000, 152),
                                                (1, 70000, 100, 152), (1, 1, 2**31 - 1, 152)])
def test_shared_plan(lib, batch, total, kv, sms):
    plan = binding.mla_shared_plan(batch, total, kv, sms)
    assert 1 <= plan.workers <= sms and plan.split in (0, 1) and plan.start >= 0
    assert batch <= 1024 or plan.split == 0
    rows = 2 * plan.workers * 64 if plan.split else 0
    assert plan.ws_lse_offset == 256 and plan.ws_partial_offset % 256 == 0
    assert plan.ws_partial_offset >= 256 + 4 * rows and plan.ws_bytes >= plan.ws_partial_offset + 2 * 512 * rows


def test_shared_plan_refusals(lib):
    for args in [(0, 1, 1, 1), (65537, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1)]:
        with pytest.raises(binding.MlaError):
            binding.mla_shared_plan(*args)
    assert lib.mla_shared_plan(1, 1, 1, 1, None) == INVALID


@pytest.mark.parametrize("name,extra", [("mla_decode_fwd", 6), ("mla_decode_fwd_bf16kv", 5)])
def test_decode_lse_refusals(lib, name, extra):
    plan = binding.mla_decode_plan(2, 300, 152)
    args = [ptr(), ptr(), ptr(), ptr(), ptr(), ptr(), None, ctypes.byref(plan), None, 0, 300, ptr(), plan.ws_bytes]
    if "bf16kv" in name:
        del args[2]
    call = getattr(lib, name + "_lse")
    for lse in (None, ptr(2)):
        assert call(*args[:extra], lse, *args[extra:]) == INVALID
    args[-1] = 16
    assert call(*args[:extra], ptr(), *args[extra:]) == WS_SMALL


def test_mxfp4_lse_refusals(lib):
    plan = binding.mla_decode_plan(2, 300, 152)
    for lse in (None, ptr(2)):
        assert lib.mla_decode_fwd_mxfp4_lse(ptr(), ptr(), ptr(), 0, ptr(), ptr(), ptr(), lse, None, ctypes.byref(plan), 300,
                                            ptr(), plan.ws_bytes) == INVALID


MEANS = dict(kv=ptr(), scale=ptr(), rows=4096, slots=ptr(), tokens=8, means=ptr(), pages=64, page=64, ws=ptr(), ws_bytes=256)


@pytest.mark.parametrize("change,status", [
    (dict(kv=None), INVALID), (dict(kv=ptr(8)), INVALID), (dict(scale=None), INVALID), (dict(scale=ptr(2)), INVALID),
    (dict(rows=0), INVALID), (dict(rows=2**31), INVALID), (dict(slots=None), INVALID), (dict(slots=ptr(2)), INVALID),
    (dict(tokens=-1), INVALID), (dict(tokens=2**31), INVALID), (dict(means=None), INVALID), (dict(means=ptr(8)), INVALID),
    (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(ws=None), INVALID), (dict(ws=ptr(64)), INVALID),
    (dict(ws_bytes=255), WS_SMALL)])
def test_means_refusals(lib, change, status):
    args = {**MEANS, **change}
    assert lib.mla_block_means(*args.values(), None) == status
    if "scale" not in change:
        del args["scale"]
        assert lib.mla_block_means_bf16kv(*args.values(), None) == status


def test_means_of_no_tokens_launch_nothing(lib):
    assert lib.mla_block_means(*{**MEANS, "tokens": 0, "slots": None, "kv": None}.values(), None) == 0


SCORES = dict(q=ptr(), total=4, means=ptr(), pages=64, table=ptr(), row=16, width=16, qo=ptr(), kv=ptr(), batch=4, page=64,
              scores=ptr(), out_row=16, ws=ptr(), ws_bytes=256)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(q=ptr(8)), INVALID), (dict(total=-1), INVALID), (dict(means=None), INVALID),
    (dict(means=ptr(4)), INVALID), (dict(pages=0), INVALID), (dict(table=None), INVALID), (dict(table=ptr(2)), INVALID),
    (dict(row=15), INVALID), (dict(row=1 << 36), INVALID), (dict(width=0), INVALID), (dict(qo=None), INVALID),
    (dict(kv=None), INVALID), (dict(qo=ptr(1)), INVALID), (dict(kv=ptr(1)), INVALID), (dict(batch=0), INVALID),
    (dict(batch=16385), INVALID), (dict(page=0), INVALID), (dict(scores=None), INVALID), (dict(scores=ptr(2)), INVALID),
    (dict(out_row=15), INVALID), (dict(out_row=1 << 36), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=8), WS_SMALL),
    (dict(width=(1 << 30) + 1, row=1 << 31, out_row=1 << 31), INVALID)])
def test_scores_refusals(lib, change, status):
    assert lib.mla_block_scores(*{**SCORES, **change}.values(), None) == status


SELECT = dict(scores=ptr(), in_row=16, table=ptr(), row=16, width=16, kv=ptr(), batch=4, page=64, pages=64, blocks=8, sink=1,
              recent=2, ptr=ptr(), indices=ptr(), room=2048, chosen=None, ws=ptr(), ws_bytes=256)


@pytest.mark.parametrize("change,status", [
    (dict(scores=None), INVALID), (dict(scores=ptr(2)), INVALID), (dict(in_row=8), INVALID), (dict(in_row=1 << 36), INVALID),
    (dict(table=None), INVALID), (dict(table=ptr(2)), INVALID), (dict(row=15), INVALID), (dict(row=1 << 36), INVALID),
    (dict(width=0), INVALID), (dict(kv=None), INVALID), (dict(kv=ptr(2)), INVALID), (dict(batch=0), INVALID),
    (dict(batch=16385), INVALID), (dict(page=0), INVALID), (dict(pages=0), INVALID), (dict(page=1 << 16, pages=1 << 15), INVALID),
    (dict(blocks=0), INVALID), (dict(blocks=8193), INVALID), (dict(sink=-1), INVALID), (dict(recent=0), INVALID),
    (dict(sink=7), INVALID), (dict(sink=2**31 - 1), INVALID), (dict(recent=9), INVALID), (dict(recent=2**31 - 1), INVALID),
    (dict(ptr=None), INVALID), (dict(ptr=ptr(2)), INVALID), (dict(indices=None), INVALID), (dict(indices=ptr(2)), INVALID),
    (dict(room=-1), INVALID), (dict(room=2**31), INVALID), (dict(chosen=ptr(2)), INVALID), (dict(ws=None), INVALID),
    (dict(ws_bytes=0), WS_SMALL), (dict(width=(1 << 30) + 1, row=1 << 31, in_row=1 << 31), INVALID)])
def test_select_refusals(lib, change, status):
    assert lib.mla_block_select(*{**SELECT, **change}.values(), None) == status


def test_the_binding_takes_no_cpu_tensors(lib):
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    q, pool, means = (torch.zeros(4, 16, 576, dtype=torch.bfloat16), torch.zeros(64, 576, dtype=torch.uint8),
                      torch.zeros(4, 576, dtype=torch.bfloat16))
    plan, scale, ws = binding.mla_shared_plan(1, 4, 64, 152), torch.ones(1), torch.zeros(256, dtype=torch.uint8)
    calls = [lambda: binding.mla_shared_fwd(q, pool, scale, i32(2), i32(2), q[..., :512], plan=plan, workspace=ws),
             lambda: binding.mla_block_means(pool, scale, i32(4), means, page_size=16, workspace=ws),
             lambda: binding.mla_block_means_bf16kv(means, i32(4), means, page_size=16, workspace=ws),
             lambda: binding.mla_block_scores(q, means, i32(4, 4), i32(5), i32(5), torch.zeros(4, 4), page_size=16, workspace=ws),
             lambda: binding.mla_block_select(torch.zeros(4, 4), i32(4, 4), i32(5), i32(5), i32(99), page_size=16, num_pages=4,
                                              blocks=4, sink=0, recent=1, workspace=ws),
             lambda: binding.mla_decode_fwd(q, pool, scale, i32(5), i32(5), q[..., :512], plan=binding.mla_decode_plan(4, 16, 152),
                                            workspace=ws, lse=torch.zeros(4, 16))]
    for call in calls:
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        binding.mla_block_means(means, scale, i32(4), means, page_size=16, workspace=ws)
    with pytest.raises(TypeError):
        binding.mla_block_means_bf16kv(pool, i32(4), means, page_size=16, workspace=ws)
    with pytest.raises(ValueError):
        binding.mla_block_means(pool[:, :512], scale, i32(4), means, page_size=16, workspace=ws)


# ---------------------------------------------------------------- the oracle itself
def test_shared_ref_is_the_decode_step_for_one_token_a_group():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 120, size=(50, 576)).astype(np.uint8)
    q, index = rng.standard_normal((3, 16, 576)), rng.permutation(50)
    out, lse = shared_ref(q, e4m3fn_decode(codes) * 0.25, [0, 1, 2, 3], [0, 7, 7, 40], index)
    assert np.allclose(out, mla_decode_ref(q, codes, np.float32(0.25), [0, 1, 2, 3], [0, 7, 7, 40], index), atol=1e-12)
    s = q[0] @ (e4m3fn_decode(codes) * 0.25)[index[:7]].T / 24
    assert np.allclose(lse[0], np.log(np.exp(s).sum(axis=1))) and (lse[1] == -np.inf).all()


def test_two_pieces_joined_by_their_lse_are_the_whole():
    rng = np.random.default_rng(1)
    q, keys = rng.standard_normal((2, 16, 576)), rng.standard_normal((30, 576))
    (a, la), (b, lb), (out, lse) = attend_ref(q, keys[:11]), attend_ref(q, keys[11:]), attend_ref(q, keys)
    total = np.logaddexp(la, lb)
    assert np.allclose(total, lse) and np.allclose(np.exp(la - total)[..., None] * a + np.exp(lb - total)[..., None] * b, out)


def test_written_pages():
    assert written_pages([5, 6, 7, 8, 9, 40, 3, -1, -1], 4) == [(1, 4), (2, 2), (10, 1), (0, 4)]
    assert written_pages([7, 8], 8) == [(0, 8), (1, 1)] and written_pages([], 4) == [] and written_pages([-1], 4) == []


def test_means_scores_and_choice_by_hand():
    values = np.arange(12)[:, None] * np.ones(576)
    means = block_means_ref(values, [4, 5, 6], np.full((3, 576), 9.0), 4)
    assert (means[0] == 9).all() and (means[1] == 5.0).all() and (means[2] == 9).all()
    q = np.zeros((1, 16, 576))
    q[0, 3, 0], q[0, 5, 0] = 24.0, -48.0
    assert block_scores_ref(q, means, [[2, 1, 7]], [0, 1], [0, 6], 4).tolist() == [[9.0, 5.0, -np.inf]]
    got = block_select_ref(np.array([[0, 3, 3, 1, 3, 9, 0]]), np.arange(7)[None] + 10, [0, 19], 3, 4, 1, 1)
    assert got["chosen"].tolist() == [[0, 1, 5, 6]]  # of equal scores the lower page
    assert got["indptr"].tolist() == [0, 10] and got["indices"].tolist() == [30, 31, 32, 33, 34, 35, 45, 46, 47, 48]
