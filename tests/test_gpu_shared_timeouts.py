"""Waits of mla_shared_fwd that run out, in every form of the call: keys in a row or by a page table (other roles read a
job, and the copies have their own way out), blocks cut (the join writes the outputs) or whole (the first kernel does).
No copy is issued, so each wait gives up by itself and the call returns with its error word set."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from tests.test_gpu_shared import TIMEOUT, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("q_lens,kv_lens", [([6], [500]), ([9, 2, 5], [300, 129, 700])])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("split", [0, 1])
def test_outputs_stay_and_the_next_call_is_right(q_lens, kv_lens, paged, split):
    c = Case(q_lens, kv_lens, paged, seed=50, lead=1, tail=1)
    if not split:  # (told of short keys and one SM, the plan takes whole blocks)
        c.plan = binding.mla_shared_plan(len(q_lens), c.q.shape[0], 1, 1)
        c.ws = binding.new_workspace(c.plan)
    assert c.plan.split == split
    i32 = lambda a: torch.from_numpy(a.astype(np.int32)).cuda()
    if split:  # parts of an earlier call are in the workspace
        assert c.run() == 0
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
    binding.mla_shared_fwd_stall_stream(c.q, c.codes, c.scale, i32(c.qo), i32(c.kv), c.out, plan=c.plan, workspace=c.ws,
                                        kv_indices=c.indices, lse=c.lse)
    torch.cuda.synchronize()
    assert binding.mla_decode_read_error(c.ws) == TIMEOUT
    assert (c.out == 7).all() and (c.lse == 7).all()
    assert c.run() == 0
    c.check()
    for t in (0, -1):
        assert (c.out[t] == 7).all() and (c.lse[t] == 7).all()
