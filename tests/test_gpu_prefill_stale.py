"""mla_prefill_fwd with cut keys writes nothing that the call itself has not computed: not for rows that
offsets going back leave out, and not after waits that ran out."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from .test_gpu_prefill import QO_INDPTR, TIMEOUT, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def stale(c, value):
    """Parts of an earlier call in the workspace: outputs of ``value`` with log-sum-exps of zero."""
    n = c.plan.splits * c.q.shape[0] * c.heads
    at = c.plan.ws_lse_offset
    c.ws[at:at + 4 * n].view(torch.float32).zero_()
    at = c.plan.ws_partial_offset
    c.ws[at:at + 4 * 128 * n].view(torch.float32).fill_(value)


def test_rows_that_offsets_going_back_leave_out():
    """The first 1024 queries twice: 8 + 8 + 1 blocks of 128 queries, where rows in order have at most 12, so
    the short row with the fewest keys is not computed."""
    c = Case([1024, 0, 0, 48], [4000, 3999, 3998, 60], heads=1)
    assert c.plan.splits > 1 and c.q.shape[0] == 1072
    c.d_qo.copy_(torch.tensor([0, 1024, 0, 1024, 1072], dtype=torch.int32))
    stale(c, 1000.0)
    c.run()
    assert binding.mla_decode_read_error(c.ws) == QO_INDPTR
    assert (c.out == 7.0).all() and (c.lse == 7.0).all()
    # the same workspace, rows in order again
    c.d_qo.copy_(torch.tensor(c.qo.tolist(), dtype=torch.int32))
    stale(c, 1000.0)
    c.run()
    c.check()


@pytest.mark.parametrize("batch", [4, 40])
def test_replayed_with_offsets_that_go_back_and_come_right(batch):
    q = [3] * batch
    kv = (4000 - 7 * np.arange(batch)).tolist()
    c = Case(q, kv, heads=1, tail=2)
    assert c.plan.splits > 1
    c.run()
    c.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    good = c.d_qo.clone()
    for _ in range(2):
        c.d_qo[1] = 9                                   # past the second row's end
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        graph.replay()
        assert binding.mla_decode_read_error(c.ws) == QO_INDPTR
        assert (c.out == 7.0).all() and (c.lse == 7.0).all()
        c.d_qo.copy_(good)
        graph.replay()
        c.check()


def test_a_call_whose_waits_ran_out():
    c = Case([64], [4000], heads=2, tail=3)
    assert c.plan.splits > 1
    stale(c, 1000.0)
    c.run(fn=binding.mla_prefill_fwd_stall_stream)
    assert binding.mla_decode_read_error(c.ws) == TIMEOUT
    assert (c.out == 7.0).all() and (c.lse == 7.0).all()
    c.run()
    c.check()
