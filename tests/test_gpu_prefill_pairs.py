"""mla_prefill_fwd's two walks.  Batches whose rows have at most 128 queries, or that leave SMs
idle: the key tiles alternate between the two softmax warpgroups, whose accumulators are
joined at a job's end.  Numbers of key tiles odd and even, jobs that start with either
warpgroup, rows that see keys in one of the two only.  And batches planned for one SM, whose
jobs are of two query tiles.  Tolerances as derived for the other prompt tests: the joining multiplies
each float32 accumulator by a power-of-two exponential (2^-22) and adds, far below the
2^-16 (spread + 1) that they allow beside the two bf16 roundings."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from .test_gpu_prefill import QO_INDPTR, TIMEOUT, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,length", [(1, 128), (1, 129), (128, 256), (100, 257), (128, 384), (33, 400), (97, 513),
                                      (128, 130), (128, 3), (127, 1290)])
def test_tiles_of_one_row(n, length, causal):
    c = Case([n], [length], heads=3, causal=causal, seed=n + length, lead=2, tail=3, sms=1)
    c.run()
    c.check()


@pytest.mark.parametrize("sms", [1, 5, 152])
@pytest.mark.parametrize("causal", [True, False])
def test_jobs_start_with_either_warpgroup(sms, causal):
    """Few blocks work through jobs of 0, 1, 2, 3, ... key tiles."""
    kv = [100, 1, 300, 0, 129, 513, 128, 70, 900, 384, 20, 256, 0, 640, 90]
    q = [100, 1, 17, 5, 128, 128, 64, 70, 2, 0, 20, 128, 0, 99, 128]
    c = Case(q, kv, heads=5, causal=causal, seed=sms, lead=1, tail=4, sms=sms)
    c.run()
    c.check()
    out, lse = c.out.clone(), c.lse.clone()
    c.run()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q,kv", [([128], [8000]), ([3, 128, 40], [4000, 2500, 1]), ([1], [1152])])
def test_split_and_paired(q, kv, causal):
    c = Case(q, kv, heads=2, causal=causal, seed=sum(kv), lead=1, tail=2)
    assert c.plan.splits > 1
    c.run()
    c.check()


@pytest.mark.parametrize("batch,sms", [(33, 152), (50, 3), (300, 152), (64, 1)])
def test_many_short_rows(batch, sms):
    rng = np.random.default_rng(batch + sms)
    q = rng.integers(0, 129, batch)
    kv = q + rng.integers(0, 400, batch) * (rng.random(batch) < 0.5)
    c = Case(q.tolist(), kv.tolist(), heads=2, seed=batch, tail=1, sms=sms)
    c.run()
    c.check()


@pytest.mark.parametrize("first_large", [True, False])
def test_maxima_far_apart(first_large):
    """One warpgroup's scores exceed the other's by hundreds: its weight alone is left."""
    c = Case([64], [512], heads=2, causal=False, seed=3, sms=1)
    keys = (torch.arange(512, device="cuda") // 128 % 2 == 0) == first_large
    c.q[:] = c.q.abs()
    c.k_nope[keys] = c.k_nope[keys].abs() * 8
    c.run()
    c.check()


def test_rows_that_see_one_tile_beside_rows_that_see_two():
    """Causal rows whose second key tile is masked as a whole: its maximum is the lowest."""
    c = Case([128], [256], heads=2, seed=5, sms=1)
    c.run()
    c.check()
    c = Case([128], [129], heads=2, seed=6, sms=1, tail=4)
    c.run()
    c.check()


def test_a_row_of_129_queries_beside_short_ones():
    c = Case([128, 129, 1], [500, 700, 300], heads=3, seed=9, tail=2)
    c.run()
    c.check()


@pytest.mark.parametrize("q,kv", [([300, 5], [700, 40]), ([300, 5], [4000, 3000])])
def test_replayed_graph_switches_between_the_forms(q, kv):
    """One captured call over rows that the device finds short, then long, then short."""
    c = Case(q, kv, heads=2, seed=4)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    for qo in ([0, 300, 305], [0, 128, 200], [0, 177, 305], [0, 1, 1], [0, 300, 305]):
        c.d_qo.copy_(torch.tensor(qo, dtype=torch.int32))
        c.qo = np.array(qo, dtype=np.int64)
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        graph.replay()
        c.check()


def test_waits_that_run_out_are_reported():
    c = Case([64, 3], [700, 300], heads=2, seed=1)
    c.run(fn=binding.mla_prefill_fwd_stall_stream)
    torch.cuda.synchronize()
    assert binding.mla_decode_read_error(c.ws) == TIMEOUT
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    c.run()
    c.check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q,kv,heads,sms", [([300, 200], [4000, 1500], 2, 19),    # parts over several rounds
                                            ([400], [3000], 8, 152),              # many rows to join
                                            ([303], [2000], 8, 152)])             # the last that join at once
def test_parts_joined(q, kv, heads, sms, causal):
    c = Case(q, kv, heads=heads, causal=causal, seed=sum(kv) + sms, lead=1, tail=1 if len(q) > 1 else 0, sms=sms)
    assert c.plan.splits > 1
    if sms == 19:
        assert (c.q.shape[0] // 128 + len(q)) * heads * c.plan.splits > sms
    c.run()
    c.check()


# ---- planned for one SM: jobs of two query tiles, which larger GPUs only use for more work
SIZES = [129, 191, 255, 256, 257, 383, 384, 512, 700]


@pytest.mark.parametrize("n", SIZES)
def test_one_prompt_in_jobs_of_two_tiles(n):
    c = Case([n], [n], heads=2, seed=n, tail=n % 3, sms=1)
    c.run()
    c.check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("layout", ["thd", "htd"])
@pytest.mark.parametrize("q,kv", [([130], [1000]), ([256], [640]), ([300], [300]), ([200], [70]), ([400], [129]),
                                  ([260], [0]), ([5, 0, 300, 128, 1, 77, 0, 513, 2], [5, 9, 300, 500, 0, 80, 0, 513, 700])])
def test_rows_in_jobs_of_two_tiles(q, kv, layout, causal):
    c = Case(q, kv, heads=3, causal=causal, layout=layout, seed=sum(q) + sum(kv), lead=2, tail=3, sms=1)
    assert c.plan.splits == 1
    c.run()
    c.check()


def test_both_walks_give_the_same_attention():
    a, b = (Case([700, 300], [900, 300], heads=2, seed=12, sms=sms) for sms in (1, 152))
    a.run()
    b.run()
    a.check()
    b.check()


def test_waits_of_jobs_of_two_tiles_that_run_out_are_reported():
    c = Case([300, 10], [300, 40], heads=2, sms=1)
    c.run(fn=binding.mla_prefill_fwd_stall_stream)
    torch.cuda.synchronize()
    assert binding.mla_decode_read_error(c.ws) == TIMEOUT
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    c.run()
    c.check()


@pytest.mark.parametrize("batch,sms", [(20, 152), (20, 1), (400, 152), (400, 1)])
def test_offsets_that_go_back_and_forth_are_reported_and_end(batch, sms):
    """Every second row is the whole of the tokens: many times the blocks that rows in order have."""
    c = Case([300] + [0] * (batch - 1), [300] + [0] * (batch - 1), heads=2, seed=1, tail=4, sms=sms)
    c.d_qo.copy_(torch.tensor([0, 300] * (batch // 2) + [0], dtype=torch.int32))
    c.run()
    assert binding.mla_decode_read_error(c.ws) & QO_INDPTR
    assert (c.out[300:] == 7.0).all() and (c.lse[300:] == 7.0).all()
    d = Case([300], [300], heads=2, seed=1, sms=sms)
    d.run()
    d.check()
