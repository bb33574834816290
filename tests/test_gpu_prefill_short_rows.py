"""mla_prefill_fwd on batches that make one block run through many jobs of one key tile each that the
row's end cuts: the two MMA issuers can then be a tile apart while V behind the rows' ends is
zeroed.  Tolerances as derived for the other prompt tests."""
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from .test_gpu_prefill import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sms", [1, 4])
@pytest.mark.parametrize("q,kv", [
    ([300] + [60] * 25, [300] + list(range(61, 86))),                 # one row of two query tiles, then one-tile jobs
    ([129, 5, 100, 1, 127] * 6, [129, 5, 100, 127, 1] * 6),           # both kinds in turn
    ([150] * 20, list(range(1, 21))),                                 # causal: only the second query tile sees keys
    ([200] + [3] * 60, [520] + [3 + i % 125 for i in range(60)]),     # more rows than lanes
])
def test_jobs_of_one_cut_tile_in_a_row(q, kv, sms, causal):
    c = Case(q, kv, heads=3, causal=causal, lead=1, tail=3, seed=len(q) + sms, sms=sms)
    assert c.plan.splits == 1
    for _ in range(3):
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        c.run()
        c.check()


def test_many_calls_repeat_themselves():
    c = Case([300] + [60] * 25, [300] + list(range(61, 86)), heads=16, tail=3, sms=152)
    c.run()
    c.check()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(50):
        c.out.fill_(7.0)
        c.run()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    assert binding.mla_decode_read_error(c.ws) == 0
