"""Shared keys in plans that cut no block, over groups as unlike as a long document's and short prompts': whole blocks
are dealt out by their key tiles, so a worker's share may begin inside a block, or hold no block's start at all."""
import pytest

from mla_decode_attention_08_gb300 import binding
from tests.test_gpu_shared import KV_INDPTR, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("sms", [3, 152])
def test_one_long_group_among_many(paged, sms):
    q = [1] * 550 + [61] + [1, 0, 3] * 183
    kv = [n % 211 for n in range(550)] + [4001] + [(7 * n) % 130 for n in range(549)]
    c = Case(q, kv, paged, seed=40, lead=2, tail=3, sms=sms)
    assert c.plan.split == 0 and c.plan.start > 0
    for _ in range(2):
        assert c.run() == 0
        c.check()
    for t in (0, 1, -3, -2, -1):
        assert (c.out[t] == 7).all() and (c.lse[t] == 7).all()


@pytest.mark.parametrize("paged", [False, True])
def test_few_groups_of_many_blocks(paged):
    """Longer than the plan was told, so that blocks that it does not cut are longer than a share."""
    c = Case([9, 1, 40, 6], [40, 1000, 700, 0], paged, seed=41)
    c.plan = binding.mla_shared_plan(4, 56, 100, 7)
    c.plan.start = 4  # (not what the plan chooses for so few groups, and runs all the same)
    c.ws = binding.new_workspace(c.plan)
    assert c.plan.split == 0
    assert c.run() == 0
    c.check()


def test_groups_without_tokens_keys_or_sense():
    c = Case([0] * 700 + [61] + [0] * 700 + [2, 2], [3] * 700 + [900] + [0] * 700 + [0, 300], True, seed=42, sms=40)
    assert c.plan.split == 0 and c.plan.start > 0
    assert c.run() == 0
    c.check()
    c.kv[1402] = c.kv[1401] - 1  # a group that ends before it begins
    c.out.fill_(7.0)
    assert c.run() == KV_INDPTR
    assert (c.out[61:63] == 7).all() and not (c.out[:61] == 7).all() and not (c.out[63:] == 7).all()
