"""A score that is NaN reaches its query's output and log-sum-exp, whatever the plan: queries that see a key
of NaN, or are NaN, get NaN, and every other query what it gets without it.  (Values and masked keys stay
finite, as the call asks; tolerances as derived for the other prompt tests.)"""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from .test_gpu_prefill import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def check(c, bad):
    """``bad[t, h]``: queries that have to be NaN."""
    assert bool(torch.isnan(c.out)[bad].all()) and bool(torch.isnan(c.lse)[bad].all())
    assert not bool(torch.isnan(c.out)[~bad].any()) and not bool(torch.isnan(c.lse)[~bad].any())


# walks and parts: two query tiles, alternating key tiles, and cut keys
SHAPES = [([300], [700], 1), ([100], [700], 1), ([100], [6000], 152), ([5, 300, 40], [90, 700, 400], 1)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q,kv,sms", SHAPES)
@pytest.mark.parametrize("key", [0, 130, -1])
def test_a_key_of_nan(q, kv, sms, causal, key):
    c = Case(q, kv, heads=2, causal=causal, seed=3, sms=sms, tail=2)
    assert (c.plan.splits > 1) == (sms > 1)
    c.run()
    want_out, want_lse = c.out.clone(), c.lse.clone()
    row = len(q) // 2
    at = kv[row] - 1 if key < 0 else key
    c.k_nope[int(c.kv[row]) + at, 1, 17] = float("nan")
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    c.run()
    assert binding.mla_decode_read_error(c.ws) == 0
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    for i in range(q[row]):
        bad[int(c.qo[row]) + i, 1] = not causal or kv[row] - q[row] + i >= at
    assert bool(bad.any())
    check(c, bad)
    assert torch.equal(c.out[~bad], want_out[~bad]) and torch.equal(c.lse[~bad], want_lse[~bad])


@pytest.mark.parametrize("q,kv,sms", SHAPES)
def test_a_query_of_nan(q, kv, sms):
    c = Case(q, kv, heads=2, seed=4, sms=sms)
    at = int(c.qo[len(q) // 2]) + 3
    c.q[at, 0, 5] = float("nan")
    c.run()
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[at, 0] = True
    check(c, bad)


def test_a_piece_of_nan_joins_to_nan():
    """The log-sum-exp of such a piece does not say that it saw no key."""
    c = Case([64], [200], heads=2, causal=False, seed=5)
    c.run()
    clean, clean_lse = c.out.clone(), c.lse.clone()
    c.k_rope[7, 3] = float("nan")
    c.run()
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    binding.mla_attn_merge(torch.stack([clean, c.out]), torch.stack([clean_lse, c.lse]), out, lse_out=lse)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


def test_nan_of_other_rows_and_of_masked_rows_does_not():
    """Queries of another row are NaN, and a row without keys still gets zeros."""
    c = Case([40, 3, 90], [300, 0, 300], heads=2, seed=6)
    c.q[:40] = float("nan")
    c.run()
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[:40] = True
    check(c, bad)
    assert bool((c.out[40:43] == 0).all()) and bool(torch.isneginf(c.lse[40:43]).all())
    assert np.isfinite(c.lse[43:].cpu().numpy()).all()
