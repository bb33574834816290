"""mla_shared_fwd up to the largest scores that it takes, 2^24: there a float32 score has no fraction left, so that the softmax
is one of whole steps, but its weights are still weights: outputs are finite and among the keys' values.

The reference is one rounding of the maximum away from it, 1 ulp of 1.4427 x 2^24 < 2^25, 2 at most in powers of two, and
probabilities of two powers above or below the reference's 2^4 have their two terms.  A term pair is off by 2^-8 and 2^-11 of its
probability and by 2^-10 where it is not zero, next to the 2^2 of the maximum at least: with n keys
|out| <= max |v| (1 + 2^-8 + 2^-10 + n 2^-12) before it is rounded to bf16, 2^-8 of itself."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from tests.test_gpu_shared import Case, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("power", [12, 20, 23])
@pytest.mark.parametrize("q_lens,kv_lens", [([5], [300]), ([3, 8], [40, 129])])
def test_weights_stay_weights(q_lens, kv_lens, power, paged):
    c = Case(q_lens, kv_lens, paged, seed=60 + power, amp=1.0)
    for g in range(len(q_lens)):  # each query's largest score lies in (2^(power - 1), 2^power] x (1 +- 2^-7)
        a, b = int(c.qo[g]), int(c.qo[g + 1])
        top = np.abs(f64(c.q[a:b]) @ c.keys(g).T / 24).max(axis=2)
        up = np.exp2(np.floor(power - np.log2(top)))
        c.q[a:b] *= torch.from_numpy(up).to("cuda", torch.bfloat16)[..., None]
    assert c.run() == 0
    out, lse = f64(c.out), f64(c.lse)
    for g in range(len(q_lens)):
        a, b = int(c.qo[g]), int(c.qo[g + 1])
        k = c.keys(g)
        most = np.abs(k[:, :512]).max(axis=0)
        limit = most * (1 + 2.0**-8 + 2.0**-10 + len(k) * 2.0**-12) * (1 + 2.0**-8)
        assert np.isfinite(out[a:b]).all() and (np.abs(out[a:b]) <= limit).all()
        s = f64(c.q[a:b]) @ k.T / 24
        spread = (np.abs(f64(c.q[a:b])) @ np.abs(k).T / 24).max(axis=2)
        low = np.abs(f64(c.q[a:b])).max(axis=2) * np.abs(k).sum(axis=1).max() / 24
        e = 2.0**-14 * spread + 2.0**-20 * low + 2.0**-20
        ref = np.log(np.exp(s - s.max(axis=2, keepdims=True)).sum(axis=2)) + s.max(axis=2)
        assert (np.abs(lse[a:b] - ref) <= e + 2.0**-22 * np.abs(ref) + 2.0).all()
