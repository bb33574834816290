"""The operators around the decode step where offsets pass 32 bits, with queries shared by the heads, and with
many heads.  Tolerances as derived for the other tests of each operator."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.ops import prefill_ref
from .test_gpu_attn_merge import check as check_merge
from .test_gpu_kv_append import Case as AppendCase
from .test_gpu_prefill import Case, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def test_prompt_behind_two_to_the_31_elements():
    """Rows at the end of a million query tokens (2^31 elements of out) and of 600,000 keys."""
    tq, tk, heads = 1_048_700, 600_000, 16
    qo, kv = [tq - 150, tq - 20, tq], [tk - 700, tk - 400, tk]
    q = torch.zeros((tq, heads, 192), dtype=torch.bfloat16, device="cuda")
    expanded = torch.zeros((tk, heads, 256), dtype=torch.bfloat16, device="cuda")
    latent = torch.zeros((tk, 576), dtype=torch.bfloat16, device="cuda")
    q[qo[0]:] = rand(1, 150, heads, 192)
    expanded[kv[0]:] = rand(2, 700, heads, 256)
    latent[kv[0]:] = rand(3, 700, 576)
    out = torch.zeros((tq, heads, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((tq, heads), device="cuda")
    plan = binding.mla_prefill_plan(2, tq, 400, heads, 152)
    ws = binding.new_workspace(plan)
    d_qo, d_kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (qo, kv))
    binding.mla_prefill_fwd(q, expanded[..., :128], latent[:, 512:], expanded[..., 128:], d_qo, d_kv, out, plan=plan,
                            workspace=ws, lse=lse)
    assert binding.mla_decode_read_error(ws) == 0
    assert int((out[:qo[0]] != 0).any(dim=2).sum()) == 0 and int((lse[:qo[0]] != 0).sum()) == 0
    want, want_lse, reach, spread = prefill_ref(
        f64(q[qo[0]:]), f64(expanded[kv[0]:, :, :128]), f64(latent[kv[0]:, 512:]), f64(expanded[kv[0]:, :, 128:]),
        [x - qo[0] for x in qo], [x - kv[0] for x in kv], 192 ** -0.5, True)
    e = 2.0 ** -16 * (spread + 1)
    got = f64(out[qo[0]:])
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + e[..., None]) * reach).all()
    assert (np.abs(f64(lse[qo[0]:]) - want_lse) <= e + 2.0 ** -22 * np.abs(want_lse)).all()


def test_merge_of_more_than_two_to_the_31_elements():
    """The last rows of three pieces of 6,000,000 rows of 128."""
    rows = 6_000_000
    parts = torch.zeros((3, rows, 128), dtype=torch.bfloat16, device="cuda")
    lses = torch.full((3, rows), -float("inf"), device="cuda")
    parts[:, -40:] = rand(4, 3, 40, 128)
    lses[:, -40:] = rand(5, 3, 40).float()
    out = torch.full((rows, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(rows, device="cuda")
    binding.mla_attn_merge(parts, lses, out, lse_out=lse)
    check_merge(parts[:, -40:], lses[:, -40:], out[-40:], lse[-40:])
    assert int((out[:-40] != 0).any(dim=1).sum()) == 0 and bool(torch.isneginf(lse[:-40]).all())


@pytest.mark.parametrize("heads", [64, 128])
def test_prompt_of_many_heads(heads):
    c = Case([70, 3], [200, 140], heads=heads, seed=heads, tail=1)
    c.run()
    c.check()


@pytest.mark.parametrize("heads", [3, 128])
def test_append_with_one_query_for_all_heads(heads):
    """A query that is one tensor for all heads (head stride 0)."""
    c = AppendCase(17, heads)
    c.q_pe = rand(6, 17, 1, 64).expand(17, heads, 64)
    c.q0 = c.q_pe.clone()
    c.run()
    c.check()


def test_append_past_two_to_the_31_elements_of_queries():
    """Queries and their outputs whose element offsets pass 32 bits (the last tokens of 40,000 with wide rows)."""
    tokens, heads = 40_000, 4
    c = AppendCase(tokens, heads, e4m3=False, dense=False, kv_pad=0)
    wide = torch.zeros((tokens, heads, 16384), dtype=torch.bfloat16, device="cuda")
    wide[..., 16320:] = rand(7, tokens, heads, 64)
    c.q_pe = wide[..., 16320:]
    c.q0 = c.q_pe.clone()
    c.q_out = wide[..., 64:128]
    c.slots[:-50] = -1
    w = np.arange(tokens) >= tokens - 50
    c.run()
    c.check(written=w)
    assert int((wide[:-50, :, 64:128] != 0).sum()) == 0
