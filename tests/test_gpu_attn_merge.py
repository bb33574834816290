"""mla_attn_merge against the float64 definition.

Tolerance: the result is rounded once to bf16 (2^-8 relative).  Before that a
weight exp(lse - top) carries the rounding of its argument (2^-24 of |lse - top|,
and |d| exp(-d) < 1/2, so below 2^-24 of the largest weight) and expf's 2 ulp; at
most 64 float32 additions and the division follow: within 2^-17 of the weighted
mean of magnitudes.  The lse: 64 additions and logf's ulps, 2^-17, and the rounding
of the sum, 2^-23 of its size."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.ops import merge_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def make(pieces, shape, dim, seed=0, empty=0.2, spread=6.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    parts = torch.randn((pieces, *shape, dim), generator=g, device="cuda").bfloat16()
    lses = spread * torch.randn((pieces, *shape), generator=g, device="cuda")
    lses[torch.rand(lses.shape, generator=g, device="cuda") < empty] = -float("inf")
    return parts, lses


def check(parts, lses, out, lse):
    want, want_lse, reach = merge_ref(parts.double().cpu().numpy(), lses.double().cpu().numpy())
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * reach).all()
    if lse is not None:
        gl = lse.double().cpu().numpy()
        unseen = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(gl), unseen)
        assert (np.abs(gl[~unseen] - want_lse[~unseen]) <= 2.0 ** -17 + 2.0 ** -23 * np.abs(want_lse[~unseen])).all()
        assert (got[unseen] == 0).all()


def run(parts, lses, with_lse=True, stream=None):
    out = torch.full(parts.shape[1:], float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full(lses.shape[1:], float("nan"), device="cuda") if with_lse else None
    assert binding.mla_attn_merge(parts, lses, out, stream, lse_out=lse) is out
    return out, lse


@pytest.mark.parametrize("pieces", [1, 2, 3, 4, 5, 9, 64])
@pytest.mark.parametrize("shape,dim", [((1, 1), 128), ((7, 3), 128), ((33, 16), 128), ((5,), 8), ((50, 16), 512),
                                       ((3, 5), 1024), ((301,), 40)])
def test_matches_the_definition(pieces, shape, dim):
    parts, lses = make(pieces, shape, dim, seed=pieces)
    check(parts, lses, *run(parts, lses, with_lse=pieces % 2 == 1))


def test_pieces_far_apart_and_rows_nobody_saw():
    parts, lses = make(3, (40, 2), 128, empty=0.0, spread=80.0)
    lses[:, 5] = -float("inf")
    lses[0, 6], lses[1, 6], lses[2, 6] = 1e30, -1e30, -float("inf")
    lses[:, 7] = -1e4                                     # far below zero, and alike
    check(parts, lses, *run(parts, lses))


def test_an_unseen_piece_is_not_read():
    parts, lses = make(3, (64,), 128, empty=0.0)
    lses[1, ::2] = -float("inf")
    clean = run(parts, lses)[0]
    parts[1, ::2] = float("nan")
    assert torch.equal(run(parts, lses)[0], clean)


def test_over_one_of_its_parts():
    parts, lses = make(2, (30, 16), 128)
    want, _ = run(parts, lses)
    binding.mla_attn_merge(parts, lses, parts[0])
    assert torch.equal(parts[0], want)


def test_graph_replay_and_another_stream():
    parts, lses = make(4, (100, 16), 128)
    out, lse = run(parts, lses)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.mla_attn_merge(parts, lses, out, lse_out=lse)
    p2, l2 = make(4, (100, 16), 128, seed=9)
    parts.copy_(p2)
    lses.copy_(l2)
    g.replay()
    torch.cuda.synchronize()
    check(p2, l2, out, lse)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(parts, lses, stream=s)
    s.synchronize()
    check(p2, l2, *got)


def test_binding_refusals():
    parts, lses = make(2, (4, 2), 128)
    out = torch.empty((4, 2, 128), dtype=torch.bfloat16, device="cuda")
    for bad in [(parts.float(), lses, out), (parts, lses.double(), out), (parts, lses, out.float())]:
        with pytest.raises(TypeError):
            binding.mla_attn_merge(*bad)
    for bad in [(parts, lses[:1], out), (parts, lses, out[:2]), (parts.transpose(1, 2), lses.transpose(1, 2), out)]:
        with pytest.raises(ValueError):
            binding.mla_attn_merge(*bad)
    with pytest.raises(binding.MlaError):
        binding.mla_attn_merge(parts[..., :4].contiguous(), lses, out[..., :4].contiguous())
