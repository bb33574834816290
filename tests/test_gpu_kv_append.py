"""mla_kv_append and its bf16 form against the float64 definition.

Tolerances, from the operator's arithmetic.  A float32 value v reaches its stored
type by one rounding: bf16 moves it by at most 2^-8 |v|, e4m3 by at most
max(2^-4 |v|, 2^-10) in code units.  Before it, float32 arithmetic: the sum of 512
squares (16 in a lane, five exchanges: at most 21 additions deep, all terms
positive), a reciprocal square root within 2 ulp and two products lie within
2^-18 of the exact value; a rotated value within 2^-22 (|a| + |b|) of it."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.fp8 import e4m3fn_decode
from oracle.ops import e4m3_target, kv_row_ref, rotate_ref

pytestmark = pytest.mark.gpu

KV_INDEX, POSITION = 4, 512
EPS = 1e-5
MAX_POS = 300


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def f64(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, tokens, heads=16, interleaved=True, e4m3=True, dense=True, kv_pad=64, seed=0, scale=0.02,
                 magnitude=1.0, q_layout="bhd"):
        g = torch.Generator(device="cuda").manual_seed(seed)
        def rand(*s):
            return torch.randn(s, generator=g, device="cuda")
        self.tokens, self.heads, self.interleaved, self.e4m3 = tokens, heads, interleaved, e4m3
        self.kv = (rand(tokens, 576 + kv_pad) * magnitude).bfloat16()[:, kv_pad:]
        self.weight = (1 + 0.3 * rand(512)).bfloat16()
        angle = torch.arange(MAX_POS, device="cuda")[:, None] * 10000.0 ** (-torch.arange(32, device="cuda") / 32)
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        self.positions = torch.randint(0, MAX_POS, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        self.rows = 2 * tokens + 7
        self.slots = torch.randperm(self.rows, generator=g, device="cuda")[:tokens].int()
        self.scale = torch.tensor([scale], device="cuda")
        if e4m3:
            self.cache = torch.randint(0, 0x7F, (self.rows, 576), generator=g, device="cuda", dtype=torch.uint8)
        else:
            self.cache = rand(self.rows, 576).bfloat16()
        if q_layout == "bhd":                       # the tail of [T, H, 192] queries, into [T, H, 576] ones
            self.q_pe = rand(tokens, heads, 192).bfloat16()[..., 128:]
            self.q_buf = rand(tokens, heads, 576).bfloat16()
            self.q_out = self.q_buf[..., 512:]
        else:                                       # heads outermost on both sides
            self.q_pe = rand(heads, tokens, 64).bfloat16().transpose(0, 1)
            self.q_buf = rand(heads, tokens, 64).bfloat16()
            self.q_out = self.q_buf.transpose(0, 1)
        self.dense = rand(tokens, 576).bfloat16() if dense else None
        self.ws = torch.zeros(binding.STEP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        self.before = [f64(self.cache), f64(self.q_buf), None if self.dense is None else f64(self.dense)]
        self.kv0, self.q0 = self.kv.clone(), self.q_pe.clone()

    def run(self, stream=None, **kw):
        args = [self.kv, self.weight, self.table, self.positions, self.slots, self.cache]
        more = dict(workspace=self.ws, eps=EPS, interleaved=self.interleaved, latent_out=self.dense,
                    q_pe=self.q_pe if self.heads else None, q_out=self.q_out if self.heads else None)
        if self.e4m3:
            binding.mla_kv_append(*args, self.scale, stream, **{**more, **kw})
        else:
            binding.mla_kv_append_bf16kv(*args, stream, **{**more, **kw})

    def check(self, error=0, written=None):
        """Tokens ``written`` (all by default) match the definition, everything else is as it was."""
        assert binding.mla_decode_read_error(self.ws) == error
        w = np.ones(self.tokens, bool) if written is None else np.asarray(written)
        pos = self.positions.cpu().numpy()[w]
        slots = self.slots.cpu().numpy()[w]
        turn = f64(self.table)[pos]
        cos, sin = turn[:, :32], turn[:, 32:]
        kv = f64(self.kv0)[w]
        row = kv_row_ref(kv, f64(self.weight), EPS, cos, sin, self.interleaved)
        slack = 2.0 ** -18 * np.abs(row)
        slack[:, 512:] = 2.0 ** -22 * 2 * np.abs(kv[:, 512:]).max(initial=0)
        cache = self.cache.cpu().numpy() if self.e4m3 else f64(self.cache)
        others = np.setdiff1d(np.arange(self.rows), slots)
        assert np.array_equal(cache[others], self.before[0][others])
        if self.e4m3:
            s = float(self.scale.item())
            want, got = e4m3_target(row, s), e4m3fn_decode(cache[slots])
            slack_q = slack / s + 2.0 ** -22 * np.abs(want)
            bound = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) * (1 + 2.0 ** -10) + slack_q
        else:
            want, got, bound = row, cache[slots], 2.0 ** -8 * np.abs(row) + slack
        assert (np.abs(got - want) <= bound).all()
        if self.dense is not None:
            d = f64(self.dense)
            assert (np.abs(d[w] - row) <= 2.0 ** -8 * np.abs(row) + slack).all()
            if self.before[2] is not None:
                assert np.array_equal(d[~w], self.before[2][~w])
        if self.heads:
            q = f64(self.q0)[w]
            want = rotate_ref(q, cos[:, None], sin[:, None], self.interleaved)
            got = f64(self.q_out)
            assert (np.abs(got[w] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * np.abs(q).max(initial=0)).all()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("tokens,heads", [(1, 16), (2, 1), (3, 0), (5, 7), (33, 8), (64, 16), (257, 9), (1000, 24)])
def test_matches_the_definition(tokens, heads, e4m3, interleaved):
    c = Case(tokens, heads, interleaved, e4m3, dense=tokens % 2 == 1, seed=tokens)
    c.run()
    c.check()
    if heads:                                    # the first 512 dims of the decode query stay
        assert np.array_equal(f64(c.q_buf)[..., :512], c.before[1][..., :512])


@pytest.mark.parametrize("e4m3", [True, False])
def test_heads_outermost(e4m3):
    c = Case(21, 5, False, e4m3, q_layout="hbd")
    c.run()
    c.check()


def test_values_past_the_range_saturate():
    c = Case(9, 0, scale=0.001, magnitude=3.0)    # normalised values near 1 / 0.001: past 448
    c.run()
    c.check()
    got = e4m3fn_decode(c.cache.cpu().numpy()[c.slots.cpu().numpy()])
    assert np.isfinite(got).all() and (np.abs(got) == 448).mean() > 0.3


def test_tiny_and_zero_latents():
    """Zero rows stay zero (eps keeps the norm finite), rows of 1e-20 do too."""
    c = Case(4, 2, e4m3=False)
    c.kv[0] = 0
    c.kv[1] = 1e-20
    c.kv0 = c.kv.clone()
    c.run()
    c.check()


def test_in_place():
    c = Case(37, 16, True, e4m3=False, kv_pad=0)
    c.before[2] = None
    c.dense = c.kv                                 # the dense copy over its source
    c.q_out = c.q_pe                               # the queries over themselves
    c.run()
    c.check()


def test_padding_tokens_are_skipped():
    c = Case(50, 16)
    c.slots[::3] = -1
    c.positions[::3] = -123                        # not looked at
    w = np.arange(50) % 3 != 0
    c.run()
    c.check(written=w)
    assert np.array_equal(f64(c.q_buf)[~w], c.before[1][~w])
    c.slots.fill_(-1)
    before = c.cache.clone()
    c.run()
    assert torch.equal(c.cache, before) and binding.mla_decode_read_error(c.ws) == 0


@pytest.mark.parametrize("e4m3", [True, False])
def test_bad_slots_and_positions_skip_their_token(e4m3):
    c = Case(20, 4, e4m3=e4m3)
    c.slots[3] = c.rows
    c.slots[7] = 2 ** 31 - 1
    w = np.ones(20, bool)
    w[[3, 7]] = False
    c.run()
    c.check(KV_INDEX, w)
    c = Case(20, 4, e4m3=e4m3)
    c.positions[0] = MAX_POS
    c.positions[19] = -1
    w = np.ones(20, bool)
    w[[0, 19]] = False
    c.run()
    c.check(POSITION, w)
    assert np.array_equal(f64(c.q_buf)[~w], c.before[1][~w])


def test_a_pool_past_2_to_31_bytes():
    """Rows whose byte offset passes 32 bits (4.6 GB of bf16 rows)."""
    c = Case(6, 2, e4m3=False)
    rows = 4_000_000
    pool = torch.zeros((rows, 576), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, rows - 1, 1_864_136, 3_728_271, 3_728_272, 2_000_003], dtype=torch.int32, device="cuda")
    small, c.cache = c.cache, pool
    keep, c.slots = c.slots, slots
    c.run()
    got = pool[slots.long()].clone()
    assert int((pool != 0).any(dim=1).sum()) == 6
    c.cache, c.slots = small, keep
    c.run()
    assert torch.equal(got, c.cache[keep.long()])


def test_graph_replay_and_streams():
    c = Case(40, 16, seed=11)
    c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.kv.copy_(torch.randn_like(c.kv.float()).bfloat16())
    c.positions.copy_((c.positions + 17) % MAX_POS)
    c.kv0 = c.kv.clone()
    g.replay()
    torch.cuda.synchronize()
    c.check()
    a, b = Case(300, 16, seed=12), Case(300, 16, seed=13)
    b.ws = a.ws
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a.run(sa)
    b.run(sb)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_bf16_rows_agree_with_the_per_tensor_quantiser():
    """The e4m3 rows are the library's own codes of the float32 row: with the dense
    bf16 copy quantised at the same scale they differ only where bf16 rounding moved a
    value across a code boundary."""
    c = Case(64, 0, e4m3=True)
    c.run()
    c.check()
    dense = f64(c.dense)
    codes = e4m3fn_decode(c.cache.cpu().numpy()[c.slots.cpu().numpy()]) * float(c.scale.item())
    assert (np.abs(codes - dense) <= (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -10) * np.abs(dense) + 2.0 ** -10 * 0.0201).all()


def test_binding_refusals():
    c = Case(8, 4)
    for name, value, err in [("kv", c.kv[:, :512], ValueError), ("weight", c.weight.float(), TypeError),
                             ("table", c.table[:, :32].contiguous(), ValueError), ("slots", c.slots[:4], ValueError),
                             ("q_pe", c.q_pe[..., ::2], ValueError), ("q_out", None, ValueError),
                             ("dense", c.dense[:4], ValueError), ("kv", c.kv.cpu(), TypeError),
                             ("cache", c.cache.bfloat16(), TypeError)]:
        keep = getattr(c, name)
        setattr(c, name, value)
        with pytest.raises(err):
            c.run()
        setattr(c, name, keep)
