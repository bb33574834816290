"""mla_prefill_fwd against the float64 definition.

Tolerances, from the operator's arithmetic.  The output is rounded to bf16 (2^-8
relative), each probability too before the second product (2^-8 of the
attention-weighted mean of |v|, ``reach``, at worst).  Scores accumulate 192 float32
products: within 2^-16 of ``spread`` = max_j scale sum |q||k|, which is absolute in
the exponent and so relative in a probability; exp2's approximation and the float32
sums stay below 2^-16.  So |out - exact| <= 2^-8 |exact| + (2^-8 + e) reach with
e = 2^-16 (spread + 1), at every element; the lse is within e and its own rounding.
Those are worst cases; rounding errors have independent signs, so in the 2-norm the
two bf16 roundings stay below 2^-8 of the result each: 2^-7 bounds the relative
2-norm error, where one wrong key of a thousand costs 3 %."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.ops import prefill_ref

pytestmark = pytest.mark.gpu

QO_INDPTR, KV_INDPTR, TIMEOUT = 1, 2, 8


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def f64(t):
    return t.double().cpu().numpy()


def indptr(lens, start=0):
    return np.concatenate([[start], start + np.cumsum(lens)]).astype(np.int64)


class Case:
    """Ragged rows of ``q_lens`` queries over ``kv_lens`` keys.  ``lead``/``tail`` tokens that
    belong to no row hold NaN on the key side; ``layout`` orders heads and tokens."""

    def __init__(self, q_lens, kv_lens, heads=2, causal=True, seed=0, lead=0, tail=0, layout="thd", sms=152,
                 amp=1.5, scale=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        def rand(*s):
            return torch.randn(s, generator=g, device="cuda")
        self.heads, self.causal, self.scale = heads, causal, scale
        self.qo, self.kv = indptr(q_lens, lead), indptr(kv_lens, lead)
        tq, tk = int(self.qo[-1]) + tail, int(self.kv[-1]) + tail
        if layout == "thd":
            self.q = (amp * rand(tq, heads, 192)).bfloat16()
            e = rand(tk, heads, 256).bfloat16()
            self.k_nope, self.v = e[..., :128], e[..., 128:]
            self.k_rope = rand(tk, 576).bfloat16()[:, 512:]
        else:
            self.q = (amp * rand(heads, tq, 200)).bfloat16()[..., :192].transpose(0, 1)
            self.k_nope = rand(heads, tk, 128).bfloat16().transpose(0, 1)
            self.v = rand(heads, tk + 3, 136).bfloat16()[:, :tk, :128].transpose(0, 1)
            self.k_rope = rand(tk, 64).bfloat16()
        for t in (self.k_nope, self.v, self.k_rope):
            t[:lead] = float("nan")
            t[int(self.kv[-1]):] = float("nan")
        self.out = torch.full((tq, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((tq, heads), 7.0, device="cuda")
        self.d_qo, self.d_kv = (torch.tensor(x.tolist(), dtype=torch.int32, device="cuda") for x in (self.qo, self.kv))
        self.plan = binding.mla_prefill_plan(len(q_lens), tq, max(kv_lens), heads, sms)
        self.ws = binding.new_workspace(self.plan)

    def run(self, stream=None, fn=None, lse=True):
        (fn or binding.mla_prefill_fwd)(self.q, self.k_nope, self.k_rope, self.v, self.d_qo, self.d_kv, self.out, stream,
                                        plan=self.plan, workspace=self.ws, scale=self.scale, causal=self.causal,
                                        lse=self.lse if lse else None)

    def check(self):
        assert binding.mla_decode_read_error(self.ws) == 0
        want, lse, reach, spread = prefill_ref(f64(self.q), f64(self.k_nope), f64(self.k_rope), f64(self.v), self.qo,
                                               self.kv, self.scale or 192 ** -0.5, self.causal)
        got, got_lse = f64(self.out), f64(self.lse)
        inside = np.zeros(got.shape[0], bool)
        inside[self.qo[0]:self.qo[-1]] = True
        assert (got[~inside] == 7.0).all() and (got_lse[~inside] == 7.0).all()
        got, got_lse, want, lse, reach, spread = (x[inside] for x in (got, got_lse, want, lse, reach, spread))
        e = 2.0 ** -16 * (spread + 1)
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + e[..., None]) * reach).all()
        norm = np.linalg.norm(want)
        assert np.linalg.norm(got - want) <= 2.0 ** -7 * norm
        unseen = np.isneginf(lse)
        assert np.array_equal(np.isneginf(got_lse), unseen) and (got[unseen] == 0).all()
        assert (np.abs(got_lse[~unseen] - lse[~unseen]) <= (e + 2.0 ** -22 * np.abs(lse))[~unseen]).all()


SIZES = [1, 2, 64, 127, 128, 129, 191, 255, 256, 257, 383, 512, 700]


@pytest.mark.parametrize("n", SIZES)
def test_one_prompt(n):
    c = Case([n], [n], heads=2, seed=n, tail=n % 3)
    c.run()
    c.check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,length", [(1, 1), (1, 300), (5, 129), (128, 128), (130, 1000), (256, 640), (300, 300),
                                      (3, 2), (200, 70), (400, 129), (1, 0), (260, 0)])
def test_queries_over_more_or_fewer_keys(n, length, causal):
    """Prefixes, and (last four) queries that see no key at all."""
    c = Case([n], [length], heads=3, causal=causal, seed=n + length, tail=2)
    c.run()
    c.check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("layout", ["thd", "htd"])
def test_ragged_rows(causal, layout):
    q = [5, 0, 300, 128, 1, 77, 0, 513, 2]
    kv = [5, 9, 300, 500, 0, 80, 0, 513, 700]
    c = Case(q, kv, heads=4, causal=causal, layout=layout, lead=3, tail=5, seed=8)
    c.run()
    c.check()


@pytest.mark.parametrize("heads", [1, 5, 16, 40])
def test_head_counts(heads):
    c = Case([200, 31], [200, 60], heads=heads, seed=heads)
    c.run()
    c.check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q,kv", [([1], [5000]), ([64], [3001]), ([7, 1, 130], [2000, 10, 2900]), ([300], [1025]),
                                  ([2, 0, 5], [4000, 70, 0])])
def test_split_keys(q, kv, causal):
    c = Case(q, kv, heads=1, causal=causal, seed=sum(kv), lead=1, tail=4)
    assert c.plan.splits > 1
    c.run()
    c.check()
    whole = Case(q, kv, heads=1, causal=causal, seed=sum(kv), lead=1, tail=4, sms=1)
    assert whole.plan.splits == 1
    whole.run()
    whole.check()


def test_rows_longer_than_planned():
    """max_kv_len sizes the split only."""
    c = Case([64], [3000], heads=1)
    c.plan = binding.mla_prefill_plan(1, c.q.shape[0], 600, 1, 152)
    c.ws = binding.new_workspace(c.plan)
    c.run()
    c.check()


def test_peaked_scores_rescale():
    """Scores of wide range, growing along the keys: the running maximum moves many times."""
    c = Case([300], [900], heads=2, amp=6.0, seed=3)
    ramp = torch.linspace(0, 4, 900, device="cuda")[:, None, None]
    c.k_nope.copy_((c.k_nope.float() * ramp).bfloat16())
    c.run()
    c.check()


def test_large_negative_and_equal_scores():
    c = Case([140], [260], heads=1, causal=False)
    c.q.fill_(-4.0)
    c.k_nope.fill_(8.0)
    c.k_rope.copy_(torch.full_like(c.k_rope, 8.0))
    c.run()
    c.check()


@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_scale(scale):
    c = Case([150], [280], heads=2, scale=scale, amp=0.5)
    c.run()
    c.check()


def test_without_lse_and_repeated():
    c = Case([300, 20], [300, 400], heads=4)
    c.run(lse=False)
    first = c.out.clone()
    assert (c.lse == 7.0).all()
    for _ in range(3):
        c.out.zero_()
        c.run()
        assert torch.equal(c.out, first)
    c.check()


def test_long_prompt_sampled():
    """Rows sampled from a 5000-token prompt and its last query's keys."""
    n = 5000
    c = Case([n], [n], heads=2, seed=6)
    c.run()
    assert binding.mla_decode_read_error(c.ws) == 0
    for i in (0, 1, 127, 128, 255, 256, 2559, 4095, 4096, n - 1):
        want, lse, reach, spread = prefill_ref(f64(c.q[i:i + 1]), f64(c.k_nope[:i + 1]), f64(c.k_rope[:i + 1]),
                                               f64(c.v[:i + 1]), [0, 1], [0, i + 1], 192 ** -0.5, False)
        e = 2.0 ** -16 * (spread[0] + 1)
        got = f64(c.out[i])
        assert (np.abs(got - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + (2.0 ** -8 + e[:, None]) * reach[0]).all(), i
        assert (np.abs(f64(c.lse[i]) - lse[0]) <= e + 2.0 ** -22 * np.abs(lse[0])).all(), i


def test_rows_outside_the_tensors_are_reported():
    c = Case([40, 50, 60], [40, 50, 60], heads=1)
    c.d_qo[3] = c.q.shape[0] + 1
    c.run()
    assert binding.mla_decode_read_error(c.ws) == QO_INDPTR
    assert (c.out[90:] == 7.0).all()
    c = Case([40, 50, 60], [40, 50, 60], heads=1)
    c.d_kv[3] = c.v.shape[0] + 1
    c.run()
    assert binding.mla_decode_read_error(c.ws) == KV_INDPTR
    assert (c.out[90:] == 7.0).all()
    c = Case([40, 50, 60], [40, 50, 60], heads=1)
    c.d_kv[0] = -1
    c.run()
    assert binding.mla_decode_read_error(c.ws) == KV_INDPTR
    assert (c.out[:40] == 7.0).all()


@pytest.mark.parametrize("q,kv", [([300, 5], [300, 40]), ([3], [4000])])
def test_replayed_graph_follows_new_rows(q, kv):
    c = Case(q, kv, heads=2)
    c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    other = [max(0, x - 2) for x in kv]
    c.kv = indptr(other)
    c.d_kv.copy_(torch.tensor(c.kv.tolist(), dtype=torch.int32))
    c.q.copy_(torch.randn_like(c.q.float()).bfloat16())
    c.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_two_streams_with_their_own_workspaces():
    a, b = Case([600], [900], heads=16, seed=1), Case([4], [6000], heads=2, seed=2)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(sa)
        b.run(sb)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_a_wait_that_runs_out_is_reported_and_leaves_the_device_usable():
    c = Case([300, 10], [300, 40], heads=2)
    c.run(fn=binding.mla_prefill_fwd_stall_stream)
    torch.cuda.synchronize()
    assert binding.mla_decode_read_error(c.ws) == TIMEOUT
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    c.run()
    c.check()


def test_binding_refusals():
    c = Case([20], [20], heads=2)
    for name, value, err in [("q", c.q[..., :128], ValueError), ("k_nope", c.k_nope[:10], ValueError),
                             ("k_rope", c.k_rope.float(), TypeError), ("v", c.v[:, :1], ValueError),
                             ("out", c.out[:10], ValueError), ("d_qo", c.d_qo[:1], ValueError),
                             ("d_kv", c.d_kv.long(), TypeError), ("lse", c.lse.double(), TypeError),
                             ("q", c.q.cpu(), TypeError),
                             ("q", torch.zeros(20, 2, 384, dtype=torch.bfloat16, device="cuda")[..., ::2], ValueError)]:
        keep = getattr(c, name)
        setattr(c, name, value)
        with pytest.raises(err):
            c.run()
        setattr(c, name, keep)
    with pytest.raises(binding.MlaError):                            # one tensor for all heads: stride 0
        c.v = c.v[:, :1].expand(-1, 2, -1)
        c.run()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sms", [1, 2, 7])
def test_a_block_works_through_many_jobs(sms, causal):
    """A plan for few SMs: each persistent block takes rows of every shape in turn, among
    them queries that see nothing and rows that end inside a key tile."""
    q = [5, 300, 0, 128, 129, 77, 260, 513, 2, 1, 400]
    kv = [5, 300, 70, 500, 0, 80, 30, 513, 700, 128, 401]
    c = Case(q, kv, heads=3, causal=causal, lead=2, tail=3, seed=sms, sms=sms)
    for _ in range(2):                      # the second call finds the counters as the first did
        c.out.fill_(7.0)
        c.lse.fill_(7.0)
        c.run()
        c.check()


def test_output_aligned_to_16_bytes_only():
    c = Case([300], [300], heads=1)
    flat = torch.full((300 * 128 + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    c.out = flat[8:].view(300, 1, 128)
    assert c.out.data_ptr() % 32 == 16
    c.run()
    c.check()


@pytest.mark.parametrize("batch,sms", [(33, 152), (40, 3), (200, 152), (1000, 152), (130, 1)])
def test_many_rows(batch, sms):
    """More rows than lanes of the scheduler's warp: runs of rows, walked from the last."""
    rng = np.random.default_rng(batch)
    q = rng.integers(0, 5, batch) * (rng.random(batch) > 0.3)
    q[rng.integers(0, batch, 3)] = [300, 140, 1]
    kv = q + rng.integers(0, 200, batch)
    c = Case(q.tolist(), kv.tolist(), heads=2, seed=batch, sms=sms, lead=1, tail=1)
    c.run()
    c.check()


def test_rows_outside_the_tensors_are_not_written_by_the_joining_kernel():
    c = Case([2, 3, 4], [2000, 1500, 3000], heads=1)
    assert c.plan.splits > 1
    c.run()                                       # leaves parts of every row in the workspace
    c.check()
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    c.d_kv[3] = c.v.shape[0] + 1
    c.run()
    assert binding.mla_decode_read_error(c.ws) == KV_INDPTR
    assert (c.out[5:] == 7.0).all() and (c.lse[5:] == 7.0).all() and (c.out[:5] != 7.0).all()
    c.d_kv[3] = c.v.shape[0]
    c.out.fill_(7.0)
    c.lse.fill_(7.0)
    c.d_qo[0] = -1
    c.run()
    assert binding.mla_decode_read_error(c.ws) == QO_INDPTR
    assert (c.out[:2] == 7.0).all() and (c.lse[:2] == 7.0).all() and (c.out[2:] != 7.0).all()
