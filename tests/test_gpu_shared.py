"""mla_shared_fwd against the float64 definition.

Tolerances, from the operator's arithmetic.  Scores: float32 sums of 2 x 576 products, within
2^-14 of ``spread`` = sum |q||k| / 24, and the query's two terms, off by 2^-20 of its head's
largest magnitude at most (half a step of the low term, 2^-10 / 8, where the largest is 224
or more): e = max_j (2^-14 spread + 2^-20 max|q| sum |k| / 24) + 2^-20 for exp2, relative in a
probability and absolute in the lse.  A probability's two terms: 2^-8 of it (twice half a
step of e4m3, 2^-4), 2^-11 by way of half precision, and half the smallest step, 2^-10, where
the row's reference, which is not above its maximum, stands at 2^4: 2^-14 of the maximum's
probability.  Parts of split keys are half precision in units of codes: 2^-11, and 2^-25 codes.
The output is rounded to bf16, 2^-8.  So with reach = sum_j p_j |v_j| / z and
z the sum of probabilities relative to the largest,
|out - exact| <= 2^-8 |exact| + (2^-8 + 2^-10 + 2 e) reach + 2^-14 sum_j |v_j| / z + 2^-25 kv_scale.
Those are worst cases; rounding errors have independent signs, so in the 2-norm the two
roundings of 2^-8 stay below 2^-8 of the result each: 2^-7 bounds the relative error."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.long_context import attend_ref

pytestmark = pytest.mark.gpu

QO_INDPTR, KV_INDPTR, KV_INDEX, TIMEOUT = 1, 2, 4, 8


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def f64(t):
    return t.double().cpu().numpy()


def indptr(lens, start=0):
    return np.concatenate([[start], start + np.cumsum(lens)]).astype(np.int64)


class Case:
    """Groups of ``q_lens`` query tokens over ``kv_lens`` keys.  ``lead``/``tail``: query tokens and
    keys that belong to no group; cache rows of no group's keys hold NaN codes."""

    def __init__(self, q_lens, kv_lens, paged=False, seed=0, lead=0, tail=0, amp=1.5, sms=152, ramp=0.0, scale=1 / 60):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.qo, self.kv = indptr(q_lens, lead), indptr(kv_lens, lead)
        tq, tk = int(self.qo[-1]) + tail, int(self.kv[-1]) + tail
        rows = max(1, tk) + (37 if paged else 0)
        x = torch.randn(rows, 576, generator=g, device="cuda") * 60
        if ramp:  # keys, and with them the scores' spread, grow along the row
            x *= (torch.arange(rows, device="cuda") * ramp)[:, None].exp()
        codes = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.indices = None
        used = torch.zeros(rows, dtype=torch.bool, device="cuda")
        if paged:
            self.indices = torch.randperm(rows, generator=g, device="cuda")[:tk].to(torch.int32)
            used[self.indices[lead:tk - tail].long()] = True
        else:
            used[lead:tk - tail] = True
        codes[~used] = 0x7F
        self.codes = codes
        self.scale = torch.full((1,), scale, device="cuda")
        self.q = (amp * torch.randn(tq, 16, 576, generator=g, device="cuda")).bfloat16()
        self.out = torch.full((tq, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((tq, 16), 7.0, device="cuda")
        self.plan = binding.mla_shared_plan(len(q_lens), tq, max([0, *kv_lens]), sms)
        self.ws = binding.new_workspace(self.plan)

    def run(self, **more):
        i32 = lambda a: torch.from_numpy(a.astype(np.int32)).cuda()
        args = dict(plan=self.plan, workspace=self.ws, kv_indices=self.indices, lse=self.lse) | more
        binding.mla_shared_fwd(self.q, self.codes, self.scale, i32(self.qo), i32(self.kv), self.out, **args)
        torch.cuda.synchronize()
        return binding.mla_decode_read_error(self.ws)

    def keys(self, g):
        j = torch.arange(int(self.kv[g]), int(self.kv[g + 1]), device="cuda")
        rows = j if self.indices is None else self.indices[j].long()
        return f64(self.codes.view(torch.float8_e4m3fn)[rows].float()) * float(self.scale)

    def check(self):
        got, lse, q = f64(self.out), f64(self.lse), f64(self.q)
        for g in range(len(self.qo) - 1):
            a, b = int(self.qo[g]), int(self.qo[g + 1])
            k = self.keys(g)
            out, ref_lse = attend_ref(q[a:b], k)
            if len(k) == 0:
                assert (got[a:b] == 0).all() and (lse[a:b] == -np.inf).all()
                continue
            if a == b:
                continue
            spread = np.abs(q[a:b]) @ np.abs(k).T / 24
            low = np.abs(q[a:b]).max(axis=2) * np.abs(k).sum(axis=1).max() / 24
            e = 2.0**-14 * spread.max(axis=2) + 2.0**-20 * low + 2.0**-20
            s = q[a:b] @ k.T / 24
            p = np.exp(s - s.max(axis=2, keepdims=True))
            z = p.sum(axis=2, keepdims=True)
            reach = p @ np.abs(k[:, :512]) / z
            bound = (2.0**-8 * np.abs(out) + (2.0**-8 + 2.0**-10 + 2 * e[..., None]) * reach
                     + 2.0**-14 * np.abs(k[:, :512]).sum(axis=0) / z + 2.0**-25 * float(self.scale))
            assert (np.abs(got[a:b] - out) <= bound).all(), (g, np.abs(got[a:b] - out).max())
            assert np.linalg.norm(got[a:b] - out) <= 2.0**-7 * np.linalg.norm(out), g
            assert (np.abs(lse[a:b] - ref_lse) <= e + 2.0**-22 * np.abs(ref_lse)).all(), (g, np.abs(lse[a:b] - ref_lse).max())


CASES = [([1], [1]), ([1], [128]), ([2], [129]), ([3], [127]), ([4], [256]), ([5], [300]), ([8], [1000]), ([64], [513]),
         ([3, 0, 9, 1], [300, 50, 0, 1]), ([7, 2], [0, 0]), ([33, 4, 2], [64, 1500, 700])]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens", CASES)
def test_groups(q_lens, kv_lens, paged):
    c = Case(q_lens, kv_lens, paged, seed=len(q_lens) + sum(kv_lens))
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("sms", [1, 3, 152])
def test_blocks_work_through_jobs(sms):
    c = Case([21, 6, 1, 30], [700, 129, 2000, 40], paged=True, seed=3, sms=sms, lead=2, tail=3)
    for _ in range(2):
        assert c.run() == 0
        c.check()
    for t in (*range(2), *range(60, 63)):
        assert (c.out[t] == 7).all() and (c.lse[t] == 7).all()


@pytest.mark.parametrize("paged", [False, True])
def test_maxima_that_rise_along_the_keys(paged):
    """The reference moves many times, and the outputs of earlier tiles are scaled down."""
    c = Case([6], [900], paged, seed=5, ramp=0.0015)
    assert c.run() == 0
    c.check()


def test_one_key_far_above_the_rest():
    """The rest's probabilities are coarse, but within the stated steps."""
    c = Case([4], [1200], seed=6, amp=1.0)
    c.codes[700] = (c.q[1, 3].float() * 180).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert c.run() == 0
    c.check()


def test_equal_keys():
    c = Case([5], [1000], seed=7)
    c.codes[:] = c.codes[:1]
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("amp", [2.0**-40, 2.0**20])
def test_queries_far_from_one(amp):
    c = Case([5], [300], seed=8, amp=amp, scale=1 / 60 / max(1.0, amp))
    assert c.run() == 0
    c.check()


def test_a_query_that_is_not_finite_stays_alone():
    c = Case([9], [500], seed=9, sms=5)
    c.q[2, 4, 100], c.q[7, 0, 575] = float("nan"), float("inf")
    assert c.run() == 0
    bad = torch.zeros(9, 16, dtype=torch.bool, device="cuda")
    bad[2, 4] = bad[7, 0] = True
    assert c.out[bad].isnan().all() and c.lse[bad].isnan().all()
    good = Case([9], [500], seed=9, sms=5)
    good.run()
    assert torch.equal(c.out[~bad], good.out[~bad]) and torch.equal(c.lse[~bad], good.lse[~bad])


def test_the_same_bits_every_time_and_without_lse():
    c = Case([70, 3], [2100, 900], paged=True, seed=10)
    assert c.plan.split == 1
    c.run()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.run()
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
    c.lse.fill_(7.0)
    assert c.run(lse=None) == 0
    assert torch.equal(c.out, out) and (c.lse == 7).all()


def test_a_group_out_of_range_is_reported_and_left():
    for field, where, value, bit in [("kv", 2, 10**6, KV_INDPTR), ("qo", 3, 90, QO_INDPTR), ("kv", 0, -1, KV_INDPTR)]:
        c = Case([5, 4, 6], [200, 300, 100], seed=11, sms=1)
        assert c.plan.split == 0
        getattr(c, field)[where] = value
        assert c.run() == bit
        ok = Case([5, 4, 6], [200, 300, 100], seed=11, sms=1)
        ok.run()
        first = slice(0, 5)
        if field == "kv" and where == 0:
            assert (c.out[first] == 7).all()
            assert torch.equal(c.out[5:], ok.out[5:])
        else:
            assert torch.equal(c.out[first], ok.out[first]) and torch.equal(c.lse[first], ok.lse[first])
            assert (c.out[9:] == 7).all()


def test_decreasing_offsets_write_nothing_stale_when_keys_are_split():
    c = Case([8, 8], [600, 600], seed=12)
    assert c.plan.split == 1 and c.run() == 0
    c.qo[1] = 20
    c.out.fill_(7.0)
    assert c.run() == QO_INDPTR
    assert (c.out == 7).all()
    c.qo[1] = 8
    assert c.run() == 0
    c.check()


def test_a_bad_page_entry_is_reported():
    c = Case([4], [300], paged=True, seed=13)
    c.indices[17] = c.codes.shape[0]
    assert c.run() == KV_INDEX
    c.indices[17] = -1
    assert c.run() == KV_INDEX
    assert c.run() == KV_INDEX and binding.mla_decode_read_error(c.ws) == 0


def test_waits_that_run_out():
    c = Case([6], [500], seed=14)
    args = (c.q, c.codes, c.scale, torch.tensor([0, 6], dtype=torch.int32, device="cuda"),
            torch.tensor([0, 500], dtype=torch.int32, device="cuda"), c.out)
    binding.mla_shared_fwd_stall_stream(*args, plan=c.plan, workspace=c.ws, lse=c.lse)
    torch.cuda.synchronize()
    assert binding.mla_decode_read_error(c.ws) == TIMEOUT
    assert (c.out == 7).all() and (c.lse == 7).all()
    assert c.run() == 0
    c.check()


def test_captured_and_on_two_streams():
    """A captured call follows new queries and lengths in its buffers; two calls with their own
    workspaces do not disturb each other."""
    a, b = Case([40], [1500], paged=True, seed=15), Case([12, 9], [700, 300], seed=16)
    qo = [torch.from_numpy(c.qo.astype(np.int32)).cuda() for c in (a, b)]
    kv = [torch.from_numpy(c.kv.astype(np.int32)).cuda() for c in (a, b)]

    def call(c, i, stream=None):
        binding.mla_shared_fwd(c.q, c.codes, c.scale, qo[i], kv[i], c.out, stream, plan=c.plan, workspace=c.ws,
                               kv_indices=c.indices, lse=c.lse)

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, c in enumerate((a, b)):
            call(c, i, streams[i])
    torch.cuda.synchronize()
    a.check()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, 0)
    a.q.copy_(a.q.flip(0) * 0.5)
    a.kv[1] = 1301
    kv[0].copy_(torch.from_numpy(a.kv.astype(np.int32)))
    for _ in range(2):
        a.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        a.check()


@pytest.mark.parametrize("page", [2, 16, 24, 64, 1000])
@pytest.mark.parametrize("skew", [0, 5])
def test_rows_that_follow_one_another_in_the_cache(page, skew):
    """Pages of rows: sixteen of a tile's that are one behind the other are copied as one, others piece by piece
    (a prefix that begins inside a page, pages that end inside a tile, the cache's last rows); the same bits
    as from the same keys in any other rows."""
    q_lens, kv_lens = [9, 6], [700, 333]
    a, b = (Case(q_lens, kv_lens, paged=True, seed=17 + page, tail=2) for _ in range(2))
    tk = sum(kv_lens)
    pages = -(-(tk + skew) // page)
    order = torch.randperm(pages, generator=torch.Generator(device="cuda").manual_seed(page), device="cuda")
    order[(order == pages - 1).nonzero()[0, 0]], order[pages // 2] = order[pages // 2].clone(), pages - 1
    t = torch.arange(skew, skew + tk, device="cuda")
    rows = order[t // page] * page + t % page
    codes = torch.full((pages * page, 576), 0x7F, dtype=torch.uint8, device="cuda")
    codes[rows] = a.codes[a.indices[:tk].long()]
    last = int(rows.max()) + 1
    b.codes, b.indices = codes[:last].clone(), rows.to(torch.int32)
    assert a.run() == 0 and b.run() == 0
    b.check()
    assert torch.equal(a.out, b.out) and torch.equal(a.lse, b.lse)


def test_a_bad_page_entry_in_a_run_is_reported():
    c = Case([4], [256], paged=True, seed=18)
    c.indices = torch.arange(100, 356, dtype=torch.int32, device="cuda")
    c.codes = c.codes[torch.randint(256, (300,), device="cuda") % c.codes.shape[0]].clone()
    c.codes[c.codes == 0x7F] = 0
    assert c.run() == KV_INDEX  # rows 300 .. 355 are outside
    c.indices -= 100
    assert c.run() == 0
    c.check()
