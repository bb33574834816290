"""The operators of decode steps over long contexts where offsets pass 32 bits, with many groups, and where a
step's rows differ much.  Tolerances as derived for the other tests of each operator."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.long_context import attend_ref, block_scores_ref, block_select_ref
from .test_gpu_blocks import f64, gen, i32, indptr, workspace
from .test_gpu_shared import Case

pytestmark = pytest.mark.gpu

FAR_ROWS = 4_000_000    # rows of 576: 2.3e9 elements
FAR_TOKENS = 270_000    # tokens of 16 x 512: 2.2e9 elements
FAR_STRIDE = 2**30 + 8  # elements between rows: the third starts behind 2^31


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("sms", [1, 152])
def test_shared_behind_two_to_the_31_elements(paged, sms):
    """Two groups at the end of 270,000 query tokens and of a cache of four million rows."""
    g, keys, q_lens = gen(1), 900, [5, 6]
    codes = torch.zeros(FAR_ROWS, 576, dtype=torch.uint8, device="cuda")
    tail = (torch.randn(keys, 576, generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    codes[-keys:] = tail.view(torch.uint8)
    scale = torch.full((1,), 1 / 60, device="cuda")
    q = torch.zeros(FAR_TOKENS, 16, 576, dtype=torch.bfloat16, device="cuda")
    q[-11:] = torch.randn(11, 16, 576, generator=g, device="cuda").bfloat16()
    out = torch.zeros(FAR_TOKENS, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(FAR_TOKENS, 16, device="cuda")
    qo = FAR_TOKENS - 11 + indptr(q_lens)
    kv = indptr([400, 500]) + (0 if paged else FAR_ROWS - keys)
    indices = torch.arange(FAR_ROWS - keys, FAR_ROWS, dtype=torch.int32, device="cuda") if paged else None
    plan = binding.mla_shared_plan(2, FAR_TOKENS, 500, sms)
    ws = binding.new_workspace(plan)
    binding.mla_shared_fwd(q, codes, scale, i32(qo), i32(kv), out, plan=plan, workspace=ws, kv_indices=indices, lse=lse)
    assert binding.mla_decode_read_error(ws) == 0
    assert not out[:-11].any() and not lse[:-11].any()
    values = f64(tail.float()) / 60
    for a, b, k in ((0, 5, values[:400]), (5, 11, values[400:])):
        ref, ref_lse = attend_ref(f64(q[-11:])[a:b], k)
        assert np.linalg.norm(f64(out[-11:])[a:b] - ref) <= 2.0**-7 * np.linalg.norm(ref)
        assert np.abs(f64(lse[-11:])[a:b] - ref_lse).max() <= 2.0**-8  # 2^-14 of spreads below 40, and the query's terms


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("groups", [31, 33, 200, 1024, 1025, 3000])
def test_many_groups(groups, paged):
    """One to three tokens a group over nothing to 300 keys; from 1025 groups on the keys are not cut."""
    rng = np.random.default_rng(groups)
    q, kv = rng.integers(0, 4, groups), rng.integers(0, 300, groups)
    q[rng.random(groups) < 0.7] = 1
    c = Case([int(x) for x in q], [int(x) for x in kv], paged, seed=groups, lead=1, tail=1)
    assert groups <= 1024 or c.plan.split == 0
    assert c.run() == 0
    c.check()
    assert (c.out[0] == 7).all() and (c.out[-1] == 7).all()


def test_one_long_group_among_short_ones():
    c = Case([1, 9, 1, 0, 2], [3, 9000, 0, 128, 129], paged=True, seed=4)
    assert c.plan.split == 1 and c.run() == 0
    c.check()


def test_more_keys_than_the_plan_was_made_for():
    """max_kv_len sizes the cut only."""
    c = Case([9, 3], [2500, 1000], seed=5)
    c.plan = binding.mla_shared_plan(2, 12, 130, 152)
    c.ws = binding.new_workspace(c.plan)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("page", [1, 16])
def test_means_behind_two_to_the_31_elements(cache, page):
    rows = FAR_ROWS
    pool = torch.zeros(rows, 576, dtype=torch.uint8 if cache == "e4m3" else torch.bfloat16, device="cuda")
    x = torch.randn(40, 576, generator=gen(2), device="cuda")
    means, ws = torch.zeros(rows // page, 576, dtype=torch.bfloat16, device="cuda"), workspace()
    slots = i32(range(rows - 32 - page, rows))
    if cache == "e4m3":
        codes = (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        pool[-40:] = codes.view(torch.uint8)
        values = f64(codes.float()) / 60
        binding.mla_block_means(pool, torch.full((1,), 1 / 60, device="cuda"), slots, means, page_size=page, workspace=ws)
    else:
        pool[-40:] = x.bfloat16()
        values = f64(pool[-40:])
        binding.mla_block_means_bf16kv(pool, slots, means, page_size=page, workspace=ws)
    assert binding.mla_decode_read_error(ws) == 0
    n = 32 // page
    ref, size = (f(values[-32:]).reshape(n, page, 576).mean(axis=1) for f in (np.array, np.abs))
    assert (np.abs(f64(means[-n:]) - ref) <= 2.0**-8 * np.abs(ref) + 2.0**-13 * size).all()
    assert not means[:-n - 3].any()


def test_scores_and_choice_behind_two_to_the_31_elements():
    """Pages at the end of four million, queries at the end of 270,000, and rows of the table and of the scores
    more than 2^30 elements apart."""
    g, page, blocks, lens = gen(3), 4, 9, [300, 77, 1001]
    width = 260
    q = torch.zeros(FAR_TOKENS, 16, 576, dtype=torch.bfloat16, device="cuda")
    q[-3:] = torch.randn(3, 16, 576, generator=g, device="cuda").bfloat16()
    means = torch.zeros(FAR_ROWS, 576, dtype=torch.bfloat16, device="cuda")
    means[-600:] = (0.3 * torch.randn(600, 576, generator=g, device="cuda")).bfloat16()
    ids = FAR_ROWS - 600 + np.random.default_rng(3).permutation(600)
    host = np.full((3, width), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        host[b, :k] = ids[at:at + k]
        at += k
    far = [torch.empty(2 * FAR_STRIDE + width, dtype=t, device="cuda") for t in (torch.int32, torch.float32)]
    table, scores = (t.as_strided((3, width), (FAR_STRIDE, 1)) for t in far)
    table.copy_(i32(host))
    ws, qo, kv = workspace(), FAR_TOKENS - 3 + np.arange(4), indptr(lens)
    binding.mla_block_scores(q, means, table, i32(qo), i32(kv), scores, page_size=page, workspace=ws)
    sel, idx = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(200, dtype=torch.int32, device="cuda")
    chosen = torch.empty(3, blocks, dtype=torch.int32, device="cuda")
    binding.mla_block_select(scores, table, i32(kv), sel, idx, page_size=page, num_pages=FAR_ROWS, blocks=blocks, sink=1,
                             recent=2, chosen=chosen, workspace=ws)
    assert binding.mla_decode_read_error(ws) == 0
    got = f64(scores)
    local = np.where(host < 0, -1, host - (FAR_ROWS - 600))
    ref = block_scores_ref(f64(q[-3:]), f64(means[-600:]), local, np.arange(4), kv, page)
    on = ref > -np.inf
    spread = (np.abs(f64(q[-3:])).reshape(-1, 576) @ np.abs(f64(means[-600:])).T).max() / 24
    assert ((got > -np.inf) == on).all() and (np.abs(got[on] - ref[on]) <= 2.0**-14 * spread).all()
    want = block_select_ref(got, host, kv, page, blocks, 1, 2)
    assert np.array_equal(chosen.cpu().numpy(), want["chosen"]) and np.array_equal(sel.cpu().numpy(), want["indptr"])
    assert np.array_equal(idx.cpu().numpy()[:len(want["indices"])], want["indices"])


@pytest.mark.parametrize("batch", [600, 2000])
def test_choice_of_many_rows(batch):
    rng = np.random.default_rng(batch)
    page, width, blocks = 16, 40, 8
    lens = rng.integers(0, page * width + 1, batch)
    host = rng.integers(0, 5000, (batch, width))
    scores = torch.randn(batch, width, generator=gen(batch), device="cuda")
    want = block_select_ref(f64(scores), host, indptr(lens), page, blocks, 1, 1)
    sel = torch.empty(batch + 1, dtype=torch.int32, device="cuda")
    idx = torch.empty(len(want["indices"]), dtype=torch.int32, device="cuda")
    chosen, ws = torch.empty(batch, blocks, dtype=torch.int32, device="cuda"), workspace()
    binding.mla_block_select(scores, i32(host), i32(indptr(lens)), sel, idx, page_size=page, num_pages=5000, blocks=blocks,
                             sink=1, recent=1, chosen=chosen, workspace=ws)
    assert binding.mla_decode_read_error(ws) == 0
    assert np.array_equal(chosen.cpu().numpy(), want["chosen"]) and np.array_equal(sel.cpu().numpy(), want["indptr"])
    assert np.array_equal(idx.cpu().numpy(), want["indices"])


def test_calls_without_tokens():
    """No query tokens: nothing is written; no new tokens: no means; rows without tokens score nothing."""
    c = Case([0, 0], [100, 5], seed=6, tail=0)
    assert c.out.shape[0] == 0 and c.run() == 0
    q = torch.empty(0, 16, 576, dtype=torch.bfloat16, device="cuda")
    means, ws = torch.ones(8, 576, dtype=torch.bfloat16, device="cuda"), workspace()
    scores = torch.full((2, 4), 7.0, device="cuda")
    binding.mla_block_scores(q, means, i32([[0, 1, 2, 3], [4, 5, 6, 7]]), i32([0, 0, 0]), i32([0, 50, 60]), scores,
                             page_size=16, workspace=ws)
    assert binding.mla_decode_read_error(ws) == 0 and (scores == -np.inf).all()


def test_operands_of_the_wrong_kind_are_refused():
    c = Case([3, 2], [100, 50], paged=True, seed=7)
    qo, kv, page = i32(c.qo), i32(c.kv), dict(page_size=16, workspace=workspace())
    means, table, scores = torch.zeros(9, 576, dtype=torch.bfloat16, device="cuda"), i32([[0, 1], [2, 3]]), torch.zeros(2, 2, device="cuda")
    room, sel, pool = i32([0] * 64), i32([0] * 3), c.codes

    def shared(q=c.q, codes=c.codes, scale=c.scale, qo=qo, kv=kv, out=c.out, **more):
        args = dict(plan=c.plan, workspace=c.ws, kv_indices=c.indices, lse=c.lse) | more
        return lambda: binding.mla_shared_fwd(q, codes, scale, qo, kv, out, **args)

    def select(scores=scores, table=table, kv=kv, sel=sel, room=room, **more):
        return lambda: binding.mla_block_select(scores, table, kv, sel, room, **(page | dict(num_pages=9, blocks=2, sink=0, recent=1) | more))

    calls = [shared(q=c.q.float()), shared(q=c.q[:, :8]), shared(q=c.q.transpose(0, 1)), shared(out=c.out[..., :256]),
             shared(out=c.out[:4]), shared(qo=qo[:2]), shared(kv=kv.long()), shared(codes=c.codes[:, ::2]), shared(scale=c.scale.double()),
             shared(lse=c.lse[:4]), shared(lse=c.lse.half()), shared(kv_indices=c.indices.long()), shared(workspace=c.ws[:256].cpu()),
             lambda: binding.mla_block_means(pool, c.scale, room.long(), means, **page),
             lambda: binding.mla_block_means(pool, c.scale, room, means.float(), **page),
             lambda: binding.mla_block_means(pool, c.scale, room, means[:, ::2], **page),
             lambda: binding.mla_block_scores(c.q, means, table.long(), qo, kv, scores, **page),
             lambda: binding.mla_block_scores(c.q, means, table[:1], qo, kv, scores, **page),
             lambda: binding.mla_block_scores(c.q, means, table, qo, kv, scores.t(), **page),
             lambda: binding.mla_block_scores(c.q, means, table, qo[:2], kv, scores, **page),
             lambda: binding.mla_block_scores(c.q, means, table, qo, kv, scores[:, :1], **page),
             select(scores=scores.half()), select(table=table[:, :1]), select(sel=sel[:2]), select(room=room.long()),
             select(chosen=i32([[0], [0]])), select(chosen=i32([[0, 0]]))]
    for i, call in enumerate(calls):
        with pytest.raises((TypeError, ValueError)):
            call()
            print("taken:", i)
    torch.cuda.synchronize()
    assert (c.out == 7).all() and (c.lse == 7).all()
    for more in (dict(blocks=0), dict(blocks=2, sink=2), dict(recent=0), dict(num_pages=0)):
        with pytest.raises((ValueError, RuntimeError)):
            select(**more)()


@pytest.mark.parametrize("paged", [False, True])
def test_two_queries_over_three_hundred_thousand_keys(paged):
    """Float64 sums over the keys on the GPU; the tolerances are those of the shorter rows (the probabilities' least
    step weighs more the more keys there are: 2^-14 of the largest for each, and the others' 2^-8)."""
    n, g = 300_001, gen(8)
    rows = n + (99 if paged else 0)
    codes = (torch.randn(rows, 576, generator=g, device="cuda") * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    index = torch.randperm(rows, generator=g, device="cuda")[:n].to(torch.int32) if paged else None
    q = (1.5 * torch.randn(2, 16, 576, generator=g, device="cuda")).bfloat16()
    out, lse = torch.empty(2, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 16, device="cuda")
    plan = binding.mla_shared_plan(1, 2, n)
    ws = binding.new_workspace(plan)
    assert plan.split == 1
    binding.mla_shared_fwd(q, codes.view(torch.uint8), torch.full((1,), 1 / 60, device="cuda"), i32([0, 2]), i32([0, n]), out,
                           plan=plan, workspace=ws, kv_indices=index, lse=lse)
    assert binding.mla_decode_read_error(ws) == 0
    keys = (codes[index.long()] if paged else codes).double() / 60
    s = q.double().flatten(0, 1) @ keys.T / 24
    p = (s - s.max(dim=1, keepdim=True).values).exp()
    z = p.sum(dim=1, keepdim=True)
    ref, reach = p @ keys[:, :512] / z, p @ keys[:, :512].abs() / z
    e = 2.0**-14 * (q.double().flatten(0, 1).abs() @ keys.abs().T / 24).max(dim=1).values[:, None] + 2.0**-12
    bound = (2.0**-8 * ref.abs() + (2.0**-8 + 2.0**-10 + 2 * e) * reach + 2.0**-14 * keys[:, :512].abs().sum(dim=0) / z
             + 2.0**-25 / 60)
    assert bool(((out.double().flatten(0, 1) - ref).abs() <= bound).all())
    want = s.logsumexp(dim=1)
    assert bool(((lse.double().flatten() - want).abs() <= e[:, 0] + 2.0**-22 * want.abs()).all())


def test_scores_of_a_long_row():
    """70,001 pages of two tokens, a second row of one page beside them."""
    page, g, lens = 2, gen(9), [140_001, 2]
    pages = 70_002
    host = np.full((2, pages), -1, dtype=np.int64)
    ids = np.random.default_rng(9).permutation(pages)
    host[0, :70_001], host[1, 0] = ids[:70_001], ids[70_001]
    q = torch.randn(3, 16, 576, generator=g, device="cuda").bfloat16()
    means = (0.3 * torch.randn(pages, 576, generator=g, device="cuda")).bfloat16()
    scores, ws = torch.full((2, pages), 7.0, device="cuda"), workspace()
    binding.mla_block_scores(q, means, i32(host), i32([0, 2, 3]), i32(indptr(lens)), scores, page_size=page, workspace=ws)
    assert binding.mla_decode_read_error(ws) == 0
    ref = torch.full((2, pages), -torch.inf, dtype=torch.float64, device="cuda")
    for b, (lo, hi, n) in enumerate(((0, 2, 70_001), (2, 3, 1))):
        m = means[torch.from_numpy(host[b, :n]).cuda()].double()
        ref[b, :n] = (q[lo:hi].double().flatten(0, 1) @ m.T).max(dim=0).values / 24
    spread = float((q.double().flatten(0, 1).abs() @ means.double().abs().T).max()) / 24
    on = ref > -torch.inf
    assert bool(((scores > -torch.inf) == on).all()) and bool(((scores.double() - ref)[on].abs() <= 2.0**-14 * spread).all())


def test_twenty_thousand_groups():
    """Runs of hundreds of groups a lane of the warp that finds the jobs, some without queries or keys."""
    rng = np.random.default_rng(11)
    q, kv = rng.integers(0, 3, 20_000), rng.integers(0, 4, 20_000)
    q[[0, 5000, 19_999]] = [9, 0, 6]
    c = Case([int(x) for x in q], [int(x) for x in kv], True, seed=11, lead=1, tail=1)
    assert c.run() == 0
    got, lse, group = f64(c.out), f64(c.lse), np.repeat(np.arange(20_000), q)
    assert (got[0] == 7).all() and (got[-1] == 7).all()
    empty = kv[group] == 0
    assert (got[1:-1][empty] == 0).all() and (lse[1:-1][empty] == -np.inf).all()
    one = kv[group] == 1  # a single key's values, twice rounded
    keys = f64(c.codes.view(torch.float8_e4m3fn)[c.indices.long()].float()) / 60
    first = keys[c.kv[:-1][group[one]]]
    assert (np.abs(got[1:-1][one] - first[:, None, :512]) <= (2.0**-8 + 2.0**-8) * np.abs(first[:, None, :512]) + 2.0**-14).all()
    for g in rng.integers(0, 20_000, 300):
        a, b = int(c.qo[g]), int(c.qo[g + 1])
        if a == b or kv[g] == 0:
            continue
        ref, ref_lse = attend_ref(f64(c.q[a:b]), keys[int(c.kv[g]):int(c.kv[g + 1])])
        assert np.linalg.norm(got[a:b] - ref) <= 2.0**-7 * np.linalg.norm(ref)
        assert np.abs(lse[a:b] - ref_lse).max() <= 2.0**-8  # 2^-14 of spreads below 40, and the query's terms
