"""Block means, block scores and the choice of blocks against their float64 definitions.

Tolerances.  Means: float32 sums of up to 1024 values (2^-24 each, relative to the sum of
magnitudes) and two roundings, then bf16: |got - exact| <= 2^-8 |exact| + 2^-13 mean |v|.
Scores: products of bf16 are exact in float32, 576 of them summed: 2^-14 of the largest
sum |q||m| / 24 of the row.  The choice is of whole numbers and has to be equal."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.attention import mla_decode_ref
from oracle.long_context import block_means_ref, block_scores_ref, block_select_ref

pytestmark = pytest.mark.gpu

QO_INDPTR, KV_INDPTR, KV_INDEX, CAPACITY = 1, 2, 4, 256


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def f64(t):
    return t.double().cpu().numpy()


def i32(a):
    return torch.tensor(np.asarray(a).tolist(), dtype=torch.int32, device="cuda")


def workspace():
    return torch.zeros(binding.STEP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def indptr(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def pages_of(lens, page, seed, width=None, spare=3):
    """Block table of rows of these lengths over shuffled pages (-1 behind a row's end), and their number."""
    need = [-(-n // page) for n in lens]
    ids = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = np.full((len(lens), width or max(1, *need)), -1, dtype=np.int64)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    return table, sum(need) + spare


# ---------------------------------------------------------------- means
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("page", [1, 7, 16, 64, 1000])
@pytest.mark.parametrize("before,new", [([0], [1]), ([63], [1]), ([64, 5, 127, 0], [1, 1, 1, 1]), ([10, 0, 300], [250, 65, 3]),
                                        ([0], [3000]), ([100] * 70, [1] * 70)])
def test_means(cache, page, before, new):
    g = gen(page + sum(new))
    total = [x + y for x, y in zip(before, new)]
    table, pages = pages_of(total, page, page)
    slots = [int(table[b, t // page]) * page + t % page for b in range(len(new)) for t in range(before[b], total[b])]
    slots += [-1] * 5
    x = torch.randn(pages * page, 576, generator=g, device="cuda").bfloat16()
    means = torch.randn(pages, 576, generator=g, device="cuda").bfloat16()
    was, ws = means.clone(), workspace()
    if cache == "e4m3":
        pool, scale = (x.float() * 60).clamp(-448, 448).to(torch.float8_e4m3fn), torch.full((1,), 1 / 60, device="cuda")
        values = f64(pool.float()) * float(scale)
        binding.mla_block_means(pool.view(torch.uint8), scale, i32(slots), means, page_size=page, workspace=ws)
    else:
        values = f64(x)
        binding.mla_block_means_bf16kv(x, i32(slots), means, page_size=page, workspace=ws)
    torch.cuda.synchronize()
    assert binding.mla_decode_read_error(ws) == 0
    ref = block_means_ref(values, slots, f64(was), page)
    touched = sorted({s // page for s in slots if s >= 0})
    rest = np.setdiff1d(np.arange(pages), touched)
    assert torch.equal(means[rest], was[rest])
    size = block_means_ref(np.abs(values), slots, np.zeros((pages, 576)), page)
    assert (np.abs(f64(means) - ref) <= 2.0**-8 * np.abs(ref) + 2.0**-13 * size)[touched].all()


def test_means_of_slots_out_of_range_are_reported():
    means, ws = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda"), workspace()
    x = torch.ones(70, 576, dtype=torch.bfloat16, device="cuda")
    binding.mla_block_means_bf16kv(x, i32([3, 64, 70, 2**31 - 1]), means, page_size=16, workspace=ws)
    assert binding.mla_decode_read_error(ws) == KV_INDEX
    assert (means[0] == 1).all() and (means[1:] == 0).all()
    binding.mla_block_means_bf16kv(x, i32([]), means, page_size=16, workspace=ws)
    assert binding.mla_decode_read_error(ws) == 0


# ---------------------------------------------------------------- scores
@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("tokens,lens", [([1], [1]), ([1, 1, 1], [64, 0, 1000]), ([2, 2], [129, 4096]), ([3, 0, 5], [300, 70, 1025]),
                                         ([4] * 9, [500] * 9), ([9], [700])])
def test_scores(tokens, lens, page):
    g = gen(page)
    if page == 1:
        lens = [min(n, 300) for n in lens]
    table, pages = pages_of(lens, page, 1, width=max(1, max(-(-n // page) for n in lens)) + 5)
    q = torch.randn(sum(tokens), 16, 576, generator=g, device="cuda").bfloat16()
    means = (0.3 * torch.randn(pages, 576, generator=g, device="cuda")).bfloat16()
    wide = torch.full((len(lens), table.shape[1] + 3), 7.0, device="cuda")
    scores, ws = wide[:, :table.shape[1]], workspace()
    binding.mla_block_scores(q, means, i32(table), i32(indptr(tokens)), i32(indptr(lens)), scores, page_size=page, workspace=ws)
    torch.cuda.synchronize()
    assert binding.mla_decode_read_error(ws) == 0
    ref, got = block_scores_ref(f64(q), f64(means), table, indptr(tokens), indptr(lens), page), f64(scores)
    assert (wide[:, table.shape[1]:] == 7).all()
    assert ((got == -np.inf) == (ref == -np.inf)).all()
    spread = (np.abs(f64(q)).reshape(-1, 576) @ np.abs(f64(means)).T).max() / 24
    on = ref > -np.inf
    assert (np.abs(got[on] - ref[on]) <= 2.0**-14 * spread).all()


def test_scores_of_bad_pages_rows_and_values():
    g = gen(2)
    q = torch.randn(3, 16, 576, generator=g, device="cuda").bfloat16()
    means = torch.randn(8, 576, generator=g, device="cuda").bfloat16()
    means[2, 5] = float("nan")
    table, ws = i32([[0, 1, 2, 3], [4, 8, 5, -1], [6, 7, 0, 1]]), workspace()
    def run(qo, kv):
        scores = torch.full((3, 4), 7.0, device="cuda")
        binding.mla_block_scores(q, means, table, i32(qo), i32(kv), scores, page_size=16, workspace=ws)
        torch.cuda.synchronize()
        return scores.cpu(), binding.mla_decode_read_error(ws)
    good, err = run([0, 1, 1, 3], [0, 64, 64, 96])
    assert err == 0 and good[0, 2].isnan() and good[0, [0, 1, 3]].isfinite().all()
    assert (good[1] == -np.inf).all() and good[2, :2].isfinite().all() and (good[2, 2:] == -np.inf).all()
    scores, err = run([0, 1, 2, 3], [0, 64, 64 + 64, 160])
    assert err == KV_INDEX
    assert scores[1, [0, 2]].isfinite().all() and (scores[1, [1, 3]] == -np.inf).all()
    for qo, kv, bit in [([0, 1, 2, 3], [0, 65, 70, 80], KV_INDPTR), ([0, 1, 2, 4], [0, 16, 20, 30], QO_INDPTR),
                        ([0, 2, 1, 3], [0, 16, 20, 30], QO_INDPTR), ([0, 1, 2, 3], [0, 30, 20, 30], KV_INDPTR)]:
        scores, err = run(qo, kv)
        assert err == bit
        assert (scores == -np.inf).all(dim=1).any() and scores.isfinite().any()


# ---------------------------------------------------------------- choice
def select(scores, table, lens, page, pages, blocks, sink, recent, room=None, chosen=True):
    b, ws = len(lens), workspace()
    ref = block_select_ref(f64(scores), table, indptr(lens), page, blocks, sink, recent)
    n = len(ref["indices"]) if room is None else room
    out = [torch.full((m,), -7, dtype=torch.int32, device="cuda") for m in (b + 1, n + 4)]
    picked = torch.full((b, blocks), -7, dtype=torch.int32, device="cuda") if chosen else None
    binding.mla_block_select(scores, i32(table), i32(indptr(lens)), out[0], out[1][:n], page_size=page, num_pages=pages,
                             blocks=blocks, sink=sink, recent=recent, chosen=picked, workspace=ws)
    torch.cuda.synchronize()
    return ref, [t.cpu().numpy() for t in out] + ([picked.cpu().numpy()] if chosen else []), binding.mla_decode_read_error(ws)


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("blocks,sink,recent", [(1, 0, 1), (4, 0, 1), (4, 1, 2), (16, 2, 14), (33, 0, 3), (600, 5, 90)])
@pytest.mark.parametrize("ties", [False, True])
def test_choice(page, blocks, sink, recent, ties):
    lens = [0, 1, page * blocks, page * blocks + 1, 700 * page + 3 % page, 1300 * page, 5 * page]
    table, pages = pages_of(lens, page, blocks)
    scores = torch.randn(table.shape, generator=gen(blocks), device="cuda")
    if ties:
        scores = (scores * 2).round() / 2
        scores[scores == 0] *= -1.0  # zeros of both signs
    ref, (ptr, idx, chosen), err = select(scores, table, lens, page, pages, blocks, sink, recent)
    assert err == 0
    assert np.array_equal(ptr, ref["indptr"]) and np.array_equal(chosen, ref["chosen"])
    assert np.array_equal(idx[:-4], ref["indices"]) and (idx[-4:] == -7).all()


def test_choice_among_scores_that_are_not_finite():
    lens, page = [900], 1
    table, pages = pages_of(lens, page, 0)
    scores = torch.randn(table.shape, generator=gen(0), device="cuda")
    scores[0, 100:500] = -np.inf
    scores[0, [50, 600]] = np.inf
    scores[0, [70, 555, 899]] = np.nan
    for blocks in (3, 6, 300, 520, 899):
        ref, (ptr, idx, chosen), err = select(scores, table, lens, page, pages, blocks, 1, 1)
        assert err == 0 and np.array_equal(chosen, ref["chosen"]) and np.array_equal(idx[:-4], ref["indices"])
    scores[:] = 0.25
    ref, (ptr, idx, chosen), err = select(scores, table, lens, page, pages, 300, 0, 1, chosen=True)
    assert np.array_equal(chosen[0], [*range(299), 899])


def test_choice_of_a_long_row():
    lens, page = [70001 * 2, 9], 2
    table, pages = pages_of(lens, page, 0)
    scores = torch.randn(table.shape, generator=gen(1), device="cuda").bfloat16().float()
    ref, (ptr, idx, chosen), err = select(scores, table, lens, page, pages, 8192, 3, 100)
    assert err == 0 and np.array_equal(ptr, ref["indptr"]) and np.array_equal(chosen, ref["chosen"])
    assert np.array_equal(idx[:-4], ref["indices"])


def test_choice_that_cannot_be_laid_out_is_emptied():
    lens, page = [100, 300, 20], 16
    table, pages = pages_of(lens, page, 0)
    scores = torch.randn(table.shape, generator=gen(1), device="cuda")
    ref, (ptr, idx, chosen), err = select(scores, table, lens, page, pages, 4, 0, 1)
    assert err == 0
    need = len(ref["indices"])
    _, (ptr, idx, chosen), err = select(scores, table, lens, page, pages, 4, 0, 1, room=need - 1)
    assert err == CAPACITY and (ptr == 0).all() and (chosen == -1).all() and (idx == -7).all()
    ws = workspace()
    for kv in ([0, 100, 90, 120], [-1, 100, 200, 220], [0, 100, 100 + 305, 410]):
        out = torch.full((4,), -7, dtype=torch.int32, device="cuda")
        room = torch.full((999,), -7, dtype=torch.int32, device="cuda")
        binding.mla_block_select(scores, i32(table), i32(kv), out, room, page_size=page, num_pages=pages, blocks=4,
                                 sink=0, recent=1, workspace=ws)
        assert binding.mla_decode_read_error(ws) == KV_INDPTR
        assert (out == 0).all() and (room == -7).all()
    table[1, 18] = pages
    _, (ptr, idx, chosen), err = select(scores, table, lens, page, pages, 4, 0, 1)
    assert err == KV_INDEX
    assert (idx[ptr[2] - 12:ptr[2]] == -1).all() and (idx[:-4] == -1).sum() == 12


# ---------------------------------------------------------------- together
def test_a_sparse_decode_step():
    """Map, append, means, scores, choice and decode step over pages of 16, twice: the second step
    on the first's pages.  The decode step is checked over the pages that the float64 choice takes."""
    g, page, num_pages, batch = gen(7), 16, 400, 3
    lens = np.array([700, 33, 1500])
    table = torch.full((batch, 120), -1, dtype=torch.int32, device="cuda")
    pool = torch.zeros(num_pages * page, 576, dtype=torch.uint8, device="cuda")
    means = torch.zeros(num_pages, 576, dtype=torch.bfloat16, device="cuda")
    scale = torch.full((1,), 8 / 448, device="cuda")
    weight = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    angle = torch.arange(2048, device="cuda")[:, None] * 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    rope = torch.cat([angle.cos(), angle.sin()], dim=1).float()
    free = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    before = np.zeros(batch, dtype=np.int64)
    ws = workspace()
    for new in (lens, np.ones(batch, dtype=np.int64)):
        t = int(new.sum())
        maps = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (batch + 1, batch + 1, int((before + new).sum()), t, t, 1)]
        qo, kv, indices, slots, positions, used = maps
        binding.mla_page_map(i32(before), i32(new), table, free, *maps, page_size=page, num_pages=num_pages, workspace=ws)
        x = torch.randn(t, 576, generator=g, device="cuda").bfloat16()
        binding.mla_kv_append(x, weight, rope, positions, slots, pool, scale, workspace=ws)
        binding.mla_block_means(pool, scale, slots, means, page_size=page, workspace=ws)
        free = free[int(used):].contiguous()
        before = before + new
    q = torch.randn(batch, 16, 576, generator=g, device="cuda").bfloat16()
    scores = torch.empty(table.shape, device="cuda")
    binding.mla_block_scores(q, means, table, qo, kv, scores, page_size=page, workspace=ws)
    sel = torch.empty(batch + 1, dtype=torch.int32, device="cuda")
    sel_indices = torch.empty(3 * 24 * page, dtype=torch.int32, device="cuda")
    chosen = torch.empty(batch, 24, dtype=torch.int32, device="cuda")
    binding.mla_block_select(scores, table, kv, sel, sel_indices, page_size=page, num_pages=num_pages, blocks=24, sink=1,
                             recent=2, chosen=chosen, workspace=ws)
    out = torch.empty(batch, 16, 512, dtype=torch.bfloat16, device="cuda")
    plan = binding.mla_decode_plan(batch, 24 * page)
    step = binding.new_workspace(plan)
    binding.mla_decode_fwd(q, pool, scale, qo, sel, out, plan=plan, workspace=step, kv_indices=sel_indices)
    torch.cuda.synchronize()
    assert binding.mla_decode_read_error(ws) == 0 and binding.mla_decode_read_error(step) == 0
    values = f64(pool.view(torch.float8_e4m3fn).float()) * float(scale)
    host = table.cpu().numpy()
    full = np.zeros((num_pages, 576))
    for b in range(batch):
        for j in range(-(-int(before[b]) // page)):
            rows = values[host[b, j] * page:host[b, j] * page + min(page, int(before[b]) - j * page)]
            full[host[b, j]] = rows.mean(axis=0)
    on = host[host >= 0]
    assert (np.abs(f64(means) - full) <= 2.0**-8 * np.abs(full) + 2.0**-10)[on].all()
    # the choice is by the scores that the GPU found, which the scores' test holds to their own definition
    want = block_select_ref(f64(scores), host, indptr(before), page, 24, 1, 2)
    assert np.array_equal(chosen.cpu().numpy(), want["chosen"]) and np.array_equal(sel.cpu().numpy(), want["indptr"])
    assert np.array_equal(sel_indices.cpu().numpy()[:len(want["indices"])], want["indices"])
    ref = mla_decode_ref(f64(q), pool.cpu().numpy(), np.float32(8 / 448), np.arange(batch + 1), want["indptr"], want["indices"])
    assert np.linalg.norm(f64(out) - ref) <= 1e-2 * np.linalg.norm(ref)


def test_captured_on_another_stream():
    """The three calls in one graph follow new lengths, slots and scores in their buffers."""
    page, lens = 16, [500, 90]
    table, pages = pages_of([600, 200], page, 3)
    g, ws = gen(8), workspace()
    x = torch.randn(pages * page, 576, generator=g, device="cuda").bfloat16()
    means = torch.zeros(pages, 576, dtype=torch.bfloat16, device="cuda")
    all_slots = i32([table[b, t // page] * page + t % page for b, n in ((0, 600), (1, 200)) for t in range(n)])
    q = torch.randn(2, 16, 576, generator=g, device="cuda").bfloat16()
    scores, dev_table = torch.empty(table.shape, device="cuda"), i32(table)
    kv, qo, sel = i32(indptr(lens)), i32([0, 1, 2]), torch.empty(3, dtype=torch.int32, device="cuda")
    idx = torch.empty(1000, dtype=torch.int32, device="cuda")

    def calls():
        binding.mla_block_means_bf16kv(x, all_slots, means, page_size=page, workspace=ws)
        binding.mla_block_scores(q, means, dev_table, qo, kv, scores, page_size=page, workspace=ws)
        binding.mla_block_select(scores, dev_table, kv, sel, idx, page_size=page, num_pages=pages, blocks=8, sink=1, recent=1,
                                 workspace=ws)

    calls()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    for lens in ([600, 200], [17, 130]):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
        kv.copy_(i32(indptr(lens)))
        graph.replay()
        torch.cuda.synchronize()
        assert binding.mla_decode_read_error(ws) == 0
        want = block_select_ref(f64(scores), table, indptr(lens), page, 8, 1, 1)
        ref = block_scores_ref(f64(q), f64(means), table, [0, 1, 2], indptr(lens), page)
        on = ref > -np.inf
        assert (np.abs(f64(scores)[on] - ref[on]) <= 2.0**-14 * 40).all() and ((f64(scores) > -np.inf) == on).all()
        assert np.array_equal(sel.cpu().numpy(), want["indptr"])
        assert np.array_equal(idx.cpu().numpy()[:len(want["indices"])], want["indices"])


@pytest.mark.parametrize("tokens", [3, 4, 5, 9])
def test_scores_of_several_tokens_over_many_pages(tokens):
    """More pages than narrow blocks hold at once (wide ones for four tokens), rows of several rounds of tokens."""
    g, page, lens = gen(tokens), 2, [2 * 9001, 2 * 8000 + 1, 0, 2 * 4001]
    table, pages = pages_of(lens, page, tokens)
    q = torch.randn(4 * tokens, 16, 576, generator=g, device="cuda").bfloat16()
    means = (0.3 * torch.randn(pages, 576, generator=g, device="cuda")).bfloat16()
    scores, ws = torch.empty(table.shape, device="cuda"), workspace()
    binding.mla_block_scores(q, means, i32(table), i32(tokens * np.arange(5)), i32(indptr(lens)), scores, page_size=page, workspace=ws)
    assert binding.mla_decode_read_error(ws) == 0
    ref, got = block_scores_ref(f64(q), f64(means), table, tokens * np.arange(5), indptr(lens), page), f64(scores)
    spread = (np.abs(f64(q)).reshape(-1, 576) @ np.abs(f64(means)).T).max() / 24
    on = ref > -np.inf
    assert ((got > -np.inf) == on).all() and (np.abs(got[on] - ref[on]) <= 2.0**-14 * spread).all()


@pytest.mark.parametrize("kind", ["same", "two", "close", "far", "huge", "mixed", "steps"])
@pytest.mark.parametrize("pages", [900, 2048, 4096, 8192, 8193, 20_000])
def test_choice_where_the_steps_hold_many(pages, kind):
    """Scores alike, close together beside a few far away, over the whole range of float32, not finite: the steps
    are divided again until few pages are left."""
    g, lens, page = gen(pages), [3 * pages, 3 * (pages // 2) + 1], 3
    table, num = pages_of(lens, page, pages)
    x = torch.randn(table.shape, generator=g, device="cuda")
    if kind == "same":
        x[:] = -2.5
    elif kind == "two":
        x = torch.where(x > 0.5, 1.0, -0.0)
    elif kind == "close":
        x = 1.0 + x * 2.0**-20
        x[:, 77] = 1e20
        x[:, 78] = -1e20
    elif kind == "far":
        x = x.sign() * (x * 30).exp()
    elif kind == "huge":
        x = x.sign() * 3.3e38 * torch.rand(x.shape, generator=g, device="cuda")
    elif kind == "mixed":
        x[x > 1.0] = float("inf")
        x[x < -0.5] = -float("inf")
        x[:, 5::17] = float("nan")
    else:
        x = (x * 4).round() * 2.0**-30
    for blocks in (4, pages // 3, pages - 5):
        if blocks > 8192:
            blocks = 8192
        ref, (ptr, idx, chosen), err = select(x, table, lens, page, num, blocks, 1, 2)
        assert err == 0 and np.array_equal(ptr, ref["indptr"]) and np.array_equal(chosen, ref["chosen"]), blocks
        assert np.array_equal(idx[:-4], ref["indices"]) and (idx[-4:] == -7).all()
