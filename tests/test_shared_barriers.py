"""The barriers of mla_shared_fwd on the CPU: every order in which the scheduler, the copies of keys, the two MMA
issuers and the softmax warps can take their steps.

As in the prompt kernel's test, whose walk over all reachable states this one uses: a wait looks at the parity of
completed phases only, and each role is written down as its waits and arrivals for a list of jobs (copies and products
are taken as done at once), beside what it writes and has read.  Two panels stand for a tile's four, two warps of
a warpgroup for its four (one with the first keys of a tile, one with the last), and one or two warpgroups, of which
the second may be one without a token."""
import random
import re

import pytest

from . import test_prefill_barriers as walk

SOURCE = walk.SOURCE.replace("prefill.cu", "shared.cu")
PANELS = 2


def roles(jobs, groups=((0, 1),), absent=(), moved=()):
    """``jobs``: key tiles of each.  ``groups``: the parts of P (0 the first keys, 1 the last) that each warpgroup's
    modelled warps write.  ``absent``: warpgroups without a token.  ``moved``: tiles (of all jobs) at which the
    references move, so that O is scaled."""
    sched, keys, scores, values = [], [], [], []
    warps = [(g, part) for g, parts in enumerate(groups) for part in parts]
    here = [w for w in warps if w[0] not in absent]
    readers = ["keys", "scores", "values", *warps]
    everyone = list(enumerate([*jobs, None]))
    parts = sorted({part for _, part in warps})

    def next_job(ops, who, k):                          # next_job: the first is known when the roles start
        if k > 0:
            ops.append(("w", ("job_full", k & 1), (k - 1) >> 1))
        ops += [("use", ("job read", who, k), {("job", k)} if k > 0 else set()), ("a", ("job_empty", k & 1))]

    for k, _ in everyone:                               # run_scheduler
        if k > 1:
            sched.append(("w", ("job_empty", k & 1), (k >> 1) - 1))
        if k > 0:
            sched += [("use", ("job", k), {("job read", r, k - 2) for r in readers} if k > 1 else set()),
                      ("a", ("job_full", k & 1))]
    tile = 0
    for k, n in everyone:                               # run_producer, run_copies
        next_job(keys, "keys", k)
        for _ in range(n or 0):
            if tile > 0:
                keys.append(("w", ("rope_empty",), tile - 1))
            keys += [("use", ("rope", tile), {("rope read", tile - 1)} if tile > 0 else set()), ("a", ("rope_full",))]
            for c in range(PANELS):
                at = PANELS * (tile & 1) + c
                if tile > 1:
                    keys.append(("w", ("key_empty", at), (tile >> 1) - 1))
                keys += [("use", ("key", tile, c), {("v read", tile - 2, c)} if tile > 1 else set()), ("a", ("key_full", at))]
            tile += 1
    tile = done = 0
    for k, n in everyone:                               # run_scores
        next_job(scores, "scores", k)
        for j in range(n or 0):
            first = PANELS * (tile & 1)
            if j == 0:
                scores += [("w", ("key_full", first + c), tile >> 1) for c in range(PANELS)]
            if tile > 1:
                scores.append(("w", ("s_free", tile & 1), (tile >> 1) - 1))
            scores.append(("w", ("rope_full",), tile))
            if j == 0:
                scores.append(("w", ("q_full",), done))
            need = {("s read", w, tile - 2) for w in here} if tile > 1 else set()
            scores += [("use", ("rope read", tile), {("rope", tile)} | need | {("q", w, done) for w in here}),
                       ("a", ("rope_empty",))]
            for c in range(PANELS):
                if j > 0:
                    scores.append(("w", ("key_full", first + c), tile >> 1))
                scores.append(("use", ("k read", tile, c), {("key", tile, c)}))
            scores += [("use", ("s", tile), set()), ("a", ("s_full", tile & 1))]
            if j == n - 1:
                scores += [("use", ("q read", done), set()), ("a", ("q_empty",))]
            tile += 1
        done += bool(n)
    tile = done = 0
    for k, n in everyone:                               # run_values
        next_job(values, "values", k)
        if n and done > 0:
            values.append(("w", ("o_free",), done - 1))
        for j in range(n or 0):
            for part in parts:
                values.append(("w", ("p_full", part), tile))
                need = {("p", w, tile) for w in here if w[1] == part}
                if j == 0 and done > 0:
                    need |= {("o read", w, done - 1) for w in here}
                values.append(("use", ("o added", tile, part), need | {("scaled", w, tile) for w in here if tile in moved and j > 0}))
            values += [("use", ("v read", tile, 0), {("key", tile, 0)}), ("a", ("key_empty", PANELS * (tile & 1)))]
            for c in range(1, PANELS):
                for part in parts:
                    if c == PANELS - 1:
                        values += [("use", ("p read", part, tile), set()), ("a", ("p_free", tile & 1, part))]
                values += [("use", ("v read", tile, c), {("key", tile, c)}), ("a", ("key_empty", PANELS * (tile & 1) + c))]
            tile += 1
        done += bool(n)
    softmax = []
    for w in warps:                                     # run_softmax
        g, part = w
        ops, tile, done, votes, moves = [], 0, 0, 0, 0

        def query(number):
            if w in here:
                ops.append(("use", ("q", w, number), {("q read", number - 1)} if number > 0 else set()))
            ops.append(("a", ("q_full",)))

        next_job(ops, w, 0)
        if jobs and jobs[0]:
            query(0)
        for k, n in enumerate(jobs):
            for j in range(n):
                ops.append(("w", ("s_full", tile & 1), tile >> 1))
                if w in here:
                    ops.append(("use", ("s read", w, tile), {("s", tile)}))
                ops.append(("a", ("s_free", tile & 1)))
                if tile > 0:
                    ops.append(("w", ("p_free", (tile - 1) & 1, part), (tile - 1) >> 1))
                if w in here:
                    if j == 0 and done > 0:
                        ops.append(("w", ("o_free",), done - 1))
                    need = {("p read", part, tile - 1)} if tile > 0 else set()
                    if j == 0 and done > 0:
                        need |= {("o read", v, done - 1) for v in here}     # the rows left through P's memory
                    ops.append(("use", ("p", w, tile), need))
                    if j > 0 and tile in moved:
                        ops += [("w", ("p_free", (tile - 1) & 1, parts[-1]), (tile - 1) >> 1),
                                ("use", ("scaled", w, tile), {("p read", parts[-1], tile - 1)}),
                                ("a", ("moved", g)), ("w", ("moved", g), moves)]
                        moves += 1
                ops.append(("a", ("p_full", part)))
                tile += 1
            next_job(ops, w, k + 1)
            ops += [("a", ("vote", g)), ("w", ("vote", g), votes)]
            votes += 1
            following = jobs[k + 1] if k + 1 < len(jobs) else 0
            if following:
                if done > 0 or n > 0:
                    ops.append(("w", ("q_empty",), done + (n > 0) - 1))
                query(done + (n > 0))
            if n > 0:
                ops.append(("w", ("p_free", (tile - 1) & 1, parts[-1]), (tile - 1) >> 1))
                if w in here:
                    ops.append(("use", ("o read", w, done), {("p read", q, tile - 1) for q in parts}))
                ops.append(("a", ("o_free",)))
                done += 1
            ops += [("a", ("vote", g)), ("w", ("vote", g), votes)]          # (factor is read)
            votes += 1
        softmax.append(ops)
    counts = {"job_empty": len(readers), "s_free": len(warps), "q_full": len(warps), "o_free": len(warps),
              "p_full": len(groups), "vote": len(groups[0]), "moved": len(groups[0])}
    return [sched, keys, scores, values, *softmax], counts


@pytest.fixture
def faults(monkeypatch):
    def run(model):
        programs, counts = model
        monkeypatch.setattr(walk, "COUNT", counts)
        found, states = walk.explore(programs)
        assert states > 20
        return found
    return run


def test_the_model_has_the_kernels_barriers():
    with open(SOURCE) as f:
        text = f.read()
    body = text[text.index("struct Misc {"):text.index("uint32_t tmem_base;")]
    names = re.findall(r"(\w+)(?:\[[^;,]*\])?[;,]", re.sub(r"//[^\n]*", "", body).replace("uint64_t", ""))
    assert set(names) == {"job_full", "job_empty", "key_full", "key_empty", "rope_full", "rope_empty", "q_full", "q_empty",
                          "s_full", "s_free", "p_full", "p_free", "o_free", "mma_done"}
    assert "uint64_t p_free[2][4];" in text and "uint64_t p_full[4];" in text


@pytest.mark.parametrize("jobs", [[1], [4], [1, 1, 1], [3, 1], [0, 2, 0, 1]])
@pytest.mark.parametrize("moved", [(), (1, 2, 3)])
def test_no_order_of_steps_passes_a_phase_twice(faults, jobs, moved):
    assert not faults(roles(jobs, moved=moved))


@pytest.mark.parametrize("jobs", [[2], [1, 1], [1, 0, 2]])
def test_two_warpgroups_and_one_without_a_token(faults, jobs):
    assert not faults(roles(jobs, groups=((1,), (1,)), moved=(1, 2)))
    assert not faults(roles(jobs, groups=((1,), (1,)), absent=(1,), moved=(1, 2)))


def test_all_warps_of_two_warpgroups(faults):
    assert not faults(roles([1], groups=((0, 1), (0, 1)), absent=(1,)))


@pytest.mark.parametrize("seed", range(4))
def test_drawn_jobs(faults, seed):
    rng = random.Random(seed)
    jobs = [rng.choice([0, 1, 1, 2, 3]) for _ in range(3)]
    assert not faults(roles(jobs, moved=[t for t in range(12) if rng.random() < 0.3]))


def without(model, name):
    programs, counts = model
    return [[op for op in ops if not (op[0] == "w" and op[1][0] == name)] for ops in programs], counts


@pytest.mark.parametrize("name", ["job_empty", "key_empty", "rope_empty", "q_empty", "s_free", "p_free", "p_full", "q_full",
                                  "s_full", "moved"])
def test_a_missing_wait_would_be_seen(faults, name):
    jobs = [2, 1] if name == "p_full" else [3, 1]
    assert faults(without(roles(jobs, moved=(1, 2)), name))


def test_the_wait_for_the_other_warpgroups_output_is_needed(faults):
    """One warpgroup's warps meet at its own barriers, two only here."""
    assert faults(without(roles([1, 1], groups=((1,), (1,))), "o_free"))
