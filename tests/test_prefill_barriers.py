"""The barriers of mla_prefill_fwd on the CPU: every order in which the scheduler, the producer, the two MMA
issuers and the two softmax warpgroups can take their steps, in both walks.

An mbarrier wait looks at the parity of the completed phases only, so it is passed too early, or
never, when whoever arrives can be two phases away from whoever waits.  Each role is written
down as its sequence of waits and arrivals for a list of jobs (copies and products are taken as
done at once: the orders that let a role run furthest ahead), beside what it writes and has read in shared
memory ("use", what, what has to be done before), and all reachable states are visited.  How many v_clean barriers the kernel has is read from its source."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_decode_attention_08_gb300",
                      "csrc", "prefill.cu")
TILE = 128


def clean_barriers() -> int:
    """Barriers that say "V behind the row's end is zeroed": one a buffer of V, or one in all."""
    with open(SOURCE) as f:
        found = re.search(r"uint64_t v_clean(?:\[(\d+)\])?;", f.read())
    return int(found.group(1) or 1)


def roles(jobs, cleans):
    """The waits ("w", barrier, phase) and arrivals ("a", barrier) of each role in the walk of two query tiles.
    A job is (keys, key tiles that query tile 0 has, key tiles that query tile 1 has)."""
    sched, producer, issuers, softmax = [], [], ([], []), ([], [])
    everyone = list(enumerate([*jobs, None]))
    for k, job in everyone:                             # run_scheduler
        if k > 1:
            sched.append(("w", ("job_empty", k & 1), (k >> 1) - 1))
        sched.append(("a", ("job_full", k & 1)))
        if job is not None:
            sched.append(("w", ("claim",), k))
    def fill(f):
        """Fill f of the ring of eight slots, in place of one that both issuers have released."""
        return "use", ("fill", f), {("released", t, f - 8) for t in range(2)} if f >= 8 else set()

    tile = 0
    loads = [0, 0]
    for k, job in everyone:                             # next_job, load_job
        producer += [("w", ("job_full", k & 1), k >> 1), ("a", ("job_empty", k & 1))]
        if job is None:
            break
        n = max(job[1:])
        for j in range(n):
            if j == max(0, n - 1):
                producer.append(("a", ("claim",)))
            if tile > 1:
                producer.append(("w", ("v_empty", tile & 1), (tile >> 1) - 1))
            producer += [*(fill(5 * tile + i) for i in range(3)), ("a", ("k_full", tile & 1))]
            for t in range(2):
                if j == 0 and job[1 + t] > 0:
                    if loads[t] > 0:
                        producer.append(("w", ("q_empty", t), loads[t] - 1))
                    producer.append(("a", ("q_full", t)))
                    loads[t] += 1
            if tile > 0:
                producer.append(("w", ("k_empty", (tile - 1) & 1), (tile - 1) >> 1))
            producer += [*(fill(5 * tile + i) for i in (3, 4)), ("a", ("v_full", tile & 1))]
            tile += 1
        if n == 0:
            producer.append(("a", ("claim",)))
    for t, ops in enumerate(issuers):                   # run_mma
        tile = mine = done = 0
        turns = 0
        clean_phase = [0] * cleans
        for k, job in everyone:
            ops += [("w", ("job_full", k & 1), k >> 1), ("a", ("job_empty", k & 1))]
            if job is None:
                break
            keys, nt, n = job[0], job[1 + t], max(job[1:])
            if n == 0:
                continue
            duo = job[1] > 0 and job[2] > 0
            partial = keys // TILE if keys % TILE and keys // TILE < n else -1

            def release(at, n):
                ops.extend(("use", ("released", t, f), {("fill", f)}) for f in range(at, at + n))

            def scores(at, last, hand_over):
                if hand_over:
                    ops.append(("a", ("turn", t ^ 1)))
                release(5 * at, 3)
                ops.extend([("a", ("s_full", t)), ("a", ("k_empty", at & 1))])
                if last:
                    ops.append(("a", ("q_empty", t)))

            if nt > 0:
                ops.append(("w", ("q_full", t), done))
            ops.append(("w", ("k_full", tile & 1), tile >> 1))
            if nt > 0:
                scores(tile, nt == 1, False)
            else:
                release(5 * tile, 3)
                ops.append(("a", ("k_empty", tile & 1)))
            for j in range(n):
                following = j + 1 < nt
                ops.append(("w", ("v_full", tile & 1), tile >> 1))
                if j == partial:
                    b = tile % cleans
                    ops.append(("a", ("v_clean", b)) if t == 0 else ("w", ("v_clean", b), clean_phase[b]))
                    clean_phase[b] += 1
                if j == 0 and nt > 0 and done > 0:
                    ops.append(("w", ("o_free", t), done - 1))
                if duo:
                    if t == 1 or turns > 0:              # tile 0's first turn is its own
                        ops.append(("w", ("turn", t), turns - (t == 0)))
                    turns += 1
                if j < nt:
                    ops += [("w", ("p_head", t), mine), ("w", ("p_full", t), mine)]
                    mine += 1
                    if not following:
                        ops.append(("a", ("o_full", t)))
                release(5 * tile + 3, 2)
                ops.append(("a", ("v_empty", tile & 1)))
                if not following and duo:
                    ops.append(("a", ("turn", t ^ 1)))
                if j + 1 < n:
                    ops.append(("w", ("k_full", (tile + 1) & 1), (tile + 1) >> 1))
                    if following:
                        scores(tile + 1, j + 2 == nt, duo)
                    else:
                        release(5 * tile + 5, 3)
                        ops.append(("a", ("k_empty", (tile + 1) & 1)))
                tile += 1
            done += nt > 0
    for t, ops in enumerate(softmax):                   # softmax_job<false>
        tile = done = 0
        for k, job in everyone:
            ops += [("w", ("job_full", k & 1), k >> 1), ("a", ("job_empty", k & 1))]
            if job is None:
                break
            for _ in range(job[1 + t]):
                ops += [("w", ("s_full", t), tile), ("a", ("p_head", t)), ("y",), ("a", ("p_full", t))]
                tile += 1
            if job[1 + t] > 0:
                ops += [("w", ("o_full", t), done), ("y",), ("a", ("o_free", t))]
                done += 1
    return [sched, producer, *issuers, *softmax]


def pair_roles(jobs):
    """The same for alternating key tiles.  A job is its number of key tiles."""
    sched, producer, issuers, softmax = [], [], ([], []), ([], [])
    everyone = list(enumerate([*jobs, None]))
    for k, n in everyone:
        if k > 1:
            sched.append(("w", ("job_empty", k & 1), (k >> 1) - 1))
        sched.append(("a", ("job_full", k & 1)))
        if n is not None:
            sched.append(("w", ("claim",), k))
    tile = queries = 0
    for k, n in everyone:                               # load_pair_job
        producer += [("w", ("job_full", k & 1), k >> 1), ("a", ("job_empty", k & 1))]
        if n is None:
            break
        for j in range(n):
            b, before = tile & 1, (tile >> 1) - 1
            if j == max(0, n - 1):
                producer.append(("a", ("claim",)))
            if before >= 0:
                producer.append(("w", ("pair_k_empty", b), before))
            producer += [("use", ("k", tile), {("k read", tile - 2)} if tile > 1 else set()), ("a", ("k_full", b))]
            if j == 0:
                if queries > 0:
                    producer.append(("w", ("pair_q_empty",), queries - 1))
                last = {("q read", t, queries - 1) for t in range(2)} if queries > 0 else set()
                producer += [("use", ("q", queries), last), ("a", ("q_full", 0))]
                queries += 1
            if before >= 0:
                producer.append(("w", ("pair_v_empty", b), before))
            producer += [("use", ("v", tile), {("v read", tile - 2)} if tile > 1 else set()), ("a", ("v_full", b))]
            tile += 1
        if n == 0:
            producer.append(("a", ("claim",)))
    for t, ops in enumerate(issuers):                   # run_pair_mma
        tile = mine = done = own = 0
        for k, n in everyone:
            ops += [("w", ("job_full", k & 1), k >> 1), ("a", ("job_empty", k & 1))]
            if n is None:
                break
            if n == 0:
                continue
            first, start = (tile ^ t) & 1, tile
            tile += n
            ops.append(("w", ("q_full", 0), done))
            done += 1
            if first >= n:
                ops += [("use", ("q read", t, done - 1), {("q", done - 1)}), ("a", ("pair_q_empty",))]
                continue
            for j in range(first, n, 2):
                last = j + 2 >= n
                ops += [("w", ("k_full", t), mine), ("use", ("k read", start + j), {("k", start + j)}), ("a", ("s_full", t)),
                        ("a", ("pair_k_empty", t))]
                if last:
                    ops += [("use", ("q read", t, done - 1), {("q", done - 1)}), ("a", ("pair_q_empty",))]
                ops.append(("w", ("v_full", t), mine))
                if j == first and own > 0:
                    ops.append(("w", ("o_free", t), own - 1))
                ops += [("w", ("p_head", t), mine), ("w", ("p_full", t), mine)]
                if last:
                    ops.append(("a", ("o_full", t)))
                ops += [("use", ("v read", start + j), {("v", start + j)}), ("a", ("pair_v_empty", t))]
                mine += 1
            own += 1
    for t, ops in enumerate(softmax):                   # softmax_job<true>
        tile = done = joins = 0
        first, given = t, -1
        for k, n in everyone:
            ops += [("w", ("job_full", k & 1), k >> 1), ("a", ("job_empty", k & 1))]
            if n is None:
                break
            if first == 0 or n > 1:
                for _ in range(first, n, 2):
                    ops += [("w", ("s_full", t), tile), ("a", ("p_head", t)), ("y",), ("a", ("p_full", t))]
                    tile += 1
                if n > first:
                    ops.append(("w", ("o_full", t), done))
                    done += 1
                if n > 1 and first != 0:
                    ops += [("use", ("stats", t, k), {("stats read", t, given)} if given >= 0 else set()),
                            ("a", ("joined", t))]
                    given = k
                elif n > 1:
                    ops += [("w", ("joined", t ^ 1), joins), ("use", ("stats read", t ^ 1, k), {("stats", t ^ 1, k)}),
                            ("a", ("o_free", t)), ("a", ("o_free", t ^ 1))]
                    joins += 1
                elif n > 0:
                    ops += [("y",), ("a", ("o_free", t))]
            first ^= n & 1
    return [sched, producer, *issuers, *softmax]


COUNT = {"k_empty": 2, "v_empty": 2, "pair_q_empty": 2, "job_empty": 5}


def explore(programs):
    """(faults, states): waits that can be passed too early or can hang, as (role, barrier, phase), states from
    which nothing moves, and shared memory used before what has to come before.

    A role takes the arrivals after a wait along with it, up to a ("y",): held back they would only
    stop others."""
    steps = []                                          # per role: (the wait, "y" or None, arrivals and uses before it)
    for ops in programs:
        row, arrivals, uses = [], {}, frozenset()
        for op in ops:
            if op[0] == "a":
                arrivals = {**arrivals, op[1]: arrivals.get(op[1], 0) + 1}
            elif op[0] == "use":
                if row and row[-1][0][0] == "use" and row[-1][1] is arrivals:   # one step of uses in a row
                    row[-1] = (("use", (*row[-1][0][1], op[1]), row[-1][0][2] | op[2]), *row[-1][1:])
                else:
                    row.append((("use", (op[1],), op[2]), arrivals, uses))
                uses = uses | {op[1]}
            else:
                row.append((op, arrivals, uses))
        steps.append([*row, (None, arrivals, uses)])
    faults, seen, todo = set(), set(), [(0,) * len(steps)]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        now = [steps[r][at] for r, at in enumerate(state)]
        moved = False
        for r, (op, _, _) in enumerate(now):
            if op is None:
                continue
            go = op[0] == "y"
            if op[0] == "use":
                go = True
                if not op[2] <= frozenset().union(*(x[2] for x in now)):
                    faults.add((r, *op[1]))
            elif op[0] == "w":
                _, bar, phase = op
                phases = sum(x[1].get(bar, 0) for x in now) // COUNT.get(bar[0], 1)
                if (phases & 1) != (phase & 1):         # what the parity says
                    go = phases == phase + 1
                    moved = True
                    if not go:
                        faults.add((r, bar, phase))
                elif phases > phase:
                    faults.add((r, bar, phase))         # a phase too late: it would wait for one that is over
            if go:
                moved = True
                todo.append(tuple(at + (o == r) for o, at in enumerate(state)))
        if not moved and any(op is not None for op, _, _ in now):
            faults.add(("stuck", state))
    return faults, len(seen)


# keys, and key tiles of the two query tiles
BATCHES = {
    "short rows": [(100, 1, 0)] * 5,
    "a short row behind a long one": [(257, 3, 0), (5, 1, 0), (100, 1, 0)],
    "two tiles, then short rows": [(300, 2, 3), (60, 1, 0), (60, 1, 0), (300, 3, 3)],
    "rows of whole tiles between": [(100, 1, 0), (128, 1, 0), (100, 1, 0), (256, 2, 0), (100, 1, 0)],
    "the first tile sees nothing": [(90, 0, 1), (90, 0, 1), (200, 2, 0), (90, 0, 1)],
    "rows without keys between": [(100, 1, 0), (0, 0, 0), (100, 1, 0), (0, 0, 0), (10, 1, 0)],
    "turns kept over jobs": [(300, 3, 3), (130, 1, 2), (130, 2, 2), (40, 1, 1), (300, 0, 3)],
}


@pytest.mark.parametrize("name", BATCHES)
def test_no_order_of_steps_passes_a_phase_twice(name):
    faults, states = explore(roles(BATCHES[name], clean_barriers()))
    assert states > 50
    assert not faults


@pytest.mark.parametrize("seed", range(24))
def test_drawn_jobs(seed):
    rng = random.Random(seed)
    jobs = []
    for _ in range(rng.randint(2, 4)):
        tiles = rng.choice([(1, 0), (1, 0), (2, 0), (0, 1), (1, 1), (1, 2), (2, 3), (0, 0), (3, 3), (0, 2)])
        n = max(tiles)
        jobs.append((n and n * TILE - rng.choice([0, 5]), *tiles))
    assert not explore(roles(jobs, clean_barriers()))[0]


PAIRS = [[1, 1, 1, 1], [2, 1, 3, 1], [1, 2, 2, 3], [3, 0, 2, 1], [4, 3], [0, 1, 0, 2]]


@pytest.mark.parametrize("jobs", PAIRS)
def test_alternating_key_tiles(jobs):
    faults, states = explore(pair_roles(jobs))
    assert states > 500
    assert not faults


@pytest.mark.parametrize("seed", range(16))
def test_drawn_jobs_of_alternating_key_tiles(seed):
    rng = random.Random(seed)
    assert not explore(pair_roles([rng.choice([0, 1, 1, 2, 3, 4]) for _ in range(rng.randint(2, 4))]))[0]


def without(programs, name):
    return [[op for op in ops if not (op[0] == "w" and op[1][0] == name)] for ops in programs]


@pytest.mark.parametrize("name", ["joined", "pair_q_empty", "pair_k_empty", "job_empty", "o_free"])
def test_a_missing_wait_of_alternating_key_tiles_would_be_seen(name):
    assert explore(without(pair_roles([2, 2, 2, 2, 2]), name))[0]


@pytest.mark.parametrize("name", ["v_empty", "k_empty", "q_empty", "job_empty"])
def test_a_missing_wait_of_two_query_tiles_would_be_seen(name):
    assert explore(without(roles([(300, 3, 3), (300, 3, 3), (100, 1, 0), (100, 1, 0)], 2), name))[0]


def test_one_barrier_for_both_buffers_would_be_passed_twice():
    """The model sees it: with one barrier issuer 0 can zero a second job's V, and so complete a second phase,
    before issuer 1 has looked at the first."""
    faults, _ = explore(roles(BATCHES["short rows"], 1))
    assert any(f[1] == ("v_clean", 0) for f in faults if f[0] == 3)
