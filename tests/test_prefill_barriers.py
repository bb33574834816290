"""The barriers of mla_prefill_fwd's walk of two query tiles, on the CPU: every order in which
the scheduler, the producer and the two MMA issuers can take their steps.

An mbarrier wait looks at the parity of the completed phases only, so it is passed too early, or
never, when whoever arrives can be two phases away from whoever waits.  Each role is written
down as its sequence of waits and arrivals for a list of jobs (the softmax and the products are taken as
done at once: the orders that let an issuer run furthest ahead), and all reachable states are
visited.  How many v_clean barriers the kernel has is read from its source."""
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
    """The waits ("w", barrier, phase) and arrivals ("a", barrier) of each role.  A job is (keys, key
    tiles that query tile 0 has, key tiles that query tile 1 has)."""
    sched, producer, issuers = [], [], ([], [])
    everyone = list(enumerate([*jobs, None]))
    for k, job in everyone:                             # run_scheduler
        if k > 1:
            sched.append(("w", ("job_empty", k & 1), (k >> 1) - 1))
        sched.append(("a", ("job_full", k & 1)))
        if job is not None:
            sched.append(("w", ("claim",), k))
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
            producer.append(("a", ("k_full", tile & 1)))
            for t in range(2):
                if j == 0 and job[1 + t] > 0:
                    if loads[t] > 0:
                        producer.append(("w", ("q_empty", t), loads[t] - 1))
                    producer.append(("a", ("q_full", t)))
                    loads[t] += 1
            if tile > 0:
                producer.append(("w", ("k_empty", (tile - 1) & 1), (tile - 1) >> 1))
            producer.append(("a", ("v_full", tile & 1)))
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

            def scores(at, last, hand_over):
                if hand_over:
                    ops.append(("a", ("turn", t ^ 1)))
                ops.append(("a", ("k_empty", at & 1)))
                if last:
                    ops.append(("a", ("q_empty", t)))

            if nt > 0:
                ops.append(("w", ("q_full", t), done))
            ops.append(("w", ("k_full", tile & 1), tile >> 1))
            if nt > 0:
                scores(tile, nt == 1, False)
            else:
                ops.append(("a", ("k_empty", tile & 1)))
            for j in range(n):
                following = j + 1 < nt
                ops.append(("w", ("v_full", tile & 1), tile >> 1))
                if j == partial:
                    b = tile % cleans
                    ops.append(("a", ("v_clean", b)) if t == 0 else ("w", ("v_clean", b), clean_phase[b]))
                    clean_phase[b] += 1
                if duo:
                    if t == 1 or turns > 0:              # tile 0's first turn is its own
                        ops.append(("w", ("turn", t), turns - (t == 0)))
                    turns += 1
                ops.append(("a", ("v_empty", tile & 1)))
                if not following and duo:
                    ops.append(("a", ("turn", t ^ 1)))
                if j + 1 < n:
                    ops.append(("w", ("k_full", (tile + 1) & 1), (tile + 1) >> 1))
                    if following:
                        scores(tile + 1, j + 2 == nt, duo)
                    else:
                        ops.append(("a", ("k_empty", (tile + 1) & 1)))
                tile += 1
            done += nt > 0
    return [sched, producer, *issuers]


COUNT = {"k_empty": 2, "v_empty": 2, "job_empty": 3}


def explore(jobs, cleans):
    """(waits that can be passed too early or can hang, states): each as (role, barrier, phase).

    A role takes the arrivals after a wait along with it: held back they would only stop others."""
    programs = roles(jobs, cleans)
    steps = []                                          # per role: (the wait or None, arrivals before it)
    for ops in programs:
        row, arrivals = [], {}
        for op in ops:
            if op[0] == "a":
                arrivals = {**arrivals, op[1]: arrivals.get(op[1], 0) + 1}
            else:
                row.append((op[1:], arrivals))
        steps.append([*row, (None, arrivals)])
    faults, seen, todo = set(), set(), [(0,) * len(steps)]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        moved = False
        for r, at in enumerate(state):
            wait, _ = steps[r][at]
            if wait is None:
                continue
            bar, phase = wait
            phases = sum(steps[o][state[o]][1].get(bar, 0) for o in range(len(steps))) // COUNT.get(bar[0], 1)
            if (phases & 1) != (phase & 1):             # what the parity says
                moved = True
                if phases != phase + 1:
                    faults.add((r, bar, phase))
                else:
                    todo.append(tuple(a + (o == r) for o, a in enumerate(state)))
            elif phases > phase:
                faults.add((r, bar, phase))             # a phase too late: it would wait for one that is over
        if not moved and any(steps[r][at][0] is not None for r, at in enumerate(state)):
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
    faults, states = explore(BATCHES[name], clean_barriers())
    assert states > 50
    assert not faults


@pytest.mark.parametrize("seed", range(60))
def test_drawn_jobs(seed):
    rng = random.Random(seed)
    jobs = []
    for _ in range(rng.randint(2, 5)):
        tiles = rng.choice([(1, 0), (1, 0), (2, 0), (0, 1), (1, 1), (1, 2), (2, 3), (0, 0), (3, 3), (0, 2)])
        n = max(tiles)
        jobs.append((n and n * TILE - rng.choice([0, 5]), *tiles))
    assert not explore(jobs, clean_barriers())[0]


def test_one_barrier_for_both_buffers_would_be_passed_twice():
    """The model sees it: with one barrier issuer 0 can zero a second job's V, and so complete a second phase,
    before issuer 1 has looked at the first."""
    faults, _ = explore(BATCHES["short rows"], 1)
    assert any(f[1] == ("v_clean", 0) for f in faults if f[0] == 3)
