"""Runs the operators of decode steps over long contexts in the debug build of libmla_decode (bounds-checked
kernels) and prints, as one JSON line, the names of the runs; each run's error word and results are checked by the
operators' own tests.  Invoked in a fresh process by tests/test_gpu_debug_build_long.py (the debug library is the
only one it loads)."""
import json
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from mla_decode_attention_08_gb300 import binding  # noqa: E402
from mla_decode_attention_08_gb300.build import build  # noqa: E402
from tests import test_gpu_blocks as blocks  # noqa: E402
from tests import test_gpu_shared as shared  # noqa: E402


def main() -> None:
    binding.load_library(build(debug=True))
    done = []

    def run(name, fn, *args, **kwargs):
        fn(*args, **kwargs)
        done.append(name)

    def groups(q, kv, paged, sms):
        case = shared.Case(q, kv, paged, seed=sum(kv), lead=1, tail=2, sms=sms)
        for _ in range(2):
            assert case.run() == 0
            case.check()

    for paged in (False, True):
        for sms in (152, 3):
            for q, kv in (([1], [1]), ([5], [300]), ([3, 0, 9, 1], [300, 50, 0, 1]), ([33, 4, 2], [64, 1500, 700]),
                          ([2] * 70, [129, 0, 60, 300, 1] * 14)):
                run(f"shared q={len(q)}:{q[0]} kv={sum(kv)} paged={paged} sms={sms}", groups, q, kv, paged, sms)
    run("shared group outside", shared.test_a_group_out_of_range_is_reported_and_left)
    run("shared decreasing", shared.test_decreasing_offsets_write_nothing_stale_when_keys_are_split)
    run("shared bad page", shared.test_a_bad_page_entry_is_reported)
    for cache in ("e4m3", "bf16"):
        for page in (1, 16, 1000):
            run(f"means {cache} page={page}", blocks.test_means, cache, page, [10, 0, 300], [250, 65, 3])
    run("means slots outside", blocks.test_means_of_slots_out_of_range_are_reported)
    for page in (1, 64):
        for tokens, lens in (([1, 1, 1], [64, 0, 1000]), ([3, 0, 5], [300, 70, 1025]), ([4] * 9, [500] * 9)):
            run(f"scores page={page} tokens={sum(tokens)}", blocks.test_scores, tokens, lens, page)
    run("scores outside", blocks.test_scores_of_bad_pages_rows_and_values)
    for blocks_, sink, recent in ((1, 0, 1), (16, 2, 14), (600, 5, 90)):
        for ties in (False, True):
            run(f"choice blocks={blocks_} ties={ties}", blocks.test_choice, 16, blocks_, sink, recent, ties)
    run("choice of a long row", blocks.test_choice_of_a_long_row)
    run("choice emptied", blocks.test_choice_that_cannot_be_laid_out_is_emptied)
    run("sparse step", blocks.test_a_sparse_decode_step)
    torch.cuda.synchronize()
    print(json.dumps(done))


if __name__ == "__main__":
    main()
