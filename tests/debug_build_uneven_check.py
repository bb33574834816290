"""Runs the operators of decode steps over long contexts in the debug build of libmla_decode (bounds-checked kernels) over
unlike groups, waits that run out, wide blocks of scores and choices that divide their steps, and prints the runs' names as
one JSON line; each run's error word and results are checked by the operators' own tests.  Invoked in a fresh process by
tests/test_debug_long_named_checks.py (the debug library is the only one it loads)."""
import json
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from mla_decode_attention_08_gb300 import binding  # noqa: E402
from mla_decode_attention_08_gb300.build import build  # noqa: E402
from tests import test_gpu_blocks as blocks  # noqa: E402
from tests import test_gpu_select_widths as widths  # noqa: E402
from tests import test_gpu_shared_timeouts as timeouts  # noqa: E402
from tests import test_gpu_shared_uneven as uneven  # noqa: E402


def main() -> None:
    binding.load_library(build(debug=True))
    done = []

    def run(name, fn, *args):
        fn(*args)
        done.append(name)

    for paged in (False, True):
        for sms in (3, 152):
            run(f"uneven long paged={paged} sms={sms}", uneven.test_one_long_group_among_many, paged, sms)
        run(f"uneven few paged={paged}", uneven.test_few_groups_of_many_blocks, paged)
        for split in (0, 1):
            run(f"timeout paged={paged} split={split}", timeouts.test_outputs_stay_and_the_next_call_is_right, [9, 2, 5],
                [300, 129, 700], paged, split)
    run("uneven none", uneven.test_groups_without_tokens_keys_or_sense)
    for tokens in (3, 9):
        run(f"scores tokens={tokens}", blocks.test_scores_of_several_tokens_over_many_pages, tokens)
    for pages in (900, 4096, 8193):
        for kind in ("same", "close", "mixed", "steps"):
            run(f"choice pages={pages} {kind}", blocks.test_choice_where_the_steps_hold_many, pages, kind)
        for low, high in ((-3.4e38, 3.4e38), (0.0, 1e-38)):
            run(f"choice pages={pages} {low}..{high}", widths.test_choice, pages, True, low, high)
    torch.cuda.synchronize()
    print(json.dumps(done))


if __name__ == "__main__":
    main()
