"""Runs the operators around the decode step in the debug build of libmla_decode (bounds-checked kernels) and
prints, as one JSON line, the names of the runs; each run's error word and results are checked by the
operators' own test cases.  Invoked in a fresh process by tests/test_gpu_debug_build_ops.py (the debug
library is the only one it loads)."""
import json
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from mla_decode_attention_08_gb300 import binding  # noqa: E402
from mla_decode_attention_08_gb300.build import build  # noqa: E402
from tests import test_gpu_attn_merge as merge  # noqa: E402
from tests import test_gpu_kv_append as append  # noqa: E402
from tests import test_gpu_page_map as page_map  # noqa: E402
from tests import test_gpu_prefill as prefill  # noqa: E402

MANY = ([300, 0, 5, 128, 1] * 12, [300, 40, 129, 500, 0] * 12)


def main() -> None:
    binding.load_library(build(debug=True))
    done = []

    def run(name, case):
        case.run()
        case.check()
        done.append(name)

    for page in (1, 3, 64):
        for kv, new in (([5, 0, 7, 0, 130], [1, 0, 0, 3, 65]), (list(range(40)), [1] * 40), ([4096, 64], [1, 0])):
            run(f"map page={page} rows={len(kv)}", page_map.Step(kv, new, page, table_pad=2))
    run("map exact room", page_map.Step([128, 64], [0, 0], 64, spare=0, room=0, slot_room=0))
    step = page_map.Step([64, 10], [1, 200], 64)
    step.t["free"] = step.t["free"][:1].contiguous()
    step.run()
    step.check_emptied(page_map.FREE_PAGES)
    done.append("map too few free pages")
    for e4m3 in (True, False):
        for inter in (True, False):
            run(f"append e4m3={e4m3} interleaved={inter}", append.Case(33, 9, inter, e4m3))
    run("append heads outermost", append.Case(21, 5, False, True, q_layout="hbd"))
    c = append.Case(20, 4)
    c.slots[3] = c.rows
    c.slots[5] = -1
    written = torch.ones(20, dtype=torch.bool)
    written[[3, 5]] = False
    c.run()
    c.check(append.KV_INDEX, written.numpy())
    done.append("append bad slots")
    for causal in (True, False):
        for name, q, kv, heads, sms in (("one", [300], [300], 2, 152), ("two tiles", [300, 5, 513], [700, 129, 513], 3, 1),
                                        ("pairs", [100, 1, 128], [513, 300, 256], 3, 2), ("cut", [64, 3], [4000, 70], 2, 152),
                                        ("cut over rounds", [300, 200], [4000, 1500], 2, 19), ("many", *MANY, 2, 152),
                                        ("no keys", [200, 3], [0, 0], 2, 152)):
            case = prefill.Case(q, kv, heads=heads, causal=causal, sms=sms, lead=1, tail=2)
            run(f"prompt {name} causal={causal} parts={case.plan.splits}", case)
    c = prefill.Case([40, 50, 60], [40, 50, 60], heads=1)
    c.d_qo[3] = c.q.shape[0] + 1
    c.d_kv[0] = -1
    c.run()
    assert binding.mla_decode_read_error(c.ws) == prefill.QO_INDPTR | prefill.KV_INDPTR
    assert (c.out[:40] == 7.0).all() and (c.out[90:] == 7.0).all()
    done.append("prompt rows outside")
    parts, lses = merge.make(3, (40, 2), 128)
    merge.check(parts, lses, *merge.run(parts, lses))
    done.append("merge")
    torch.cuda.synchronize()
    print(json.dumps(done))


if __name__ == "__main__":
    main()
