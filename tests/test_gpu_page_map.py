"""mla_page_map on the GPU against the loops of its definition: every output is a
whole number and has to be equal."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.ops import page_map_ref

pytestmark = pytest.mark.gpu

SEQ_LEN, FREE_PAGES, CAPACITY, KV_INDEX = 64, 128, 256, 4
FILL = -77


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


class Step:
    """A step's inputs on both sides; ``table_pad`` widens the table's rows."""

    def __init__(self, kv_lens, new_lens, page, seed=0, spare=3, table_pad=0, room=5, slot_room=5):
        rng = np.random.default_rng(seed)
        self.page = page
        self.kv_lens, self.new_lens = np.array(kv_lens), np.array(new_lens)
        before, after = -(-self.kv_lens // page), -(-(self.kv_lens + self.new_lens) // page)
        self.num_pages = int(after.sum()) + spare
        ids = rng.permutation(self.num_pages)
        self.table = np.full((len(kv_lens), max(1, int(after.max())) + 1), FILL)
        k = 0
        for b, n in enumerate(before):
            self.table[b, :n] = ids[k:k + n]
            k += n
        self.free = ids[k:]
        self.total, self.fresh = int((self.kv_lens + self.new_lens).sum()), int(self.new_lens.sum())
        dev = dict(dtype=torch.int32, device="cuda")
        self.t = {"kv_lens": torch.tensor(kv_lens, **dev), "new_lens": torch.tensor(new_lens, **dev),
                  "free": torch.tensor(self.free.tolist(), **dev)}
        wide = torch.full((len(kv_lens), self.table.shape[1] + table_pad), FILL, **dev)
        self.dev_table = wide[:, :self.table.shape[1]]
        self.dev_table.copy_(torch.from_numpy(self.table))
        n = len(kv_lens) + 1
        sizes = {"qo_indptr": n, "kv_indptr": n, "kv_indices": self.total + room,
                 "slots": self.fresh + slot_room, "positions": self.fresh + slot_room, "pages_used": 1}
        self.out = {k: torch.full((v,), FILL, **dev) for k, v in sizes.items()}
        self.ws = torch.zeros(binding.STEP_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        binding.mla_page_map(self.t["kv_lens"], self.t["new_lens"], self.dev_table, self.t["free"],
                             *self.out.values(), stream, page_size=self.page, num_pages=self.num_pages,
                             workspace=self.ws)

    def check(self):
        want = page_map_ref(self.kv_lens, self.new_lens, self.table, self.free, self.page)
        got = {k: v.cpu().numpy() for k, v in self.out.items()}
        assert binding.mla_decode_read_error(self.ws) == 0
        assert np.array_equal(self.dev_table.cpu().numpy(), want["table"])
        for k in ("qo_indptr", "kv_indptr"):
            assert np.array_equal(got[k], want[k]), k
        assert got["pages_used"][0] == want["pages_used"]
        for k, n, rest in (("kv_indices", self.total, FILL), ("slots", self.fresh, -1), ("positions", self.fresh, 0)):
            assert np.array_equal(got[k][:n], want[k]), k
            assert (got[k][n:] == rest).all(), k

    def check_emptied(self, error):
        assert binding.mla_decode_read_error(self.ws) == error
        assert binding.mla_decode_read_error(self.ws) == 0
        assert np.array_equal(self.dev_table.cpu().numpy(), self.table)
        got = {k: v.cpu().numpy() for k, v in self.out.items()}
        for k in ("qo_indptr", "kv_indptr", "positions", "pages_used"):
            assert (got[k] == 0).all(), k
        assert (got["slots"] == -1).all() and (got["kv_indices"] == FILL).all()


@pytest.mark.parametrize("page", [1, 3, 16, 64, 1000])
@pytest.mark.parametrize("kv_lens,new_lens", [
    ([0], [1]), ([0], [0]), ([1], [0]), ([63], [1]), ([64], [1]), ([65], [200]), ([4096], [1]),
    ([0, 0, 0], [0, 0, 0]), ([5, 0, 7, 0, 0, 130], [1, 0, 0, 3, 0, 65]),
    (list(range(40)), [1] * 40), ([1000, 0, 3, 64, 128, 2047], [0, 0, 700, 64, 1, 1])])
def test_maps_equal_the_definition(page, kv_lens, new_lens):
    step = Step(kv_lens, new_lens, page, seed=len(kv_lens) + page)
    step.run()
    step.check()
    step.run()                      # inputs are not consumed
    step.check()


@pytest.mark.parametrize("batch", [511, 512, 513, 1500])
def test_many_rows(batch):
    rng = np.random.default_rng(batch)
    kv = rng.integers(0, 200, batch) * (rng.random(batch) > 0.2)
    step = Step(kv.tolist(), rng.integers(0, 3, batch).tolist(), 16, seed=1, table_pad=5)
    step.run()
    step.check()


def test_the_largest_batch():
    rng = np.random.default_rng(5)
    step = Step(rng.integers(0, 9, 16384).tolist(), rng.integers(0, 2, 16384).tolist(), 4)
    step.run()
    step.check()


def test_exact_room_and_no_free_pages():
    step = Step([128, 64], [0, 0], 64, spare=0, room=0, slot_room=0)
    assert len(step.free) == 0
    step.run()
    step.check()
    binding.mla_page_map(step.t["kv_lens"], step.t["new_lens"], step.dev_table, None, step.out["qo_indptr"],
                         step.out["kv_indptr"], step.out["kv_indices"], None, None, step.out["pages_used"],
                         page_size=64, num_pages=step.num_pages, workspace=step.ws)
    step.check()


def test_a_step_that_cannot_be_mapped_is_emptied():
    step = Step([10, 20], [5, 6], 16, spare=0)
    step.t["new_lens"][1] = -1
    step.run()
    step.check_emptied(SEQ_LEN)
    step = Step([10, 20], [5, 6], 16)
    step.t["kv_lens"][0] = 16 * step.table.shape[1]              # + 5 tokens: past the row's pages
    step.run()
    step.check_emptied(SEQ_LEN)
    step = Step([10, 20], [0, 13], 16, spare=0)
    step.t["free"] = step.t["free"][:0]
    step.run()
    step.check_emptied(FREE_PAGES)
    step = Step([10, 20], [5, 6], 16, room=-1)
    step.run()
    step.check_emptied(CAPACITY)
    step = Step([10, 20], [5, 6], 16, slot_room=-1)
    step.run()
    step.check_emptied(CAPACITY)


def test_sums_past_32_bits_are_refused_not_wrapped():
    """Three rows of 2^30 tokens each pass every row's own limit; their sum passes 2^31."""
    step = Step([1, 1, 1], [0, 0, 0], 1 << 21, spare=1000)
    step.t["kv_lens"].fill_(1 << 30)
    wide = torch.full((3, 512), FILL, dtype=torch.int32, device="cuda")
    binding.mla_page_map(step.t["kv_lens"], step.t["new_lens"], wide, step.t["free"], *step.out.values(),
                         page_size=1 << 21, num_pages=1003, workspace=step.ws)
    assert binding.mla_decode_read_error(step.ws) == CAPACITY
    assert step.out["kv_indptr"].tolist() == [0, 0, 0, 0]


def test_a_page_outside_the_pool_marks_its_tokens():
    step = Step([40, 33], [1, 2], 16)
    want = page_map_ref(step.kv_lens, step.new_lens, step.table, step.free, 16)
    step.dev_table[0, 1] = step.num_pages
    step.dev_table[1, 0] = -5
    step.run()
    assert binding.mla_decode_read_error(step.ws) == KV_INDEX
    indices = want["kv_indices"].copy()
    indices[16:32] = -1
    indices[41:41 + 16] = -1
    assert np.array_equal(step.out["kv_indices"].cpu().numpy()[:step.total], indices)
    assert np.array_equal(step.out["slots"].cpu().numpy()[:step.fresh], want["slots"])


def test_replayed_graph_follows_the_lengths():
    first, second = Step([100, 5, 31], [1, 1, 1], 16, seed=2), Step([101, 6, 32], [1, 1, 1], 16, seed=2)
    step = Step([101, 6, 32], [1, 1, 1], 16, seed=2)
    step.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run()
    for want in (first, second):
        step.kv_lens, step.new_lens = want.kv_lens, want.new_lens
        step.table, step.free = want.table, want.free
        step.total, step.fresh = want.total, want.fresh
        step.num_pages = want.num_pages
        step.t["kv_lens"].copy_(want.t["kv_lens"])
        n = min(step.table.shape[1], step.dev_table.shape[1])
        step.dev_table.fill_(FILL)
        step.dev_table[:, :n].copy_(want.dev_table[:, :n])
        step.table = step.dev_table.cpu().numpy()
        free = torch.full_like(step.t["free"], 0)
        m = min(len(want.free), free.numel())
        free[:m] = want.t["free"][:m]
        step.t["free"].copy_(free)
        for v in step.out.values():
            v.fill_(FILL)
        g.replay()
        torch.cuda.synchronize()
        step.check()


def test_on_another_stream_and_sharing_a_workspace():
    a, b = Step([1000, 3], [1, 1], 16, seed=3), Step([77] * 50, [2] * 50, 8, seed=4)
    b.ws = a.ws
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        a.run(streams[0])
        b.run(streams[1])
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_binding_refuses_wrong_shapes():
    step = Step([4, 4], [1, 1], 4)
    with pytest.raises(ValueError):                                  # positions shorter than slots
        step.out["positions"] = step.out["positions"][:-1]
        step.run()
    step = Step([4, 4], [1, 1], 4)
    with pytest.raises(TypeError):
        step.t["kv_lens"] = step.t["kv_lens"].long()
        step.run()
    step = Step([4, 4], [1, 1], 4)
    with pytest.raises(ValueError):
        step.dev_table = step.dev_table[:1]
        step.run()
    step = Step([4, 4], [1, 1], 4)
    with pytest.raises(ValueError):                                  # overlapping rows
        step.dev_table = step.dev_table[:1].expand(2, -1)
        step.run()
