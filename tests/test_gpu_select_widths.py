"""mla_block_select where the scores' range makes no steps of float32: ranges beyond its largest value, so narrow that the
steps a unit are, denormal scores, each alone and beside infinities and NaN."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from tests.test_gpu_blocks import gen, pages_of, select

pytestmark = pytest.mark.gpu

# (lowest, highest) finite scores: 255 / (highest - lowest) overflows below about 7.5e-37
RANGES = [(-3.4e38, 3.4e38), (-3.4e38, 0.1), (-1e30, 3.402823e38), (0.0, 1e-38), (-1e-38, 1e-38), (1e-38, 1.1e-38), (0.0, 7e-37),
          (0.0, 8e-37), (-7e-45, 7e-45), (0.0, 1.4e-45), (1.0, 1.0000001)]


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("low,high", RANGES)
@pytest.mark.parametrize("others", [False, True])
@pytest.mark.parametrize("pages", [200, 900, 8192, 8193])
def test_choice(pages, others, low, high):
    g, lens, page = gen(pages), [3 * pages, 3 * (pages // 2) + 1], 3
    table, num = pages_of(lens, page, pages)
    u = torch.rand(table.shape, generator=g, device="cuda", dtype=torch.float64)
    x = (low + (high - low) * u).float()
    assert bool(x.isfinite().all())
    x[:, 11], x[:, 12] = low, high
    if others:
        x[:, 20::9], x[:, 21::11], x[:, 22::40] = float("inf"), -float("inf"), float("nan")
    for blocks in (4, pages // 3, pages - 5):
        ref, (ptr, idx, chosen), err = select(x, table, lens, page, num, blocks, 1, 2)
        assert err == 0 and np.array_equal(ptr, ref["indptr"]) and np.array_equal(chosen, ref["chosen"]), blocks
        assert np.array_equal(idx[:-4], ref["indices"]) and (idx[-4:] == -7).all()
