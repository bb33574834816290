"""How mla_prefill_plan cuts a row's keys, on the CPU: never where the SMs have work, never
finer than key tiles, rounds bounded, and the workspace sized by the cut."""
import numpy as np
import pytest

from mla_decode_attention_08_gb300 import binding


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("seed", range(40))
def test_bounds(seed):
    rng = np.random.default_rng(seed)
    for _ in range(50):
        batch, sms = int(rng.integers(1, 40)), int(rng.integers(1, 200))
        total, kv = int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 17))
        heads = int(rng.integers(1, 40))
        p = binding.mla_prefill_plan(batch, total, kv, heads, sms)
        # as many rows as there may be end one query into a block of 128
        blocks, tiles = ((total - min(batch, total)) // 128 + min(batch, total)) * heads, -(-kv // 128)
        assert 1 <= p.splits <= max(1, tiles)
        if 10 * blocks >= 13 * sms:
            assert p.splits == 1
        assert blocks * p.splits <= max(blocks, 8 * sms)
        rows = p.splits * total * heads if p.splits > 1 else 0
        assert p.ws_bytes >= 256 + 4 * rows + 512 * rows


def test_no_keys_and_one_tile_are_not_cut():
    for kv in (0, 1, 128):
        assert binding.mla_prefill_plan(1, 4, kv, 1, 152).splits == 1


def test_thousands_of_empty_rows_are_not_cut():
    assert binding.mla_prefill_plan(1024, 4, 8192, 16, 152).splits > 1
    assert binding.mla_prefill_plan(1025, 4, 8192, 16, 152).splits == 1


def test_few_queries_take_a_part_for_every_free_sm():
    p = binding.mla_prefill_plan(1, 64, 8256, 16, 152)
    assert p.splits == 152 // 16


def test_blocks_on_most_of_the_sms_are_cut_over_several_rounds():
    p = binding.mla_prefill_plan(2, 800, 8500, 16, 152)
    blocks = ((800 - 2) // 128 + 2) * 16
    assert blocks < 152 < blocks * p.splits


def test_a_plan_with_other_parts_is_another_plan():
    """The parts may be chosen by the caller only together with the workspace's layout."""
    p = binding.mla_prefill_plan(1, 64, 8256, 16, 152)
    assert p.ws_bytes == p.ws_partial_offset + -(-p.splits * 64 * 16 * 512 // 256) * 256
