"""mla_kv_append: the e4m3 codes of the position parts bit for bit, and every latent within half a step.

The position parts at an angle of zero (cos 1, sin 0) are the inputs themselves, so their codes are those
of the float32 quotient by the scale, to nearest even.  The latents' float32 values lie within 2^-18 of the
exact ones (see the other append tests) and the quotient within 2^-22 more; the code is then off by at most
half its step, which is 2^-4 of the binade's lower end and 2^-10 below 2^-6."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.fp8 import e4m3fn_decode, e4m3fn_encode
from oracle.ops import e4m3_target, kv_row_ref
from .test_gpu_kv_append import EPS, Case, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


def chosen_values() -> np.ndarray:
    """e4m3's finite magnitudes, the ties between them and their bf16 neighbours, and values past the range."""
    grid = e4m3fn_decode(np.arange(1, 0x7F, dtype=np.uint8))
    ties = np.concatenate([[grid[0] / 2], (grid[1:] + grid[:-1]) / 2])
    near = np.concatenate([ties * (1 + 2.0 ** -7), ties * (1 - 2.0 ** -8)])
    far = np.array([464.0, 466.0, 480.0, 1e4, 3e38, 2.0 ** -11, 2.0 ** -20, 1e-38])
    values = np.concatenate([grid, ties, near, far])
    values = torch.tensor(values).bfloat16().double().numpy()
    return np.concatenate([values, -values])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("scale", [1.0, 0.25, 0.02, 3.1e-3, 7.0])
def test_position_parts_bit_for_bit(scale, interleaved):
    values = chosen_values()
    # At other scales: the bf16 values nearest to the chosen codes' values.
    with np.errstate(over="ignore"):
        values = torch.tensor(np.float32(values) * np.float32(scale)).bfloat16().float().numpy()
    values = values[np.isfinite(values)]
    tokens = -(-len(values) // 64)
    c = Case(tokens, 0, interleaved, scale=scale, seed=1)
    flat = np.zeros(64 * tokens, np.float32)
    flat[:len(values)] = values
    c.kv[:, 512:] = torch.tensor(flat.reshape(tokens, 64)).cuda().bfloat16()
    c.positions.zero_()
    assert (c.table[0, :32] == 1).all() and (c.table[0, 32:] == 0).all()
    c.run()
    assert binding.mla_decode_read_error(c.ws) == 0
    want = e4m3fn_encode(flat.reshape(tokens, 64) / np.float32(scale))
    got = c.cache.cpu().numpy()[c.slots.cpu().numpy()][:, 512:]
    # (the rotation adds a zero, so a negative value that rounds to zero keeps its sign and zero itself has none)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("scale", [0.02, 0.3, 0.004])
def test_latents_within_half_a_step(scale):
    c = Case(200, 0, scale=scale, seed=2)
    c.run()
    row = kv_row_ref(f64(c.kv0), f64(c.weight), EPS, np.ones((200, 32)), np.zeros((200, 32)), True)[:, :512]
    want = e4m3_target(row, float(c.scale.item()))
    got = e4m3fn_decode(c.cache.cpu().numpy()[c.slots.cpu().numpy()])[:, :512]
    half = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -30))) - 4), 2.0 ** -10)
    assert (np.abs(got - want) <= half + (2.0 ** -18 + 2.0 ** -22) * np.abs(row / float(c.scale.item()))).all()
