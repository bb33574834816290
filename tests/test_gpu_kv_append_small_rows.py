"""mla_kv_append: norms of rows whose squares float32 does not hold.

Tolerances: the float32 value lies within 2^-18 of the exact one (scaling by a power of two rounds nothing),
bf16 moves it by at most 2^-8 of it, or half its last step of 2^-133 next to zero, e4m3 by
max(2^-4 of it, 2^-10) in code units."""
import numpy as np
import pytest
import torch

from mla_decode_attention_08_gb300 import binding
from oracle.fp8 import e4m3fn_decode
from oracle.ops import e4m3_target, kv_row_ref
from .test_gpu_kv_append import Case, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30, 1e-25, 1e-12])
@pytest.mark.parametrize("magnitude", [1e-13, 1e-15, 1e-17, 1e-19, 1e-22, 1e-25, 1e-32, 1e-38])
def test_rows_whose_squares_float32_does_not_hold(magnitude, eps, e4m3):
    """The mean square of such rows is below float32's smallest values, the normalised row is not."""
    c = Case(9, 0, e4m3=e4m3, magnitude=magnitude, seed=3, kv_pad=0)
    c.kv[:, 512:] = 0.5
    c.kv[3, 1:512] = 0
    c.kv[4, :512] = torch.where(torch.arange(512, device="cuda") % 7 == 0, 1.0, magnitude).bfloat16()  # both kinds
    c.run(eps=eps)
    eps = float(np.float32(eps))
    assert binding.mla_decode_read_error(c.ws) == 0
    row = kv_row_ref(f64(c.kv), f64(c.weight), eps, np.ones((9, 32)), np.zeros((9, 32)), True)[:, :512]
    got = f64(c.dense)[:, :512]
    # (results near bf16's smallest values are held to its last step there)
    assert (np.abs(got - row) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(row) + 2.0 ** -134).all()
    if e4m3:
        s = float(c.scale.item())
        want = e4m3_target(row, s)
        codes = e4m3fn_decode(c.cache.cpu().numpy()[c.slots.cpu().numpy()])[:, :512]
        assert (np.abs(codes - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 2.0 ** -17 * np.abs(row / s)).all()
