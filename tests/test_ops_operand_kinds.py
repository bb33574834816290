"""Operands of another kind (a number for a tensor, a scalar tensor for a matrix) are refused by the binding
with its own errors."""
import pytest

from mla_decode_attention_08_gb300 import binding

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _lib(built_library):
    binding.load_library(built_library)


@pytest.mark.parametrize("scale", [0.02, None, "0.02"])
def test_a_scale_that_is_no_tensor(scale):
    i, h = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError if scale is None else TypeError, match="kv_scale"):
        binding.mla_kv_append(h, h[0, :512], torch.zeros(8, 64), i, i, h.to(torch.uint8), scale,
                              workspace=torch.zeros(256, dtype=torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [True, False])
def test_a_cache_of_no_dimension(e4m3):
    from .test_gpu_kv_append import Case
    c = Case(8, 4, e4m3=e4m3)
    c.cache = c.cache[0, 0]
    with pytest.raises(ValueError, match="576"):
        c.run()


@pytest.mark.gpu
def test_keys_of_no_dimension():
    from .test_gpu_prefill import Case
    c = Case([4], [4])
    c.k_nope = c.k_nope[0, 0, 0]
    with pytest.raises(ValueError, match="k_nope"):
        c.run()
