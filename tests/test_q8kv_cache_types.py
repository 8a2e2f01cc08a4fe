"""The pools that q8_cache makes, whatever torch's default type is."""
import pytest

torch = pytest.importorskip("torch")
import invariant_sequence_decode_gb300 as luce  # noqa: E402


@pytest.mark.parametrize("default", [torch.float32, torch.float64, torch.bfloat16])
def test_pools_have_their_types(default):
    was = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        k, v, s = luce.q8_cache(3, 2, 4, device="cpu")
    finally:
        torch.set_default_dtype(was)
    assert k.dtype == v.dtype == torch.int8 and s.dtype == torch.float32
    assert k.shape == v.shape == (3, 2, 4, 128, 128) and s.shape == (3, 2, 4, 2, 4)
