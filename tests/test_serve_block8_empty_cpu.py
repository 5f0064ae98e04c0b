"""keys_values of a served attention block that holds nothing, on the CPU."""
import pytest
from test_serve_block8_cpu import block

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", [[0, 0, 0], [0, -3, 0]])
def test_a_block_without_tokens_gives_no_rows(monkeypatch, dtype, lens):
    """Before any prompt and step, and for lengths that a step takes as 0: empty
    rows, without a call of the library, which refuses none."""
    layer, calls = block(monkeypatch, kv_bits=8)
    layer.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    k, v, starts = layer.keys_values(dtype)
    assert starts == [0] * 5 and k.shape == v.shape == (0, 1, 64)
    assert k.dtype == v.dtype == (dtype or torch.float16)
    assert "lqmm_kv_read_f8" not in calls.names()
