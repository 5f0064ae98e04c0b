"""The type that an 8-bit cache is written for, with and without queries."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve8_oracle as s8
from gpu_util import announce
from test_serve8_gpu import values
from test_serve_gpu import DEV, DT, np64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


def append(x, with_q, **kw):
    cache = [c.view(torch.uint8).zero_() for c in bq.kv_cache_empty(2, 1, 16, 64, dtype=F8)]
    cache += [s.view(torch.uint8) for s in bq.kv_scales_empty(2, 1, 16)]
    announce(f"append_norm of a type: {x.dtype} q={with_q} {kw}")
    q = bq.lqmm_kv_append_norm(x[:, :1] if with_q else None, x[:, 1:2], x[:, 2:], None,
                               torch.arange(len(x), device=DEV), *cache, **kw)
    return q, cache


def vectors(tin):
    r = np.random.default_rng(1)
    x = np.ldexp(r.standard_normal((9, 3, 64)), r.integers(-4, 15 if tin == "f16" else 40, (9, 3, 1)))
    return torch.from_numpy(np.clip(x, -6e4, 6e4) if tin == "f16" else x).to(DT[tin]).to(DEV)


@pytest.mark.parametrize("tin", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_keys_and_values_alone_are_held_as_beside_queries(tin, t):
    """Large vectors: the same codes and scales with q, with q_out and without q,
    those of the type's range."""
    x = vectors(tin)
    want = append(x, True, q_out=torch.empty(9, 1, 64, dtype=DT[t], device=DEV))[1]
    q, both = append(x, True, dtype=DT[t])
    none, alone = append(x, False, dtype=DT[t])
    assert q.dtype == DT[t] and none is None
    for got in (both, alone):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    v, e = s8.quant(np64(x[:, 2]), t)
    got = values(want[1]).transpose(0, 1, 2, 4, 3).reshape(32, 64)
    assert np.array_equal(got[:9], v) and np.array_equal(want[3].cpu().numpy().reshape(32)[:9], e + 127)
    assert tin == "f16" or (e.max() > 7) == (t == "bf16")


def test_the_type_by_default():
    """k's when that is 16-bit, else float16."""
    for tin, t in (("f32", "f16"), ("bf16", "bf16"), ("f16", "f16")):
        x = vectors(tin)
        assert all(torch.equal(a, b) for a, b in zip(append(x, False)[1], append(x, False, dtype=DT[t])[1]))


def test_types_that_do_not_fit_are_refused():
    x = vectors("f32")
    for dtype in (torch.float32, F8, "float16", 1):
        with pytest.raises(TypeError):
            append(x, False, dtype=dtype)
    with pytest.raises(TypeError):
        append(x, True, dtype=torch.bfloat16, q_out=torch.empty(9, 1, 64, dtype=torch.float16, device=DEV))
    k, v = bq.kv_cache_empty(2, 1, 16, 64)
    slots = torch.arange(9, device=DEV)
    with pytest.raises(TypeError):
        bq.lqmm_kv_append_norm(None, x[:, 1:2], x[:, 2:], None, slots, k, v, dtype=torch.bfloat16)
    bq.lqmm_kv_append_norm(None, x[:, 1:2], x[:, 2:], None, slots, k, v, dtype=torch.float16)
