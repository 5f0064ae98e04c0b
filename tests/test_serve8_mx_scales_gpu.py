"""MXFP4 products with scales at both ends of their byte (2^-127 is every zero
block's), against 64 bits."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve8_oracle as s8
import serve_oracle as so
from gpu_util import announce
from test_serve8_gpu import up
from test_serve_gpu import DT

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
MOST = {"f16": 65504.0, "bf16": 2.0 ** 128 - 2.0 ** 120, "f32": 2.0 ** 128 - 2.0 ** 104}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M, N, K", [(1, 130, 96), (16, 300, 4128), (40, 200, 544), (64, 6144, 1056), (100, 1001, 288),
                                     (300, 700, 416), (2049, 4100, 256)])
@pytest.mark.parametrize("of_w, of_x", [
    ((0, 1), (253, 254)), ((253, 254), (0, 1)),  # ends against each other: ordinary products
    ((0, 127), (0, 127)),                        # beside zero blocks' scale
    ((0, 254), (100, 127)),                      # far apart, some past the largest number
    ((60, 66), (60, 66)), ((57, 60), (50, 53)),  # products around fp32's least normal number, and below it
    ((190, 195), (60, 66)), ((0, 1), (0, 1)),
])
def test_products_of_far_scales(M, N, K, t, of_w, of_x):
    """Where no sum leaves the output's range. Beside check_mx's bound, each of the
    K / 128 + 10 roundings may be at fp32's smallest step, 2^-149 (half of it)."""
    r = np.random.default_rng(M)
    make = lambda n, of: (r.integers(0, 16, (n, K)).astype(np.uint8), r.choice(of, (n, K // 32)).astype(np.uint8))  # noqa: E731
    (w, ws), (x, xs) = make(N, of_w), make(M, of_x)
    announce(f"gemm_mxfp4 {M}x{N}x{K} {t} scales {of_w} {of_x}")
    got = bq.lqmm_gemm_mxfp4(up(s8.mx_pack(w)), up(ws), up(s8.mx_pack(x)), up(xs), out_dtype=DT[t]).double()
    W, X = up(s8.mx_values(w, ws)), up(s8.mx_values(x, xs))
    want = torch.matmul(X, W.t().contiguous())
    total = torch.matmul(X.abs(), W.abs().t().contiguous())
    n = K / 128 + 10
    bound = so.U[t] * want.abs() + so.TINY[t] + n * 2.0 ** -24 * (1 + so.U[t]) * total + n * 2.0 ** -150
    held = (total * (1 + n * 2.0 ** -23) < MOST["f32"]) & (want.abs() + bound < MOST[t])
    assert of_w == (0, 254) or t == "f16" or held.all()
    assert (((got - want).abs() <= bound) | ~held).all()
    assert not torch.isnan(got[held]).any()
