"""serve8_dense.attention against serve8_oracle.attention, row by row."""
import numpy as np
import pytest

import serve8_dense
import serve8_oracle as s8
import serve_oracle as so


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("lens, news, prefix", [([1], [1], 0), ([20, 0, 9], [3, 1, 9], 0), ([5, 33], [2, 30], 13), ([0, 4], [0, 1], 7),
                                                ([2], [5], 0), ([0], [2], 3)])
def test_the_same_as_row_by_row(lens, news, prefix, t):
    r = np.random.default_rng(sum(lens))
    P, hkv, hq, ps, d = 9, 2, 6, 8, 16
    code = lambda s: so.E4M3[np.where((c := r.integers(0, 256, s)) & 0x7f == 0x7f, 3, c)]  # noqa: E731
    cache = [code((P, hkv, ps, d)), code((P, hkv, ps // 8, d, 8)),
             *(r.integers(110, 130, (P, hkv, ps)).astype(np.uint8) for _ in range(2))]
    pages = r.integers(-1, P + 1, (len(lens), 6))
    start = np.concatenate(([0], np.cumsum(news)))
    q = r.standard_normal((int(start[-1]) + 1, hq, d))
    args = (q, cache, pages, lens, r.integers(0, P, 3), prefix, start, -0.3, t)
    for got, want in zip(serve8_dense.attention(*args), s8.attention(*args)):
        assert np.allclose(got, want, rtol=1e-10, atol=1e-300)
