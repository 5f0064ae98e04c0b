"""Attention over the 8-bit cache with many rows: calls large enough that the
kernels for 128 and 256 rows a workgroup take them (16 rows are the estimate's
choice below some 3e7 keys x heads x rows, or 1e6 for many short sequences),
against 64 bits inside the bounds of serve8_oracle.py."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve8_dense
from test_serve8_gpu import Batch, compare, up, values
from test_serve_gpu import DEV, DT, np64, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


class Wide(Batch):
    def want(self, scale=None):
        kc, vc, ks, vs = self.cache
        return serve8_dense.attention(np64(self.q), (values(kc), values(vc), ks, vs), self.table, self.lens, self.pids,
                                      self.prefix, self.start, self.d ** -0.5 if scale is None else scale, self.t, DEV)


LENS = [90, 5, 0, 64] + [17 + 29 * i % 70 for i in range(28)]
NEWS = [32, 5, 0, 32] + [min(n, 1 + 13 * i % 32) for i, n in enumerate(LENS[4:])]
SHORT = (LENS, NEWS, 32, 8, 0)                        # 128 rows
LONG = ([3000, 900], [600, 300], 16, 2, 0)            # 256 rows; 128 with 96 and 256 dimensions
BEHIND = ([60 - i for i in range(30)], [30 - i // 3 for i in range(30)], 64, 8, 1500)  # the prefix 256 or 128, the others 128
CASES = [(*c[:4], d, c[4], t) for c in (SHORT, LONG, BEHIND) for d in (64, 96, 128, 256) for t in ("f16", "bf16")]
SOME = [(*SHORT[:4], 64, 0, "f16"), (*SHORT[:4], 128, 0, "bf16"), (*SHORT[:4], 256, 0, "f16"), (*LONG[:4], 64, 0, "f16"),
        (*LONG[:4], 128, 0, "f16"), (*LONG[:4], 128, 0, "bf16"), (*LONG[:4], 96, 0, "bf16"), (*BEHIND[:4], 64, 1500, "bf16")]


def batch(case, seed=0, **kw):
    lens, news, hq, hkv, d, prefix, t = case
    return Wide(lens, news, hq, hkv, d, 16, prefix, t, seed=seed + d, **kw)


@pytest.mark.parametrize("case", CASES + [([16000], [256], 128, 16, 96, 0, "bf16")])
def test_many_rows(case):
    b = batch(case)
    compare(*b.run(), b.want())


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("case", SOME[:6])
def test_many_rows_scale(case, scale):
    b = batch(case, 1)
    compare(*b.run(scale=scale), b.want(scale))


@pytest.mark.parametrize("case", SOME)
def test_many_rows_scales_far_apart(case):
    b = batch(case, 2)
    ks, vs = b.cache[2:]
    ks[ks != 255] = 120
    keep = vs != 255
    vs[keep] = np.random.default_rng(1).choice([67, 100, 127, 187 if b.t == "bf16" else 134], keep.sum())
    compare(*b.run(), b.want())


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("case", SOME)
def test_many_rows_behind_a_nan_code(case, what):
    """A NaN in the last new token reaches that token's rows and no others."""
    b = batch(case, 3)
    want = b.want()
    last = len(b.lens) - 1
    j = b.lens[last] - 1
    page, place = b.table[last, j // 16], j % 16
    if what == "k":
        b.cache[0][page, :, place, 3] = 0x7f
    else:
        b.cache[1][page, :, place // 8, :, place % 8] = 0xff
    nan = np.zeros(len(b.q), dtype=bool)
    nan[b.start[last + 1] - 1] = True
    out, lse = b.run()
    assert np.isnan(out[nan]).all()
    compare(out[~nan], lse[~nan], [w[~nan] for w in want])
    if what == "v":  # lse knows nothing of the values
        within(lse[nan], want[1][nan], want[3][nan], "lse")
    else:
        assert np.isnan(lse[nan]).all()


@pytest.mark.parametrize("case", SOME[:6])
def test_many_rows_with_a_nan_query(case):
    b = batch(case, 4)
    want = b.want()
    nan = np.zeros(b.q.shape[:2], dtype=bool)
    nan[-1, 0] = nan[len(nan) // 2, -1] = True
    b.q[torch.from_numpy(nan)] = float("nan")
    compare(*b.run(), want, nan & np.isfinite(want[1]))


@pytest.mark.parametrize("case", [SOME[0], SOME[1], SOME[4], SOME[7]])
def test_many_rows_and_rows_of_no_sequence(case):
    b = batch(case, 5)
    want = b.want()
    before, after, max_q = 3, 40, max(b.news) - 5
    T = before + sum(b.news) + after
    q = torch.full((T, *b.q.shape[1:]), 3.0, dtype=DT[b.t])
    q[before:before + len(b.q)] = b.q
    of = np.full(T, -1)
    for s, n in zip(b.start, b.news):
        of[before + s:before + s + min(n, max_q)] = np.arange(s, s + min(n, max_q))
    b.q, b.start = q, b.start + np.int32(before)
    out, lse = b.run(max_q=max_q, q_start=up(b.start))
    live = of >= 0
    assert (out[~live] == 0).all() and np.isneginf(lse[~live]).all()
    compare(out[live], lse[live], [w[of[live]] for w in want])


@pytest.mark.parametrize("case", [SOME[0], SOME[3], SOME[5]])
def test_many_rows_in_a_captured_graph(case):
    b = batch(case, 6)
    a, kw = b.args()
    eager = [t.clone() for t in bq.lqmm_attn_prefix_f8(*a, **kw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        got = bq.lqmm_attn_prefix_f8(*a, **kw)
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        other = bq.lqmm_attn_prefix_f8(*a, **kw)  # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) and torch.equal(z, y) for x, z, y in zip(got, other, eager))
