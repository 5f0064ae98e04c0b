"""Attention over the 8-bit cache with scales as far apart as its bytes let them
be, against 64 bits inside the bounds of serve8_oracle.py."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve_oracle as so
from test_serve8_gpu import Batch, compare
from test_serve8_wide_gpu import BEHIND, LONG, SHORT, Wide

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
LN2 = float(np.log(2.0))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


def code_of(v):
    return np.abs(np.nan_to_num(so.E4M3, nan=1e9) - v).argmin().astype(np.uint8)


def set_logits(b, z):
    """Logits (base 2, of scale ln 2) of every used key: its first dimension, with
    a query that is 1 there and 0 elsewhere. z: [P][H][ps], exact in e4m3."""
    used = b.cache[3] != 255
    b.q.zero_()
    b.q[..., 0] = 1.0
    b.cache[2][used] = 127
    codes = {v: code_of(v) for v in np.unique(z[used])}
    for p, h, o in np.argwhere(used):
        b.cache[0][p, h, o, 0] = codes[z[p, h, o]]


def slot_of(b, seq, j):
    """Page and place of a sequence's key, or of the prefix's (seq None)."""
    ids = b.pids if seq is None else b.table[seq]
    return ids[j // b.ps], j % b.ps


FAR = [
    # lens, new tokens, heads, dimensions, prefix, keys at the largest scale
    ([30], [1], 2, 1, 64, 0, [(0, 3)]),               # one wave
    ([200, 97], [1, 1], 4, 2, 128, 0, [(0, 150), (1, 0)]),  # several waves
    ([130], [1], 2, 1, 96, 0, [(0, 129)]),
    ([61], [3], 4, 2, 256, 0, [(0, 20)]),
    ([2700], [1], 2, 1, 128, 0, [(0, 2000)]),         # several parts
    ([9001], [1], 8, 8, 64, 0, [(0, 17)]),
    ([40, 300], [1, 1], 4, 1, 128, 1500, [(1, 5)]),   # a prefix beside it
    ([40, 300], [1, 1], 4, 1, 64, 1500, [(None, 1400)]),
    ([150, 64], [140, 64], 2, 1, 128, 0, [(0, 30)]),  # many rows
    ([100], [90], 2, 2, 64, 50, [(None, 7)]),
]


@pytest.mark.parametrize("case", FAR)
def test_a_key_at_the_largest_scale_beside_keys_at_the_least(case):
    """V's scales 2^120 apart: keys that vanish beside the large one in the
    numerator still count in the sum of the weights."""
    lens, news, hq, hkv, d, prefix, far = case
    b = Batch(lens, news, hq, hkv, d, 16, prefix, "bf16", seed=sum(lens) + d)
    r = np.random.default_rng(d)
    vs = b.cache[3]
    used = vs != 255
    z = -2.0 * r.integers(3, 7, vs.shape)  # -6 .. -12
    vs[used] = 67
    for seq, j in far:
        p, o = slot_of(b, seq, j)
        vs[p, :, o], z[p, :, o] = 187, 0.0
    set_logits(b, z)
    compare(*b.run(scale=LN2), b.want(LN2))


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("byte", [1, 11, 25, 66])
@pytest.mark.parametrize("lens, news, hq, hkv, d", [([97], [1], 4, 2, 64), ([3000], [1], 2, 1, 128), ([80], [60], 2, 1, 128)])
def test_least_scales_leave_the_sums_whole(t, byte, lens, news, hq, hkv, d):
    """Values as small as scale bytes can say. Beside the oracle's bound: bf16
    drops terms below its least normal number, 2^-126 of a code of at most 448
    for each key, of a sum of weights of at least 1."""
    b = Batch(lens, news, hq, hkv, d, 16, 0, t, seed=byte)
    b.cache[3][b.cache[3] != 255] = byte
    wo, wl, bo, bl = b.want()
    compare(*b.run(), (wo, wl, bo + max(lens) * 448 * 2.0 ** -126, bl))


HIDDEN = [([90], [70], 2, 2, 96, 0), ([80], [60], 2, 1, 256, 50), ([150], [140], 2, 1, 128, 0),
          ([400, 390], [200, 390], 2, 1, 128, 200), ([300], [300], 2, 1, 64, 40), ([41, 33], [3, 2], 4, 2, 64, 0)]
HIDDEN += [(*c[:4], d, c[4]) for c, d in ((SHORT, 64), (SHORT, 96), (SHORT, 256), (LONG, 64), (LONG, 128), (BEHIND, 128))]


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("byte", [0, 135, 200, 253, 254, 255])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("case", HIDDEN)
def test_a_scale_past_the_type_stays_behind_the_mask(case, what, byte, t):
    """The last new token has a scale past fp16's values, or a byte that stands for
    nothing: the rows before it, whose mask leaves it out, are as without it."""
    lens, news, hq, hkv, d, prefix = case
    b = Wide(lens, news, hq, hkv, d, 16, prefix, t, seed=sum(lens))
    want = b.want()
    last = len(lens) - 1
    p, o = slot_of(b, last, lens[last] - 1)
    b.cache[2 if what == "k" else 3][p, :, o] = byte
    out, lse = b.run()
    rows = np.arange(sum(news)) != b.start[last + 1] - 1
    compare(out[rows], lse[rows], [w[rows] for w in want])


@pytest.mark.parametrize("case", HIDDEN + [([97, 5], [1, 1], 4, 2, 128, 0), ([300], [1], 2, 1, 64, 40)])
@pytest.mark.parametrize("byte", [135, 140, 187, 253])
def test_fp16_takes_larger_scales_as_its_largest(case, byte):
    """A bf16 call's cache under fp16 queries: scales past 2^7 count as 2^7."""
    lens, news, hq, hkv, d, prefix = case
    b = Wide(lens, news, hq, hkv, d, 16, prefix, "f16", seed=sum(lens) + 1)
    b.q *= 2.0 ** -14  # (logits stay ordinary)
    r = np.random.default_rng(byte)
    for c in b.cache[2:]:
        c[(c != 255) & (r.random(c.shape) < 0.2)] = byte
    got = b.run()
    for c in b.cache[2:]:
        c[(c > 134) & (c != 255)] = 134
    compare(*got, b.want())


def test_attention_repeats_itself():
    """Sums have one order: the same call again gives the same bits."""
    for case in (([3000, 40], [1, 1], 8, 2, 128, 700, "f16"), ([150, 64], [140, 64], 2, 1, 128, 30, "bf16")):
        lens, news, hq, hkv, d, prefix, t = case
        b = Batch(lens, news, hq, hkv, d, 16, prefix, t)
        first = b.run()
        for _ in range(3):
            assert all(np.array_equal(x, y) for x, y in zip(b.run(), first))
