"""Edges of the serving operators: what NaN, infinite and very large values, rows
of no sequence and products that cancel must come to, against the 64-bit forms
and the bounds of serve_oracle.py."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve_oracle as so
from gpu_util import announce
from test_serve_gpu import DEV, DT, f8_dev, make_attn, np64, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


# ---- NaN logits ------------------------------------------------------------------
# Sizes that take every way through the kernels: the 16-row and the wide kernel,
# one part (written directly) and several (joined).
SHAPES = [
    # lens, new tokens, heads, dimensions, prefix, type
    ([97], [1], 2, 1, 64, 0, "f16"), ([70, 3], [1, 1], 4, 2, 128, 70, "bf16"),
    ([2700], [1], 2, 1, 64, 0, "f16"), ([41, 33], [3, 2], 4, 2, 256, 0, "bf16"),
    ([90], [70], 2, 2, 96, 0, "f16"), ([150, 64], [140, 64], 2, 1, 128, 0, "bf16"),
    ([100, 64], [90, 64], 2, 2, 64, 50, "bf16"), ([80], [60], 2, 1, 256, 50, "f16"),
    ([int(n) for n in range(35)], [1] * 35, 4, 1, 128, 130, "f16"),
]


class Batch:
    """One batch on the host, run through the library and the 64-bit form."""

    def __init__(self, lens, news, hq, hkv, d, prefix, t, what):
        announce(f"attn {what} lens={lens[:4]} new={news[:4]} h={hq}/{hkv} d={d} prefix={prefix} {t}")
        self.lens, self.news, self.prefix, self.t, self.d = lens, news, prefix, t, d
        (self.q, self.kc, self.vc, self.table, self.ln, self.pids,
         self.start) = make_attn(lens, news, hq, hkv, d, 16, prefix, t, sum(lens) + d)

    def want(self):
        return so.attention(np64(self.q), np64(self.kc), np64(self.vc), self.table, self.lens, self.pids,
                            self.prefix, self.start, self.d ** -0.5, self.t)

    def run(self, **kw):
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        if any(n != 1 for n in self.news):
            kw = dict(q_start=up(self.start), max_q=max(self.news)) | kw
        out, lse = bq.lqmm_attn_prefix(self.q.to(DEV), self.kc.to(DEV), self.vc.to(DEV), up(self.table),
                                       up(self.ln), prefix_pages=up(self.pids) if self.prefix else None,
                                       prefix_len=self.prefix, return_lse=True, **kw)
        return np64(out), np64(lse)

    def keys_of(self, b, j0, j1):
        """(page, place) of sequence b's keys j0 .. j1 - 1."""
        return [(self.table[b, j // 16], j % 16) for j in range(j0, min(j1, self.lens[b]))]

    def first_seen(self, b, j):
        """The first row of sequence b that sees its key j."""
        return self.start[b] + max(0, j - (self.lens[b] - self.news[b]))


def compare(out, lse, want, nan):
    """Rows in `nan` (tokens, or tokens x heads) are NaN, out and lse; the others
    within their bounds."""
    wo, wl, bo, bl = want
    nan = np.broadcast_to(nan if nan.ndim == 2 else nan[:, None], wl.shape)
    assert np.isnan(out[nan]).all() and np.isnan(lse[nan]).all()
    within(out[~nan], wo[~nan], bo[~nan], "out")
    empty = np.isneginf(wl) & ~nan
    assert np.array_equal(np.isneginf(lse), empty)
    some = ~nan & ~empty
    within(lse[some], wl[some], bl[some], "lse")


@pytest.mark.parametrize("case", SHAPES)
def test_a_nan_query_gives_nan(case):
    """A row whose every logit is NaN is not a row that sees no key, however its
    keys are split."""
    b = Batch(*case, "NaN queries")
    want = b.want()
    nan = np.zeros(b.q.shape[:2], dtype=bool)
    nan[-1, 0] = nan[len(nan) // 2, -1] = True
    b.q[torch.from_numpy(nan)] = float("nan")
    sees = np.isfinite(want[1])  # a row without keys has no logit
    compare(*b.run(), want, nan & sees)


@pytest.mark.parametrize("part", ["sequence", "a wave's keys", "prefix"])
@pytest.mark.parametrize("case", SHAPES)
def test_keys_that_are_all_nan_give_nan(case, part):
    """A part, or the keys that one wave takes, whose logits are all NaN."""
    b = Batch(*case, f"NaN keys: {part}")
    want = b.want()
    nan = np.zeros(len(b.q), dtype=bool)
    if part == "prefix":
        if not b.prefix:
            pytest.skip("no prefix")
        b.kc[b.pids.astype(np.int64)] = float("nan")
        nan[:] = True
    else:
        last = len(b.lens) - 1
        j0, j1 = (0, b.lens[last]) if part == "sequence" else (32, 64)
        if j0 >= b.lens[last]:
            j0, j1 = 0, 32
        for page, place in b.keys_of(last, j0, j1):
            b.kc[page, :, place] = float("nan")
        nan[b.first_seen(last, j0):b.start[last + 1]] = True
    compare(*b.run(), want, nan)


@pytest.mark.parametrize("case", [c for c in SHAPES if max(c[1]) > 1])
def test_a_nan_query_among_rows_done_again(case):
    """The rows of a mask's edge that are computed by themselves, because a value
    behind it is infinite, keep the NaN of their queries."""
    b = Batch(*case, "NaN query beside an infinite value")
    want = b.want()
    n, new = b.lens[0], b.news[0]
    page, place = b.keys_of(0, n - 1, n)[0]
    b.vc[page, :, place // 8, :, place % 8] = float("inf")
    seen = np.zeros(len(b.q), dtype=bool)
    seen[b.start[1] - 1] = True  # the only row that sees the infinite value
    nan = np.zeros(b.q.shape[:2], dtype=bool)
    nan[b.start[1] - 2, 0] = True
    b.q[torch.from_numpy(nan)] = float("nan")
    out, lse = b.run()
    keep = ~seen
    compare(out[keep], lse[keep], [w[keep] for w in want], nan[keep])


# ---- more new tokens than max_q --------------------------------------------------
@pytest.mark.parametrize("lens, news, max_q, hq, hkv, d, prefix, t", [
    ([50, 30], [9, 4], 5, 4, 2, 64, 0, "f16"), ([50, 30], [9, 4], 5, 4, 2, 256, 40, "bf16"),
    ([120, 60], [100, 50], 77, 2, 2, 96, 60, "f16"), ([120], [100], 60, 4, 1, 128, 0, "bf16"),
    ([5, 40], [9, 3], 6, 2, 1, 64, 0, "f16"),
])
def test_rows_below_max_q_keep_their_masks(lens, news, max_q, hq, hkv, d, prefix, t):
    """Leaving out a sequence's rows past max_q changes nothing of the others:
    token i of n still sees the keys 0 .. len - n + i."""
    b = Batch(lens, news, hq, hkv, d, prefix, t, f"max_q {max_q}")
    want = b.want()
    rows = np.concatenate([np.arange(s, s + min(n, max_q)) for s, n in zip(b.start, news)])
    out, lse = b.run(max_q=max_q)
    compare(out[rows], lse[rows], [w[rows] for w in want], np.zeros(len(rows), dtype=bool))


# ---- rows of no sequence ---------------------------------------------------------
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("lens, news, max_q, before, after, hq, hkv, d, prefix, t", [
    ([20, 9], [3, 2], 3, 0, 4, 2, 1, 64, 0, "f16"), ([20, 9], [3, 2], 3, 5, 4, 4, 2, 128, 40, "bf16"),
    ([50, 30], [9, 4], 5, 2, 0, 4, 2, 64, 0, "f16"), ([50, 30], [9, 4], 5, 2, 300, 4, 2, 256, 40, "bf16"),
    ([120, 60], [100, 50], 100, 3, 7, 2, 1, 128, 0, "f16"), ([120, 60], [100, 50], 77, 0, 40, 2, 2, 96, 60, "f16"),
    ([2700], [2], 2, 1, 5, 2, 1, 64, 0, "bf16"), ([120], [100], 60, 40, 3, 4, 1, 64, 0, "bf16"),
    ([0, 7], [0, 2], 2, 3, 3, 2, 1, 64, 30, "f16"),
])
def test_rows_of_no_sequence(lens, news, max_q, before, after, hq, hkv, d, prefix, t, given):
    """Rows of q before q_start[0], from q_start[batch] on and past max_q of a
    sequence's come out as rows without keys do, whatever the workspace and the
    output held; nothing around them is written."""
    b = Batch(lens, news, hq, hkv, d, prefix, t, "rows of no sequence")
    wo, wl, bo, bl = b.want()
    T = before + sum(news) + after
    q = torch.full((T, hq, d), 3.0, dtype=DT[t])
    q[before:before + sum(news)] = b.q
    of = np.full(T, -1)  # the row of b.q that a row is
    for s, n in zip(b.start, news):
        of[before + s:before + s + min(n, max_q)] = np.arange(s, s + min(n, max_q))
    b.q, b.start = q, b.start + np.int32(before)
    args = dict(max_q=max_q, q_start=torch.from_numpy(b.start).to(DEV))
    if given:
        whole = torch.full((T + 2, hq, d), 7.0, dtype=DT[t], device=DEV)
        lses = torch.full((T + 2, hq), 7.0, device=DEV)
        need = bq.lqmm_attn_prefix_workspace_bytes(prefix, b.table.shape[1], max_q, T, len(lens), hq, hkv, d, 16)
        ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)  # (NaN in fp32)
        args |= dict(out=whole[1:-1], lse=lses[1:-1], workspace=ws[:need])
    out, lse = b.run(**args)
    if given:
        assert (whole[[0, -1]] == 7).all() and (lses[[0, -1]] == 7).all() and (ws[need:] == 0xFF).all()
    live = of >= 0
    assert (out[~live] == 0).all() and np.isneginf(lse[~live]).all()
    compare(out[live], lse[live], [w[of[live]] for w in (wo, wl, bo, bl)], np.zeros(live.sum(), dtype=bool))


# ---- 8-bit float products: sums in 32 bits ---------------------------------------
@pytest.mark.parametrize("t", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["outlier", "cancel"])
@pytest.mark.parametrize("M, N, K", [
    (1, 130, 272), (16, 130, 400), (9, 12301, 272), (20, 300, 144), (32, 4000, 272), (45, 4127, 400),
    (64, 3000, 1040), (100, 1001, 272), (300, 3000, 400), (700, 8300, 272), (1500, 9000, 272),
    (2900, 9100, 400),
])
def test_f8_sums_keep_small_products(M, N, K, kind, t):
    """Products far below a block's largest count in full, for every output type
    and tile: behind one large product, and behind two that cancel. Bound of each
    output: half a step of the type, and for the fp32 sum of a block's 128 products
    and of the blocks, in any order, 2^-23 of the sum of absolute products for
    each addition and scaling."""
    r = np.random.default_rng(M + N)
    x, w = r.choice([1.75, 2.0], (M, K)), r.choice([3.5, 3.75], (N, K))
    for k in range(0, K, 128):
        at = k + r.permutation(min(128, K - k))[:2]
        x[:, at[0]], w[:, at[0]] = 448.0, 448.0
        if kind == "cancel":
            x[:, at[1]], w[:, at[1]] = 448.0, -448.0
    s = 2.0 ** -9  # (fp16 outputs stay in range)
    nb, kb = -(-N // 128), -(-K // 128)
    ws, xs = s * np.exp2(r.integers(0, 2, (nb, kb))), np.exp2(r.integers(0, 2, (kb, M)))
    announce(f"gemm_f8b128 {kind} {M}x{N}x{K} {t}")
    dev = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    X, W = dev(x), dev(w)
    f8 = torch.float8_e4m3fn
    got = bq.lqmm_gemm_f8b128(W.to(f8), dev(ws).float(), X.to(f8), dev(xs).float(), out_dtype=DT[t]).double()
    of = torch.arange(K, device=DEV) // 128
    X, W = X * dev(xs)[of].t(), W * dev(ws)[torch.arange(N, device=DEV) // 128][:, of]
    want = torch.matmul(X, W.t().contiguous())
    total = torch.matmul(X.abs(), W.abs().t().contiguous())
    sums = (128 + kb + 4) * 2.0 ** -23 * total
    bound = so.U[t] * torch.exp2(torch.floor(torch.log2(want.abs() + sums))) + sums
    over = (got - want).abs() - bound
    assert torch.isfinite(got).all() and float(over.max()) <= 0, float(over.max())


# ---- very large values -----------------------------------------------------------
@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("case", [c[:6] + ("bf16",) for c in SHAPES] + [([9000], [1], 1, 1, 64, 0, "bf16")])
def test_values_near_the_type_s_largest(case, again):
    """The mean of finite values is finite: bf16 values up to 3.3e38, with and
    without the rows of a mask's edge done by themselves."""
    b = Batch(*case, "large values")
    keep = ~np.isnan(np64(b.vc))
    r = np.random.default_rng(1)
    big = r.uniform(1e38, 3.3e38, b.vc.shape) * r.choice([-1.0, 1.0, 1.0, 1.0], b.vc.shape[-2])[:, None]
    b.vc = torch.from_numpy(np.where(keep, big, np.nan)).to(DT["bf16"])
    want = b.want()
    rows = np.ones(len(b.q), dtype=bool)
    if again:
        if b.news[0] < 2:
            pytest.skip("one new token")
        page, place = b.keys_of(0, b.lens[0] - 1, b.lens[0])[0]
        b.vc[page, :, place // 8, :, place % 8] = float("inf")
        rows[b.start[1] - 1] = False  # sees the infinite value
    out, lse = b.run()
    compare(out[rows], lse[rows], [w[rows] for w in want], np.zeros(rows.sum(), dtype=bool))


# ---- more workgroups than one launch takes ---------------------------------------
# (a launch counts its threads in 32 bits)
@pytest.mark.parametrize("M, N", [(1, 2 ** 27 + 37), (2 ** 28 + 35, 1)])
def test_f8_product_of_very_many_rows(M, N):
    announce(f"gemm_f8b128 {M}x{N}x16")
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    code = lambda n: torch.randint(0x30, 0x40, (n, 16), device=DEV, generator=g, dtype=torch.uint8)  # noqa: E731
    w, x = code(N), code(M)
    ws, xs = torch.ones(-(-N // 128), 1, device=DEV), torch.ones(1, M, device=DEV)
    y = bq.lqmm_gemm_f8b128(w, ws, x, xs, out_dtype=torch.float32).view(-1)
    big, one = (w, x) if N > M else (x, w)
    f8 = torch.float8_e4m3fn
    for i in range(0, max(M, N), 2 ** 24):  # sums of products of 4 bits each: exact
        want = (big[i:i + 2 ** 24].view(f8).float() * one.view(f8).float()).sum(1)
        assert torch.equal(y[i:i + 2 ** 24], want)


def test_quant_of_very_many_rows():
    M = 2 ** 28 + 19
    announce(f"quant {M}x16")
    x = torch.empty(M, 16, dtype=torch.float16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    for i in range(0, M, 2 ** 24):
        x[i:i + 2 ** 24] = torch.randint(-7, 8, x[i:i + 2 ** 24].shape, device=DEV, generator=g, dtype=torch.int8)
    x[:, 3] = 7.0  # the scale is 2^-6, and codes are exact
    codes, scales = bq.lqmm_quant_f8b128(x)
    assert (scales == 2.0 ** -6).all()
    for i in range(0, M, 2 ** 24):
        assert torch.equal(codes[i:i + 2 ** 24].float(), x[i:i + 2 ** 24].float() * 64)


def test_append_of_very_many_tokens():
    T, ps = 2 ** 24 + 11, 1024
    P = -(-T // ps)
    announce(f"append {T} tokens")
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    k = torch.randint(-99, 100, (T, 1, 64), device=DEV, generator=g, dtype=torch.int16).half()
    v = torch.randint(-99, 100, (T, 1, 64), device=DEV, generator=g, dtype=torch.int16).half()
    kc, vc = (c.zero_() for c in bq.kv_cache_empty(P, 1, ps, 64))
    bq.lqmm_kv_append(None, k, v, None, torch.arange(T, device=DEV), kc, vc)
    assert torch.equal(kc.view(-1, 64)[:T], k.view(T, 64)) and not kc.view(-1, 64)[T:].any()
    got = vc.view(-1, 64, 8).transpose(1, 2).reshape(-1, 64)
    assert torch.equal(got[:T], v.view(T, 64)) and not got[T:].any()


def test_attention_of_very_many_sequences():
    B, H = 2 ** 20 + 3, 16
    announce(f"attn {B} sequences of one key, {H} heads")
    kc, vc = bq.kv_cache_empty(3, H, 8, 64)
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    for c in (kc, vc):
        c.copy_(torch.randn(c.shape, device=DEV, generator=g))
    pages = torch.randint(0, 3, (B, 1), device=DEV, generator=g, dtype=torch.int32)
    lens = torch.ones(B, dtype=torch.int32, device=DEV)
    q = torch.ones(B, H, 64, dtype=torch.float16, device=DEV)
    out = bq.lqmm_attn_prefix(q, kc, vc, pages, lens)
    values = vc[:, :, 0, :, 0]  # one key: its value
    for i in range(0, B, 2 ** 17):
        assert torch.equal(out[i:i + 2 ** 17], values[pages[i:i + 2 ** 17, 0].long()])


# ---- activations to e4m3: very small groups --------------------------------------
@pytest.mark.parametrize("lo, hi", [(-149, -120), (-126, -110), (-112, -90), (-90, -60), (-66, -55), (100, 127)])
def test_quant_rounds_small_and_large_groups_correctly(lo, hi):
    """Codes are those of the correctly rounded quotient, ties and their
    neighbours included, whatever the group's exponent."""
    r = np.random.default_rng(hi - lo)
    x = np.ldexp(r.standard_normal((4096, 1024)), r.integers(lo, hi, (4096, 8)).repeat(128, 1))
    x = np.clip(x, -3e38, 3e38).astype(np.float32)
    v = np.sort(np.unique(np.abs(so.E4M3[np.isfinite(so.E4M3)])))
    mid = ((v[:-1] + v[1:]) / 2).astype(np.float32)
    for m in range(0, 4096, 2):
        top = np.float32(np.ldexp(1 + r.random(), int(r.integers(lo, hi))))
        s = max(np.float32(top / np.float32(448.0)), np.float32(2.0 ** -126))
        t = r.choice(mid, 127) * s
        up = np.nextafter(t, np.float32(np.inf))
        t = np.choose(r.integers(0, 3, 127), (t, up, np.nextafter(t, np.float32(-np.inf))))
        x[m, :127], x[m, 127] = np.clip(t, -top, top), top
    announce(f"quant of groups of 2^{lo} .. 2^{hi}")
    codes, scales = bq.lqmm_quant_f8b128(torch.from_numpy(x).to(DEV))
    want, ws = so.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(np64(codes), want)


# ---- lse --------------------------------------------------------------------------
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -24, 0.01])
@pytest.mark.parametrize("case", [c[:6] for c in SHAPES])
def test_lse_of_nearly_equal_logits(case, scale, t):
    """lse has fp32's accuracy at its own size, whatever weights and parts are
    scaled by: 2^-20 and 2^-22 of it beside the logits' error."""
    b = Batch(*case, t, f"lse at scale {scale}")
    want = so.attention(np64(b.q), np64(b.kc), np64(b.vc), b.table, b.lens, b.pids, b.prefix, b.start, scale, t)
    out, lse = b.run(scale=scale)
    compare(out, lse, want, np.zeros(len(b.q), dtype=bool))
