"""The serving operators in fewer bits on the GPU against their 64-bit forms,
inside the bounds of serve8_oracle.py."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve8_oracle as s8
import serve_oracle as so
from gpu_util import announce
from test_serve_gpu import DEV, DT, np64, rnd, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def values(codes):
    """Code values in 64 bits of a tensor or array of e4m3 bytes."""
    if isinstance(codes, torch.Tensor):
        codes = codes.view(torch.uint8).cpu().numpy()
    return so.E4M3[codes]


def random_cache(r, P, hkv, ps, d, spread=3):
    """Host codes (no NaN) and scale bytes."""
    code = lambda s: np.where((c := r.integers(0, 256, s)) & 0x7f == 0x7f, 0x30, c).astype(np.uint8)  # noqa: E731
    scale = lambda: (127 - 7 + r.integers(-spread, spread + 1, (P, hkv, ps))).astype(np.uint8)  # noqa: E731
    return code((P, hkv, ps, d)), code((P, hkv, ps // 8, d, 8)), scale(), scale()


# ---- append ----------------------------------------------------------------------
def run_append(T, hq, hkv, d, ps, P, rot, inter, tin, t, slots, seed, normed="qk", bits=8, far=100000,
               eps=1e-6, x=None, stream=None):
    r = np.random.default_rng(seed)
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot) if rot else np.zeros(0)
    qkv = rnd(r, (T, hq + 2 * hkv, d), tin) * 3 if x is None else x
    pos = r.integers(0, far, T).astype(np.int32)
    wq, wk = ((1 + 0.3 * r.standard_normal(d)).astype(np.float32) if n in normed else None for n in "qk")
    announce(f"append_norm T={T} hq={hq} hkv={hkv} d={d} ps={ps} rot={rot} inter={inter} {tin}->{t} {bits} {normed}")
    g = qkv.to(DEV)
    if bits == 8:
        kc, vc, ks, vs = random_cache(r, P, hkv, ps, d)
        dev = [up(a) for a in (kc, vc, ks, vs)]
    else:
        kc, vc = rnd(r, (P, hkv, ps, d), t), rnd(r, (P, hkv, ps // 8, d, 8), t)
        dev = [kc.to(DEV), vc.to(DEV), None, None]
    wide = torch.full((T + 2, hq, d), 7.0, dtype=DT[t], device=DEV)
    weights = [up(w) if w is not None else None for w in (wq if hq else None, wk)]
    args = (g[:, :hq] if hq else None, g[:, hq:hq + hkv], g[:, hq + hkv:], up(pos), up(slots), *dev)
    kw = dict(q_norm=weights[0], k_norm=weights[1], eps=eps, rope_turns=bq.lqmm_rope_turns(inv) if rot else None,
              interleaved=inter, q_out=wide[1:-1] if hq else None)
    torch.cuda.synchronize()
    qo = bq.lqmm_kv_append_norm(*args, **kw, stream=stream)
    torch.cuda.synchronize()
    a = np64(qkv)
    q, qe = s8.norm_rotate(a[:, :hq], wq, eps, pos, inv, inter)
    k, ke = s8.norm_rotate(a[:, hq:hq + hkv], wk, eps, pos, inv, inter)
    v = a[:, hq + hkv:]
    if hq:
        within(qo, q, so.U[t] * np.abs(q) + so.TINY[t] + (1 + so.U[t]) * qe, "q")
        assert (wide[[0, -1]] == 7).all()
    else:
        assert qo is None
    if bits == 16:
        wk_, wv_, bk, bv = np64(kc), np64(vc), np.zeros(kc.shape), np.zeros(vc.shape)
        so.place(wk_, wv_, k, v, slots)
        so.place(bk, bv, so.U[t] * np.abs(k) + so.TINY[t] + (1 + so.U[t]) * ke,
                 so.U[t] * np.abs(v) + so.TINY[t], slots)
        within(dev[0], wk_, bk, "k_cache")
        within(dev[1], wv_, bv, "v_cache")
        return
    # exponents: those of the value, or of a neighbour of it within its error
    got = [x.cpu().numpy() for x in dev]
    (kv, kx), (vv, vx) = s8.quant(k, t), s8.quant(v, t)
    lo, hi = s8.exponent(np.abs(k).max(-1) * (1 - 2e-6), t), s8.exponent(np.abs(k).max(-1) * (1 + 2e-6), t)
    for tok, s in enumerate(slots):
        if 0 <= s < P * ps:
            e = got[2][s // ps, :, s % ps].astype(int) - 127
            assert ((e >= lo[tok]) & (e <= hi[tok])).all(), (tok, e, kx[tok])
            kx[tok] = e
    # what no token's slot names is as before, bit for bit; V is exact
    want = [values(kc), values(vc), ks.copy(), vs.copy()]
    s8.place(*want, kv, vv, kx + 127, vx + 127, slots)
    assert np.array_equal(got[2], want[2]) and np.array_equal(got[3], want[3])
    assert np.array_equal(values(got[1]), want[1], equal_nan=True)
    bound, zero, one = np.zeros(kc.shape), np.zeros(vc.shape), np.ones((P, hkv, ps))
    s8.place(bound, zero, one, one.copy(), s8.held_bound(k, ke, kx, t), v, kx, vx, slots)
    exact = values(kc)
    s8.place(exact, zero, one, one.copy(), k, v, kx, vx, slots)
    scale = np.ones((P, hkv, ps))
    s8.place(np.zeros(kc.shape), zero, scale, one, k, v, np.exp2(kx.astype(float)), vx, slots)
    within(values(got[0]) * scale[..., None], exact, bound, "k_cache")


def scattered(T, ps, seed):
    P = max(2, 90 // ps + 1)
    slots = np.random.default_rng(seed).permutation(P * ps)[:T].astype(np.int64)
    slots[2::7] = -1
    slots[4::11] = P * ps + 3
    slots[5::13] = 1 << 40
    return P, slots


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("T, hq, hkv, d, ps, rot, inter, tin, t, normed", [
    (1, 4, 1, 128, 16, 128, False, "f16", "f16", "qk"), (1, 1, 1, 64, 8, 16, True, "f32", "bf16", "qk"),
    (5, 6, 2, 96, 8, 96, False, "bf16", "bf16", "k"), (9, 7, 7, 64, 32, 32, True, "f16", "f16", "q"),
    (33, 40, 8, 128, 1024, 64, True, "f32", "f16", ""), (17, 8, 1, 256, 64, 256, False, "f32", "bf16", "qk"),
    (8, 0, 3, 128, 16, 128, False, "bf16", "f16", "k"), (40, 2, 2, 256, 16, 0, False, "f16", "bf16", "qk"),
    (23, 3, 5, 96, 16, 48, True, "f16", "f16", "qk"), (11, 64, 64, 64, 16, 64, False, "f16", "f16", "qk"),
])
def test_append_scattered(T, hq, hkv, d, ps, rot, inter, tin, t, normed, bits):
    P, slots = scattered(T, ps, T + d)
    run_append(T, hq, hkv, d, ps, P, rot, inter, tin, t, slots, 3 * T + d, normed, bits)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("first", [0, 1, 5, 7, 8])
@pytest.mark.parametrize("T, d", [(7, 64), (8, 128), (9, 96), (23, 256), (64, 128)])
def test_append_runs(first, T, d, bits):
    """Consecutive tokens from any place in a page: whole groups and their ends."""
    ps, P = 16, 8
    tok = np.arange(T) + first
    order = np.random.default_rng(first).permutation(P)
    slots = (order[tok // ps] * ps + tok % ps).astype(np.int64)
    run_append(T, 3, 5, d, ps, P, 64, False, "f16", "f16", slots, 100 * first + T, bits=bits)


@pytest.mark.parametrize("bits", [8, 16])
def test_append_broken_runs(bits):
    slots = np.arange(40, dtype=np.int64)
    slots[3], slots[12], slots[13] = 63, 13, 12
    slots[20] = -1
    slots[32:40] = np.arange(72, 80)
    run_append(40, 2, 1, 128, 16, 5, 128, False, "bf16", "bf16", slots, 9, bits=bits)


def test_append_far_positions():
    run_append(16, 4, 1, 128, 16, 2, 128, False, "f32", "f16", np.arange(16, dtype=np.int64), 5,
               far=2 ** 31 - 1)


def test_append_on_another_stream():
    run_append(19, 4, 2, 64, 16, 2, 64, False, "f16", "f16", np.arange(19, dtype=np.int64), 6,
               stream=torch.cuda.Stream())


@pytest.mark.parametrize("tin, lo, hi", [("f32", -149, -100), ("f32", -75, -50), ("f32", -20, 4), ("f32", 50, 90),
                                         ("f32", 90, 127), ("bf16", -126, -110), ("bf16", 90, 127), ("f16", -24, 15)])
@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("normed", ["", "qk"])
def test_append_small_and_large_vectors(tin, lo, hi, t, normed):
    """Vectors of any size, whole ones of zeros among them: the norm is that of the
    value, and the scale is bounded."""
    r = np.random.default_rng(hi - lo)
    x = np.ldexp(r.standard_normal((24, 6, 64)), r.integers(lo, hi, (24, 6, 1)))
    lim = {"f32": 3e38, "bf16": 3e38, "f16": 6e4}[tin]
    x = torch.from_numpy(np.clip(x, -lim, lim).astype(np.float32)).to(DT[tin])
    x[5] = 0.0
    if t == "f16" and not normed:
        x[:, :2] = x[:, :2].float().clamp(-3e4, 3e4).to(DT[tin])  # q goes to fp16
    run_append(24, 2, 2, 64, 16, 3, 0, False, tin, t, np.arange(24, dtype=np.int64), 7, normed, x=x,
               eps=1e-6 if hi > -50 else 0.0 if normed == "" else 1e-30)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_append_infinities_and_nan(d):
    """Without a norm an infinity or NaN is held as NaN, and the vector's other
    values as without it; a token's odd values reach no other vector."""
    r = np.random.default_rng(d)
    x = rnd(r, (16, 3, d), "f32")
    clean = x.clone()
    x[3, 1, d // 2], x[7, 2, 5], x[9, 1, 0], x[9, 2, d - 1] = float("inf"), float("-inf"), float("nan"), float("nan")
    out = []
    for a in (x, clean):
        kc, vc = (c.view(torch.uint8).zero_() for c in bq.kv_cache_empty(1, 1, 16, d, dtype=F8))
        ks, vs = bq.kv_scales_empty(1, 1, 16)
        g = a.to(DEV)
        announce(f"append_norm infinities d={d}")
        bq.lqmm_kv_append_norm(None, g[:, 1:2], g[:, 2:3], None, torch.arange(16, device=DEV), kc, vc, ks, vs)
        out.append([values(kc), values(vc), ks.view(torch.uint8).cpu().numpy(), vs.view(torch.uint8).cpu().numpy()])
    for i, name in ((1, 0), (2, 1)):
        v, e = s8.quant(np64(x[:, i]), "f16")
        got = out[0][name][0, 0] if name == 0 else out[0][name][0, 0].transpose(0, 2, 1).reshape(16, d)
        assert np.array_equal(got, v, equal_nan=True) and np.array_equal(out[0][2 + name][0, 0], e + 127)
        assert np.isnan(got).sum() == 2


def test_append_refuses():
    kc, vc = bq.kv_cache_empty(2, 1, 16, 64, dtype=F8)
    ks, vs = bq.kv_scales_empty(2, 1, 16)
    x = torch.zeros(3, 1, 64, dtype=torch.float16, device=DEV)
    slots = torch.arange(3, device=DEV)
    call = lambda **kw: bq.lqmm_kv_append_norm(  # noqa: E731
        kw.pop("q", None), x, x, None, slots, kw.pop("kc", kc), kw.pop("vc", vc), **(dict(k_scales=ks, v_scales=vs) | kw))
    with pytest.raises(TypeError):
        call(k_scales=None)
    with pytest.raises(TypeError):
        call(v_scales=vs.float())
    with pytest.raises(ValueError):
        call(k_scales=ks[:1])
    with pytest.raises(ValueError):
        call(k_norm=torch.ones(32, device=DEV))
    with pytest.raises(TypeError):
        call(k_norm=torch.ones(64, device=DEV).half())
    with pytest.raises(ValueError):
        call(q_norm=torch.ones(64, device=DEV))  # without q
    with pytest.raises(bq.LqmmError):
        call(eps=-1.0)
    with pytest.raises(TypeError):
        call(q=x, q_out=torch.empty(3, 1, 64, device=DEV))
    k16, v16 = bq.kv_cache_empty(2, 1, 16, 64)
    with pytest.raises(ValueError):
        call(kc=k16, vc=v16)  # scales beside 16-bit caches
    with pytest.raises(TypeError):
        call(vc=v16)


# ---- reading back ------------------------------------------------------------------
@pytest.mark.parametrize("hkv, d, ps, t", [(1, 64, 8, "f16"), (3, 96, 16, "bf16"), (8, 128, 64, "f32"),
                                           (5, 256, 16, "f16"), (9, 64, 128, "f32"), (7, 96, 8, "f32")])
@pytest.mark.parametrize("lens, before, after", [([1], 0, 0), ([7, 8, 9, 0, 17], 0, 0), ([0], 3, 2), ([40, 3], 5, 11),
                                                 ([1] * 70, 0, 1), ([0, 0, 130, 0], 1, 0), (list(range(130)), 2, 3)])
def test_read(hkv, d, ps, t, lens, before, after):
    r = np.random.default_rng(sum(lens) + d)
    n_pages = [-(-n // ps) for n in lens]
    P = sum(n_pages) + 3
    kc, vc, ks, vs = random_cache(r, P, hkv, ps, d, 30 if t == "f32" else 6)
    mp = max(1, max(n_pages))
    ids = r.permutation(P)
    table = r.choice(np.array([-1, 1 << 30, P]), (len(lens), mp)).astype(np.int32)
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = ids[at:at + n]
        at += n
    starts = (before + np.concatenate(([0], np.cumsum(lens)))).astype(np.int32)
    T = int(starts[-1]) + after
    if T == 0:
        pytest.skip("no rows")
    announce(f"read lens={lens[:5]} hkv={hkv} d={d} ps={ps} {t}")
    whole = [torch.full((T + 2, hkv, d), 7.0, dtype=DT[t], device=DEV) for _ in range(2)]
    k, v = bq.lqmm_kv_read_f8(up(kc), up(vc), up(ks), up(vs), up(table), up(starts), T, dtype=DT[t],
                              k_out=whole[0][1:-1], v_out=whole[1][1:-1])
    wk, wv = np.zeros((T, hkv, d)), np.zeros((T, hkv, d))
    for b, n in enumerate(lens):
        a, c, _ = s8.tokens_of(values(kc), values(vc), ks, vs, table[b], n)
        wk[starts[b]:starts[b] + n], wv[starts[b]:starts[b] + n] = a.transpose(1, 0, 2), c.transpose(1, 0, 2)
    if t != "f32":
        wk, wv = s8.to_type(wk, t), s8.to_type(wv, t)
    assert np.array_equal(np64(k), wk) and np.array_equal(np64(v), wv)
    assert all((w[[0, -1]] == 7).all() for w in whole)
    if before == 0 and lens == [7, 8, 9, 0, 17]:  # its own outputs, another stream
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        k2, v2 = bq.lqmm_kv_read_f8(up(kc), up(vc), up(ks), up(vs), up(table), up(starts), T, dtype=DT[t],
                                    k_out=torch.empty_like(k), v_out=torch.empty_like(v), stream=s)
        s.synchronize()
        assert torch.equal(k2, k) and torch.equal(v2, v)


def test_read_page_numbers_and_starts_out_of_bounds():
    """Page numbers outside the cache read page 0, tokens past the page table are
    zeros, starts outside the rows are cut off."""
    r = np.random.default_rng(3)
    kc, vc, ks, vs = random_cache(r, 2, 2, 8, 64)
    table = np.array([[5, -3]], dtype=np.int32)
    announce("read out of bounds")
    k, v = bq.lqmm_kv_read_f8(up(kc), up(vc), up(ks), up(vs), up(table), up(np.array([0, 20], np.int32)), 20,
                              dtype=torch.float32)
    a, c, _ = s8.tokens_of(values(kc), values(vc), ks, vs, [0, 0], 16)
    assert np.array_equal(np64(k)[:16], a.transpose(1, 0, 2)) and np.array_equal(np64(v)[:16], c.transpose(1, 0, 2))
    assert not k[16:].any() and not v[16:].any()
    for starts in ([-5, 1000], [3, 2 ** 31 - 1], [-2 ** 31, 0]):
        k, v = bq.lqmm_kv_read_f8(up(kc), up(vc), up(ks), up(vs), up(table), up(np.array(starts, np.int32)), 20)
        torch.cuda.synchronize()


def test_read_far_into_a_large_cache():
    """Offsets past 32 bits."""
    P, hkv, ps, d = 2 ** 14 + 9, 16, 64, 256
    announce("read far")
    kc, vc = (c.view(torch.uint8) for c in bq.kv_cache_empty(P, hkv, ps, d, dtype=F8))
    ks, vs = bq.kv_scales_empty(P, hkv, ps)
    x = torch.randn(2 * ps, hkv, d, device=DEV).half()
    slots = torch.cat((torch.arange((P - 1) * ps, P * ps, device=DEV), torch.arange(5 * ps, 6 * ps, device=DEV)))
    bq.lqmm_kv_append_norm(None, x, -x, None, slots, kc, vc, ks, vs)
    table = torch.tensor([[P - 1, 5]], dtype=torch.int32, device=DEV)
    k, v = bq.lqmm_kv_read_f8(kc, vc, ks, vs, table, torch.tensor([0, 2 * ps], dtype=torch.int32, device=DEV), 2 * ps)
    want, e = s8.quant(np64(x), "f16")
    want = want * np.exp2(e.astype(float))[..., None]
    assert np.array_equal(np64(k), s8.to_type(want, "f16")) and np.array_equal(np64(v), -s8.to_type(want, "f16"))


# ---- attention -----------------------------------------------------------------------
class Batch:
    """One batch on the host; memory that no row may see holds NaN codes and the
    scale byte 255, unused page-table entries numbers outside the cache."""

    def __init__(self, lens, news, hq, hkv, d, ps, prefix, t, seed=0, spread=3, extra=3):
        announce(f"attn_f8 lens={list(lens)[:6]} new={list(news)[:6]} h={hq}/{hkv} d={d} ps={ps} prefix={prefix} {t}")
        r = np.random.default_rng(seed)
        self.lens, self.news, self.prefix, self.t, self.d, self.ps = list(lens), list(news), prefix, t, d, ps
        n_pages, pp = [-(-n // ps) for n in lens], -(-prefix // ps)
        P = sum(n_pages) + pp + extra
        ids = r.permutation(P).astype(np.int32)
        mp = max(1, max(n_pages)) + 1
        self.table = r.choice(np.array([-1, 1 << 30, -(1 << 31), P], dtype=np.int64), (len(lens), mp)).astype(np.int32)
        kc, vc, ks, vs = random_cache(r, P, hkv, ps, d, spread)
        used = np.zeros(P * ps, dtype=bool)
        at = pp
        for b, n in enumerate(n_pages):
            self.table[b, :n] = ids[at:at + n]
            for j in range(lens[b]):
                used[ids[at + j // ps] * ps + j % ps] = True
            at += n
        for j in range(prefix):
            used[ids[j // ps] * ps + j % ps] = True
        u = ~used.reshape(P, 1, ps)
        kc[np.broadcast_to(u[..., None], kc.shape)] = 0x7f
        vc[np.broadcast_to(u.reshape(P, 1, ps // 8, 1, 8), vc.shape)] = 0xff
        ks[np.broadcast_to(u, ks.shape)] = vs[np.broadcast_to(u, vs.shape)] = 255
        self.cache = [kc, vc, ks, vs]
        self.pids = ids[:pp]
        self.start = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
        self.q = rnd(r, (sum(news), hq, d), t) * 1.5

    def want(self, scale=None):
        kc, vc, ks, vs = self.cache
        return s8.attention(np64(self.q), (values(kc), values(vc), ks, vs), self.table, self.lens, self.pids,
                            self.prefix, self.start, self.d ** -0.5 if scale is None else scale, self.t)

    def args(self, **kw):
        if any(n != 1 for n in self.news):
            kw = dict(q_start=up(self.start), max_q=max(self.news)) | kw
        q = self.q if self.q.is_cuda else self.q.to(DEV)
        return (q, *map(up, self.cache), up(self.table), up(np.array(self.lens, dtype=np.int32))), dict(
            prefix_pages=up(self.pids) if self.prefix else None, prefix_len=self.prefix, return_lse=True) | kw

    def run(self, **kw):
        a, k = self.args(**kw)
        out, lse = bq.lqmm_attn_prefix_f8(*a, **k)
        return np64(out), np64(lse)


def compare(out, lse, want, nan=None):
    wo, wl, bo, bl = want
    nan = np.zeros(wl.shape, dtype=bool) if nan is None else np.broadcast_to(nan if nan.ndim == 2 else nan[:, None], wl.shape)
    assert np.isnan(out[nan]).all() and np.isnan(lse[nan]).all()
    within(out[~nan], wo[~nan], bo[~nan], "out")
    empty = np.isneginf(wl) & ~nan
    assert np.array_equal(np.isneginf(lse), empty) and not out[empty].any()
    some = ~nan & ~empty
    within(lse[some], wl[some], bl[some], "lse")


@pytest.mark.parametrize("lens", [[1], [7, 8, 9], [31, 32, 33], [127, 128, 129], [0, 1], [0], [300, 0, 17]])
@pytest.mark.parametrize("prefix", [0, 1, 40, 129])
def test_attention_lengths(lens, prefix):
    b = Batch(lens, [1] * len(lens), 4, 2, 64, 16, prefix, "f16", seed=len(lens) + prefix)
    compare(*b.run(), b.want())


@pytest.mark.parametrize("hq, hkv, d, ps, t", [
    (1, 1, 64, 8, "bf16"), (8, 1, 128, 32, "f16"), (7, 1, 96, 16, "f16"), (16, 1, 128, 64, "bf16"),
    (20, 1, 64, 8, "f16"), (6, 3, 256, 16, "bf16"), (40, 1, 128, 128, "f16"), (4, 4, 256, 1024, "f16"),
    (14, 2, 96, 8, "bf16"), (4, 4, 128, 16, "f16"),
])
@pytest.mark.parametrize("prefix", [0, 70])
def test_attention_heads(hq, hkv, d, ps, t, prefix):
    b = Batch([45, 3, 160], [1, 1, 1], hq, hkv, d, ps, prefix, t, seed=hq + d)
    compare(*b.run(), b.want())


@pytest.mark.parametrize("lens, news", [
    ([5], [5]), ([33], [33]), ([40, 9, 1], [3, 9, 1]), ([130, 64], [17, 64]), ([2, 70], [5, 33]),
    ([100, 3, 80], [1, 0, 2]), ([260], [130]),
])
@pytest.mark.parametrize("hq, hkv, d, prefix, t", [
    (4, 2, 64, 0, "f16"), (8, 1, 128, 50, "bf16"), (3, 1, 96, 130, "f16"), (2, 1, 256, 33, "f16"), (2, 2, 128, 0, "bf16"),
])
def test_attention_new_tokens(lens, news, hq, hkv, d, prefix, t):
    b = Batch(lens, news, hq, hkv, d, 16, prefix, t, seed=sum(lens))
    compare(*b.run(), b.want())


@pytest.mark.parametrize("lens, news, hq, hkv, d, prefix, t", [
    ([3000], [1], 8, 1, 128, 0, "f16"), ([2700, 5], [1, 1], 2, 1, 64, 1500, "bf16"),
    ([int(n) for n in range(35)], [1] * 35, 4, 1, 128, 1300, "f16"), ([700], [300], 2, 1, 64, 0, "bf16"),
    ([400, 390], [200, 390], 2, 1, 128, 200, "f16"),
])
def test_attention_many_keys_and_rows(lens, news, hq, hkv, d, prefix, t):
    b = Batch(lens, news, hq, hkv, d, 32, prefix, t, seed=sum(lens))
    compare(*b.run(), b.want())


SHAPES = [
    # lens, new tokens, heads, dimensions, prefix, type
    ([97], [1], 2, 1, 64, 0, "f16"), ([70, 3], [1, 1], 4, 2, 128, 70, "bf16"),
    ([2700], [1], 2, 1, 64, 0, "f16"), ([41, 33], [3, 2], 4, 2, 256, 0, "bf16"),
    ([90], [70], 2, 2, 96, 0, "f16"), ([150, 64], [140, 64], 2, 1, 128, 0, "bf16"),
    ([100, 64], [90, 64], 2, 2, 64, 50, "bf16"), ([80], [60], 2, 1, 256, 50, "f16"),
    ([int(n) for n in range(35)], [1] * 35, 4, 1, 128, 130, "f16"),
]


def shape_batch(case, seed=0, **kw):
    lens, news, hq, hkv, d, prefix, t = case
    return Batch(lens, news, hq, hkv, d, 16, prefix, t, seed=seed + sum(lens), **kw)


@pytest.mark.parametrize("case", SHAPES)
@pytest.mark.parametrize("spread", [0, 14, 50])
def test_attention_scales_far_apart(case, spread):
    """Scales of neighbouring tokens up to 2^100 apart (K's kept near 1, so that
    logits stay ordinary); a zero vector's least scale beside them."""
    b = shape_batch(case, spread=spread)
    kc, vc, ks, vs = b.cache
    ks[ks != 255] = 120
    if spread == 50:
        keep = vs != 255
        vs[keep] = np.random.default_rng(1).choice([67, 100, 127, 150 if b.t == "bf16" else 130], keep.sum())
    want = b.want()
    compare(*b.run(), want)


@pytest.mark.parametrize("case", SHAPES)
def test_a_nan_query_gives_nan(case):
    b = shape_batch(case, 1)
    want = b.want()
    nan = np.zeros(b.q.shape[:2], dtype=bool)
    nan[-1, 0] = nan[len(nan) // 2, -1] = True
    b.q[torch.from_numpy(nan)] = float("nan")
    compare(*b.run(), want, nan & np.isfinite(want[1]))


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("case", SHAPES)
def test_a_nan_code_reaches_the_rows_that_see_it(case, what):
    """A NaN among the new tokens' keys or values does not reach the rows whose
    mask leaves it out."""
    b = shape_batch(case, 2)
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
    if what == "v":  # lse knows nothing of the values
        rows = ~nan
        assert np.isnan(out[nan]).all()
        compare(out[rows], lse[rows], [w[rows] for w in want])
        within(lse[nan], want[1][nan], want[3][nan], "lse")
    else:
        compare(out, lse, want, nan)


@pytest.mark.parametrize("case", SHAPES)
def test_values_at_the_ends_of_the_range(case):
    """Largest codes at the largest scale, and zeros at the least one."""
    b = shape_batch(case, 3)
    seen = b.cache[3] != 255
    vc = b.cache[1].transpose(0, 1, 2, 4, 3)  # [P][H][ps / 8][8][D]
    P, H, ps = seen.shape
    vc = vc.reshape(P, H, ps, b.d).copy()
    vc[seen] = 0x7e
    b.cache[3][seen] = 127 + 7 if b.t == "f16" else 127 + 60
    b.cache[1] = np.ascontiguousarray(vc.reshape(P, H, ps // 8, 8, b.d).transpose(0, 1, 2, 4, 3))
    compare(*b.run(), b.want())
    vc[seen] = 0
    b.cache[3][seen] = 67
    b.cache[1] = np.ascontiguousarray(vc.reshape(P, H, ps // 8, 8, b.d).transpose(0, 1, 2, 4, 3))
    compare(*b.run(), b.want())


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("case", SHAPES)
def test_attention_scale(case, scale):
    b = shape_batch(case, 4)
    compare(*b.run(scale=scale), b.want(scale))


@pytest.mark.parametrize("lens, news, max_q, before, after, hq, hkv, d, prefix, t", [
    ([20, 9], [3, 2], 3, 0, 4, 2, 1, 64, 0, "f16"), ([20, 9], [3, 2], 3, 5, 4, 4, 2, 128, 40, "bf16"),
    ([50, 30], [9, 4], 5, 2, 300, 4, 2, 256, 40, "bf16"), ([120, 60], [100, 50], 77, 0, 40, 2, 2, 96, 60, "f16"),
    ([2700], [2], 2, 1, 5, 2, 1, 64, 0, "bf16"), ([0, 7], [0, 2], 2, 3, 3, 2, 1, 64, 30, "f16"),
    ([120], [100], 60, 40, 3, 4, 1, 128, 0, "bf16"),
])
def test_rows_of_no_sequence(lens, news, max_q, before, after, hq, hkv, d, prefix, t):
    b = Batch(lens, news, hq, hkv, d, 16, prefix, t, seed=5)
    want = b.want()
    T = before + sum(news) + after
    q = torch.full((T, hq, d), 3.0, dtype=DT[t])
    q[before:before + sum(news)] = b.q
    of = np.full(T, -1)
    for s, n in zip(b.start, news):
        of[before + s:before + s + min(n, max_q)] = np.arange(s, s + min(n, max_q))
    b.q, b.start = q, b.start + np.int32(before)
    whole = torch.full((T + 2, hq, d), 7.0, dtype=DT[t], device=DEV)
    lses = torch.full((T + 2, hq), 7.0, device=DEV)
    need = bq.lqmm_attn_prefix_f8_workspace_bytes(prefix, b.table.shape[1], max_q, T, len(lens), hq, hkv, d, 16)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    out, lse = b.run(max_q=max_q, q_start=up(b.start), out=whole[1:-1], lse=lses[1:-1], workspace=ws[:need])
    assert (whole[[0, -1]] == 7).all() and (lses[[0, -1]] == 7).all() and (ws[need:] == 0xFF).all()
    live = of >= 0
    assert (out[~live] == 0).all() and np.isneginf(lse[~live]).all()
    compare(out[live], lse[live], [w[of[live]] for w in want])


def test_attention_strided_q_and_another_stream():
    b = Batch([45, 3, 160], [1, 1, 1], 4, 2, 128, 16, 40, "f16", seed=8)
    want = b.want()
    wide = torch.full((3, 9, 128), float("nan"), dtype=torch.float16, device=DEV)
    wide[:, 2:6] = b.q.to(DEV)
    b.q = wide[:, 2:6]
    a, kw = b.args()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, lse = bq.lqmm_attn_prefix_f8(*a, **kw, stream=s)
    s.synchronize()
    compare(np64(out), np64(lse), want)


def test_attention_lengths_and_pages_out_of_bounds():
    """A length past the table's is cut, a negative one is 0, a page outside the
    cache reads page 0."""
    b = Batch([30, 30], [1, 1], 2, 1, 64, 8, 0, "f16", seed=9)
    a, kw = b.args()
    a = list(a)
    announce("attn_f8 bad lengths")
    table = a[5][:, :4].contiguous()
    for lens in ([1000, -7], [2 ** 31 - 1, -2 ** 31]):
        out, lse = bq.lqmm_attn_prefix_f8(*a[:5], table, up(np.array(lens, np.int32)), return_lse=True)
        torch.cuda.synchronize()
        assert not out[1].any() and torch.isneginf(lse[1]).all()


def test_attention_in_a_captured_graph():
    b = Batch([200, 31, 0], [1, 1, 1], 4, 2, 64, 16, 300, "f16", seed=10)
    a, kw = b.args()
    eager = [t.clone() for t in bq.lqmm_attn_prefix_f8(*a, **kw)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bq.lqmm_attn_prefix_f8(*a, **kw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    announce("attn_f8 graph")
    with torch.cuda.graph(graph, stream=side):
        out, lse = bq.lqmm_attn_prefix_f8(*a, **kw)
    for _ in range(3):
        out.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        other = bq.lqmm_attn_prefix_f8(*a, **kw)  # eager work between the replays
        assert torch.equal(other[0], eager[0])


def test_attention_refuses():
    b = Batch([20], [1], 2, 1, 64, 16, 0, "f16")
    a, kw = b.args()
    a = list(a)
    with pytest.raises(TypeError):
        bq.lqmm_attn_prefix_f8(a[0].float(), *a[1:])
    with pytest.raises(TypeError):
        bq.lqmm_attn_prefix_f8(a[0], a[1].half(), *a[2:])
    with pytest.raises(ValueError):
        bq.lqmm_attn_prefix_f8(*a[:3], a[3][:1], *a[4:])
    with pytest.raises(TypeError):
        bq.lqmm_attn_prefix_f8(*a[:4], a[4].float(), *a[5:])


# ---- microscaled 4-bit floats ----------------------------------------------------------
@pytest.mark.parametrize("M, K, t", [(1, 32, "f32"), (3, 96, "f16"), (33, 4096, "bf16"), (5, 11008 + 32, "f16"),
                                     (1000, 64, "f32"), (257, 2080, "bf16"), (2, 32 * 4097, "f32")])
@pytest.mark.parametrize("lo, hi", [(-3, 4), (-149, -110), (100, 127)])
def test_mx_quant(M, K, t, lo, hi):
    """Bit for bit, ties and zero blocks included."""
    if t == "f16":
        lo, hi = (-24, -12) if lo < -100 else (10, 15) if lo > 50 else (lo, hi)
    r = np.random.default_rng(M + K)
    x = np.ldexp(r.standard_normal((M, K)), r.integers(lo, hi, (M, K // 32)).repeat(32, 1))
    # multiples of an eighth of a power of two: half of them are ties
    e = np.ldexp(1.0, r.integers(lo, hi, (M, K // 32)).repeat(32, 1) - 1)
    x[M // 2:] = (np.round(r.standard_normal((M, K)) * 8) / 8 * e)[M // 2:]
    x[0, :32] = 0.0
    lim = {"f16": 6e4, "bf16": 3e38, "f32": 3e38}[t]
    x = torch.from_numpy(np.clip(x, -lim, lim).astype(np.float32)).to(DT[t])
    announce(f"quant_mxfp4 {M}x{K} {t}")
    wide = torch.zeros(M, K + 64, dtype=DT[t], device=DEV)
    wide[:, 32:32 + K] = x.to(DEV)
    codes, scales = bq.lqmm_quant_mxfp4(wide[:, 32:32 + K])
    c, s = s8.mx_quant(np64(x))
    assert np.array_equal(scales.view(torch.uint8).cpu().numpy(), s)
    got = codes.cpu().numpy()
    want = s8.mx_pack(c)
    assert np.array_equal(got, want), np.argwhere(got != want)[:3]


def test_mx_quant_infinities_and_nan():
    x = torch.randn(4, 128, device=DEV)
    x[0, 40], x[1, 3], x[2, 127] = float("inf"), float("nan"), float("-inf")
    codes, scales = bq.lqmm_quant_mxfp4(x)
    c, s = s8.mx_quant(np64(x))
    assert np.array_equal(codes.cpu().numpy(), s8.mx_pack(c))
    assert np.array_equal(scales.view(torch.uint8).cpu().numpy(), s) and (s == 255).sum() == 3


def mx_random(r, n, k, lo=-6, hi=3):
    return r.integers(0, 16, (n, k)).astype(np.uint8), (127 + r.integers(lo, hi, (n, k // 32))).astype(np.uint8)


def check_mx(M, N, K, t, seed=0, make=mx_random, out=None):
    r = np.random.default_rng(seed + M + N)
    (w, ws), (x, xs) = make(r, N, K), make(r, M, K)
    announce(f"gemm_mxfp4 {M}x{N}x{K} {t}")
    got = bq.lqmm_gemm_mxfp4(up(s8.mx_pack(w)), up(ws), up(s8.mx_pack(x)), up(xs), out_dtype=DT[t]).double()
    W, X = up(s8.mx_values(w, ws)), up(s8.mx_values(x, xs))
    want = torch.matmul(X, W.t().contiguous())
    # one rounding of the sum for each 128 of K, and of the sums that waves share
    total = torch.matmul(X.abs(), W.abs().t().contiguous())
    bound = so.U[t] * want.abs() + so.TINY[t] + (K / 128 + 10) * 2.0 ** -24 * (1 + so.U[t]) * total
    over = (got - want).abs() - bound
    assert torch.isfinite(got).all() and float(over.max()) <= 0, float(over.max())


@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M, N, K", [
    (1, 1, 32), (1, 130, 96), (2, 16, 128), (16, 17, 160), (16, 300, 4128), (17, 33, 512), (45, 4127, 544),
    (64, 200, 1024), (65, 129, 2080), (100, 1001, 288), (128, 256, 8192), (300, 700, 416), (513, 1029, 1056),
    (1, 28672, 1024), (33, 9000, 64), (1500, 2100, 672), (2049, 4100, 256),
])
def test_mx_product(M, N, K, t):
    check_mx(M, N, K, t)


@pytest.mark.parametrize("M, N, K", [(1, 50, 1056), (20, 300, 544), (70, 500, 1024), (300, 3000, 416), (2900, 4100, 288)])
def test_mx_sums_keep_small_products(M, N, K):
    """Beside products 2^15 above them that cancel, the others (all positive)
    count in full: the sums are fp32's. A cut 14 bits below the largest product
    would lose all of them, (K - 32) 9 2^-15 or over 80 bounds."""
    def make(r, n, k):
        c, s = r.integers(1, 8, (n, k)).astype(np.uint8), np.full((n, k // 32), 119 if n == N else 120, np.uint8)
        c[:, :16], c[:, 16:32], s[:, 0] = 7, 15 if n == N else 7, 127
        return c, s
    check_mx(M, N, K, "f32", make=make)


def test_mx_nan_scales():
    """A block of scale 255 makes its row's outputs NaN, and no others."""
    r = np.random.default_rng(2)
    for M, N, K in ((3, 40, 160), (40, 90, 1056), (300, 400, 640)):
        (w, ws), (x, xs) = mx_random(r, N, K), mx_random(r, M, K)
        xs[1, K // 32 - 1], ws[7, 0] = 255, 255
        announce(f"gemm_mxfp4 NaN {M}x{N}x{K}")
        y = np64(bq.lqmm_gemm_mxfp4(up(s8.mx_pack(w)), up(ws), up(s8.mx_pack(x)), up(xs), out_dtype=torch.float32))
        nan = np.zeros((M, N), dtype=bool)
        nan[1], nan[:, 7] = True, True
        assert np.array_equal(np.isnan(y), nan)


def test_mx_quant_then_product():
    """Both together against 64 bits on the same codes."""
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x, w = torch.randn(37, 1056, device=DEV, generator=g).half(), torch.randn(515, 1056, device=DEV, generator=g)
    (xc, xs), (wc, ws) = bq.lqmm_quant_mxfp4(x), bq.lqmm_quant_mxfp4(w)
    y = bq.lqmm_gemm_mxfp4(wc, ws, xc, xs, out_dtype=torch.float32)
    X, W = (s8.mx_values(*s8.mx_quant(np64(a))) for a in (x, w))
    want = X @ W.T
    assert np.abs(np64(y) - want).max() <= 20 * 2.0 ** -24 * (np.abs(X) @ np.abs(W).T).max()


def test_mx_refuses():
    w, ws = torch.zeros(4, 32, dtype=torch.uint8, device=DEV), torch.zeros(4, 2, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        bq.lqmm_gemm_mxfp4(w, ws, w[:, :16].contiguous(), ws)
    with pytest.raises(ValueError):
        bq.lqmm_gemm_mxfp4(w, ws[:, :1].contiguous(), w, ws)
    with pytest.raises(TypeError):
        bq.lqmm_gemm_mxfp4(w, ws.float(), w, ws)
    with pytest.raises(ValueError):
        bq.lqmm_quant_mxfp4(torch.zeros(3, 48, device=DEV))
    with pytest.raises(TypeError):
        bq.lqmm_quant_mxfp4(torch.zeros(3, 64, device=DEV, dtype=torch.int32))
