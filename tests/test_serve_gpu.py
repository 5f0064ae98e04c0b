"""The serving operators on the GPU against their 64-bit forms, inside the
bounds of serve_oracle.py: sizes from one token up, ragged and empty rows,
pages that end inside a tile, NaN in memory that no row sees, strided inputs,
other streams, offsets past 32 bits, captured graphs."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve_oracle as so
from gpu_util import announce

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


def np64(t):
    return t.detach().cpu().double().numpy()


def within(got, want, bound, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    over = np.abs(got - want) - bound
    assert not np.isnan(over).any(), f"{what}: NaN"
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over the bound, at {np.unravel_index(over.argmax(), over.shape)}"


def rnd(r, shape, t):
    """Seeded normal values of type t on the host (a torch tensor)."""
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(DT[t])


# ---- append --------------------------------------------------------------------
def run_append(T, hq, hkv, d, ps, P, rot, inter, tin, t, slots, seed, base=10000.0, far=100000):
    r = np.random.default_rng(seed)
    inv = base ** (-np.arange(0, rot, 2) / rot) if rot else np.zeros(0)
    qkv = rnd(r, (T, hq + 2 * hkv, d), tin)
    kc, vc = rnd(r, (P, hkv, ps, d), t), rnd(r, (P, hkv, ps // 8, d, 8), t)
    pos = r.integers(0, far, T).astype(np.int32)
    announce(f"append T={T} hq={hq} hkv={hkv} d={d} ps={ps} rot={rot} inter={inter} {tin}->{t}")
    g = qkv.to(DEV)
    kg, vg = kc.to(DEV), vc.to(DEV)
    turns = bq.lqmm_rope_turns(inv) if rot else None
    qo = bq.lqmm_kv_append(g[:, :hq] if hq else None, g[:, hq:hq + hkv], g[:, hq + hkv:],
                           torch.from_numpy(pos).to(DEV), torch.from_numpy(slots).to(DEV), kg, vg,
                           rope_turns=turns, interleaved=inter)
    x = np64(qkv)
    n = rot // 2
    y = so.rotate(x, pos, inv, inter)
    b = so.rotate_bound(x, y, n, inter, t)
    if hq:
        within(qo, y[:, :hq], b[:, :hq], "q")
    else:
        assert qo is None
    wk, wv, bk, bv = np64(kc), np64(vc), np.zeros(kc.shape), np.zeros(vc.shape)
    v = x[:, hq + hkv:]
    so.place(wk, wv, y[:, hq:hq + hkv], v, slots)
    so.place(bk, bv, b[:, hq:hq + hkv], so.U[t] * np.abs(v) + so.TINY[t], slots)
    within(kg, wk, bk, "k_cache")
    within(vg, wv, bv, "v_cache")


@pytest.mark.parametrize("T, hq, hkv, d, ps, rot, inter, tin, t", [
    (1, 4, 1, 128, 16, 128, False, "f16", "f16"),
    (1, 1, 1, 64, 8, 16, True, "f32", "bf16"),
    (5, 6, 2, 96, 8, 96, False, "bf16", "bf16"),
    (9, 7, 7, 64, 32, 32, True, "f16", "f16"),
    (33, 40, 8, 128, 1024, 64, True, "f32", "f16"),
    (17, 8, 1, 256, 64, 256, False, "f32", "bf16"),
    (8, 0, 3, 128, 16, 128, False, "bf16", "f16"),
    (40, 2, 2, 256, 16, 0, False, "f16", "bf16"),
])
def test_append_scattered(T, hq, hkv, d, ps, rot, inter, tin, t):
    """Any slots, some negative or past the cache (not appended)."""
    P = max(2, 90 // ps + 1)
    r = np.random.default_rng(T + d)
    slots = r.permutation(P * ps)[:T].astype(np.int64)
    slots[2::7] = -1
    slots[4::11] = P * ps + 3
    slots[5::13] = 1 << 40
    run_append(T, hq, hkv, d, ps, P, rot, inter, tin, t, slots, 3 * T + d)


@pytest.mark.parametrize("first", [0, 1, 5, 7, 8])
@pytest.mark.parametrize("T", [7, 8, 9, 23, 64])
def test_append_runs(first, T):
    """Consecutive tokens from any place in a page: whole groups and their ends."""
    ps, P = 16, 8
    tok = np.arange(T) + first
    order = np.random.default_rng(first).permutation(P)
    slots = (order[tok // ps] * ps + tok % ps).astype(np.int64)
    run_append(T, 3, 2, 64, ps, P, 64, False, "f16", "f16", slots, 100 * first + T)


def test_append_broken_runs():
    """Runs with a gap, an out-of-order pair, or a dropped token in a group."""
    slots = np.arange(40, dtype=np.int64)
    slots[3], slots[12], slots[13] = 63, 13, 12
    slots[20] = -1
    slots[32:40] = np.arange(72, 80)  # the last group ends at the cache's end
    run_append(40, 2, 1, 128, 16, 5, 128, False, "bf16", "bf16", slots, 9)


def test_append_far_positions():
    run_append(16, 4, 1, 128, 16, 2, 128, False, "f32", "f16", np.arange(16, dtype=np.int64), 5,
               far=2 ** 31 - 1)


# ---- attention -----------------------------------------------------------------
def make_attn(lens, news, hq, hkv, d, ps, prefix, t, seed, poison=True, extra=3):
    """Host tensors of a batch; memory that no row may see holds NaN, and unused
    page-table entries hold numbers outside the cache."""
    r = np.random.default_rng(seed)
    B = len(lens)
    n_pages = [-(-n // ps) for n in lens]
    pp = -(-prefix // ps)
    P = sum(n_pages) + pp + extra
    ids = r.permutation(P).astype(np.int32)
    mp = max(1, max(n_pages)) + 1
    table = r.choice(np.array([-1, 1 << 30, -(1 << 31), P], dtype=np.int64), (B, mp)).astype(np.int32)
    kc = rnd(r, (P, hkv, ps, d), t)
    vc = rnd(r, (P, hkv, ps // 8, d, 8), t)
    used = np.zeros(P * ps, dtype=bool)
    at = pp
    for b in range(B):
        table[b, :n_pages[b]] = ids[at:at + n_pages[b]]
        for j in range(lens[b]):
            used[ids[at + j // ps] * ps + j % ps] = True
        at += n_pages[b]
    for j in range(prefix):
        used[ids[j // ps] * ps + j % ps] = True
    if poison:
        u = torch.from_numpy(used).view(P, 1, ps, 1)
        kc = kc.masked_fill(~u, float("nan"))
        vc = vc.masked_fill(~u.view(P, 1, ps // 8, 1, 8), float("nan"))
    T = sum(news)
    q = rnd(r, (T, hq, d), t) * 1.5
    start = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    return q, kc, vc, table, np.array(lens, dtype=np.int32), ids[:pp], start


def check_attn(lens, news, hq, hkv, d, ps, prefix, t, seed=0, scale=None, ldq=None, stream=None):
    q, kc, vc, table, ln, pids, start = make_attn(lens, news, hq, hkv, d, ps, prefix, t, seed)
    announce(f"attn lens={list(lens)[:6]} new={list(news)[:6]} h={hq}/{hkv} d={d} ps={ps} prefix={prefix} {t}")
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    qg = q.to(DEV)
    if ldq:  # rows of a wider tensor
        wide = torch.full((q.shape[0], ldq, d), float("nan"), dtype=q.dtype, device=DEV)
        wide[:, 1:1 + hq] = qg
        qg = wide[:, 1:1 + hq]
    one = all(n == 1 for n in news)
    args = (qg, kc.to(DEV), vc.to(DEV), up(table), up(ln))
    kw = dict(prefix_pages=up(pids) if prefix else None, prefix_len=prefix,
              q_start=None if one else up(start), max_q=1 if one else max(news), scale=scale,
              return_lse=True)
    if stream is not None:
        torch.cuda.synchronize()
        out, lse = bq.lqmm_attn_prefix(*args, **kw, stream=stream)
        stream.synchronize()
    else:
        out, lse = bq.lqmm_attn_prefix(*args, **kw)
    wo, wl, bo, bl = so.attention(np64(q), np64(kc), np64(vc), table, list(lens), pids, prefix, start,
                                  d ** -0.5 if scale is None else scale, t)
    within(out, wo, bo, "out")
    lse = np64(lse)
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(lse), empty)
    within(np.where(empty, 0, lse), np.where(empty, 0, wl), bl, "lse")
    return args, kw, out


@pytest.mark.parametrize("lens", [[1], [7, 8, 9], [31, 32, 33], [127, 128, 129], [0, 1], [0], [300, 0, 17]])
@pytest.mark.parametrize("prefix", [0, 1, 40, 129])
def test_attention_lengths(lens, prefix):
    check_attn(lens, [1] * len(lens), 4, 2, 64, 16, prefix, "f16", seed=len(lens) + prefix)


@pytest.mark.parametrize("hq, hkv, d, ps, t", [
    (1, 1, 64, 8, "bf16"), (8, 1, 128, 32, "f16"), (7, 1, 96, 16, "f16"), (16, 1, 128, 64, "bf16"),
    (20, 1, 64, 8, "f16"), (6, 3, 256, 16, "bf16"), (40, 1, 128, 128, "f16"), (4, 4, 256, 1024, "f16"),
    (14, 2, 96, 8, "bf16"), (4, 4, 128, 16, "f16"),
])
@pytest.mark.parametrize("prefix", [0, 70])
def test_attention_heads(hq, hkv, d, ps, t, prefix):
    check_attn([45, 3, 160], [1, 1, 1], hq, hkv, d, ps, prefix, t, seed=hq + d)


@pytest.mark.parametrize("lens, news", [
    ([5], [5]), ([33], [33]), ([40, 9, 1], [3, 9, 1]), ([130, 64], [17, 64]), ([2, 70], [5, 33]),
    ([100, 3, 80], [1, 0, 2]), ([260], [130]),
])
@pytest.mark.parametrize("prefix", [0, 50])
@pytest.mark.parametrize("hq, hkv, d, t", [(2, 1, 64, "f16"), (8, 2, 128, "bf16")])
def test_attention_new_tokens(lens, news, prefix, hq, hkv, d, t):
    """Several new tokens a sequence, causal among themselves; a sequence with
    more new tokens than keys has rows that see only the prefix, or nothing."""
    check_attn(lens, news, hq, hkv, d, 8, prefix, t, seed=sum(lens))


@pytest.mark.parametrize("batch, hq, hkv, d, prefix, t", [
    (33, 4, 1, 128, 300, "f16"), (70, 8, 2, 64, 257, "bf16"), (9, 16, 1, 256, 500, "f16"),
    (40, 7, 1, 96, 200, "bf16"),
])
def test_attention_many_rows_share_a_prefix(batch, hq, hkv, d, prefix, t):
    r = np.random.default_rng(batch)
    lens = [int(x) for x in r.integers(0, 40, batch)]
    check_attn(lens, [1] * batch, hq, hkv, d, 16, prefix, t, seed=batch)


@pytest.mark.parametrize("value", ["nan", "inf"])
@pytest.mark.parametrize("lens, news, hq, hkv, d, t", [
    ([9], [7], 2, 1, 64, "f16"), ([140, 40], [9, 3], 4, 2, 128, "bf16"), ([90], [70], 2, 2, 96, "f16"),
    ([300, 64], [290, 64], 2, 2, 64, "bf16"), ([300, 64], [290, 64], 2, 1, 128, "f16"),
    ([200], [100], 2, 1, 256, "bf16"),
])
@pytest.mark.parametrize("prefix", [0, 50])
def test_attention_later_tokens_are_not_seen(lens, news, hq, hkv, d, t, prefix, value):
    """A value vector that is not finite reaches only the rows that see its key:
    not the new tokens before it, whose mask leaves it out."""
    q, kc, vc, table, ln, pids, start = make_attn(lens, news, hq, hkv, d, 16, prefix, t, 5)
    announce(f"attn {value} behind the mask lens={lens} new={news} h={hq}/{hkv} d={d} prefix={prefix} {t}")
    wo, _, bo, _ = so.attention(np64(q), np64(kc), np64(vc), table, list(lens), pids, prefix, start,
                                d ** -0.5, t)
    clear = np.zeros(len(q), dtype=bool)  # rows that see no such value
    for b, (n, new) in enumerate(zip(lens, news)):
        at = n - 1 - new // 3
        kc[table[b, at // 16], :, at % 16] = float(value)
        vc[table[b, at // 16], :, at % 16 // 8, :, at % 8] = float(value)
        clear[start[b]:start[b] + at - (n - new)] = True
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    out = bq.lqmm_attn_prefix(q.to(DEV), kc.to(DEV), vc.to(DEV), up(table), up(ln),
                              prefix_pages=up(pids) if prefix else None, prefix_len=prefix,
                              q_start=up(start), max_q=max(news))
    assert clear.any() and not clear.all()
    got = np64(out)
    within(got[clear], wo[clear], bo[clear], "out")
    if value == "nan":
        assert np.isnan(got[~clear]).all()


def test_attention_large_logits_and_ties():
    """A scale that makes one weight of each row nearly 1, and a scale of zero
    (all seen keys weigh the same)."""
    check_attn([90, 17], [1, 1], 4, 1, 64, 16, 33, "f16", scale=3.0)
    check_attn([90, 17], [1, 1], 4, 1, 64, 16, 33, "bf16", scale=0.0)


def test_attention_strided_queries():
    check_attn([50, 20, 3], [2, 1, 3], 4, 2, 128, 16, 20, "f16", ldq=9)
    check_attn([50, 20, 3], [1, 1, 1], 4, 2, 64, 16, 0, "bf16", ldq=6)


def test_attention_long():
    """Many chunks and their join: one sequence, a long cache of its own."""
    check_attn([5003], [1], 2, 1, 64, 32, 0, "f16")
    check_attn([17], [1], 2, 1, 128, 32, 4097, "bf16")


def test_attention_other_stream_and_repeats():
    s = torch.cuda.Stream()
    args, kw, out = check_attn([200, 33], [1, 1], 8, 2, 128, 16, 700, "f16", stream=s)
    for _ in range(3):
        again, _ = bq.lqmm_attn_prefix(*args, **kw)
        assert torch.equal(again, out)


def test_attention_lengths_are_bounded():
    """Lengths past the page table and offsets outside q: cut, nothing else is
    read or written (guard values around out stay)."""
    q, kc, vc, table, ln, pids, start = make_attn([40, 24], [1, 1], 2, 1, 64, 8, 0, "f16", 4,
                                                 poison=False)
    table = np.ascontiguousarray(table[:, :3])  # 24 tokens
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    dev = [x.to(DEV) for x in (q, kc, vc)]
    announce("attn lengths past the page table")
    whole = torch.full((4, 2, 64), 7.0, dtype=torch.float16, device=DEV)
    bq.lqmm_attn_prefix(*dev, up(table), up(np.array([1 << 30, -5], dtype=np.int32)), out=whole[1:3])
    want, _, b, _ = so.attention(np64(q), np64(kc), np64(vc), table, [24, 0], [], 0, [0, 1, 2], 0.125, "f16")
    within(whole[1:3], want, b, "cut lengths")
    assert (whole[0] == 7).all() and (whole[3] == 7).all()
    announce("attn offsets outside q")
    whole.fill_(7.0)
    bad = up(np.array([-9, 1, 1 << 30], dtype=np.int32))
    bq.lqmm_attn_prefix(*dev, up(table), up(np.array([24, 24], dtype=np.int32)), q_start=bad, max_q=5,
                        out=whole[1:3])
    assert (whole[0] == 7).all() and (whole[3] == 7).all()


def test_cache_offsets_past_32_bits():
    """Pages whose elements lie past 2^32 bytes and 2^31 elements."""
    P, hkv, ps, d = 2200, 8, 1024, 128  # 2.3e9 elements
    kc, vc = bq.kv_cache_empty(P, hkv, ps, d, dtype=torch.float16)
    r = np.random.default_rng(0)
    T, ids = 1100, [P - 1, P - 3]
    k, v = rnd(r, (T, hkv, d), "f16"), rnd(r, (T, hkv, d), "f16")
    slots = np.array([ids[j // ps] * ps + j % ps for j in range(T)], dtype=np.int64)
    announce("append and attention past 2^31 elements")
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    bq.lqmm_kv_append(None, k.to(DEV), v.to(DEV), None, up(slots), kc, vc)
    small_k, small_v = kc[ids].cpu(), vc[ids].cpu()
    q = rnd(r, (1, hkv, d), "f16")
    for prefix in (0, 1050):
        table = np.array([[ids[0], ids[1]]], dtype=np.int32)
        out = bq.lqmm_attn_prefix(q.to(DEV), kc, vc, up(table), up(np.array([T], dtype=np.int32)),
                                  prefix_pages=up(table[0]) if prefix else None, prefix_len=prefix)
        want, _, b, _ = so.attention(np64(q), np64(small_k), np64(small_v), [[0, 1]], [T], [0, 1],
                                     prefix, [0, 1], d ** -0.5, "f16")
        within(out, want, b, f"prefix {prefix}")


def test_attention_workspace_rules():
    q, kc, vc, table, ln, pids, start = make_attn([40], [1], 2, 1, 64, 8, 100, "f16", 4)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    args = [x.to(DEV) for x in (q, kc, vc)] + [up(table), up(ln)]
    kw = dict(prefix_pages=up(pids), prefix_len=100)
    need = bq.lqmm_attn_prefix_workspace_bytes(100, table.shape[1], 1, 1, 1, 2, 1, 64, 8)
    assert need > 0
    with pytest.raises(bq.LqmmError) as e:
        bq.lqmm_attn_prefix(*args, **kw, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    assert e.value.status == 4
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device=DEV)
    a = bq.lqmm_attn_prefix(*args, **kw, workspace=ws[:need])
    assert (ws[need:] == 0xAB).all()
    assert torch.equal(a, bq.lqmm_attn_prefix(*args, **kw))
    with pytest.raises(TypeError):
        bq.lqmm_attn_prefix(args[0].float(), *args[1:], **kw)
    with pytest.raises(ValueError):
        bq.lqmm_attn_prefix(*args, prefix_pages=up(pids), prefix_len=105)


# ---- 8-bit floats --------------------------------------------------------------
@pytest.mark.parametrize("t", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M, K", [(1, 16), (1, 4096), (3, 128), (16, 144), (17, 1040), (200, 272)])
def test_quant_codes(M, K, t):
    r = np.random.default_rng(M + K)
    x = rnd(r, (M, K), t) * torch.exp(2 * rnd(r, (K,), "f32")).to(DT[t])
    if M > 1:
        x[1] = 0.0
        x[0, :16] = torch.finfo(DT[t]).max / 2
    announce(f"quant {M}x{K} {t}")
    codes, scales = bq.lqmm_quant_f8b128(x.to(DEV))
    want, ws = so.quantize(x.float().numpy())
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(np64(codes), want)


def test_quant_every_quotient():
    """Codes equal those of the correctly rounded quotient: random mantissas and
    scales over the exponent range, and values on and next to the ties."""
    r = np.random.default_rng(11)
    x = r.standard_normal((4096, 1024)).astype(np.float32)
    x *= np.exp2(r.integers(-60, 60, (4096, 8))).astype(np.float32).repeat(128, 1)
    # ties of e4m3 times a group's scale, moved by at most one ulp
    v = np.sort(np.unique(np.abs(so.E4M3[np.isfinite(so.E4M3)])))
    mid = ((v[:-1] + v[1:]) / 2).astype(np.float32)
    for m in range(0, 4096, 2):
        top = np.float32(1 + r.random())
        s = np.float32(top / np.float32(448.0))
        t = (r.choice(mid, 127) * s).astype(np.float32)
        t = np.nextafter(t, t + r.integers(-1, 2, 127).astype(np.float32) * np.float32(1e30)).astype(np.float32)
        x[m, :127], x[m, 127] = np.clip(t, -top, top), top
    announce("quant: every quotient")
    codes, scales = bq.lqmm_quant_f8b128(torch.from_numpy(x).to(DEV))
    want, ws = so.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(np64(codes), want)


def test_quant_strided_and_special():
    r = np.random.default_rng(3)
    x = rnd(r, (5, 400), "f16")
    x[2, 130] = float("nan")
    x[3, 5] = float("inf")
    g = x.to(DEV)[:, 16:288]  # rows of a wider tensor
    codes, scales = bq.lqmm_quant_f8b128(g)
    plain, ps = bq.lqmm_quant_f8b128(g.contiguous())
    assert torch.equal(codes.view(torch.uint8), plain.view(torch.uint8)) and torch.equal(scales, ps)
    got = np64(codes)
    assert np.isnan(got[2, 130 - 16]) and np.isnan(got).sum() == 1  # (column 5 is outside)
    g2, s2 = bq.lqmm_quant_f8b128(x.to(DEV)[:, :128])
    assert torch.isinf(s2[0, 3]) and np.isnan(np64(g2)[3, 5])


def make_f8(M, N, K, seed):
    r = np.random.default_rng(seed)
    fine = np.array([c for c in range(256) if (c & 127) != 127], dtype=np.uint8)
    w, x = r.choice(fine, (N, K)), r.choice(fine, (M, K))
    nb, kb = -(-N // 128), -(-K // 128)
    ws = np.exp(r.standard_normal((nb, kb))).astype(np.float32) * np.float32(0.01)
    xs = np.exp(r.standard_normal((kb, M))).astype(np.float32)
    return w, ws, x, xs


def f8_dev(a):
    return torch.from_numpy(a).to(DEV).view(torch.float8_e4m3fn)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 130, 300])
@pytest.mark.parametrize("N, K, t", [
    (1, 16, "f32"), (127, 128, "f16"), (129, 144, "bf16"), (256, 1024, "f32"), (515, 2064, "f16"),
    (1024, 400, "f16"),
])
def test_f8_product(M, N, K, t):
    """fp32 outputs to the fp32 limits of the library's tests; 16-bit outputs to
    one rounding more."""
    w, ws, x, xs = make_f8(M, N, K, 7 * M + N + K)
    announce(f"gemm_f8b128 {M}x{N}x{K} {t}")
    y = bq.lqmm_gemm_f8b128(f8_dev(w), torch.from_numpy(ws).to(DEV), f8_dev(x),
                            torch.from_numpy(xs).to(DEV), out_dtype=torch.float32 if t == "f32" else DT[t])
    got, want = np64(y), so.f8_product(so.E4M3[w], ws, so.E4M3[x], xs)
    if t == "f16":  # values past the type's range become infinite
        big = np.abs(want) > 65504
        assert np.isinf(got[np.abs(want) > 65536]).all()
        got, want = np.where(big, 0, got), np.where(big, 0, want)
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    top = np.abs(got - want).max() / np.abs(want).max()
    u = 0.0 if t == "f32" else so.U[t]
    assert rel <= 1e-5 + u and top <= 1e-4 + u, (rel, top)


@pytest.mark.parametrize("M, N, K, t", [
    (300, 3000, 1040, "bf16"), (300, 3000, 144, "f16"), (700, 8300, 400, "bf16"),
    (700, 8300, 272, "f32"), (1500, 9000, 384, "bf16"), (1500, 9000, 256, "f16"),
    (2900, 9100, 400, "bf16"), (2900, 9100, 272, "f16"), (16, 12300, 144, "f16"),
    (9, 12301, 1040, "bf16"), (32, 4000, 2064, "f32"), (20, 300, 16, "bf16"),
    (45, 4127, 4112, "f32"), (64, 3000, 1040, "f16"), (100, 1001, 272, "bf16"),
    (2200000, 1, 16, "f16"), (1, 2200000, 16, "bf16"),
])
def test_f8_product_large(M, N, K, t):
    """Every tile size, ends in all three directions; expected values in 64
    bits on the GPU."""
    w, ws, x, xs = make_f8(M, N, K, M + N + K)
    announce(f"gemm_f8b128 {M}x{N}x{K} {t}")
    dw, dx = f8_dev(w), f8_dev(x)
    dws, dxs = torch.from_numpy(ws).to(DEV), torch.from_numpy(xs).to(DEV)
    got = bq.lqmm_gemm_f8b128(dw, dws, dx, dxs, out_dtype=DT[t]).double()
    kb = torch.arange(K, device=DEV) // 128
    W = dw.double() * dws.double()[torch.arange(N, device=DEV) // 128][:, kb]
    want = torch.matmul(dx.double() * dxs.double()[kb].t(), W.t().contiguous())
    if t == "f16":
        big = want.abs() > 65504
        assert torch.isinf(got[want.abs() > 65536]).all()
        got, want = got.masked_fill(big, 0), want.masked_fill(big, 0)
    rel = float((got - want).norm() / want.norm())
    top = float((got - want).abs().max() / want.abs().max())
    u = 0.0 if t == "f32" else so.U[t]
    assert rel <= 1e-5 + u and top <= 1e-4 + u, (rel, top)


def test_f8_product_is_exact_on_integers():
    """Products and sums that fp32 holds exactly come out exactly."""
    r = np.random.default_rng(5)
    w, x = r.integers(-4, 5, (300, 512)).astype(np.float64), r.integers(-4, 5, (70, 512)).astype(np.float64)
    f8 = lambda a: torch.from_numpy(a).to(torch.float8_e4m3fn).to(DEV)  # noqa: E731
    ws, xs = 2.0 ** r.integers(-2, 3, (3, 4)), 2.0 ** r.integers(-2, 3, (4, 70))
    dev = lambda a: torch.from_numpy(a.astype(np.float32)).to(DEV)  # noqa: E731
    announce("gemm_f8b128 exact integers")
    for m in (1, 20, 70):
        y = bq.lqmm_gemm_f8b128(f8(w), dev(ws), f8(x[:m]), dev(xs[:, :m]), out_dtype=torch.float32)
        assert np.array_equal(np64(y), so.f8_product(w, ws, x[:m], xs[:, :m]))


def test_f8_nan_stays_in_its_row():
    """A NaN code of one row of X reaches that row only; a NaN weight its column."""
    w, ws, x, xs = make_f8(40, 200, 272, 1)
    x[3, 271], w[130, 0] = 0x7F, 0xFF
    announce("gemm_f8b128 NaN codes")
    y = np64(bq.lqmm_gemm_f8b128(f8_dev(w), torch.from_numpy(ws).to(DEV), f8_dev(x),
                                 torch.from_numpy(xs).to(DEV), out_dtype=torch.float32))
    want = np.zeros(y.shape, dtype=bool)
    want[3], want[:, 130] = True, True
    assert np.array_equal(np.isnan(y), want)


def test_guarded_outputs():
    """Nothing is written outside the outputs (odd sizes, guard rows)."""
    w, ws, x, xs = make_f8(21, 131, 144, 2)
    g = torch.full((23, 131), 5.0, dtype=torch.float32, device=DEV)
    flat = g.view(-1)
    # rows 1..21 start 4-byte aligned only: refused; whole buffers are fine
    with pytest.raises(bq.LqmmError):
        bq.lqmm_gemm_f8b128(f8_dev(w), torch.from_numpy(ws).to(DEV), f8_dev(x),
                            torch.from_numpy(xs).to(DEV), out=g[1:22])
    big = torch.full((21 * 131 + 256,), 5.0, dtype=torch.float32, device=DEV)
    out = big[128:128 + 21 * 131].view(21, 131)
    bq.lqmm_gemm_f8b128(f8_dev(w), torch.from_numpy(ws).to(DEV), f8_dev(x),
                        torch.from_numpy(xs).to(DEV), out=out)
    assert (big[:128] == 5).all() and (big[128 + 21 * 131:] == 5).all() and (flat == 5).all()
    xf = torch.randn(21, 144, device=DEV)
    raw = torch.full((21 * 144 + 64,), 9, dtype=torch.uint8, device=DEV)
    sc = torch.full((2 * 21 + 8,), 9.0, device=DEV)
    bq.lqmm_quant_f8b128(xf, out=raw[32:32 + 21 * 144].view(21, 144), scales=sc[4:46].view(2, 21))
    assert (raw[:32] == 9).all() and (raw[-32:] == 9).all() and (sc[:4] == 9).all() and (sc[46:] == 9).all()
