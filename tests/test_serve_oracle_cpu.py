"""The 64-bit forms that the serving kernels are tested against, and the host
parts of the library behind them, against hand-worked values and closed forms."""
import ctypes
import math
import os

import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve_oracle as so


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bq.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return bq.load()


def test_e4m3_values():
    assert so.e4m3_value(0x00) == 0.0 and so.e4m3_value(0x01) == 2.0 ** -9
    assert so.e4m3_value(0x38) == 1.0 and so.e4m3_value(0xB8) == -1.0
    assert so.e4m3_value(0x7E) == 448.0 and math.isnan(so.e4m3_value(0x7F))
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, so.E4M3, equal_nan=True)


def test_e4m3_rounding():
    fine = so.E4M3[np.isfinite(so.E4M3)]
    assert np.array_equal(so.e4m3_round(fine), fine)
    pos = np.sort(np.unique(np.abs(fine)))
    mid = (pos[:-1] + pos[1:]) / 2
    even = np.where(np.arange(len(mid)) % 2 == 0, pos[:-1], pos[1:])  # codes count up from 0
    assert np.array_equal(so.e4m3_round(mid), even)
    assert np.array_equal(so.e4m3_round(mid * (1 + 1e-9)), pos[1:])
    assert np.array_equal(so.e4m3_round(-mid * (1 - 1e-9)), -pos[:-1])


def test_quantize_by_hand():
    x = np.zeros((2, 144), dtype=np.float32)
    x[0, :4] = [448.0, -224.0, 17.0, 17.9]
    x[0, 128] = -2.0
    v, s = so.quantize(x)
    assert s.tolist() == [[1.0, 2.0 ** -126], [np.float32(2.0) / np.float32(448.0), 2.0 ** -126]]
    assert v[0, :4].tolist() == [448.0, -224.0, 16.0, 18.0] and v[0, 128] == -448.0
    assert not v[1].any()


def test_f8_product_against_loops():
    r = np.random.default_rng(0)
    w, x = r.choice(so.E4M3[:126], (130, 144)), r.choice(so.E4M3[:126], (3, 144))
    ws, xs = r.random((2, 2)), r.random((2, 3))
    y = so.f8_product(w, ws, x, xs)
    for m, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
        want = sum(x[m, k] * xs[k // 128, m] * w[n, k] * ws[n // 128, k // 128] for k in range(144))
        assert abs(y[m, n] - want) <= 1e-9 * abs(want)


def test_rotation_is_a_rotation():
    r = np.random.default_rng(1)
    x, f = r.standard_normal((5, 2, 64)), 10.0 ** -np.arange(16.0)
    for inter in (False, True):
        y = so.rotate(x, np.array([0, 1, 2, 1000, -7]), f, inter)
        assert np.allclose(y[0], x[0], atol=0) and np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        # turning back
        back = np.stack([so.rotate(y[i:i + 1], [-p], f, inter)[0] for i, p in enumerate([0, 1, 2, 1000, -7])])
        assert np.allclose(back, x)
    one = np.zeros((1, 1, 64))
    one[0, 0, 0] = 1.0
    y = so.rotate(one, [1], [math.pi / 2] + [0.0] * 15, False)
    assert abs(y[0, 0, 16] - 1) < 1e-15 and abs(y[0, 0, 0]) < 1e-15


def test_attention_closed_forms():
    """Equal keys average the values they see; a far larger logit picks its value."""
    r = np.random.default_rng(2)
    P, H, ps, D = 4, 1, 8, 4
    k, v = np.zeros((P, H, ps, D)), np.zeros((P, H, ps // 8, D, 8))
    vals = r.standard_normal((20, D))
    so.place(k, v, np.zeros((20, H, D)), vals[:, None], [8 + j if j < 8 else 24 + j - 8 if j < 16 else j - 16 for j in range(20)])
    q = r.standard_normal((2, 2, D))
    out, lse, _, _ = so.attention(q, k, v, [[3, 0]], [11], [1], 5, [0, 2], 0.5, "f16")
    # prefix: tokens 0..4; own tokens 8.. (page 3) and 16.. (page 0); 2 new of 11
    see0 = np.concatenate((vals[:5], vals[8:18]))
    assert np.allclose(out[0, 1], see0.mean(0)) and np.allclose(lse[0], math.log(15))
    assert np.allclose(out[1, 0], np.concatenate((vals[:5], vals[8:19])).mean(0))
    k[3, 0, 2] = 100 * q[1, 0]
    out, _, _, _ = so.attention(q, k, v, [[3, 0]], [11], [1], 5, [0, 2], 1.0, "f16")
    assert np.allclose(out[1, 0], vals[10])


def test_rope_turns_matches_exact_fractions(lib):
    f = np.concatenate((10000.0 ** (-np.arange(64) / 64), [0.0, 1e-30, 2 * np.pi, 7.5, -0.25, 1e6]))
    out = np.zeros(f.size, dtype=np.uint64)
    assert lib.lqmm_rope_turns(f.ctypes.data, f.size, out.ctypes.data) == 0
    assert out.tolist() == so.turns_of(f)
    # the angle it gives at a far position, against 64-bit arithmetic
    for i in (0, 10, 63):
        turn = (123456789 * int(out[i])) % 2 ** 64 / 2.0 ** 64
        want = 123456789 * f[i] / (2 * math.pi) % 1.0
        assert min(abs(turn - want), 1 - abs(turn - want)) < 1e-7
    bad = np.array([1.0, np.nan])
    assert lib.lqmm_rope_turns(bad.ctypes.data, 2, out.ctypes.data) == 2
    assert lib.lqmm_rope_turns(None, 2, out.ctypes.data) == 1
    assert lib.lqmm_rope_turns(bad.ctypes.data, 0, out.ctypes.data) == 2


# ---- refusals: invalid arguments never reach the device ---------------------------
A16, A4 = 0x10000, 0x10004
NULL, SHAPE, ALIGN, DEVICE, TYPE = 1, 2, 3, 5, 7
NO_GPU = not os.path.exists("/dev/kfd")


def _append(lib, **kw):
    a = dict(q=A16, k=A16, v=A16, in_type=1, ldq=512, ldk=128, ldv=128, positions=A16, slots=A16,
             turns=A16, rot=128, inter=0, q_out=A16, kc=A16, vc=A16, ctype=1, tokens=3, hq=4,
             hkv=1, d=128, ps=16, pages=4, stream=None)
    a.update(kw)
    return lib.lqmm_kv_append(*a.values())


@pytest.mark.parametrize("change, want", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(kc=None), NULL),
    (dict(vc=None), NULL), (dict(q=None), NULL), (dict(q_out=None), NULL),
    (dict(positions=None), NULL), (dict(turns=None), NULL),
    (dict(in_type=3), TYPE), (dict(in_type=-1), TYPE), (dict(ctype=0), TYPE), (dict(ctype=9), TYPE),
    (dict(tokens=0), SHAPE), (dict(tokens=-1), SHAPE), (dict(pages=0), SHAPE), (dict(d=80), SHAPE),
    (dict(ps=12), SHAPE), (dict(ps=4), SHAPE), (dict(ps=2048), SHAPE), (dict(hkv=0), SHAPE),
    (dict(hq=-1), SHAPE), (dict(rot=8), SHAPE), (dict(rot=144), SHAPE), (dict(rot=-16), SHAPE),
    (dict(ldq=504), SHAPE), (dict(ldk=120), SHAPE), (dict(ldv=0), SHAPE),
    (dict(ldk=132), ALIGN), (dict(k=A4), ALIGN), (dict(kc=A4), ALIGN), (dict(q=A4), ALIGN),
    (dict(slots=A4), ALIGN), (dict(turns=A4), ALIGN), (dict(positions=0x10002), ALIGN),
])
def test_append_refusals(lib, change, want):
    assert _append(lib, **change) == want


def _attn(lib, **kw):
    a = dict(q=A16, ldq=512, kc=A16, vc=A16, type=1, pp=A16, plen=5, pages=A16, mp=3, lens=A16,
             start=None, max_q=1, out=A16, lse=None, scale=ctypes.c_float(0.1), tokens=2, batch=2,
             hq=4, hkv=1, d=128, ps=16, npages=9, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    return lib.lqmm_attn_prefix(*a.values())


@pytest.mark.parametrize("change, want", [
    (dict(q=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(pages=None), NULL),
    (dict(lens=None), NULL), (dict(out=None), NULL), (dict(pp=None), NULL),
    (dict(type=0), TYPE), (dict(type=5), TYPE),
    (dict(tokens=0), SHAPE), (dict(batch=0), SHAPE), (dict(mp=0), SHAPE), (dict(max_q=0), SHAPE),
    (dict(plen=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hq=5, hkv=2), SHAPE), (dict(d=32), SHAPE),
    (dict(ps=24), SHAPE), (dict(npages=0), SHAPE), (dict(tokens=3), SHAPE), (dict(max_q=2), SHAPE),
    (dict(mp=1 << 30), SHAPE), (dict(plen=1 << 31), SHAPE), (dict(tokens=1 << 30, start=A16), SHAPE),
    (dict(scale=ctypes.c_float(float("nan"))), SHAPE), (dict(ldq=384), SHAPE),
    (dict(ldq=516), ALIGN), (dict(q=A4), ALIGN), (dict(out=A4), ALIGN), (dict(lens=0x10002), ALIGN),
    (dict(ws=A4, ws_bytes=1 << 20), ALIGN),
])
def test_attention_refusals(lib, change, want):
    assert _attn(lib, **change) == want


@pytest.mark.parametrize("change, want", [
    (dict(W=None), NULL), (dict(ws=None), NULL), (dict(X=None), NULL), (dict(xs=None), NULL),
    (dict(Y=None), NULL), (dict(t=3), TYPE), (dict(M=0), SHAPE), (dict(N=0), SHAPE),
    (dict(K=0), SHAPE), (dict(K=24), SHAPE), (dict(K=1 << 22), SHAPE), (dict(M=(1 << 31) + 1), SHAPE),
    (dict(W=A4), ALIGN), (dict(X=A4), ALIGN), (dict(Y=A4), ALIGN), (dict(xs=A4), ALIGN),
])
def test_f8_product_refusals(lib, change, want):
    a = dict(W=A16, ws=A16, X=A16, xs=A16, Y=A16, t=1, M=3, N=5, K=32, stream=None)
    a.update(change)
    assert lib.lqmm_gemm_f8b128(*a.values()) == want


@pytest.mark.parametrize("change, want", [
    (dict(X=None), NULL), (dict(Xq=None), NULL), (dict(xs=None), NULL), (dict(t=-1), TYPE),
    (dict(M=0), SHAPE), (dict(K=40), SHAPE), (dict(ld=16), SHAPE), (dict(ld=36), ALIGN),
    (dict(X=A4), ALIGN), (dict(Xq=A4), ALIGN),
])
def test_quant_refusals(lib, change, want):
    a = dict(X=A16, t=1, ld=32, Xq=A16, xs=A16, M=3, K=32, stream=None)
    a.update(change)
    assert lib.lqmm_quant_f8b128(*a.values()) == want


@pytest.mark.skipif(not NO_GPU, reason="needs a machine without a GPU")
def test_well_formed_calls_need_a_device(lib):
    assert _append(lib) == DEVICE and _append(lib, q=None, q_out=None, hq=0, ldq=0) == DEVICE
    assert _append(lib, rot=0, positions=None, turns=None) == DEVICE
    assert _attn(lib) == DEVICE and _attn(lib, plen=0, pp=None) == DEVICE
    assert lib.lqmm_gemm_f8b128(A16, A16, A16, A16, A16, 0, 3, 5, 32, None) == DEVICE
    assert lib.lqmm_quant_f8b128(A16, 0, 32, A16, A16, 3, 32, None) == DEVICE
    assert bq.lqmm_attn_prefix_workspace_bytes(5, 3, 1, 2, 2, 4, 1, 128, 16) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 32)
    with pytest.raises(ValueError):
        bq.lqmm_quant_f8b128(x)
    with pytest.raises(ValueError):
        bq.lqmm_gemm_f8b128(x.to(torch.float8_e4m3fn), x, x.to(torch.float8_e4m3fn), x)
    with pytest.raises(TypeError):
        bq.lqmm_gemm_f8b128(x, x, x, x)
    k, v = bq.kv_cache_empty(2, 1, 16, 64, device="cpu")
    assert k.shape == (2, 1, 16, 64) and v.shape == (2, 1, 2, 64, 8)
    with pytest.raises(ValueError):
        bq.lqmm_kv_append(None, x, x, None, x, k, v)
    with pytest.raises(ValueError):
        bq.lqmm_attn_prefix(x, k, v, x, x)
    with pytest.raises(ValueError):
        bq.kv_cache_empty(2, 1, 12, 64, device="cpu")
