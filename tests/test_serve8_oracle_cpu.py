"""The 64-bit forms of serve8_oracle.py against hand-worked values, and what the
entry points of the serving operators in fewer bits refuse (no GPU)."""
import ctypes
import os

import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve8_oracle as s8

NO_GPU = not os.path.exists("/dev/kfd")
NULL, SHAPE, ALIGN, WORKSPACE, DEVICE, TYPE = 1, 2, 3, 4, 5, 7
A16, A4 = 0x10000, 0x10004


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bq.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return bq.load()


def test_status_numbers(lib):
    names = {NULL: "NULL", SHAPE: "SHAPE", ALIGN: "ALIGN", WORKSPACE: "WORKSPACE", DEVICE: "DEVICE", TYPE: "TYPE"}
    for n, name in names.items():
        assert name in bq.lqmm_status_string(n)


def test_exponents():
    f = lambda x, t="bf16": int(s8.exponent(np.array([x]), t)[0])  # noqa: E731
    assert f(448.0) == 0 and f(448.0001) == 1 and f(224.0) == -1 and f(1.0) == -8 and f(1.75) == -8
    assert f(1.7500001) == -7 and f(0.0) == -60 and f(1e-30) == -60 and f(1e30) == 60 and f(1e30, "f16") == 7


def test_codes():
    c, e = s8.quant(np.array([[448.0, 17.0, 18.0, 19.0, -1.0, 0.0]]), "f16")
    assert e[0] == 0 and c[0].tolist() == [448, 16, 18, 20, -1, 0]
    c, e = s8.quant(np.array([[np.inf, 2.0, np.nan, -3.5]]), "f16")
    assert e[0] == -7 and np.isnan(c[0, [0, 2]]).all() and c[0, 1] == 256 and c[0, 3] == -448
    c, e = s8.quant(np.array([[65504.0, 1.0]]), "f16")
    assert e[0] == 7 and c[0, 0] == 448


def test_norm():
    y = s8.norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, np.array([[3, 8]]) / np.sqrt(12.5))
    assert np.array_equal(s8.norm(np.array([[3.0]]), None, 1.0), [[3.0]])


def test_mx():
    x = np.zeros((2, 32))
    x[0, :8] = [6, -0.25, 0.75, 1.25, 5, 3.5, 2.5, 0.26]
    x[1, 0] = 7.9
    c, s = s8.mx_quant(x)
    assert s.tolist() == [[127], [127]]
    assert s8.mx_values(c, s)[0, :8].tolist() == [6, 0, 1, 1, 4, 4, 2, 0.5]
    assert s8.mx_values(c, s)[1, 0] == 6 and s8.mx_pack(c).shape == (2, 16)
    assert s8.mx_pack(np.array([[1, 2]]))[0, 0] == 0x21
    c, s = s8.mx_quant(np.full((1, 32), np.inf))
    assert s[0, 0] == 255 and not c.any()
    c, s = s8.mx_quant(np.zeros((1, 32)))
    assert s[0, 0] == 0


def test_attention_of_two_keys():
    kc, vc = np.zeros((1, 1, 8, 64)), np.zeros((1, 1, 1, 64, 8))
    ks, vs = np.full((1, 1, 8), 127, np.uint8), np.full((1, 1, 8), 127, np.uint8)
    kc[0, 0, 1, 0], ks[0, 0, 1] = 2.0, 126  # 1.0
    vc[0, 0, 0, :, 0], vc[0, 0, 0, :, 1], vs[0, 0, 1] = 1.0, 1.0, 129  # 1 and 4
    q = np.zeros((1, 1, 64))
    q[0, 0, 0] = np.log(3.0)
    o, lse, *_ = s8.attention(q, (kc, vc, ks, vs), [[0]], [2], [], 0, [0, 1], 1.0, "bf16")
    assert np.allclose(o, (1 + 3 * 4) / 4) and np.allclose(lse, np.log(4.0))


# ---- refusals --------------------------------------------------------------------
def _append(lib, **kw):
    a = dict(q=A16, k=A16, v=A16, in_type=1, ldq=512, ldk=128, ldv=128, positions=A16, slots=A16,
             turns=A16, rot=128, inter=0, qn=A16, kn=A16, eps=ctypes.c_float(1e-6), q_out=A16, kc=A16,
             vc=A16, ks=A16, vs=A16, type=1, tokens=3, hq=4, hkv=1, d=128, ps=16, pages=4, stream=None)
    a.update(kw)
    return lib.lqmm_kv_append_norm(*a.values())


@pytest.mark.parametrize("change, want", [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(kc=None), NULL),
    (dict(vc=None), NULL), (dict(q=None), NULL), (dict(q_out=None), NULL), (dict(ks=None), NULL),
    (dict(vs=None), NULL), (dict(positions=None), NULL), (dict(turns=None), NULL),
    (dict(in_type=3), TYPE), (dict(type=0), TYPE), (dict(type=9), TYPE),
    (dict(tokens=0), SHAPE), (dict(pages=0), SHAPE), (dict(d=80), SHAPE), (dict(ps=12), SHAPE),
    (dict(ps=2048), SHAPE), (dict(hkv=0), SHAPE), (dict(hq=-1), SHAPE), (dict(rot=8), SHAPE),
    (dict(rot=144), SHAPE), (dict(ldq=504), SHAPE), (dict(ldk=120), SHAPE),
    (dict(eps=ctypes.c_float(-1e-6)), SHAPE), (dict(eps=ctypes.c_float(float("inf"))), SHAPE),
    (dict(eps=ctypes.c_float(float("nan"))), SHAPE),
    (dict(ldk=132), ALIGN), (dict(k=A4), ALIGN), (dict(kc=A4), ALIGN), (dict(q=A4), ALIGN),
    (dict(slots=A4), ALIGN), (dict(qn=A4), ALIGN), (dict(kn=A4), ALIGN), (dict(ks=A4), ALIGN),
    (dict(vs=A4), ALIGN),
])
def test_append_refusals(lib, change, want):
    assert _append(lib, **change) == want


def _read(lib, **kw):
    a = dict(kc=A16, vc=A16, ks=A16, vs=A16, pages=A16, mp=3, starts=A16, ko=A16, vo=A16, type=1,
             tokens=5, batch=2, hkv=1, d=128, ps=16, npages=9, stream=None)
    a.update(kw)
    return lib.lqmm_kv_read_f8(*a.values())


@pytest.mark.parametrize("change, want", [
    *[({n: None}, NULL) for n in ("kc", "vc", "ks", "vs", "pages", "starts", "ko", "vo")],
    (dict(type=3), TYPE), (dict(tokens=0), SHAPE), (dict(batch=0), SHAPE), (dict(mp=0), SHAPE),
    (dict(hkv=0), SHAPE), (dict(d=32), SHAPE), (dict(ps=4), SHAPE), (dict(npages=0), SHAPE),
    (dict(tokens=1 << 31), SHAPE), (dict(batch=1 << 31), SHAPE),
    *[({n: A4}, ALIGN) for n in ("kc", "vc", "ks", "vs", "ko", "vo")], (dict(pages=0x10002), ALIGN),
    (dict(starts=0x10002), ALIGN),
])
def test_read_refusals(lib, change, want):
    assert _read(lib, **change) == want


def _attn(lib, **kw):
    a = dict(q=A16, ldq=512, kc=A16, vc=A16, ks=A16, vs=A16, type=1, pp=A16, plen=5, pages=A16, mp=3,
             lens=A16, start=None, max_q=1, out=A16, lse=None, scale=ctypes.c_float(0.1), tokens=2,
             batch=2, hq=4, hkv=1, d=128, ps=16, npages=9, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    return lib.lqmm_attn_prefix_f8(*a.values())


@pytest.mark.parametrize("change, want", [
    *[({n: None}, NULL) for n in ("q", "kc", "vc", "ks", "vs", "pages", "lens", "out", "pp")],
    (dict(type=0), TYPE), (dict(type=5), TYPE),
    (dict(tokens=0), SHAPE), (dict(batch=0), SHAPE), (dict(mp=0), SHAPE), (dict(max_q=0), SHAPE),
    (dict(plen=-1), SHAPE), (dict(hq=5, hkv=2), SHAPE), (dict(d=32), SHAPE), (dict(ps=24), SHAPE),
    (dict(npages=0), SHAPE), (dict(tokens=3), SHAPE), (dict(mp=1 << 30), SHAPE),
    (dict(scale=ctypes.c_float(float("nan"))), SHAPE), (dict(ldq=384), SHAPE),
    (dict(ldq=516), ALIGN), (dict(q=A4), ALIGN), (dict(out=A4), ALIGN), (dict(lens=0x10002), ALIGN),
    (dict(ws=A4, ws_bytes=1 << 20), ALIGN), (dict(ks=A4), ALIGN), (dict(vs=A4), ALIGN),
])
def test_attention_refusals(lib, change, want):
    assert _attn(lib, **change) == want


@pytest.mark.parametrize("change, want", [
    *[({n: None}, NULL) for n in ("W", "ws", "X", "xs", "Y")], (dict(t=3), TYPE), (dict(M=0), SHAPE),
    (dict(N=0), SHAPE), (dict(K=0), SHAPE), (dict(K=48), SHAPE), (dict(K=1 << 22), SHAPE),
    (dict(M=(1 << 31) + 1), SHAPE), *[({n: A4}, ALIGN) for n in ("W", "X", "Y")],
])
def test_product_refusals(lib, change, want):
    a = dict(W=A16, ws=A16, X=A16, xs=A16, Y=A16, t=1, M=3, N=5, K=64, stream=None)
    a.update(change)
    assert lib.lqmm_gemm_mxfp4(*a.values()) == want


@pytest.mark.parametrize("change, want", [
    (dict(X=None), NULL), (dict(Xq=None), NULL), (dict(xs=None), NULL), (dict(t=-1), TYPE),
    (dict(M=0), SHAPE), (dict(K=40), SHAPE), (dict(ld=16), SHAPE), (dict(ld=36), ALIGN),
    (dict(X=A4), ALIGN), (dict(Xq=A4), ALIGN),
])
def test_quant_refusals(lib, change, want):
    a = dict(X=A16, t=1, ld=32, Xq=A16, xs=A16, M=3, K=32, stream=None)
    a.update(change)
    assert lib.lqmm_quant_mxfp4(*a.values()) == want


@pytest.mark.skipif(not NO_GPU, reason="needs a machine without a GPU")
def test_well_formed_calls_need_a_device(lib):
    assert _append(lib) == DEVICE and _append(lib, ks=None, vs=None) == DEVICE
    assert _append(lib, qn=None, kn=None, q=None, q_out=None, hq=0, ldq=0) == DEVICE
    assert _read(lib) == DEVICE and _read(lib, type=0) == DEVICE
    assert _attn(lib) == DEVICE and _attn(lib, plen=0, pp=None) == DEVICE
    assert lib.lqmm_gemm_mxfp4(A16, A4 + 1, A16, A4 + 2, A16, 0, 3, 5, 32, None) == DEVICE
    assert lib.lqmm_quant_mxfp4(A16, 0, 32, A16, A4 + 3, 3, 32, None) == DEVICE
    assert bq.lqmm_attn_prefix_f8_workspace_bytes(5, 3, 1, 2, 2, 4, 1, 128, 16) == 0


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        bq.lqmm_quant_mxfp4(x)
    with pytest.raises(TypeError):
        bq.lqmm_gemm_mxfp4(x, x, x, x)
    with pytest.raises(ValueError):
        bq.lqmm_gemm_mxfp4(x.byte(), x, x.byte(), x)
    k, v = bq.kv_cache_empty(2, 1, 16, 64, dtype=torch.float8_e4m3fn, device="cpu")
    ks, vs = bq.kv_scales_empty(2, 1, 16, device="cpu")
    assert k.dtype == torch.float8_e4m3fn and ks.shape == (2, 1, 16) and ks.dtype == torch.float8_e8m0fnu
    assert (ks.float() == 1).all() and ks.data_ptr() != vs.data_ptr()
    with pytest.raises(ValueError):
        bq.kv_scales_empty(2, 1, 12, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        bq.lqmm_kv_append_norm(None, x, x, None, x, k, v, ks, vs)
    with pytest.raises(ValueError):
        bq.lqmm_kv_read_f8(k, v, ks, vs, i, i, 3)
    with pytest.raises(ValueError):
        bq.lqmm_attn_prefix_f8(x, k, v, ks, vs, i, i)
    with pytest.raises(TypeError):
        bq.lqmm_attn_prefix_f8(x, x, x, ks, vs, i, i)
