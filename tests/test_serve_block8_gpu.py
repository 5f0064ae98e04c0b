"""The serving operators in fewer bits together, as the served attention block
runs them: a prompt, decode steps, eager and from a replayed HIP graph.

Each operator's results inside the block are held to its own bound, from what the
block gave it; replays equal eager steps bit for bit; and the whole is compared
with the block in 64 bits.

Tolerance of the whole: what fp16 rounds differently before a quantization
(2^-11) moves a share of about 2^-11 / s of the codes to a neighbour s away
(relative to the value; s 2^-3 for e4m3, 2^-1 at most for the 4-bit floats), an
error of sqrt(2^-11 s) of the norm: 1.6e-2 at each of two products in 4 bits,
0.8e-2 in e4m3 (1.1e-2 as test_serve_layer_gpu.py counts it), and 0.8e-2 for each
of K and V in an 8-bit cache. Added up without cancellation: 3.2e-2 + 1.6e-2.
5e-2 is allowed."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve8_oracle as s8
import serve_oracle as so
from gpu_util import announce
from test_serve8_gpu import values
from test_serve_gpu import np64, within

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


def make(weight_bits, kv_bits, hidden=288, hq=4, hkv=2, d=64, batch=5, prompt_pages=5, max_pages=3, ps=8, seed=1):
    from block_quantized_matmul_amd.serve import SharedPromptAttention
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    wqkv, wo = r((hq + 2 * hkv) * d, hidden) / hidden ** 0.5, r(hidden, hq * d) / (hq * d) ** 0.5
    norms = [1 + 0.2 * r(d) for _ in range(2)]
    layer = SharedPromptAttention(wqkv, wo, hq, hkv, d, batch, prompt_pages=prompt_pages, max_pages=max_pages,
                                  page_size=ps, weight_bits=weight_bits, kv_bits=kv_bits, q_norm=norms[0],
                                  k_norm=norms[1], eps=EPS)
    return layer, (wqkv, wo, *norms), lambda n: r(n, hidden).half()


class Plain:
    """The block in 64 bits, with dense caches."""

    def __init__(self, layer, weights):
        self.l = layer
        self.wqkv, self.wo = (self.quant(np64(w)) if layer.weight_bits == 4 else self.f8(w) for w in weights[:2])
        self.norms = [np64(w) for w in weights[2:]]
        self.inv = 10000.0 ** (-np.arange(0, layer.d, 2) / layer.d)

    def f8(self, w):
        from block_quantized_matmul_amd.serve import quantize_weight_f8b128
        c, s = quantize_weight_f8b128(w)
        return np64(c.float()) * np64(s).repeat(128, 0).repeat(128, 1)[:w.shape[0], :w.shape[1]]

    def quant(self, x):
        if self.l.weight_bits == 4:
            return s8.mx_values(*s8.mx_quant(x))
        v, s = so.quantize(x.astype(np.float32))
        return v * s.T.astype(np.float64).repeat(128, 1)[:, :x.shape[1]]

    def project(self, x, pos):
        hq, hkv, d = self.l.hq, self.l.hkv, self.l.d
        y = (self.quant(x) @ self.wqkv.T).reshape(len(x), hq + 2 * hkv, d)
        q, k = (so.rotate(s8.norm(a, w, EPS), pos, self.inv, False)
                for a, w in zip((y[:, :hq], y[:, hq:hq + hkv]), self.norms))
        return q, self.held(k), self.held(y[:, hq + hkv:])

    def held(self, x):
        if self.l.kv_bits == 16:
            return x
        v, e = s8.quant(x, "f16")
        return v * np.exp2(e.astype(np.float64))[..., None]

    def attend(self, q, k, v):
        out = np.zeros(q.shape)
        for h in range(self.l.hq):
            z = k[:, h * self.l.hkv // self.l.hq] @ q[h] / np.sqrt(self.l.d)
            p = np.exp(z - z.max())
            out[h] = p @ v[:, h * self.l.hkv // self.l.hq] / p.sum()
        return out

    def output(self, o):
        return self.quant(o.reshape(len(o), -1)) @ self.wo.T


def close(got, want, what):
    rel = np.linalg.norm(np64(got) - want) / np.linalg.norm(want)
    print(f"{what}: {rel:.2e}", flush=True)
    assert rel <= 5e-2, (what, rel)


@pytest.mark.parametrize("weight_bits, kv_bits", [(4, 8), (4, 16), (8, 8), (8, 16)])
def test_prompt_and_decode_steps(weight_bits, kv_bits):
    layer, weights, x_of = make(weight_bits, kv_bits)
    plain, n, batch = Plain(layer, weights), 37, 5
    announce(f"serving block {weight_bits}/{kv_bits}: prompt")
    xp = x_of(n)
    got = layer.prompt(xp)
    q, k, v = plain.project(np64(xp), np.arange(n))
    close(got, plain.output(np.stack([plain.attend(q[i], k[:i + 1], v[:i + 1]) for i in range(n)])), "prompt")
    ks, vs = [k] * batch, [v] * batch
    x = x_of(batch)
    announce(f"serving block {weight_bits}/{kv_bits}: capture")
    graph, out = layer.capture(x)
    for t in range(13):
        x.copy_(x_of(batch))
        if t % 3 == 0:  # eager steps between the replays
            got = layer.step(x)
        else:
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone()
        q, k, v = plain.project(np64(x), np.full(batch, n + t))
        ks = [np.concatenate((a, k[b:b + 1])) for b, a in enumerate(ks)]
        vs = [np.concatenate((a, v[b:b + 1])) for b, a in enumerate(vs)]
        close(got, plain.output(np.stack([plain.attend(q[b], ks[b], vs[b]) for b in range(batch)])), f"step {t}")
    assert layer.lens.tolist() == [13] * batch


@pytest.mark.parametrize("d, hq, hkv, ps, prompt", [(64, 4, 2, 8, 37), (128, 16, 2, 16, 300), (96, 6, 6, 32, 1), (256, 4, 1, 8, 70)])
def test_each_operator_inside_the_block(monkeypatch, d, hq, hkv, ps, prompt):
    """What each call of a prompt and of three steps returned, against 64 bits of
    what it was given."""
    layer, _, x_of = make(4, 8, hidden=416, hq=hq, hkv=hkv, d=d, batch=3, ps=ps, prompt_pages=-(-prompt // ps), max_pages=2)
    calls = []
    for name in ("lqmm_quant_mxfp4", "lqmm_gemm_mxfp4", "lqmm_kv_append_norm", "lqmm_attn_prefix_f8"):
        def record(*args, name=name, call=getattr(bq, name), **kw):
            out = call(*args, **kw)
            keep = lambda x: x.clone() if isinstance(x, torch.Tensor) else x  # noqa: E731
            calls.append((name, [keep(a) for a in args], {k: keep(a) for k, a in kw.items()},
                          [keep(a) for a in (out if isinstance(out, tuple) else (out,))]))
            return out
        monkeypatch.setattr(bq, name, record)
    announce(f"serving block d={d} heads {hq}/{hkv} prompt {prompt}")
    layer.prompt(x_of(prompt))
    for _ in range(3):
        layer.step(x_of(3))
    torch.cuda.synchronize()
    assert len(calls) == 24
    inv = 10000.0 ** (-np.arange(0, d, 2) / d)
    for name, a, kw, out in calls:
        if name == "lqmm_quant_mxfp4":
            c, s = s8.mx_quant(np64(a[0]))
            assert np.array_equal(out[0].cpu().numpy(), s8.mx_pack(c))
            assert np.array_equal(out[1].view(torch.uint8).cpu().numpy(), s)
        elif name == "lqmm_gemm_mxfp4":
            def held(codes, scales):
                b = codes.cpu().numpy()
                c = np.stack((b & 15, b >> 4), -1).reshape(len(b), -1)
                return s8.mx_values(c, scales.view(torch.uint8).cpu().numpy())
            W, X = held(a[0], a[1]), held(a[2], a[3])
            want, total = X @ W.T, np.abs(X) @ np.abs(W).T
            bound = so.U["f16"] * np.abs(want) + so.TINY["f16"]
            bound += (X.shape[1] / 128 + 10) * 2.0 ** -24 * (1 + so.U["f16"]) * total
            within(out[0], want, bound, "product")
        elif name == "lqmm_kv_append_norm":
            q, k, v, pos, slots, kc, vc, ks, vs = a
            pos, slots = pos.cpu().numpy(), slots.tolist()
            want, e = s8.norm_rotate(np64(q), np64(kw["q_norm"]), EPS, pos, inv, False)
            within(out[0], want, so.U["f16"] * np.abs(want) + so.TINY["f16"] + (1 + so.U["f16"]) * e, "q")
            want, e = s8.norm_rotate(np64(k), np64(kw["k_norm"]), EPS, pos, inv, False)
            kc, ks = values(kc), ks.view(torch.uint8).cpu().numpy().astype(np.float64)
            vc, vs = values(vc), vs.view(torch.uint8).cpu().numpy().astype(np.float64)
            vv, vx = s8.quant(np64(v), "f16")
            for t, s in enumerate(slots):
                p, o = s // ps, s % ps
                x = ks[p, :, o].astype(int) - 127
                within(kc[p, :, o] * np.exp2(x.astype(float))[:, None], want[t], s8.held_bound(want[t], e[t], x, "f16"), "k")
                assert np.array_equal(vc[p, :, o // 8, :, o % 8], vv[t]) and np.array_equal(vs[p, :, o], vx[t] + 127.0)
        else:
            q, kc, vc, ks, vs, pages, lens = a
            cache = (values(kc), values(vc), *(x.view(torch.uint8).cpu().numpy() for x in (ks, vs)))
            lens = lens.tolist()
            start = kw["q_start"].tolist() if "q_start" in kw else list(range(len(lens) + 1))
            pre = kw.get("prefix_pages")
            wo, _, bo, _ = s8.attention(np64(q), cache, pages.cpu().numpy(), lens, [] if pre is None else pre.tolist(),
                                        kw.get("prefix_len", 0), start, d ** -0.5, "f16")
            within(out[0], wo, bo, "attention")


@pytest.mark.parametrize("weight_bits, kv_bits", [(4, 8), (8, 8), (4, 16)])
def test_replays_equal_eager_steps(weight_bits, kv_bits):
    layer, _, x_of = make(weight_bits, kv_bits, hidden=512, hq=16, hkv=2, d=128, batch=7, prompt_pages=70, max_pages=2, ps=16)
    layer.prompt(x_of(1111))
    x = x_of(7)
    announce(f"serving block {weight_bits}/{kv_bits}: capture and replay")
    graph, out = layer.capture(x)
    for t in range(5):
        x.copy_(x_of(7))
        eager = layer.step(x).clone()
        layer.lens -= 1
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert eager.isfinite().all() and torch.equal(out, eager), t


def test_keys_values_are_those_of_the_cache():
    layer, _, x_of = make(4, 8)
    layer.prompt(x_of(37))
    for _ in range(4):
        layer.step(x_of(5))
    layer.lens[2] = 0  # a conversation with nothing of its own
    announce("serving block: keys_values")
    for dtype in (None, torch.float32):
        k, v, starts = layer.keys_values(dtype)
        torch.cuda.synchronize()
        assert starts == [0, 37, 41, 45, 45, 49, 53] and k.dtype == v.dtype == (dtype or torch.float16)
        cache = [values(layer.k_cache), values(layer.v_cache),
                 *(x.view(torch.uint8).cpu().numpy() for x in layer.cache[2:])]
        tables = [layer.prompt_pages] + list(layer.pages)
        for i, ids in enumerate(tables):
            n = starts[i + 1] - starts[i]
            kk, vv, _ = s8.tokens_of(*cache, ids.tolist(), n)
            for got, want in ((k, kk), (v, vv)):
                want = want.transpose(1, 0, 2)
                want = s8.to_type(want, "f16") if dtype is None else want
                assert np.array_equal(np64(got)[starts[i]:starts[i + 1]], want)


@pytest.mark.parametrize("replayed", [False, True])
def test_full_conversations_write_nothing(replayed):
    """Steps past a conversation's last slot: its pages and scales stay, its
    output is NaN, the others' are those of a batch in which it is not full."""
    got = []
    for lens in ([3, 9, 5], [3, 16, 5]):
        layer, _, x_of = make(4, 8, hidden=128, batch=3, prompt_pages=5, max_pages=2)
        layer.prompt(x_of(17))
        layer.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        for c in layer.cache:  # (what earlier steps would have left)
            c.view(torch.uint8)[layer.pages.long().flatten()] = 0x38 if c.dim() > 3 else 120
        kept = [c.view(torch.uint8).clone() for c in layer.cache]
        x = x_of(3)
        announce(f"serving block in fewer bits: lengths {lens}, replayed {replayed}")
        if replayed:
            graph, out = layer.capture(x)
        ys = []
        for _ in range(3):
            x.copy_(x_of(3))
            if replayed:
                graph.replay()
            else:
                out = layer.step(x)
            torch.cuda.synchronize()
            ys.append(out.clone())
        got.append((layer, torch.stack(ys), kept))
    (_, yf, _), (full, yn, kept) = got
    assert full.lens.tolist() == [6, 16, 8]
    assert yn[:, 1].isnan().all() and torch.equal(yn[:, ::2], yf[:, ::2])
    mine = full.pages[1].long()
    assert all(torch.equal(c.view(torch.uint8)[mine], k[mine]) for c, k in zip(full.cache, kept))
