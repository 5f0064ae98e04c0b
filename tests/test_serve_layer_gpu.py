"""The serving operators together: a shared prompt, conversations behind it and
their decode steps, eager and from a replayed HIP graph, against the same block
in 64 bits on the dequantized weights.

Tolerance: the inputs of the two products are e4m3 (4 significant bits). What
fp16 rounds differently before a quantization (2^-11) moves at most a share of
about 2^-11 / 2^-4 of the codes to their neighbour, 2^-3 away: an error of
sqrt(2^-7) 2^-3 = 1.1e-2 of the norm for each of the two quantizations, 1.6e-2
together; 2e-2 is allowed."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve_oracle as so
from gpu_util import announce

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


class Plain:
    """The block in 64 bits, with dense caches, for the rows it is given."""

    def __init__(self, layer):
        self.h = (layer.hq, layer.hkv, layer.d)
        deq = lambda w, s: (w.double().cpu().numpy()  # noqa: E731
                            * s.double().cpu().numpy().repeat(128, 0).repeat(128, 1)[:w.shape[0], :w.shape[1]])
        self.wqkv, self.wo = deq(layer.wqkv, layer.wqkv_scale), deq(layer.wo, layer.wo_scale)
        self.inv = 10000.0 ** (-np.arange(0, layer.d, 2) / layer.d)

    def project(self, x, pos):
        hq, hkv, d = self.h
        v, s = so.quantize(x)
        y = (v * s.T.astype(np.float64).repeat(128, 1)[:, :x.shape[1]]) @ self.wqkv.T
        y = y.reshape(len(x), hq + 2 * hkv, d)
        return so.rotate(y[:, :hq], pos, self.inv, False), so.rotate(y[:, hq:hq + hkv], pos, self.inv, False), y[:, hq + hkv:]

    def attend(self, q, k, v):
        """q (hq, d) over k, v (n, hkv, d)."""
        hq, hkv, d = self.h
        out = np.zeros((hq, d))
        for h in range(hq):
            z = k[:, h * hkv // hq] @ q[h] / np.sqrt(d)
            p = np.exp(z - z.max())
            out[h] = p @ v[:, h * hkv // hq] / p.sum()
        return out

    def output(self, o):
        o = o.reshape(len(o), -1).astype(np.float32)
        v, s = so.quantize(o)
        return (v * s.T.astype(np.float64).repeat(128, 1)[:, :o.shape[1]]) @ self.wo.T


def close(got, want, what):
    got = got.double().cpu().numpy()
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= 2e-2, (what, rel)


def test_prompt_and_decode_steps():
    from block_quantized_matmul_amd.serve import SharedPromptAttention
    hidden, hq, hkv, d, batch, n = 272, 4, 2, 64, 5, 37
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    announce("serving block: prompt")
    layer = SharedPromptAttention(r((hq + 2 * hkv) * d, hidden) / hidden ** 0.5,
                                  r(hidden, hq * d) / (hq * d) ** 0.5, hq, hkv, d, batch,
                                  prompt_pages=5, max_pages=3, page_size=8)
    plain = Plain(layer)
    xp = r(n, hidden).half()
    got = layer.prompt(xp)
    q, k, v = plain.project(xp.float().cpu().numpy(), np.arange(n))
    close(got, plain.output(np.stack([plain.attend(q[i], k[:i + 1], v[:i + 1]) for i in range(n)])), "prompt")

    ks, vs = [k for _ in range(batch)], [v for _ in range(batch)]
    x = torch.empty(batch, hidden, dtype=torch.float16, device="cuda")
    x.copy_(r(batch, hidden))
    announce("serving block: capture")
    graph, out = layer.capture(x)
    for t in range(20):
        x.copy_(r(batch, hidden))
        announce(f"serving block: step {t}")
        if t % 3 == 0:  # eager steps between the replays
            got = layer.step(x)
        else:
            graph.replay()
            got = out.clone()
            torch.cuda.synchronize()
        q, k, v = plain.project(x.float().cpu().numpy(), np.full(batch, n + t))
        o = []
        for b in range(batch):
            ks[b], vs[b] = np.concatenate((ks[b], k[b:b + 1])), np.concatenate((vs[b], v[b:b + 1]))
            o.append(plain.attend(q[b], ks[b], vs[b]))
        close(got, plain.output(np.stack(o)), f"step {t}")
    assert layer.lens.tolist() == [20] * batch


def test_replays_equal_eager_steps():
    """A replay gives the bits of an eager step from the same state."""
    from block_quantized_matmul_amd.serve import SharedPromptAttention
    hidden, hq, hkv, d, batch = 512, 16, 2, 128, 7
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    layer = SharedPromptAttention(r((hq + 2 * hkv) * d, hidden) / hidden ** 0.5,
                                  r(hidden, hq * d) / (hq * d) ** 0.5, hq, hkv, d, batch,
                                  prompt_pages=70, max_pages=2, page_size=16)
    layer.prompt(r(1111, hidden).half())
    x = r(batch, hidden).half()
    announce("serving block: capture and replay")
    graph, out = layer.capture(x)
    for t in range(5):
        x.copy_(r(batch, hidden))
        eager = layer.step(x).clone()
        layer.lens -= 1
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), t
