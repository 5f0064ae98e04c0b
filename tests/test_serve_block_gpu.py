"""The served attention block at its edges: conversations that fill their pages,
graphs and their prompts, workspaces of graphs and threads."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
from gpu_util import announce

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


def small_layer(prompt_pages=5, max_pages=2, batch=3):
    from block_quantized_matmul_amd.serve import SharedPromptAttention
    hidden, hq, hkv, d = 128, 4, 2, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    layer = SharedPromptAttention(r((hq + 2 * hkv) * d, hidden) / hidden ** 0.5,
                                  r(hidden, hq * d) / (hq * d) ** 0.5, hq, hkv, d, batch,
                                  prompt_pages=prompt_pages, max_pages=max_pages, page_size=8)
    for c in (layer.k_cache, layer.v_cache):
        c.copy_(r(*c.shape))
    return layer, lambda n: r(n, hidden).half()


@pytest.mark.parametrize("replayed", [False, True])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_full_conversations_write_nothing(at, replayed):
    """Steps past a conversation's last free slot, eager and replayed: no page
    changes for it, the other conversations' outputs and pages are those of a
    batch in which it is not full."""
    got = []
    for lens in ([3, 9, 5], [3, 9, 5][:at] + [16] + [3, 9, 5][at + 1:]):
        layer, x_of = small_layer()
        layer.prompt(x_of(17))
        layer.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        k, v = layer.k_cache.clone(), layer.v_cache.clone()
        x = x_of(3)
        announce(f"serving block: conversation {at} at {lens[at]} of 16 tokens, replayed {replayed}")
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
        got.append((layer, torch.stack(ys), k, v))
    (free, yf, _, _), (full, yn, k, v) = got
    rest = [b for b in range(3) if b != at]
    assert full.lens.tolist() == [16 if b == at else [6, 12, 8][b] for b in range(3)]
    assert yn[:, at].isnan().all() and torch.equal(yn[:, rest], yf[:, rest])
    mine = full.pages[at].long()
    assert torch.equal(full.k_cache[mine], k[mine]) and torch.equal(full.v_cache[mine], v[mine])
    others = [p for p in range(len(k)) if p not in mine.tolist()]
    assert torch.equal(full.k_cache[others], free.k_cache[others])
    assert torch.equal(full.v_cache[others], free.v_cache[others])
