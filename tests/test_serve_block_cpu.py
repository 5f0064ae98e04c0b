"""Host logic of the served attention block on the CPU: the library's calls are
replaced by plain ones that record what they are given."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


class Calls:
    """Stands in for the library: a cache in plain form, outputs of ones."""

    def __init__(self):
        self.slots, self.lens = [], []

    def kv_cache_empty(self, pages, heads, page_size, dim, device):
        self.used = torch.zeros(pages * page_size, dtype=torch.int64)
        return torch.zeros(pages, heads, page_size, dim), torch.zeros(pages, heads, page_size // 8, dim, 8)

    def lqmm_rope_turns(self, inv_freq, device):
        return torch.zeros(len(inv_freq), dtype=torch.int64)

    def lqmm_quant_f8b128(self, x):
        return x, None

    def lqmm_gemm_f8b128(self, w, ws, x, xs):
        return torch.ones(x.shape[0], w.shape[0])

    def lqmm_kv_append(self, q, k, v, positions, slots, k_cache, v_cache, turns):
        assert slots.dtype == torch.int64 and positions.dtype == torch.int32
        self.slots.append(slots.tolist())
        self.positions = positions.tolist()
        for s in slots.tolist():
            if 0 <= s < len(self.used):
                self.used[s] += 1
        return q

    def lqmm_attn_prefix(self, q, k_cache, v_cache, pages, lens, **kw):
        self.lens.append(lens.tolist())
        return q.contiguous()


def block(monkeypatch, batch=3, max_pages=2, page_size=8, prompt_pages=1):
    import block_quantized_matmul_amd as bq
    from block_quantized_matmul_amd.serve import SharedPromptAttention
    calls = Calls()
    for name in ("kv_cache_empty", "lqmm_rope_turns", "lqmm_quant_f8b128", "lqmm_gemm_f8b128",
                 "lqmm_kv_append", "lqmm_attn_prefix"):
        monkeypatch.setattr(bq, name, getattr(calls, name))
    layer = SharedPromptAttention(torch.ones(3 * 64, 64), torch.ones(64, 64), 1, 1, 64, batch,
                                  prompt_pages=prompt_pages, max_pages=max_pages, page_size=page_size)
    return layer, calls


def test_steps_fill_a_conversation_s_own_pages(monkeypatch):
    layer, calls = block(monkeypatch)
    layer.prompt(torch.ones(5, 64))
    for t in range(16):
        y = layer.step(torch.ones(3, 64))
        assert y.isfinite().all()
        assert calls.slots[-1] == [8 + 16 * b + t for b in range(3)]
        assert calls.positions == [5 + t] * 3 and calls.lens[-1] == [t + 1] * 3
    assert calls.used.tolist() == [1] * 5 + [0] * 3 + [1] * 48


def test_a_full_conversation_leaves_the_others_pages_alone(monkeypatch):
    """At max_pages * page_size tokens a conversation's next one is not appended
    anywhere, its length stays and its output is NaN; the others go on."""
    layer, calls = block(monkeypatch)
    layer.lens.copy_(torch.tensor([16, 3, 15], dtype=torch.int32))
    for t, full in enumerate(([0], [0, 2], [0, 2])):
        y = layer.step(torch.ones(3, 64))
        want = [8 + 16 * b + int(n) + t for b, n in enumerate([16, 3, 15])]
        assert calls.slots[-1] == [-1 if b in full else s for b, s in enumerate(want)]
        assert calls.lens[-1] == [16, 4 + t, 16] and layer.lens.tolist() == calls.lens[-1]
        assert [b for b in range(3) if y[b].isnan().all()] == full
        assert [b for b in range(3) if y[b].isfinite().all()] == [b for b in range(3) if b not in full]
    assert int(calls.used.max()) == 1 and calls.used[8:24].sum() == 0


@pytest.mark.parametrize("bad", [-1, -100, 17, 2 ** 31 - 1])
def test_lengths_out_of_range_reach_no_page(monkeypatch, bad):
    layer, calls = block(monkeypatch)
    layer.lens[1] = bad
    layer.step(torch.ones(3, 64))
    slots = calls.slots[-1]
    assert slots[0] == 8 and slots[2] == 40 and (slots[1] == -1 or 24 <= slots[1] < 40)
    assert 0 <= calls.lens[-1][1] <= 16


def test_workspaces_are_allocated_for_each_call_on_its_stream(monkeypatch):
    """What a call on another stream than the current one works in is new, and
    that stream's: nothing is kept and handed to another call."""
    import contextlib
    from types import SimpleNamespace

    import block_quantized_matmul_amd as bq
    on = [None]

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    cuda = SimpleNamespace(stream=stream, default_stream=lambda i: ("default", i),
                           ExternalStream=lambda h, device: ("external", h, device))
    fake = SimpleNamespace(cuda=cuda, uint8="u8", device=lambda *a: a,
                           empty=lambda n, dtype, device: [n, dtype, device, on[-1]])
    monkeypatch.setattr(bq, "_torch", lambda: fake)
    held = SimpleNamespace(cuda_stream=9)
    a, b = bq._workspace_on(1, held, 64), bq._workspace_on(1, held, 64)
    assert a is not b and a == [64, "u8", ("cuda", 1), held]
    assert bq._workspace_on(0, 77, 8)[3] == ("external", 77, 0)
    assert bq._workspace_on(0, 0, 8)[3] == ("default", 0) and on == [None]
