"""Host logic of the served attention block in fewer bits, on the CPU: the
library's calls are replaced by plain ones that record what they are given."""
import pytest

torch = pytest.importorskip("torch")


class Calls:
    def __init__(self):
        self.seen = []

    def __getattr__(self, name):
        def call(*args, **kw):
            self.seen.append((name, args, kw))
            return getattr(self, "_" + name)(*args, **kw)
        return call

    def names(self):
        return [n for n, _, _ in self.seen]

    def last(self, name):
        return [c for c in self.seen if c[0] == name][-1]

    def _kv_cache_empty(self, pages, heads, ps, dim, device, dtype=torch.float16):
        return tuple(torch.zeros(s, dtype=torch.uint8).view(dtype) if dtype.itemsize == 1 else torch.zeros(s, dtype=dtype)
                     for s in ((pages, heads, ps, dim), (pages, heads, ps // 8, dim, 8)))

    def _kv_scales_empty(self, pages, heads, ps, device):
        return torch.zeros(pages, heads, ps), torch.zeros(pages, heads, ps)

    def _lqmm_rope_turns(self, inv_freq, device):
        return torch.zeros(len(inv_freq), dtype=torch.int64)

    def _lqmm_quant_f8b128(self, x):
        return x, "e4m3"

    _lqmm_quant_mxfp4 = lambda self, x: (x, "mxfp4")  # noqa: E731

    def _lqmm_gemm_f8b128(self, w, ws, x, xs):
        assert xs == "e4m3"
        return torch.ones(x.shape[0], w.shape[0])

    def _lqmm_gemm_mxfp4(self, w, ws, x, xs):
        assert ws == xs == "mxfp4"
        return torch.ones(x.shape[0], w.shape[0])

    def _lqmm_kv_append(self, q, *rest):
        return q

    _lqmm_kv_append_norm = lambda self, q, *rest, **kw: q  # noqa: E731
    _lqmm_attn_prefix = lambda self, q, *rest, **kw: q.contiguous()  # noqa: E731
    _lqmm_attn_prefix_f8 = _lqmm_attn_prefix

    def _lqmm_kv_read_f8(self, kc, vc, ks, vs, pages, starts, tokens, dtype):
        return torch.zeros(tokens, 1, 64), torch.zeros(tokens, 1, 64)


def block(monkeypatch, **kw):
    import block_quantized_matmul_amd as bq
    from block_quantized_matmul_amd.serve import SharedPromptAttention
    calls = Calls()
    for name in dir(Calls):
        if name.startswith(("_lqmm", "_kv")):
            monkeypatch.setattr(bq, name[1:], getattr(calls, name[1:]))
    return SharedPromptAttention(torch.ones(3 * 64, 64), torch.ones(64, 64), 1, 1, 64, 3, prompt_pages=2,
                                 max_pages=2, page_size=8, **kw), calls


NORM = torch.full((64,), 0.5, dtype=torch.float64)


@pytest.mark.parametrize("weight_bits", [8, 4])
@pytest.mark.parametrize("kv_bits", [16, 8])
@pytest.mark.parametrize("norms", [dict(), dict(q_norm=NORM), dict(k_norm=NORM, q_norm=NORM, eps=1e-5)])
def test_a_step_calls_the_operators_of_its_form(monkeypatch, weight_bits, kv_bits, norms):
    layer, calls = block(monkeypatch, weight_bits=weight_bits, kv_bits=kv_bits, **norms)
    layer.prompt(torch.ones(5, 64))
    calls.seen.clear()
    y = layer.step(torch.ones(3, 64))
    assert y.isfinite().all() and layer.lens.tolist() == [1] * 3
    of = "mxfp4" if weight_bits == 4 else "f8b128"
    norm = kv_bits == 8 or norms
    append = "lqmm_kv_append_norm" if norm else "lqmm_kv_append"
    attn = "lqmm_attn_prefix" + ("_f8" if kv_bits == 8 else "")
    assert calls.names() == [f"lqmm_quant_{of}", f"lqmm_gemm_{of}", append, attn, f"lqmm_quant_{of}", f"lqmm_gemm_{of}"]
    caches = 4 if kv_bits == 8 else 2
    _, args, kw = calls.last(append)
    assert args[3].tolist() == [5] * 3 and args[4].tolist() == [16, 32, 48]
    assert len(layer.cache) == caches and all(a is b for a, b in zip(args[5:], layer.cache))
    if norm:
        for name in ("q_norm", "k_norm"):
            assert (kw[name] is None) == (name not in norms)
            assert kw[name] is None or kw[name].dtype == torch.float32 and (kw[name] == 0.5).all()
        assert kw["eps"] == norms.get("eps", 1e-6) and kw["rope_turns"] is layer.turns
    _, args, kw = calls.last(attn)
    assert all(a is b for a, b in zip(args[1:], layer.cache)) and args[1 + caches] is layer.pages
    assert kw["prefix_len"] == 5 and args[2 + caches].tolist() == [1] * 3


def test_a_full_conversation_is_not_appended(monkeypatch):
    layer, calls = block(monkeypatch, kv_bits=8, weight_bits=4)
    layer.lens.copy_(torch.tensor([16, 3, 15], dtype=torch.int32))
    for full in ([0], [0, 2]):
        y = layer.step(torch.ones(3, 64))
        slots = calls.last("lqmm_kv_append_norm")[1][4].tolist()
        assert [b for b in range(3) if slots[b] == -1] == full
        assert [b for b in range(3) if y[b].isnan().all()] == full


def test_keys_values_names_the_prompt_and_every_conversation(monkeypatch):
    layer, calls = block(monkeypatch, kv_bits=8)
    layer.prompt(torch.ones(11, 64))
    layer.lens.copy_(torch.tensor([16, 0, 9], dtype=torch.int32))
    k, v, starts = layer.keys_values(torch.float32)
    assert starts == [0, 11, 27, 27, 36] and k.shape == v.shape == (36, 1, 64)
    _, args, kw = calls.last("lqmm_kv_read_f8")
    assert args[4].tolist() == [[0, 1], [2, 3], [4, 5], [6, 7]] and args[4].dtype == torch.int32
    assert args[5].tolist() == starts and args[5].dtype == torch.int32 and args[6] == 36
    assert kw["dtype"] == torch.float32


def test_forms_that_are_not_there_are_refused(monkeypatch):
    for kw in (dict(weight_bits=16), dict(kv_bits=4), dict(weight_bits=None)):
        with pytest.raises(ValueError):
            block(monkeypatch, **kw)
    layer, _ = block(monkeypatch)
    with pytest.raises(ValueError, match="8-bit"):
        layer.keys_values()


def test_keys_values_takes_lengths_as_a_step_does(monkeypatch):
    layer, calls = block(monkeypatch, kv_bits=8)
    layer.prompt(torch.ones(3, 64))
    layer.lens.copy_(torch.tensor([-7, 2 ** 31 - 1, 5], dtype=torch.int32))
    assert layer.keys_values()[2] == [0, 3, 3, 19, 24]


@pytest.mark.parametrize("change", [lambda w: w.double(), lambda w: w.t().contiguous().t(), lambda w: w.half()])
def test_weights_are_taken_in_any_float_type_and_order(monkeypatch, change):
    import block_quantized_matmul_amd as bq
    from block_quantized_matmul_amd.serve import SharedPromptAttention
    calls = Calls()
    for name in dir(Calls):
        if name.startswith(("_lqmm", "_kv")):
            monkeypatch.setattr(bq, name[1:], getattr(calls, name[1:]))
    w = [torch.randn(n, 64, generator=torch.Generator().manual_seed(n)).half().float() for n in (192, 64)]
    SharedPromptAttention(change(w[0]), change(w[1]), 1, 1, 64, 2, 1, 1, weight_bits=4)
    seen = [a[0] for n, a, _ in calls.seen if n == "lqmm_quant_mxfp4"]
    assert len(seen) == 2 and all(s.is_contiguous() and s.dtype == torch.float32 and torch.equal(s, x) for s, x in zip(seen, w))
