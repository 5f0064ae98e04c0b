"""The served attention block at its edges: conversations that fill their pages,
graphs and their prompts, workspaces of graphs and threads."""
import gc

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


# ---- workspaces that the caller does not pass ------------------------------------
def split_call(seed, batch=24, prefix=700):
    """Arguments of an attention call whose keys are split, and its output by itself."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g).half()  # noqa: E731
    pp, hkv, d, ps = -(-prefix // 16), 2, 128, 16
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (r(batch, 8, d), r(pp + 4 * batch, hkv, ps, d), r(pp + 4 * batch, hkv, ps // 8, d, 8),
            pp + torch.arange(4 * batch, **i32).view(batch, 4), torch.arange(batch, **i32) % 60 + 1)
    kw = dict(prefix_pages=torch.arange(pp, **i32), prefix_len=prefix)
    assert bq.lqmm_attn_prefix_workspace_bytes(prefix, 4, 1, batch, batch, 8, hkv, d, ps) > 0
    out = bq.lqmm_attn_prefix(*args, **kw)
    torch.cuda.synchronize()
    return args, kw, out


@pytest.mark.parametrize("where", ["current", "stream", "handle", "default"])
def test_a_call_keeps_no_workspace(where):
    announce(f"attn workspace of a call on {where}")
    args, kw, want = split_call(1)
    out, s = torch.empty_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    gc.collect()  # (what earlier tests left is not freed in between)
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        if where == "default":  # (the stream's handle is 0)
            with torch.cuda.stream(s):
                bq.lqmm_attn_prefix(*args, **kw, out=out, stream=0)
        else:
            bq.lqmm_attn_prefix(*args, **kw, out=out, stream={"current": None, "stream": s, "handle": s.cuda_stream}[where])
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.cuda.memory_allocated() == before


def test_graphs_of_one_capture_stream_run_beside_each_other():
    """Two graphs captured on one stream, replayed on two, beside eager calls on
    the capture stream: each gives what it gives alone."""
    s, calls = torch.cuda.Stream(), [split_call(seed) for seed in (1, 2, 3)]
    graphs = []
    for args, kw, _ in calls[:2]:
        announce("attn graphs of one capture stream")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = [bq.lqmm_attn_prefix(*args, **kw) for _ in range(8)]
        graphs.append((graph, outs))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(10):
        torch.cuda.synchronize()
        for (graph, outs), on in zip(graphs, streams):
            with torch.cuda.stream(on):
                for o in outs:
                    o.zero_()
                graph.replay()
        with torch.cuda.stream(s):
            eager = [bq.lqmm_attn_prefix(*calls[2][0], **calls[2][1]) for _ in range(8)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, calls[2][2]) for o in eager)
        for (_, outs), (_, _, want) in zip(graphs, calls):
            assert all(torch.equal(o, want) for o in outs), i


def test_threads_of_one_stream_do_not_share_a_workspace():
    import threading
    calls, wrong = [split_call(seed) for seed in (4, 5, 6)], []

    def work(args, kw, want):
        outs = [bq.lqmm_attn_prefix(*args, **kw) for _ in range(200)]
        wrong.append(sum(not torch.equal(o, want) for o in outs))

    announce("attn from three threads on one stream")
    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0, 0]


def test_a_graph_is_not_replayed_behind_another_prompt_length():
    """A graph holds the prompt length of its capture: after a prompt of another
    length its replay is refused, and takes no step; one captured then is right."""
    layer, x_of = small_layer()
    layer.prompt(x_of(17))
    x = x_of(3)
    announce("serving block: prompt after capture")
    graph, _ = layer.capture(x)
    graph.replay()
    layer.prompt(x_of(23))
    torch.cuda.synchronize()
    before = layer.lens.tolist()
    with pytest.raises(RuntimeError, match="prompt"):
        graph.replay()
    torch.cuda.synchronize()
    assert layer.lens.tolist() == before
    graph, out = layer.capture(x)
    eager = layer.step(x).clone()
    layer.lens -= 1
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)
    layer.prompt(x_of(23))  # the same length: the graph stays good
    graph.replay()
    torch.cuda.synchronize()


@pytest.mark.parametrize("bad", [1 << 64, 1 << 90, -1, -(1 << 70)])
def test_numbers_that_are_no_stream_handle_are_refused(bad):
    """An integer outside a pointer's range raises, and nothing runs."""
    announce(f"stream handle {bad}")
    x = torch.ones(3, 128, device="cuda")
    codes = torch.full((3, 128), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((1, 3), 9.0, device="cuda")
    with pytest.raises(OverflowError):
        bq.lqmm_quant_f8b128(x, out=codes, scales=scales, stream=bad)
    torch.cuda.synchronize()
    assert (codes == 9).all() and (scales == 9).all()
